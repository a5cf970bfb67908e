"""Attention over a paged key-value cache, operator by operator: cases, inputs, plain forms.

Three operators of the library:

  append   the position rotation of new queries and keys; keys and values into the paged cache
  decode   attention of one new token of each sequence over its cache
  prefill  causal attention of the new tokens of prompts (or of chunks of prompts) over the cache

Both attentions may have a sliding window, with a few first tokens that stay visible.

The cache is a pool of pages of ``page`` tokens, a list of page numbers for each sequence.  In a page, each
key-value head has ``page * D`` elements of K and of V:

  K  [page / 16][D / c][16][c]   token t, column d at [t / 16][d / c][t % 16][d % c], c = 16 bytes of elements
  V  [page / 32][4][D][8]        token t, column d at [t / 32][t % 16 / 4][d][t % 32 / 16 * 4 + t % 4]

Elements are float16, bfloat16, or e4m3 with one fp32 scale for each token and head ([page] of K and of V):
the scale is the largest magnitude of the row over 448, at least 2^-126, and the values are e4m3(v / scale).

``own`` chooses what ``run`` measures: the plain forms below, or the library's calls.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126
FP8 = torch.float8_e4m3fn
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
THETA = 1e6


# ---------------------------------------------------------------- cases
#
# B sequences; lens: the longest cache, spread: its ratio to the shortest; new: the most new tokens of a sequence
# (append, prefill; 0: the whole cache is new); x: type of q, k, v; c8: the cache is e4m3; out8: the output is e4m3

def listed():
    return [
        # a single user's next token: rotation and cache write, latency
        dict(name="append_t1", op="append", B=1, lens=777, spread=1, new=1, Hq=32, Hkv=8, D=128, page=32, x="bf16",
             c8=False, rot=128, inter=False),
        # the decode step of a batch, half of each head rotated, pairs side by side
        dict(name="append_decode_b256", op="append", B=256, lens=900, spread=4, new=1, Hq=16, Hkv=4, D=256, page=64,
             x="f16", c8=False, rot=128, inter=True),
        # a chunk of three prompts into an 8-bit cache
        dict(name="append_chunk_c8", op="append", B=3, lens=2200, spread=2, new=1900, Hq=32, Hkv=8, D=128, page=64,
             x="bf16", c8=True, rot=128, inter=False),
        # long prompts of a model with 48 query heads
        dict(name="append_prompts", op="append", B=5, lens=6001, spread=3, new=0, Hq=48, Hkv=8, D=128, page=128,
             x="f16", c8=False, rot=128, inter=False),
        # a single user's next token after a short prompt: latency
        dict(name="decode_b1_short", op="decode", B=1, lens=601, spread=1, Hq=32, Hkv=8, D=128, page=32, x="bf16",
             c8=False, out8=False, window=0, sinks=0),
        # one very long context
        dict(name="decode_b1_long", op="decode", B=1, lens=131072, spread=1, Hq=48, Hkv=8, D=128, page=128, x="f16",
             c8=False, out8=False, window=0, sinks=0),
        # a serving batch of very uneven lengths
        dict(name="decode_b64_uneven", op="decode", B=64, lens=16000, spread=100, Hq=32, Hkv=8, D=128, page=32,
             x="bf16", c8=False, out8=False, window=0, sinks=0),
        # a large serving batch on an 8-bit cache, the output in 8 bits for the projection behind it
        dict(name="decode_b200_c8_out8", op="decode", B=200, lens=2600, spread=3, Hq=32, Hkv=8, D=128, page=64,
             x="bf16", c8=True, out8=True, window=0, sinks=0),
        # long conversations, a window of 4096 tokens and four first tokens, a key head for each query head
        dict(name="decode_b24_window", op="decode", B=24, lens=30000, spread=20, Hq=16, Hkv=16, D=64, page=64,
             x="f16", c8=False, out8=False, window=4096, sinks=4),
        # a few short prompts, an 8-bit cache
        dict(name="prefill_short_c8", op="prefill", B=7, lens=120, spread=30, new=0, Hq=32, Hkv=8, D=128, page=32,
             x="f16", c8=True, window=0, sinks=0),
        # one prompt
        dict(name="prefill_8192", op="prefill", B=1, lens=8192, spread=1, new=0, Hq=32, Hkv=8, D=128, page=64,
             x="bf16", c8=False, window=0, sinks=0),
        # chunks of long documents behind what is in the cache already: the largest
        dict(name="prefill_chunk_window", op="prefill", B=3, lens=20011, spread=2, new=6000, Hq=48, Hkv=8, D=128,
             page=128, x="bf16", c8=False, window=8192, sinks=16),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "prefill"])
    D, page = rng.choice([64, 128, 128, 256]), rng.choice([32, 64, 128, 256])
    Hkv, G = rng.choice([1, 2, 3, 4, 8, 8, 16]), rng.choice([1, 2, 3, 4, 4, 5, 6, 8, 12, 16])
    x, spread = rng.choice(["f16", "bf16"]), rng.choice([1, 1, 2, 7, 40])
    c = dict(op=op, Hq=Hkv * G, Hkv=Hkv, D=D, page=page, x=x, spread=spread, c8=rng.random() < 0.4)
    if op == "append":
        most = max(1, 60_000_000 // (Hkv * (G + 2) * D))  # rows
        c["B"] = _log_int(rng, 1, min(256, most))
        c["new"] = rng.choice([1, _log_int(rng, 1, max(1, most // c["B"]))])
        c["lens"] = c["new"] + _log_int(rng, 1, 500)
        return dict(c, rot=rng.choice([0, 32, D // 2, D, D]), inter=rng.random() < 0.4)
    window = rng.choice([0, 0, _log_int(rng, 8, 8192)])
    c["window"], c["sinks"] = window, rng.choice([0, rng.randint(1, 200)]) if window else 0
    if op == "decode":
        most = max(40, 250_000_000 // (Hkv * D))  # tokens
        c["B"] = _log_int(rng, 1, 256)
        c["lens"] = _log_int(rng, 1, max(1, min(131072, most // c["B"])))
        return dict(c, out8=D % 128 == 0 and rng.random() < 0.4)
    c["B"] = _log_int(rng, 1, 12)
    pairs = 3.0e12 / (4 * D * c["Hq"] * c["B"])
    c["lens"] = _log_int(rng, 1, max(1, min(24000, int(math.sqrt(pairs)))))
    c["new"] = rng.choice([0, _log_int(rng, 1, c["lens"])])
    return c


def _lens(c):
    """Tokens in each cache: spread evenly over their logarithm, in an order that is neither sorted nor random."""
    B, hi = c["B"], c["lens"]
    lo = max(1, hi // c["spread"])
    step = next(s for s in range(max(1, int(B * 0.618)), 2 * B + 2) if math.gcd(s, B) == 1)
    return [int(round(hi * (lo / hi) ** ((i * step % B) / max(1, B - 1)))) for i in range(B)]


def _news(c):
    if c["op"] == "decode":
        return [1] * c["B"]
    return [n if c["new"] == 0 else min(n, c["new"]) for n in _lens(c)]


# ---------------------------------------------------------------- inputs

def _pack_k(x, size):
    """[..., page, D] -> the order of K in a page; size: bytes of an element."""
    c = 16 // size
    *lead, page, D = x.shape
    x = x.reshape(*lead, page // 16, 16, D // c, c)
    return x.transpose(-3, -2).reshape(*lead, page * D)


def _pack_v(x):
    *lead, page, D = x.shape
    x = x.reshape(*lead, page // 32, 2, 4, 4, D)  # tile, half, group, token, column
    n = x.dim()
    return x.permute(*range(n - 4), n - 3, n - 1, n - 4, n - 2).reshape(*lead, page * D)


def _pool(gen, c, n_pages, spread):
    """Pages of random rows (stale ones too: a pool is used over and over), packed; (elements, scales)."""
    data, scale = [], []
    for kind in range(2):
        elem = torch.uint8 if c["c8"] else TYPES[c["x"]]
        d = torch.empty((n_pages, c["Hkv"], c["page"] * c["D"]), dtype=elem, device=DEV)
        s = torch.empty((n_pages, c["Hkv"], c["page"]), device=DEV) if c["c8"] else None
        gain = 0.4 + 1.2 * torch.rand((c["Hkv"], 1, c["D"]), generator=gen, device=DEV)
        mean = 0.5 * torch.randn((c["Hkv"], 1, c["D"]), generator=gen, device=DEV)
        step = max(1, 50_000_000 // (c["Hkv"] * c["page"] * c["D"]))
        for p in range(0, n_pages, step):
            n = min(step, n_pages - p)
            r = torch.randn((n, c["Hkv"], c["page"], c["D"]), generator=gen, device=DEV) * gain * spread[kind] + mean
            if c["c8"]:
                s[p : p + n] = (r.abs().amax(dim=3) / E4M3_MAX).clamp_min(SCALE_MIN)
                r = (r / s[p : p + n, :, :, None]).to(FP8).view(torch.uint8)
            d[p : p + n] = (_pack_v(r) if kind else _pack_k(r, d.element_size())).to(elem)
        data.append(d.view(FP8) if c["c8"] else d)
        scale.append(s)
    return data, scale


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    c, s = case, {"case": dict(case)}
    lens, news, page = _lens(c), _news(c), c["page"]
    need = [-(-n // page) for n in lens]
    n_pages, width = sum(need) + 2, max(need)
    ids = torch.randperm(n_pages, generator=gen, device=DEV).int()
    table = torch.zeros((c["B"], width), dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at : at + n]
        at += n
    offsets = [0]
    for n in news:
        offsets.append(offsets[-1] + n)
    s["host"] = {"lens": lens, "offsets": offsets}  # the program's own scheduling
    s["table"] = table
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    one = all(n == 1 for n in news) and c["op"] != "prefill"
    s["offsets"] = None if one else torch.tensor(offsets, dtype=torch.int32, device=DEV)
    (s["k"], s["v"]), (s["k_scale"], s["v_scale"]) = _pool(gen, c, n_pages, (1.0, 1.0))
    T, D, x = offsets[-1], c["D"], TYPES[c["x"]]
    if c["op"] != "append":
        # scores with a standard deviation of about 2.5: a few tokens have most of the weight
        s["q"] = (2.5 * torch.randn((T, c["Hq"] * D), generator=gen, device=DEV)).to(x)
        return s
    # one projection gives a token's queries, keys and values in one row
    s["qkv"] = (1.5 * torch.randn((T, (c["Hq"] + 2 * c["Hkv"]) * D), generator=gen, device=DEV)).to(x)
    if c["rot"]:
        pos = torch.arange(max(lens), device=DEV, dtype=torch.float64)
        f = THETA ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])
        a = pos[:, None] * f
        s["rope"] = torch.cat([a.cos(), a.sin()], dim=1).float()  # [positions][cosines, sines]
    return s


def _parts(s, c):
    q, k = c["Hq"] * c["D"], c["Hkv"] * c["D"]
    return s["qkv"][:, :q], s["qkv"][:, q : q + k], s["qkv"][:, q + k :]


# ---------------------------------------------------------------- plain forms

def _rows_k(d, c):
    """Rows [..., page, D] of packed K."""
    n = 16 // d.element_size()
    return d.view(*d.shape[:-1], c["page"] // 16, c["D"] // n, 16, n).transpose(-3, -2).reshape(
        *d.shape[:-1], c["page"], c["D"])


def _rows_v(d, c):
    v = d.view(*d.shape[:-1], c["page"] // 32, 4, c["D"], 2, 4)
    n = v.dim()
    return v.permute(*range(n - 4), n - 2, n - 4, n - 1, n - 3).reshape(*d.shape[:-1], c["page"], c["D"])


def _values(d, scale, c, rows):
    """fp32 rows of pages; d: [..., page * D]."""
    if scale is None:
        return rows(d, c).float()
    return rows(d.view(torch.uint8), c).view(FP8).float() * scale[..., None]


def _gathered(s, c, pages):
    """K and V [..., Hkv, tokens, D] in fp32 of lists of pages [..., n]."""
    out = []
    for name, rows in (("k", _rows_k), ("v", _rows_v)):
        d, sc = s[name], s[name + "_scale"]
        d = d.view(torch.uint8)[pages.long()].view(FP8) if c["c8"] else d[pages.long()]
        r = _values(d, None if sc is None else sc[pages.long()], c, rows)
        r = r.transpose(-4, -3)
        out.append(r.reshape(*r.shape[:-3], r.shape[-3] * r.shape[-2], r.shape[-1]))
    return out


def _visible(pos, j, c):
    m = j <= pos
    return m & ((pos - j < c["window"]) | (j < c["sinks"])) if c["window"] else m


def _attend(q, k, v, seen, scale):
    """q [..., R, D], k, v [..., N, D], seen [..., R, N]: softmax(scale q k) v, zeros where nothing is seen."""
    z = (q @ k.transpose(-1, -2)).mul_(scale).masked_fill_(~seen, -math.inf)
    m = z.amax(dim=-1, keepdim=True)
    p = z.sub_(torch.where(torch.isinf(m), torch.zeros_like(m), m)).exp_()
    return p @ v / p.sum(dim=-1, keepdim=True).clamp_min(1e-38)


def _out(o, c):
    """[T, Hq * D] fp32 -> the output's type; 8 bits as the values they stand for."""
    x = TYPES[c["x"]]
    if not c.get("out8"):
        return o.to(x)
    g = o.view(o.shape[0], -1, 128)
    sc = (g.abs().amax(dim=2, keepdim=True) / E4M3_MAX).clamp_min(SCALE_MIN)
    return ((g / sc).to(FP8).float() * sc).view(o.shape).to(x)


def _plain_decode(s, c):
    lens, D, Hkv = s["host"]["lens"], c["D"], c["Hkv"]
    G = c["Hq"] // Hkv
    o = torch.empty((c["B"], c["Hq"] * D), device=DEV)
    b = 0
    while b < c["B"]:  # as many sequences at once as their padded caches take 4 GB
        e, top = b + 1, lens[b]
        while e < c["B"] and (e + 1 - b) * max(top, lens[e]) * Hkv * D * 8 < 1 << 32:
            top = max(top, lens[e])
            e += 1
        k, v = _gathered(s, c, s["table"][b:e, : -(-top // c["page"])])
        q = s["q"][b:e].float().view(e - b, Hkv, G, D)
        j = torch.arange(k.shape[-2], device=DEV)
        seen = _visible((s["lens"][b:e] - 1)[:, None, None, None], j, c)
        o[b:e] = _attend(q, k, v, seen, D ** -0.5).reshape(e - b, -1)
        b = e
    return _out(o, c)


def _plain_prefill(s, c):
    lens, at, D, Hkv = s["host"]["lens"], s["host"]["offsets"], c["D"], c["Hkv"]
    G = c["Hq"] // Hkv
    o = torch.empty((at[-1], c["Hq"] * D), device=DEV)
    for b in range(c["B"]):
        n, new = lens[b], at[b + 1] - at[b]
        k, v = _gathered(s, c, s["table"][b, : -(-n // c["page"])])
        rows = max(1, (1 << 29) // (c["Hq"] * n))  # 2 GB of scores at once
        for r in range(0, new, rows):
            e = min(new, r + rows)
            end = n - new + e  # keys behind the last query of the part are left out
            q = s["q"][at[b] + r : at[b] + e].float().view(e - r, Hkv, G, D).permute(1, 2, 0, 3)
            pos = torch.arange(n - new + r, end, device=DEV)[:, None]
            seen = _visible(pos, torch.arange(end, device=DEV), c)
            part = _attend(q.reshape(Hkv, G * (e - r), D), k[:, :end], v[:, :end], seen.repeat(G, 1), D ** -0.5)
            o[at[b] + r : at[b] + e] = part.view(Hkv, G, e - r, D).permute(2, 0, 1, 3).reshape(e - r, -1)
    return _out(o, c)


def _rotate(x, cos, sin, c):
    """x [T, heads, D] in 64 bits: a value next to a border of its type must fall on the same side."""
    h = c["rot"] // 2
    if not h:
        return x
    r, rest = x[..., : 2 * h], x[..., 2 * h :]
    a, b = (r[..., 0::2], r[..., 1::2]) if c["inter"] else (r[..., :h], r[..., h:])
    u, w = a * cos - b * sin, a * sin + b * cos
    r = torch.stack([u, w], dim=-1).flatten(-2) if c["inter"] else torch.cat([u, w], dim=-1)
    return torch.cat([r, rest], dim=-1)


def _tokens(s):
    """Sequence and position of each row, from the batch's offsets and lengths."""
    lens = s["lens"].long()
    if s["offsets"] is None:
        seq = torch.arange(lens.shape[0], device=DEV)
        return seq, lens - 1
    off = s["offsets"].long()
    t = torch.arange(s["host"]["offsets"][-1], device=DEV)
    seq = (t[:, None] >= off[None, 1:]).sum(dim=1)
    return seq, lens[seq] - off[seq + 1] + t


def _round8(v):
    """v (64 bits) rounded once to e4m3's values: through fp32 a quotient next to a border would fall on the border."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return ((v / step).round() * step).float()


def _plain_append(s, c):
    T, D, Hkv, page = s["qkv"].shape[0], c["D"], c["Hkv"], c["page"]
    q, k, v = (p.double().view(T, -1, D) for p in _parts(s, c))
    seq, pos = _tokens(s)
    if c["rot"]:
        cos, sin = s["rope"][pos].double()[:, None, :].chunk(2, dim=-1)
        q, k = _rotate(q, cos, sin, c), _rotate(k, cos, sin, c)
    pages, t = s["table"][seq, pos // page].long(), pos % page
    out = {"q": q.to(TYPES[c["x"]]).view(T, -1)}
    for name, rows in (("k", k), ("v", v)):
        pool, sc = s[name], s[name + "_scale"]
        if c["c8"]:
            scale = (rows.abs().amax(dim=2) / E4M3_MAX).float().clamp_min(SCALE_MIN)
            rows = _round8(rows / scale[:, :, None].double()).to(FP8).view(torch.uint8)
            sc[pages, :, t] = scale
            pool = pool.view(torch.uint8)
        rows = rows.to(pool.dtype)
        n = 16 // pool.element_size()
        if name == "k":
            view = pool.view(-1, Hkv, page // 16, D // n, 16, n)
            view[pages, :, t // 16, :, t % 16] = rows.view(T, Hkv, D // n, n)
        else:
            view = pool.view(-1, Hkv, page // 32, 4, D, 8)
            view[pages, :, t // 32, t % 16 // 4, :, t % 32 // 16 * 4 + t % 4] = rows
        out[name] = _whole(s, c, name)
    return out


def _whole(s, c, name):
    """The updated pool, in its own order: 8 bits as the values they stand for."""
    d, sc = s[name], s[name + "_scale"]
    if sc is None:
        return d
    D, page = c["D"], c["page"]
    if name == "k":
        f = sc.view(*sc.shape[:2], page // 16, 1, 16, 1)
        return (d.float().view(*d.shape[:2], page // 16, D // 16, 16, 16) * f).view(d.shape)
    f = sc.view(*sc.shape[:2], page // 32, 2, 4, 4).transpose(3, 4).reshape(*sc.shape[:2], page // 32, 4, 1, 8)
    return (d.float().view(*d.shape[:2], page // 32, 4, D, 8) * f).view(d.shape)


# ---------------------------------------------------------------- one pass

_ctx = None


def _library():
    global _ctx
    import any_precision_weight_amd as apw
    if _ctx is None:
        _ctx = apw.Context(torch.cuda.current_device())
    return apw, _ctx


def _own(s, c):
    apw, ctx = _library()
    T, D, x = s["host"]["offsets"][-1], c["D"], TYPES[c["x"]]
    if "buf" not in s:  # a program's own plan and buffers, kept from step to step
        cache = apw.KvCache(s["k"], s["v"], c["page"], c["Hkv"], D, s["k_scale"], s["v_scale"])
        batch = apw.KvBatch(s["table"], s["lens"], T, s["offsets"], max_len=max(s["host"]["lens"]))
        out = torch.empty((T, c["Hq"] * D), dtype=x, device=DEV)
        o8 = osc = ws = None
        if c["op"] != "append":
            ws = torch.empty(apw.attn_workspace(ctx, cache, batch, c["Hq"]), dtype=torch.uint8, device=DEV)
        if c.get("out8"):
            o8 = torch.empty((T, c["Hq"] * D), dtype=FP8, device=DEV)
            osc = torch.empty((T, c["Hq"] * D // 128), device=DEV)
        s["buf"] = cache, batch, ws, out, o8, osc
    cache, batch, ws, out, o8, osc = s["buf"]
    if c["op"] == "append":
        q, k, v = _parts(s, c)
        apw.kv_append(ctx, cache, batch, q, k, v, c["Hq"], s.get("rope"), c["rot"], c["inter"], out)
        return {"q": out, "k": _whole(s, c, "k"), "v": _whole(s, c, "v")}
    call = apw.attn_decode if c["op"] == "decode" else apw.attn_prefill
    if o8 is None:
        call(ctx, cache, batch, s["q"], c["Hq"], D ** -0.5, c["window"], c["sinks"], ws, out)
        return out
    call(ctx, cache, batch, s["q"], c["Hq"], D ** -0.5, c["window"], c["sinks"], ws, None, o8, osc)
    return (o8.float().view(T, -1, 128) * osc[:, :, None]).view(T, -1).to(x)


def run(state):
    c = state["case"]
    if own:
        return _own(state, c)
    if c["op"] == "append":
        return _plain_append(state, c)
    return _plain_decode(state, c) if c["op"] == "decode" else _plain_prefill(state, c)


# ---------------------------------------------------------------- work

def _seen(p, c):
    """Keys that a query at position p sees."""
    if not c["window"]:
        return p + 1
    first = max(0, p + 1 - c["window"])
    return p + 1 - first + min(c["sinks"], first)


def work(case):
    c = case
    lens, news, D = _lens(c), _news(c), c["D"]
    T, e = sum(news), 1 if c["c8"] else 2
    row = 2 * c["Hkv"] * (D * e + (4 if c["c8"] else 0))  # a token's K and V in the cache
    meta = 4 * sum(-(-n // c["page"]) for n in lens) + 8 * c["B"]
    if c["op"] == "append":
        b = T * (2 * D * (2 * c["Hq"] + 2 * c["Hkv"]) + row) + 4 * T * c["rot"] + meta
        return {"bytes": b, "flops": 3 * T * c["rot"] * (c["Hq"] + c["Hkv"])}
    pairs = tokens = 0
    for n, new in zip(lens, news):
        if not c["window"]:
            pairs += sum(range(n - new + 1, n + 1))
            tokens += n
        else:
            pairs += sum(_seen(p, c) for p in range(n - new, n))
            first = max(0, n - new + 1 - c["window"])
            tokens += n - first + min(c["sinks"], first)
    out = T * c["Hq"] * (D + D // 32) if c.get("out8") else 2 * T * c["Hq"] * D
    return {"bytes": tokens * row + 2 * T * c["Hq"] * D + out + meta, "flops": 4 * pairs * c["Hq"] * D}


# ---------------------------------------------------------------- 64 bits

def _e4m3(v):
    """The nearest e4m3 value of each v, found among all of them; between two the one with an even code."""
    code = torch.arange(127, device=DEV, dtype=torch.float64)
    e, f = torch.floor(code / 8), code % 8
    values = torch.where(e == 0, f * 2.0 ** -9, (8 + f) * torch.exp2(e - 10))
    middles = (values[1:] + values[:-1]) / 2
    a = v.abs()
    i = torch.searchsorted(middles, a.contiguous())
    tie = (i < 126) & (middles[i.clamp_max(125)] == a)
    return values[i + (tie & (i % 2 == 1))] * torch.sign(v)


def _place(c, name, size):
    """[page, D] place of each token's columns in a page's elements."""
    t = torch.arange(c["page"], device=DEV)[:, None]
    d = torch.arange(c["D"], device=DEV)[None, :]
    if name == "k":
        n = 16 // size
        return ((t // 16 * (c["D"] // n) + d // n) * 16 + t % 16) * n + d % n
    return ((t // 32 * 4 + t % 16 // 4) * c["D"] + d) * 8 + t % 32 // 16 * 4 + t % 4


def _exact_rows(s, c, name, pages, head, n):
    """Rows [n, D] of one head of one sequence."""
    d, sc = s[name], s[name + "_scale"]
    if c["c8"]:
        d = d.view(torch.uint8)
    d = d[pages, head][:, _place(c, name, d.element_size())]
    if not c["c8"]:
        return d.reshape(-1, c["D"])[:n].double()
    return d.view(FP8).double().view(-1, c["D"])[:n] * sc[pages, head].double().reshape(-1, 1)[:n]


def _exact_attention(s, c):
    lens, at, D = s["host"]["lens"], s["host"]["offsets"], c["D"]
    G = c["Hq"] // c["Hkv"]
    o = torch.zeros((at[-1], c["Hq"], D), dtype=torch.float64, device=DEV)
    for b in range(c["B"]):
        n, new = lens[b], at[b + 1] - at[b]
        pages = s["table"][b, : -(-n // c["page"])].long()
        p = torch.arange(n - new, n, device=DEV).view(-1, 1, 1)
        j = torch.arange(n, device=DEV).view(1, 1, -1)
        for h in range(c["Hkv"]):
            k, v = (_exact_rows(s, c, name, pages, h, n) for name in ("k", "v"))
            rows = max(1, 200_000_000 // (G * n))
            for r in range(0, new, rows):
                e = min(new, r + rows)
                q = s["q"][at[b] + r : at[b] + e].double().view(-1, c["Hq"], D)[:, h * G : (h + 1) * G]
                z = (q.reshape(-1, D) @ k.T).view(e - r, G, n) / math.sqrt(D)
                gone = j > p[r:e]
                if c["window"]:
                    gone = gone | ((j <= p[r:e] - c["window"]) & (j >= c["sinks"]))
                z = torch.softmax(z.masked_fill(gone, -math.inf), dim=2)
                o[at[b] + r : at[b] + e, h * G : (h + 1) * G] = (z.view(-1, n) @ v).view(e - r, G, D)
    o = o.view(at[-1], -1)
    if not c.get("out8"):
        return o
    for c0 in range(0, o.shape[1], 128):
        part = o[:, c0 : c0 + 128]
        sc = torch.clamp(part.abs().max(dim=1, keepdim=True).values / E4M3_MAX, min=SCALE_MIN).float().double()
        o[:, c0 : c0 + 128] = _e4m3(part / sc) * sc
    return o


def _exact_append(s, c):
    D, Hkv, Hq, page = c["D"], c["Hkv"], c["Hq"], c["page"]
    x = s["qkv"].double().view(-1, Hq + 2 * Hkv, D).clone()
    seq, pos = [], []
    for b, (n, at) in enumerate(zip(s["host"]["lens"], s["host"]["offsets"])):
        new = s["host"]["offsets"][b + 1] - at
        seq += [b] * new
        pos += range(n - new, n)
    seq, pos = torch.tensor(seq, device=DEV), torch.tensor(pos, device=DEV)
    h = c["rot"] // 2
    for i in range(h):
        a, b = (2 * i, 2 * i + 1) if c["inter"] else (i, i + h)
        co, si = s["rope"][pos, i].double()[:, None], s["rope"][pos, h + i].double()[:, None]
        u, w = x[:, : Hq + Hkv, a].clone(), x[:, : Hq + Hkv, b].clone()
        x[:, : Hq + Hkv, a] = u * co - w * si
        x[:, : Hq + Hkv, b] = w * co + u * si
    out = {"q": x[:, :Hq].reshape(-1, Hq * D)}
    pages, t = s["table"][seq, pos // page].long(), pos % page
    for name, rows in (("k", x[:, Hq : Hq + Hkv]), ("v", x[:, Hq + Hkv :])):
        pool, sc = s[name], s[name + "_scale"]
        place = _place(c, name, pool.element_size())
        full = pool.double()
        if c["c8"]:
            full[:, :, place.view(-1)] *= sc.double().repeat_interleave(D, dim=2)
            f = torch.clamp(rows.abs().max(dim=2, keepdim=True).values / E4M3_MAX, min=SCALE_MIN).float().double()
            rows = _e4m3(rows / f) * f
        for g in range(Hkv):
            full[pages[:, None], g, place[t]] = rows[:, g]
        out[name] = full
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s, case) if case["op"] == "append" else _exact_attention(s, case)
