"""The 8-bit path of the MoE layer, operator by operator: cases, inputs, plain forms.

Four operators of the library:

  norm       root-mean-square norm of x + residual, written in x's type and / or as e4m3 with scales
  gemm       the experts' product (or, with one expert, a dense one) in e4m3 with fp32 scales:
             one for each row and 128 columns of the input, one for each 128 x 128 block of the weight
  gemm_act   the gate_up product with SiLU(gate) * up, written as e4m3 with scales
  layer      routing, gate_up, down and the weighted sum over a token's experts

A row in 8 bits: for each group of 128 columns (the last may be shorter) the scale s is the largest magnitude
over 448, at least 2^-126, and the values are e4m3(v / s).

``own`` chooses what ``run`` measures: the plain forms below, or the library's calls.
"""
import math

import torch

own = False

DEV = "cuda"
BLK = 128
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126
FP8 = torch.float8_e4m3fn
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token's hidden row between two layers of a decode step: residual in, residual and row out
        dict(name="norm_decode_t1", op="norm", T=1, H=4096, x="f16", res="f16", y=True, q=True),
        # a decode batch with ragged rows (704 = 5.5 groups), 8-bit output only, no residual
        dict(name="norm_q_t333_h704", op="norm", T=333, H=704, x="bf16", res="none", y=False, q=True),
        # a prefill chunk with an fp32 residual stream
        dict(name="norm_prefill_t8192", op="norm", T=8192, H=6144, x="bf16", res="f32", y=True, q=False),
        # dense projection of a decode batch (E = 1)
        dict(name="gemm_dense_decode_t8", op="gemm", T=8, topk=1, E=1, N=6144, K=4096, gather=True, out="bf16", zipf=0.0),
        # dense projection of a prefill chunk
        dict(name="gemm_dense_prefill_t4096", op="gemm", T=4096, topk=1, E=1, N=6144, K=4096, gather=True, out="f16",
             zipf=0.0),
        # down product of many small experts, a few rows each
        dict(name="gemm_experts_decode_t64", op="gemm", T=64, topk=4, E=60, N=2048, K=1408, gather=False, out="f32",
             zipf=0.0),
        # down product of eight large experts, unevenly loaded
        dict(name="gemm_experts_prefill_t2048", op="gemm", T=2048, topk=2, E=8, N=4096, K=14336, gather=False,
             out="f32", zipf=0.8),
        # gate_up of a decode batch: every expert's weights are read for a few rows
        dict(name="act_decode_t16", op="gemm_act", T=16, topk=2, E=8, F=14336, K=4096, zipf=0.0),
        # gate_up of a prompt over many small experts
        dict(name="act_prefill_t2048", op="gemm_act", T=2048, topk=4, E=60, F=1408, K=2048, zipf=0.0),
        # one token through a layer of many small experts: latency
        dict(name="layer_t1_small", op="layer", T=1, topk=4, shared=4, E=60, H=2048, F=1408, renorm=False, zipf=0.0),
        # a few tokens (speculative or small-batch decode) through a layer of large experts
        dict(name="layer_t4_large", op="layer", T=4, topk=2, shared=0, E=8, H=4096, F=14336, renorm=True, zipf=0.0),
        # a prompt through the same layer, unevenly routed: the largest
        dict(name="layer_prefill_t4096", op="layer", T=4096, topk=2, shared=0, E=8, H=4096, F=14336, renorm=True,
             zipf=0.8),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "gemm", "gemm", "gemm_act", "layer", "layer"])
    if op == "norm":
        H = 8 * _log_int(rng, 4, 1500)
        T = _log_int(rng, 1, max(1, 48_000_000 // H))
        q = rng.random() < 0.6
        return dict(op=op, T=T, H=H, x=rng.choice(["f16", "bf16", "f32"]), res=rng.choice(["none", "f16", "bf16", "f32"]),
                    y=(not q) or rng.random() < 0.5, q=q)
    if op == "gemm":
        E = rng.choice([1, 1, 1, rng.randint(2, 16), rng.randint(17, 128)])
        K = 16 * _log_int(rng, 4, 900)
        N = _log_int(rng, 33, max(34, min(28672, 900_000_000 // (E * K))))
        topk = rng.randint(1, min(E, 8))
        T = _log_int(rng, 1, max(1, min(8192, int(5e11 / (N * K * topk)))))
        return dict(op=op, T=T, topk=topk, E=E, N=N, K=K, gather=rng.random() < 0.5,
                    out=rng.choice(["f16", "bf16", "f32"]), zipf=rng.choice([0.0, 0.0, 0.8, 1.2]))
    E = rng.choice([rng.randint(1, 8), rng.randint(9, 32), rng.randint(33, 128)])
    H = 16 * _log_int(rng, 8, 400)
    F = 16 * _log_int(rng, 4, max(5, min(1024, 28_000_000 // (E * H))))
    topk = rng.randint(1, min(E, 8))
    zipf = rng.choice([0.0, 0.0, 0.8, 1.2])
    if op == "gemm_act":
        T = _log_int(rng, 1, max(1, min(8192, int(2e11 / (F * H * topk)))))
        return dict(op=op, T=T, topk=topk, E=E, F=F, K=H, zipf=zipf)
    shared = rng.choice([0, 0, rng.randint(1, 4)])
    # half of them a few tokens
    T = _log_int(rng, 1, rng.choice([16, max(1, min(8192, int(1.5e11 / (F * H * (topk + shared)))))]))
    return dict(op=op, T=T, topk=topk, shared=shared, E=E, H=H, F=F, renorm=rng.random() < 0.5, zipf=zipf)


# ---------------------------------------------------------------- inputs

def _weights(gen, experts, halves, rows, K):
    """e4m3 weights [experts][halves * rows][K] of N(0, 0.02^2) values, and the scales of their 128 x 128 blocks
    (each half blocked by itself)."""
    nb, kb = -(-rows // BLK), -(-K // BLK)
    w8 = torch.empty((experts, halves, rows, K), dtype=FP8, device=DEV)
    sc = torch.empty((experts, halves, nb, kb), dtype=torch.float32, device=DEV)
    for e in range(experts):
        for h in range(halves):
            w = torch.zeros((nb * BLK, kb * BLK), device=DEV)
            w[:rows, :K] = torch.randn((rows, K), generator=gen, device=DEV) * 0.02
            b = w.view(nb, BLK, kb, BLK)
            s = (b.abs().amax(dim=(1, 3)) / E4M3_MAX).clamp_min(SCALE_MIN)
            w8[e, h] = (b / s[:, None, :, None]).reshape(nb * BLK, kb * BLK)[:rows, :K].to(FP8)
            sc[e, h] = s
    return w8.view(experts, halves * rows, K), sc


def _activations(gen, rows, C):
    """Rows of a hidden state: a few channels are much larger than the others."""
    x = torch.randn((rows, C), generator=gen, device=DEV)
    x *= 0.5 + torch.rand((C,), generator=gen, device=DEV)
    x[:, torch.randperm(C, generator=gen, device=DEV)[: max(1, C // 200)]] *= 12.0
    return x


def _rows8(x):
    R, C = x.shape
    g = -(-C // BLK)
    p = torch.zeros((R, g * BLK), device=DEV)
    p[:, :C] = x
    p = p.view(R, g, BLK)
    s = (p.abs().amax(dim=2) / E4M3_MAX).clamp_min(SCALE_MIN)
    return (p / s[:, :, None]).view(R, g * BLK)[:, :C].contiguous().to(FP8), s


def _bias(gen, E, zipf):
    if not zipf:
        return None
    p = torch.arange(1, E + 1, device=DEV, dtype=torch.float64) ** -zipf
    return torch.log(p / p.sum())[torch.randperm(E, generator=gen, device=DEV)].float()


def _assign(gen, T, topk, E, zipf):
    """What the router leaves: each token's distinct experts, and the assignments grouped by expert."""
    z = torch.randn((T, E), generator=gen, device=DEV)
    b = _bias(gen, E, zipf)
    ids = (z if b is None else z + b).argsort(dim=1, descending=True)[:, :topk].reshape(-1)
    perm = ids.argsort(stable=True).int()
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.bincount(ids, minlength=E).cumsum(0)
    return perm, offsets


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    c, s = case, {"case": dict(case)}
    if c["op"] == "norm":
        s["x"] = _activations(gen, c["T"], c["H"]).to(TYPES[c["x"]])
        s["gamma"] = (1.0 + 0.2 * torch.randn((c["H"],), generator=gen, device=DEV)).to(TYPES[c["x"]])
        if c["res"] != "none":
            s["residual"] = (4.0 * _activations(gen, c["T"], c["H"])).to(TYPES[c["res"]])
        return s
    if c["op"] in ("gemm", "gemm_act"):
        act = c["op"] == "gemm_act"
        s["perm"], s["offsets"] = _assign(gen, c["T"], c["topk"], c["E"], c["zipf"])
        rows = c["T"] if act or c["gather"] else c["T"] * c["topk"]
        s["x8"], s["xs"] = _rows8(_activations(gen, rows, c["K"]))
        s["w8"], s["ws"] = _weights(gen, c["E"], 2 if act else 1, c["F"] if act else c["N"], c["K"])
        return s
    E = c["E"] + c["shared"]
    x = _activations(gen, c["T"], c["H"])
    s["x"] = x.half()
    s["x8"], s["xs"] = _rows8(s["x"].float())
    s["router"] = (torch.randn((c["E"], c["H"]), generator=gen, device=DEV) * 0.02).half()
    s["bias"] = _bias(gen, c["E"], c["zipf"])
    s["gate_up"], s["gate_up_s"] = _weights(gen, E, 2, c["F"], c["H"])
    s["down"], s["down_s"] = _weights(gen, E, 1, c["H"], c["F"])
    return s


# ---------------------------------------------------------------- plain forms

def _values(q, s):
    """The values that e4m3 rows with a scale for each 128 columns stand for."""
    return q.float() * s.repeat_interleave(BLK, dim=1)[:, : q.shape[1]]


def _weight_values(w8, s):
    """[N][K] values of one expert's matrix; s [halves][row blocks][column blocks]."""
    N, K = w8.shape
    rows = N // s.shape[0]
    f = s.repeat_interleave(BLK, dim=1)[:, :rows].reshape(N, s.shape[2])
    return w8.float() * f.repeat_interleave(BLK, dim=1)[:, :K]


def _to_8bit(v):
    R, C = v.shape
    g = -(-C // BLK)
    p = torch.nn.functional.pad(v, (0, g * BLK - C)).view(R, g, BLK)
    s = (p.abs().amax(dim=2) / E4M3_MAX).float().clamp_min(SCALE_MIN)
    return (p / s[:, :, None]).view(R, g * BLK)[:, :C].float().to(FP8), s


def _plain_norm(s, c):
    x = s["x"].float()
    out = {}
    if c["res"] != "none":
        out["residual"] = (x + s["residual"].float()).to(TYPES[c["res"]])
        x = out["residual"].float()
    # in 64 bits: a value next to a border of e4m3 must fall on the same side
    h = x.double()
    y = h * torch.rsqrt(h.square().mean(dim=1, keepdim=True) + 1e-5) * s["gamma"].double()
    if c["y"]:
        out["y"] = y.to(s["x"].dtype)
    if c["q"]:
        q, sc = _to_8bit(y)
        out["q"], out["scale"] = _values(q, sc).to(s["x"].dtype), sc
    return out


def _plain_product(xv, w8, ws, offsets, rows_of):
    """[rows][N] of every expert's product, 32-bit sums; rows_of: the input row of each output row."""
    out = torch.zeros((rows_of.shape[0], w8.shape[1]), device=DEV)
    at = offsets.tolist()
    for e in range(w8.shape[0]):  # the experts' row counts are the router's
        if at[e + 1] > at[e]:
            out[at[e] : at[e + 1]] = xv[rows_of[at[e] : at[e + 1]]] @ _weight_values(w8[e], ws[e]).T
    return out


def _rows_of(perm, topk, gather):
    return (perm // topk if gather else torch.arange(perm.shape[0], device=DEV)).long()


def _plain_act(h, F):
    g, u = h[:, :F], h[:, F:]
    return _to_8bit(g / (1.0 + torch.exp(-g)) * u)


def _plain_layer(s, c):
    T, E, kt = c["T"], c["E"], c["topk"] + c["shared"]
    z = s["x"].double() @ s["router"].double().T
    if s["bias"] is not None:
        z = z + s["bias"].double()
    z, ids = torch.sort(z, dim=1, descending=True, stable=True)
    e = torch.exp(z - z[:, :1])
    w = e[:, : c["topk"]] / (e[:, : c["topk"]] if c["renorm"] else e).sum(dim=1, keepdim=True)
    ids = torch.cat([ids[:, : c["topk"]], torch.arange(E, E + c["shared"], device=DEV).expand(T, -1)], dim=1)
    w = torch.cat([w.float(), torch.ones((T, c["shared"]), device=DEV)], dim=1)
    perm = ids.reshape(-1).argsort(stable=True)
    offsets = torch.zeros(E + c["shared"] + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = torch.bincount(ids.reshape(-1), minlength=E + c["shared"]).cumsum(0)
    h = _plain_product(_values(s["x8"], s["xs"]), s["gate_up"], s["gate_up_s"], offsets, _rows_of(perm, kt, True))
    a = _values(*_plain_act(h, c["F"]))
    y = _plain_product(a, s["down"], s["down_s"], offsets, _rows_of(perm, kt, False))
    back = torch.empty_like(y)
    back[perm] = y
    return (back.view(T, kt, -1) * w[:, :, None]).sum(dim=1).half()


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
    if c["op"] == "norm":
        res = s.get("residual")
        if "buf" not in s:  # a program's own buffers, kept from step to step
            T, H, x = c["T"], c["H"], s["x"]
            s["buf"] = (None if res is None else torch.empty_like(res), torch.empty_like(x) if c["y"] else None,
                        torch.empty((T, H), dtype=FP8, device=DEV) if c["q"] else None,
                        torch.empty((T, -(-H // BLK)), device=DEV) if c["q"] else None)
        h, y, q, sc = s["buf"]
        out = {} if h is None else {"residual": h}
        apw.norm(ctx, s["x"], res, h, s["gamma"], 1e-5, c["T"], c["H"], y, q, sc)
        if c["y"]:
            out["y"] = y
        if c["q"]:
            out["q"], out["scale"] = _values(q, sc).to(s["x"].dtype), sc
        return out
    if c["op"] == "gemm":
        if "buf" not in s:
            s["buf"] = torch.empty((c["T"] * c["topk"], c["N"]), dtype=TYPES[c["out"]], device=DEV)
        apw.gemm_fp8(ctx, s["x8"], s["xs"], s["w8"], s["ws"], c["E"], c["N"], c["K"], c["gather"], s["perm"],
                     s["offsets"], c["T"], c["topk"], s["buf"])
        return s["buf"]
    if c["op"] == "gemm_act":
        R = c["T"] * c["topk"]
        if "buf" not in s:
            s["buf"] = (torch.empty((R, c["F"]), dtype=FP8, device=DEV),
                        torch.empty((R, -(-c["F"] // BLK)), device=DEV))
        a8, sc = s["buf"]
        apw.gemm_act_fp8(ctx, s["x8"], s["xs"], s["w8"], s["ws"], c["E"], c["F"], c["K"], True, s["perm"],
                         s["offsets"], c["T"], c["topk"], a8, sc)
        return {"a": _values(a8, sc).half(), "scale": sc}
    if "buf" not in s:
        ex = apw.Fp8Experts(s["gate_up"], s["gate_up_s"], s["down"], s["down_s"])
        n = apw.moe_workspace_fp8(ctx, ex, c["T"], c["topk"], n_shared=c["shared"])
        s["buf"] = ex, torch.empty(n, dtype=torch.uint8, device=DEV), torch.empty_like(s["x"])
    ex, ws, out = s["buf"]
    apw.moe_forward_fp8(ctx, ex, s["x"], s["x8"], s["xs"], s["router"], s["bias"], c["T"], c["topk"], c["renorm"], ws,
                        out, n_shared=c["shared"])
    return out


def run(state):
    c = state["case"]
    if own:
        return _own(state, c)
    if c["op"] == "norm":
        return _plain_norm(state, c)
    if c["op"] == "gemm":
        y = _plain_product(_values(state["x8"], state["xs"]), state["w8"], state["ws"], state["offsets"],
                           _rows_of(state["perm"], c["topk"], c["gather"]))
        return y.to(TYPES[c["out"]])
    if c["op"] == "gemm_act":
        h = _plain_product(_values(state["x8"], state["xs"]), state["w8"], state["ws"], state["offsets"],
                           _rows_of(state["perm"], c["topk"], True))
        q, sc = _plain_act(h, c["F"])
        return {"a": _values(q, sc).half(), "scale": sc}
    return _plain_layer(state, c)


# ---------------------------------------------------------------- work

def _active(tokens, topk, E):
    """Experts that a batch reaches when the choices are even (the expected number, rounded up)."""
    return min(E, math.ceil(E * (1.0 - (1.0 - topk / E) ** tokens)))


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["T"] * c["H"]
        size = {"none": 0, "f16": 2, "bf16": 2, "f32": 4}
        b = n * (size[c["x"]] * (2 if c["y"] else 1) + 2 * size[c["res"]]) + c["H"] * size[c["x"]]
        if c["q"]:
            b += n + 4 * c["T"] * -(-c["H"] // BLK)
        return {"bytes": b, "flops": 8 * n}
    if c["op"] in ("gemm", "gemm_act"):
        act = c["op"] == "gemm_act"
        N, K, R = (2 * c["F"] if act else c["N"]), c["K"], c["T"] * c["topk"]
        w = _active(c["T"], c["topk"], c["E"]) * (N * K + 4 * -(-N // BLK) * -(-K // BLK))
        rows = c["T"] if act or c["gather"] else R
        out = R * (c["F"] + 4 * -(-c["F"] // BLK)) if act else R * N * {"f16": 2, "bf16": 2, "f32": 4}[c["out"]]
        return {"bytes": w + rows * (K + 4 * -(-K // BLK)) + out, "flops": 2 * R * N * K}
    H, F, T = c["H"], c["F"], c["T"]
    R = T * (c["topk"] + c["shared"])
    w = (_active(T, c["topk"], c["E"]) + c["shared"]) * 3 * (H * F + 4 * -(-H // BLK) * -(-F // BLK))
    return {"bytes": w + 2 * c["E"] * H + T * (5 * H + 4 * -(-H // BLK)), "flops": 6 * R * H * F + 2 * T * c["E"] * H}


# ---------------------------------------------------------------- 64 bits

def _e4m3(v):
    """v rounded to the nearest e4m3 value, ties to even: 3 fraction bits, exponents down to -6, at most 448."""
    _, e = torch.frexp(v)  # |v| in [2^(e-1), 2^e)
    ulp = torch.exp2((e - 1).clamp_min(-6).double() - 3)
    return (torch.round(v / ulp) * ulp).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_8bit(v):
    """(values that the 8-bit row stands for, scales) of each row of v, in 64 bits."""
    vals, scales = torch.empty_like(v), []
    for c0 in range(0, v.shape[1], BLK):
        part = v[:, c0 : c0 + BLK]
        s = torch.clamp(part.abs().max(dim=1, keepdim=True).values / E4M3_MAX, min=SCALE_MIN).float().double()
        vals[:, c0 : c0 + BLK] = _e4m3(part / s) * s
        scales.append(s)
    return vals, torch.cat(scales, dim=1)


def _exact_rows(q, s):
    v = q.double()
    for b in range(s.shape[1]):
        v[:, b * BLK : (b + 1) * BLK] *= s[:, b : b + 1].double()
    return v


def _exact_matrix(w8, s):
    v = w8.double()
    halves, nb, kb = s.shape
    half = v.shape[0] // halves
    for h in range(halves):
        for i in range(nb):
            rows = slice(h * half + i * BLK, h * half + min(half, (i + 1) * BLK))
            v[rows] *= s[h, i].double().repeat_interleave(BLK)[: v.shape[1]]
    return v


def _exact_norm(s, c):
    x = s["x"].double()
    res = None
    if "residual" in s:
        t = s["residual"].dtype
        res = (s["x"].float() + s["residual"].float()).to(t)  # the sum is held in 32 bits, then in the residual's type
        x = res.double()
    ms = (x * x).sum(dim=1, keepdim=True) / c["H"]
    y = x / torch.sqrt(ms + 1e-5) * s["gamma"].double()
    out = {} if res is None else {"residual": res.double()}
    if c["y"]:
        out["y"] = y
    if c["q"]:
        out["q"], out["scale"] = _exact_8bit(y)
    return out


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "norm":
        return _exact_norm(s, c)
    if c["op"] == "layer":
        kt, E = c["topk"] + c["shared"], c["E"] + c["shared"]
        z = torch.stack([(s["x"].double() * r.double()).sum(dim=1) for r in s["router"]], dim=1)
        if s["bias"] is not None:
            z = z + s["bias"].double()
        p = torch.softmax(z, dim=1)
        order = torch.argsort(-z, dim=1, stable=True)[:, : c["topk"]]
        chosen = torch.gather(p, 1, order)
        if c["renorm"]:
            chosen = chosen / chosen.sum(dim=1, keepdim=True)
        weight = torch.zeros((c["T"], E), dtype=torch.float64, device=DEV)
        weight.scatter_(1, order, chosen)
        weight[:, c["E"] :] = 1.0
        x = _exact_rows(s["x8"], s["xs"])
        out = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device=DEV)
        mine = torch.zeros((c["T"], E), dtype=torch.bool, device=DEV).scatter_(1, order, True)
        mine[:, c["E"] :] = True
        for e in range(E):
            t = torch.nonzero(mine[:, e]).flatten()
            if t.numel():
                gu = x[t] @ _exact_matrix(s["gate_up"][e], s["gate_up_s"][e]).T
                g, u = gu[:, : c["F"]], gu[:, c["F"] :]
                a, _ = _exact_8bit(g * torch.sigmoid(g) * u)
                out[t] += weight[t, e, None] * (a @ _exact_matrix(s["down"][e], s["down_s"][e]).T)
        return out
    act = c["op"] == "gemm_act"
    x = _exact_rows(s["x8"], s["xs"])
    perm, off = s["perm"].long(), s["offsets"].tolist()
    parts = []
    for e in range(c["E"]):
        r = torch.arange(off[e], off[e + 1], device=DEV)
        src = perm[r] // c["topk"] if act or c["gather"] else r
        parts.append(x[src] @ _exact_matrix(s["w8"][e], s["ws"][e]).T)
    h = torch.cat(parts)
    if not act:
        return h
    g, u = h[:, : c["F"]], h[:, c["F"] :]
    a, sc = _exact_8bit(g * torch.sigmoid(g) * u)
    return {"a": a, "scale": sc}
