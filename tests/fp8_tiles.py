"""The tile product's choices in plain Python, and the cases that the tests of its kernels
run: which kernel a call takes, its tiles, and the form that each workgroup runs.  A host
test holds the cases to the forms that they are there for; a change of the kernels' rules
is made here too."""
from __future__ import annotations

XCDS, XCD_CUS, GROUP = 8, 32, 8


def cdiv(a: int, b: int) -> int:
    return -(-a // b)


def weight_tiles(N: int, act: bool) -> int:
    """N: rows of an expert's matrix; with the activation 2 F."""
    return cdiv(N // 2, 128) if act else cdiv(N, 256)


def takes_tiles(E: int, N: int, T: int, topk: int, act: bool) -> bool:
    R = T * topk
    most, served = (R if E == 1 else T), min(E, R)

    def tiles(tok):
        return ((R - served) // tok + served) * weight_tiles(N, act)
    if act:
        return most > 32 or (most > 16 and tiles(128) < 256)
    return most > 32 and tiles(32) > 64


def forms(offsets, N: int, act: bool, exact: bool):
    """[(expert, first row, rows, weight tile, parts, whole round)] of the workgroups that
    have work."""
    tok, NT = (128 if exact else 256), weight_tiles(N, act)
    units = [(e, offsets[e] + m0, min(tok, offsets[e + 1] - offsets[e] - m0))
             for e in range(len(offsets) - 1) for m0 in range(0, offsets[e + 1] - offsets[e], tok)]
    MT = len(units)
    total = MT * NT
    per = cdiv(total, XCDS)
    out = []
    for x in range(XCDS):
        first = x * per
        mine = max(0, min(per, total - first))
        rem = mine % XCD_CUS
        parts = 4 if tok >= 256 and 4 * rem <= XCD_CUS else 2 if 2 * rem <= XCD_CUS else 1
        for i in range(mine):
            whole = i < mine - rem
            k, at = divmod(first + i, GROUP * MT)
            u, j = divmod(at, min(GROUP, NT - GROUP * k))
            e, r0, m = units[u]
            n = 1 if whole else parts
            size = tok // n
            for p in range(n):
                rows = min(size, m - p * size)
                if rows > 0:
                    out.append((e, r0 + p * size, rows, k * GROUP + j, n, whole))
    return out


def width(rows: int, exact: bool) -> int:
    """Tokens of the form that a tile of so many rows takes."""
    for w in ((64, 128) if exact else (64, 128, 256)):
        if rows <= w:
            return w
    raise AssertionError(rows)


def offsets_of(loads) -> list[int]:
    o = [0]
    for m in loads:
        o.append(o[-1] + m)
    return o


# (rows of each expert, N, K): ragged N and K of several column blocks, more tiles than half
# of the CUs, so that tiles of every width are run whole; and more than all, for a whole
# round with a split rest
GEMMS = [([1100], 8720, 656), ([2100], 8720, 528), ([110, 70, 0, 128, 66], 8500, 912), ([40, 64, 3, 33, 50], 8720, 1168),
         ([300, 0, 513, 129, 5, 260], 4360, 784)]
# (rows of each expert, F, K)
ACTS = [([500], 4368, 656), ([1300], 4240, 400), ([110, 70, 0, 128, 66], 4112, 912), ([40, 64, 3, 33, 50], 3600, 528)]
