"""Plain 64-bit forms of the tree-step operators (norm + rotation + append, tree
attention, draft verification, path commit), written from their definitions.
FP8 values and codes come from the oracle."""
import numpy as np
import torch

import oracle

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
E4M3 = np.array([oracle.e4m3_value(b) for b in range(127)])


def parents_of(kind: str, n: int):
    """A chain, a wide tree, or a star; -1 for the root."""
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "star":
        return [-1] + [0] * (n - 1)
    return [-1] + [(i - 1) // 2 if i % 3 else max(0, i - 2) for i in range(1, n)]


def ancestors(parents) -> np.ndarray:
    n = len(parents)
    m = np.zeros((n, n), bool)
    for i, p in enumerate(parents):
        if p >= 0:
            m[i] = m[p]
        m[i, i] = True
    return m


def mask_words(m: np.ndarray) -> torch.Tensor:
    """bool [..., n] -> int32 words [..., ceil(n / 32)]."""
    n = m.shape[-1]
    w = np.zeros((*m.shape[:-1], (n + 31) // 32), np.uint32)
    for j in range(n):
        w[..., j // 32] |= m[..., j].astype(np.uint32) << np.uint32(j % 32)
    return torch.from_numpy(w.view(np.int32).copy())


def fp8_values(codes, scales, s) -> np.ndarray:
    """FP8 values (fp64) of NVFP4 planes [B][H][S][...] as attention reads them."""
    B, H, S, _ = codes.shape
    by = oracle.dequant_planes(codes, scales, s, np.full(B, S, np.int32))
    vals = np.concatenate([E4M3, [0.0], -E4M3, [0.0]])
    return vals[by]


def tree_attention(q, kv, vv, start, nodes, seen, scale=None):
    """One sequence: q [N][Hq][D], kv/vv [Hkv][S][D] fp64, seen bool [N][N].
    Returns (out [nodes][Hq][D], sum of p |v| / l, worst sum |q k| scale per row,
    sum of |v|)."""
    N, Hq, D = q.shape
    Hkv = kv.shape[0]
    g = Hq // Hkv
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    L = start + nodes
    out = np.zeros((nodes, Hq, D))
    mag = np.zeros_like(out)
    worst = np.zeros((nodes, Hq, 1))
    flat = np.zeros_like(out)
    for i in range(nodes):
        vis = np.ones(L, bool)
        vis[start:] = seen[i, :nodes]
        if not vis.any():
            continue
        for h in range(Hq):
            k, v = kv[h // g, :L][vis], vv[h // g, :L][vis]
            z = (k @ q[i, h]) * scale
            p = np.exp(z - z.max())
            p /= p.sum()
            out[i, h] = p @ v
            mag[i, h] = p @ np.abs(v)
            flat[i, h] = np.abs(v).sum(0)
            worst[i, h] = scale * (np.abs(k) @ np.abs(q[i, h])).max()
    return out, mag, worst, flat


def attention_tolerance(out, mag, worst, flat, tokens, bf16):
    """|error| allowed, from the roundings the kernel makes: probabilities (f16:
    2^-11; two f16 terms: 2^-21), scores (8 accumulation steps of 2^-23 of sum
    |q k|, entering numerator and denominator), the sums over tiles (8 steps of
    2^-23 a tile), exp2 and the softmax sums (2^-20), and the output (bf16: 2^-8).
    Small weights meet f16's absolute step of 2^-24: they are scaled so that the
    row's largest is 2^6 or more, so each is off by at most 2^-25 of that scale,
    2^-31 of the largest weight and hence of their sum l: 2^-31 sum |v|."""
    tiles = (tokens + 127) // 128
    rel = (2.0 ** -11 if bf16 else 2.0 ** -21) + 2 * worst * 2.0 ** -20 + tiles * 8 * 2.0 ** -23 + 2.0 ** -20
    return 2.0 ** -31 * flat + rel * mag + (2.0 ** -8 if bf16 else 2.0 ** -23) * np.abs(out) + 1e-30


def norm_rope(x, w, eps, cs, interleaved):
    """x [..., D] fp64; cs [..., R] cos and sin (R = 0: none).  Returns (y, bound
    on the fp32 result's error: 24 roundings of 2^-24 of the terms' magnitudes)."""
    D, R = x.shape[-1], cs.shape[-1]
    if eps >= 0:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        if w is not None:
            x = x * w
    y, m = x.copy(), np.abs(x)
    if R:
        i = np.arange(0, R, 2) if interleaved else np.arange(R // 2)
        j = i + 1 if interleaved else i + R // 2
        c, s = cs[..., :R // 2], cs[..., R // 2:]
        a, b = x[..., i], x[..., j]
        y[..., i], y[..., j] = a * c - b * s, b * c + a * s
        m[..., i] = np.abs(a * c) + np.abs(b * s)
        m[..., j] = np.abs(b * c) + np.abs(a * s)
    return y, 24 * 2.0 ** -24 * m


def nearest(x, grid):
    """Nearest grid value to x >= 0, ties to the even index, saturating (64 bits)."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    up, down = grid[hi] - x, x - grid[lo]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), grid[hi], grid[lo])


def check_quantized(codes, scales, y, e, s):
    """codes [..., D/2], scales [..., D/16] are what some value within e of y
    quantizes to under tensor scale s (every step is monotone in the value)."""
    D = y.shape[-1]
    blk = lambda a: a.reshape(*a.shape[:-1], D // 16, 16)
    amax, ea = np.abs(blk(y)).max(-1), blk(e).max(-1)
    sb = E4M3[scales]
    slack = 1 + 2.0 ** -22                              # the two fp32 divisions of the definition
    assert np.all(nearest(np.maximum(amax - ea, 0) / slack / (6 * s), E4M3) <= sb)
    assert np.all(sb <= nearest((amax + ea) * slack / (6 * s), E4M3))
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], D)
    val = blk(np.where(nib >= 8, -1.0, 1.0) * E2M1[nib & 7])
    den = (sb * s)[..., None]
    ok = np.broadcast_to(den > 0, val.shape)
    with np.errstate(divide="ignore", invalid="ignore"):
        lo, hi = (blk(y) - blk(e)) / den, (blk(y) + blk(e)) / den
    snap = lambda v: np.sign(v) * nearest(np.abs(v), E2M1)
    lo = snap(np.where(ok, lo - 2.0 ** -22 * np.abs(lo), 0))
    hi = snap(np.where(ok, hi + 2.0 ** -22 * np.abs(hi), 0))
    assert np.all(np.where(ok, (lo <= val) & (val <= hi), val == 0))


def verify(p, d, tokens, parents, ua, us, n):
    """One sequence, fp64: (path, next token).  p, d [N][V]; d None: point masses."""
    path, at = [0], 0
    clean = lambda r: np.where(r > 0, r, 0.0)
    w, Z = clean(p[0]), 1.0
    for c in range(1, n):
        if parents[c] != at:
            continue
        x = tokens[c]
        q = d[at] if d is not None else (np.arange(p.shape[1]) == x).astype(np.float64)
        if ua[c] * q[x] * Z < w[x]:
            path.append(c)
            at, w, Z = c, clean(p[c]), 1.0
            continue
        rest = np.maximum(w - Z * q, 0)
        if rest.sum() > 0:
            w, Z = rest, rest.sum()
    cum = np.cumsum(w)
    if not (cum[-1] > 0 and np.isfinite(cum[-1])):
        return path, -1
    return path, int(np.searchsorted(cum, us * cum[-1], side="right"))
