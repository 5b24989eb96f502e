"""Plain 64-bit forms of the attention layer's operators, for the GPU tests, written from the
definitions, and the bounds the results are held to (layer_common.check adds half a step of the
output type).

u = 2^-24 is the relative error of one fp32 operation.
"""
import numpy as np

from layer_common import U

# A sum of d squares over up to 16 values of a lane and 6 exchanges (22 u of the sum, half of it in
# rstd), a division, an addition, rsqrt within 1 ulp (2 u) and a product with the weight.
RSTD = 32 * U


def turn(x, table, pos, interleaved, back=False):
    """Rows [T, H, d] turned by their positions' angles, and the magnitudes behind every value."""
    rot = table.shape[1]
    y, mag = x.copy(), np.abs(x)
    if rot == 0:
        return y, mag
    row = table[np.clip(pos, 0, len(table) - 1)][:, None]
    c, s = row[..., :rot // 2], row[..., rot // 2:]
    s = -s if back else s
    ia = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia], mag[..., ib] = np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)
    return y, mag


def rotary_ref(x, w, table, pos, interleaved, eps, dy=None):
    """x, dy [T, H, d] in fp64, pos [T]. Returns y or, with dy, dx and dw, each with its bound."""
    pad = (pos < 0) | ((pos >= len(table)) & (table.shape[1] > 0))
    T, H, d = x.shape
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if dy is None:
        n = x if w is None else x * r * w
        y, mag = turn(n, table, pos, interleaved)
        y[pad], mag[pad] = 0, 0
        # the normed value is off by RSTD + u, then a product, a fused one and its rounding
        return y, mag * ((0 if w is None else RSTD + U) + 3 * U)
    e, mag = turn(dy, table, pos, interleaved, back=True)
    ee = 3 * U * mag
    if w is None:
        e[pad], ee[pad] = 0, 0
        return e, ee, None, None
    v = e * x * r
    # a wave's heads and tokens, its lanes, the waves, then the workgroups' partial sums
    grow = (H * (1 + T / 4096) + 6 + 3 + 32 + 32) * U
    keep = ~pad
    dw = v[keep].sum((0, 1))
    dwb = (np.abs(x * r) * ee + np.abs(v) * (RSTD + 2 * U + grow))[keep].sum((0, 1))
    g, ge = e * w, np.abs(w) * ee + U * np.abs(e * w)
    m = r * r * (g * x).mean(-1, keepdims=True)
    me = r * r * (np.abs(x) * (ge + 26 * U * np.abs(g))).mean(-1, keepdims=True) + 2 * (RSTD + U) * np.abs(m)
    dx = r * (g - x * m)
    dxe = r * (ge + np.abs(x) * me + 3 * U * (np.abs(g) + np.abs(x * m))) + np.abs(dx) * (RSTD + U)
    dx[pad], dxe[pad] = 0, 0
    return dx, dxe, dw, dwb


def attention_ref(q, k, v, scale, window, bf16):
    """One sequence: q [T, hq, d], k, v [L, hk, d] in fp64. Returns o and lse, each with its bound."""
    T, hq, d = q.shape
    L, hk, _ = k.shape
    G = hq // hk
    o, ob = np.zeros((T, hq, d)), np.zeros((T, hq, d))
    lse, lb = np.full((T, hq), -np.inf), np.zeros((T, hq))
    for t in range(T):
        p = L - T + t
        lo = max(0, p - window + 1) if window else 0
        if p < lo:
            continue
        for h in range(hk):
            kk, vv = k[lo:p + 1, h], v[lo:p + 1, h]
            n = len(kk)
            for i in range(h * G, (h + 1) * G):
                s = scale * (kk @ q[t, i])
                # a product of d terms, the scale (rounded with log2 e: 2 u) and its product; log2 e
                # itself is rounded, and so is the scale (2 u)
                se = abs(scale) * (d + 6) * U * (np.abs(kk) @ np.abs(q[t, i]))
                top = s.max()
                e = np.exp(s - top)
                total = e.sum()
                w = e / total
                # a weight: its product's error, the difference from the maximum (which cancels, but is
                # rounded), exp2 within 1 ulp
                we = se + se.max() + (2 * np.abs(s - top) + 4) * U
                if bf16:                          # held as the sum of two bf16: 2^-8 of 2^-8, twice
                    wv = we + 2.0 ** -16
                else:
                    wv = we
                # sums: a wave's keys (a quarter, or all of a short sequence), the rescaling at every
                # tile (3 u each, 16 keys or more), 4 waves, the parts
                grow = (n + 3 * (n / 16 + 1) + 128) * U
                o[t, i] = w @ vv
                ob[t, i] = (w * (wv + grow)) @ np.abs(vv) + np.abs(o[t, i]) * ((w * we).sum() + grow + 4 * U)
                lse[t, i] = top + np.log(total)
                # the logarithm and its sum with the maximum in base 2, turned to base e
                lb[t, i] = (w * we).sum() + grow + se.max() + 6 * U * (np.abs(lse[t, i]) + np.abs(top) + 1)
    return o, ob, lse, lb
