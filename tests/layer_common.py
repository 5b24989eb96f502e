"""Plain 64-bit forms of the operators around the recurrence, for the GPU tests, written one
sequence and one token at a time from the definitions, and the bounds the results are held to.

A bound is an absolute one per element, from the arithmetic: u = 2^-24 per fp32 operation on the
magnitudes that go into it, the transcendental unit's error, and half a step of the output type
(2^-8 of the value in bf16, 2^-24 in fp32).
"""
import numpy as np
import torch

U = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def f64(t):
    return None if t is None else t.detach().to("cpu").double().numpy()


def offsets(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)


def check(name, got, want, bound, dtype=torch.float32):
    """|got - want| <= bound + half a step of want, element by element."""
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert np.all(np.isfinite(got)), f"{name}: not finite"
    lim = bound + HALF_STEP[dtype] * (np.abs(want) + bound) + 1e-37
    err = np.abs(got - want)
    bad = err > lim
    worst = float((err / lim).max()) if err.size else 0.0
    print(f"[layer] {name}: largest error / bound {worst:.3f}", flush=True)
    assert not bad.any(), (name, worst, np.argwhere(bad)[:4].tolist())


def sigmoid(a):
    return 1.0 / (1.0 + np.exp(-a))


def act_err(a, da):
    """Bound on the error of silu(a) when a is off by da: slope at most 1.1; exp2 of a rounded
    product, an add and a reciprocal give a relative error of (|a| + 6) 2^-23."""
    return 1.1 * da + (np.abs(a) + 6) * 2 * U * np.abs(a)


def slope_err(a, da):
    """The same for d silu / da = s (1 + a (1 - s)): its own slope is at most 0.5."""
    return 0.5 * da + (np.abs(a) + 8) * 2 * U * (1 + np.abs(a))


# ---- short convolution -------------------------------------------------------------------


def conv_ref(x, weight, bias, state0, lens, silu, dy=None, dstate_T=None):
    """x [T, C] flat in fp64. Returns a dict: y, state_T and, with dy, the gradients; for each
    a bound under its name + "_b"."""
    T, C = x.shape
    W = weight.shape[1]
    cu = offsets(lens)
    N = len(lens)
    r = {"y": np.zeros((T, C)), "y_b": np.zeros((T, C)), "state_T": np.zeros((N, W - 1, C))}
    if dy is not None:
        r.update(dx=np.zeros((T, C)), dx_b=np.zeros((T, C)), dweight=np.zeros((C, W)),
                 dweight_b=np.zeros((C, W)), dbias=np.zeros(C), dbias_b=np.zeros(C),
                 dstate0=np.zeros((N, W - 1, C)), dstate0_b=np.zeros((N, W - 1, C)))
    b = np.zeros(C) if bias is None else bias
    for n in range(N):
        lo, hi = cu[n], cu[n + 1]
        old = np.zeros((W - 1, C)) if state0 is None else state0[n]
        seen = np.concatenate([old, x[lo:hi]])
        r["state_T"][n] = seen[hi - lo:]
        d_seen, d_b = np.zeros_like(seen), np.zeros_like(seen)
        for t in range(hi - lo):
            rows = seen[t:t + W]
            a = (rows * weight.T).sum(0) + b
            da = (W + 2) * U * ((np.abs(rows) * np.abs(weight.T)).sum(0) + np.abs(b))
            r["y"][lo + t] = a * sigmoid(a) if silu else a
            r["y_b"][lo + t] = act_err(a, da) if silu else da
            if dy is None:
                continue
            g = dy[lo + t]
            s = sigmoid(a)
            slope = s * (1 + a * (1 - s)) if silu else np.ones(C)
            e = g * slope
            eb = np.abs(g) * (slope_err(a, da) if silu else 0.0) + U * np.abs(e)
            d_seen[t:t + W] += e * weight.T
            d_b[t:t + W] += np.abs(weight.T) * (eb + (W + 2) * U * np.abs(e))
            # sums of up to 64 tokens in a lane, then of the tiles in 16 waves
            grow = (64 + T / 128 + 18) * U
            r["dweight"] += (e * rows).T
            r["dweight_b"] += (np.abs(rows) * (eb + grow * np.abs(e))).T
            r["dbias"] += e
            r["dbias_b"] += eb + grow * np.abs(e)
        if dy is not None:
            if dstate_T is not None:
                d_seen[hi - lo:] += dstate_T[n]
                d_b[hi - lo:] += U * np.abs(dstate_T[n])
            r["dstate0"][n], r["dstate0_b"][n] = d_seen[:W - 1], d_b[:W - 1]
            r["dx"][lo:hi], r["dx_b"][lo:hi] = d_seen[W - 1:], d_b[W - 1:]
    return r


# ---- selective scan ----------------------------------------------------------------------


def scan_ref(x, dt, A, B, C, D, gate, dt_bias, softplus, S0, lens, tile=128):
    """x, dt, gate [T, ch]; B, C [T, G, M]; A [ch, M]; flat, in fp64. Returns o, S_T and their
    bounds. The bounds follow the recurrence: `m` holds the magnitudes behind the state, `e` the
    error of the state."""
    T, ch = x.shape
    G, M = B.shape[1:]
    rep = ch // G
    cu = offsets(lens)
    raw = dt + (0.0 if dt_bias is None else dt_bias)
    step = np.logaddexp(0.0, raw) if softplus else raw
    # the sum dt + dt_bias, the rounded exponent of e^-|raw|, and a dozen operations of softplus
    rel = U * ((3 * np.abs(raw) + 24) if softplus else 1.0)
    r = {"o": np.zeros((T, ch)), "o_b": np.zeros((T, ch)),
         "S_T": np.zeros((len(lens), ch, M)), "S_T_b": np.zeros((len(lens), ch, M))}
    for n in range(len(lens)):
        h = np.zeros((ch, M)) if S0 is None else S0[n].copy()
        m, e = np.abs(h), np.zeros((ch, M))
        for t in range(cu[n], cu[n + 1]):
            z = step[t][:, None] * A
            a = np.exp(z)
            b = (step[t] * x[t])[:, None] * np.repeat(B[t], rep, 0)
            er = (rel[t] if softplus else rel)
            er = np.broadcast_to(er, (ch,))[:, None]
            da = a * (np.abs(z) * (er + 3 * U) + 2 * U)
            e = a * e + da * m + np.abs(b) * (er + 4 * U)
            h, m = a * h + b, a * m + np.abs(b)
            e += 2 * U * m
            c = np.repeat(C[t], rep, 0)
            # a tile's decay comes from its summed dt: an error of the sum's rounding, at most
            # tile U of it, times z e^-z <= 0.4
            et = e + 0.4 * tile * U * m
            y = (c * h).sum(-1)
            ye = (np.abs(c) * (et + (M + 3) * U * m)).sum(-1)
            if D is not None:
                y = y + D * x[t]
                ye = ye + 2 * U * np.abs(D * x[t])
            if gate is not None:
                s = gate[t] * sigmoid(gate[t])
                ye = np.abs(s) * ye + np.abs(y * s) * (np.abs(gate[t]) + 8) * 2 * U
                y = y * s
            r["o"][t], r["o_b"][t] = y, ye
        r["S_T"][n], r["S_T_b"][n] = h, e + 0.4 * tile * U * m
    return r


# ---- block norm --------------------------------------------------------------------------


def norm_ref(x, nw, gate, res, scale, nxt, eps, dh=None, dy=None):
    """Rows in fp64. Returns h, y and, with dh or dy, the gradients, each with its bound. Errors
    of row statistics are relative: a sum of d squares over 8 or 16 values and up to ten
    exchanges, a division, rsqrt and a product come to at most 32 U of rstd."""
    R = 32 * U
    rows, d = x.shape
    rx = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    p = x if nw is None else x * rx * nw
    pe = 0.0 if nw is None else np.abs(p) * R
    if gate is not None:
        s = sigmoid(gate)
        sl, se = gate * s, (np.abs(gate) + 8) * 2 * U * np.abs(gate * s)
        u, ue = p * sl, np.abs(sl) * pe + np.abs(p) * se + U * np.abs(p * sl)
    else:
        u, ue = p, pe
    sc = 1.0 if scale is None else scale
    r0 = 0.0 if res is None else res
    h = r0 + sc * u
    he = np.abs(sc) * ue + 2 * U * (np.abs(sc * u) + np.abs(r0))
    rh = 1 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    # rstd(h) moves by rh^2 |h| he / |h| at most, relative
    rhe = R + rh * rh * (np.abs(h) * he).mean(-1, keepdims=True)
    out = {"h": h, "h_b": he + 0 * h}
    if nxt is not None:
        out["y"] = h * rh * nxt
        out["y_b"] = np.abs(rh * nxt) * he + np.abs(out["y"]) * (rhe + 2 * U)
    if dh is None and dy is None:
        return out
    g = np.zeros_like(x) if dh is None else dh.copy()
    ge = np.zeros_like(x)
    # sums over rows: a workgroup's rows in a lane, then its partial sums in 16 waves
    grow = (rows / 512 + rows / 16 + 24) * U
    col = lambda v, e: (v.sum(0), (e + grow * np.abs(v)).sum(0))  # noqa: E731
    if nxt is not None:
        v = dy * h * rh
        out["dnext_weight"], out["dnext_weight_b"] = col(v, np.abs(v) * (rhe + 2 * U) + np.abs(dy * rh) * he)
        w = dy * nxt
        m = rh * rh * (w * h).mean(-1, keepdims=True)
        me = rh * rh * (np.abs(w) * (he + 32 * U * np.abs(h))).mean(-1, keepdims=True) + 2 * rhe * np.abs(m)
        inner = w - h * m
        g = g + rh * inner
        ge = rh * (np.abs(h) * me + he * np.abs(m) + 3 * U * (np.abs(w) + np.abs(h * m))) \
            + np.abs(rh * inner) * rhe + 2 * U * (np.abs(g) + np.abs(rh * inner))
    if res is not None:
        out["dresidual"], out["dresidual_b"] = g, ge
    if scale is not None:
        v = g * u
        out["dscale"], out["dscale_b"] = col(v, np.abs(u) * ge + np.abs(g) * ue + U * np.abs(v))
        g, ge = g * scale, np.abs(scale) * ge + U * np.abs(g * scale)
    if gate is not None:
        slope = s * (1 + gate * (1 - s))
        out["dgate"] = g * p * slope
        out["dgate_b"] = np.abs(p * slope) * ge + np.abs(g * slope) * pe + np.abs(g * p) * slope_err(gate, 0.0) \
            + 3 * U * np.abs(out["dgate"])
        g, ge = g * sl, np.abs(sl) * ge + np.abs(g) * se + U * np.abs(g * sl)
    if nw is not None:
        v = g * x * rx
        out["dnorm_weight"], out["dnorm_weight_b"] = col(v, np.abs(x * rx) * ge + np.abs(v) * (R + 2 * U))
        w, we = g * nw, np.abs(nw) * ge + U * np.abs(g * nw)
        m = rx * rx * (w * x).mean(-1, keepdims=True)
        me = rx * rx * (np.abs(x) * (we + 32 * U * np.abs(w))).mean(-1, keepdims=True) + 2 * R * np.abs(m)
        g = rx * (w - x * m)
        ge = rx * (we + np.abs(x) * me + 3 * U * (np.abs(w) + np.abs(x * m))) + np.abs(g) * R
    out["dx"], out["dx_b"] = g, ge
    return out


def scan_bwd_ref(x, dt, A, B, C, D, gate, dt_bias, softplus, S0, lens, dO, dS_T, tile=32):
    """Gradients of scan_ref's o and S_T and their bounds, token by token from the last to the
    first. `gm` holds the magnitudes behind the state's gradient, `ge` its error."""
    T, ch = x.shape
    G, M = B.shape[1:]
    rep = ch // G
    cu = offsets(lens)
    raw = dt + (0.0 if dt_bias is None else dt_bias)
    step = np.logaddexp(0.0, raw) if softplus else raw
    rel = U * ((3 * np.abs(raw) + 24) if softplus else np.ones_like(raw))
    sp = sigmoid(raw) if softplus else np.ones_like(raw)
    spe = (np.abs(raw) + 6) * 2 * U * sp if softplus else np.zeros_like(raw)
    skip = np.zeros(ch) if D is None else D
    z = lambda *s: np.zeros(s)  # noqa: E731
    names = {"dx": (T, ch), "ddt": (T, ch), "dgate": (T, ch), "dB": (T, G, M), "dC": (T, G, M),
             "dA": (ch, M), "dD": (ch,), "ddt_bias": (ch,), "dS0": (len(lens), ch, M)}
    r = {n: z(*s) for n, s in names.items()}
    r.update({n + "_b": z(*s) for n, s in names.items()})
    # tiles' sums in order, a few lanes' sums before them
    grow = (tile + T / tile + 8) * U
    over = (16 + ch / 32) * U                 # channels: lanes, waves, workgroups
    chan = lambda v: v.reshape(G, rep, M).sum(1)  # noqa: E731
    for n in range(len(lens)):
        lo, hi = cu[n], cu[n + 1]
        L = hi - lo
        H, HM, HE = z(L + 1, ch, M), z(L + 1, ch, M), z(L + 1, ch, M)
        a, da = z(L, ch, M), z(L, ch, M)
        H[0] = 0.0 if S0 is None else S0[n]
        HM[0] = np.abs(H[0])
        for k in range(L):
            t = lo + k
            er = rel[t][:, None]
            zz = step[t][:, None] * A
            a[k] = np.exp(zz)
            da[k] = a[k] * (np.abs(zz) * (er + 3 * U) + 2 * U)
            b = (step[t] * x[t])[:, None] * np.repeat(B[t], rep, 0)
            HE[k + 1] = a[k] * HE[k] + da[k] * HM[k] + np.abs(b) * (er + 4 * U)
            H[k + 1], HM[k + 1] = a[k] * H[k] + b, a[k] * HM[k] + np.abs(b)
            HE[k + 1] += 2 * U * HM[k + 1]
        HE = HE + 0.4 * tile * U * HM
        g = z(ch, M) if dS_T is None else dS_T[n].copy()
        gm, ge = np.abs(g), z(ch, M)
        for k in range(L - 1, -1, -1):
            t = lo + k
            er = rel[t][:, None]
            b, c = np.repeat(B[t], rep, 0), np.repeat(C[t], rep, 0)
            u = (step[t] * x[t])[:, None]
            dy, dye = dO[t], z(ch)
            if gate is not None:
                s = sigmoid(gate[t])
                sl = gate[t] * s
                y = (c * H[k + 1]).sum(-1) + skip * x[t]
                ye = (np.abs(c) * (HE[k + 1] + (M + 4) * U * HM[k + 1])).sum(-1) + 2 * U * np.abs(skip * x[t])
                slope = s * (1 + gate[t] * (1 - s))
                r["dgate"][t] = dO[t] * y * slope
                r["dgate_b"][t] = np.abs(dO[t]) * (ye * np.abs(slope) + np.abs(y) * slope_err(gate[t], 0.0)) \
                    + 3 * U * np.abs(r["dgate"][t])
                dy = dO[t] * sl
                dye = np.abs(dy) * (np.abs(gate[t]) + 9) * 2 * U
            cy = c * dy[:, None]
            gh, ghm = cy + g, np.abs(cy) + gm
            ghe = np.abs(c) * dye[:, None] + ge + 2 * U * ghm
            gt = ghe + 0.4 * tile * U * ghm
            v = dy[:, None] * H[k + 1]
            r["dC"][t] = chan(v)
            r["dC_b"][t] = chan(np.abs(dy)[:, None] * HE[k + 1] + dye[:, None] * np.abs(H[k + 1])
                                + over * np.abs(dy)[:, None] * HM[k + 1])
            r["dB"][t] = chan(gh * u)
            r["dB_b"][t] = chan(np.abs(u) * (gt + ghm * (er + over + 2 * U)))
            sB = (gh * b).sum(-1)
            sBm = (ghm * np.abs(b)).sum(-1)
            sBe = (gt * np.abs(b)).sum(-1) + (M + 3) * U * sBm
            ah, ahm = a[k] * H[k], a[k] * HM[k]
            ahe = a[k] * HE[k] + da[k] * HM[k] + U * ahm
            q = gh * ah
            qe = gt * ahm + ghm * ahe + 2 * U * ghm * ahm
            sA = (q * A).sum(-1)
            sAe = (qe * np.abs(A)).sum(-1) + (M + 5) * U * (ghm * ahm * np.abs(A)).sum(-1)
            d = step[t]
            r["dx"][t] = skip * dy + d * sB
            r["dx_b"][t] = np.abs(skip) * (dye + 2 * U * np.abs(dy)) + np.abs(d) * (sBe + (rel[t] + 2 * U) * sBm)
            full = x[t] * sB + sA
            fe = np.abs(x[t]) * sBe + sAe + 2 * U * (np.abs(x[t]) * sBm + (ghm * ahm * np.abs(A)).sum(-1))
            r["ddt"][t] = full * sp[t]
            de = fe * sp[t] + np.abs(full) * spe[t] + U * np.abs(r["ddt"][t])
            r["ddt_b"][t] = de
            r["dA"] += q * d[:, None]
            r["dA_b"] += np.abs(d)[:, None] * (qe + ghm * ahm * (er + grow))
            r["dD"] += dy * x[t]
            r["dD_b"] += np.abs(x[t]) * (dye + (grow + U) * np.abs(dy))
            r["ddt_bias"] += r["ddt"][t]
            r["ddt_bias_b"] += de + grow * np.abs(r["ddt"][t])
            g, ge = a[k] * gh, a[k] * ghe + da[k] * ghm
            gm = a[k] * ghm
            ge = ge + U * gm
        r["dS0"][n], r["dS0_b"][n] = g, ge + 0.4 * tile * U * gm
    return r
