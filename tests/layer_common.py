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
