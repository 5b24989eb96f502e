"""Scores at the ends of the types: products of -inf and of the lowest finite value (a caller's own masks,
written into the keys), over single keys, whole tiles, whole parts and whole rows, at every kind of scale;
and scores that differ by more than any weight can hold."""
import numpy as np
import pytest
import torch

import gated_delta_rule_gdn_amd as g
from attention_common import attention_ref
from layer_common import U, check, f64
from test_gpu_paged_attention import call, make

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16

# scales whose product with log2 e rounds up, down, and (powers of two) as log2 e itself; below 0; of 1
SCALES = [None, 0.125, 0.1, 0.2, 0.0884, 0.7, 1.0, -0.3, -0.125]


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g.lib()


def worst(kind, scale, dtype):
    """The value of a key that makes its scaled product -inf, or the lowest of the type, where q is 1."""
    v = float("inf") if kind == "inf" else torch.finfo(dtype).max
    return v if scale is not None and scale < 0 else -v


def mask(x, n, keys, value, page=16):
    """Value 0 of the given keys of sequence n, for all heads; q's is 1 everywhere."""
    x["q"][..., 0] = 1.0
    for j in keys:
        x["kp"][x["table"][n, j // page], :, j % page, 0] = value


def against(x, n, got, kept, scale, dtype):
    """Sequence n's rows against the 64-bit form over the keys that are kept."""
    d = x["q"].shape[-1]
    o, lse = got
    r, b, rl, lb = attention_ref(f64(x["q"][n]), f64(x["k"][n])[kept], f64(x["v"][n])[kept],
                                 d ** -0.5 if scale is None else scale, 0, dtype == BF16)
    check("o", o[n], r, b, dtype)
    check("lse", lse[n], rl, lb)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kind", ["inf", "lowest"])
@pytest.mark.parametrize("scale", SCALES)
def test_masked_keys_take_no_part(scale, kind, d, dtype):
    """The first keys of two sequences (of the second whole tiles and parts), for three new tokens; and for
    one, single keys in between and everything behind the fifth key."""
    value = worst(kind, scale, dtype)
    x = make(d, [40, 700], 3, 2, 2, d, 16, dtype)
    mask(x, 0, range(5), value)
    mask(x, 1, range(651), value)
    got = call(x, scale=scale)
    against(x, 0, got, slice(5, None), scale, dtype)
    against(x, 1, got, slice(651, None), scale, dtype)
    x = make(d + 1, [90, 700, 40], 1, 2, 3, d, 16, dtype)
    some = [[7, 8, 40, 89], list(range(5, 700)), list(range(39))]
    for n, keys in enumerate(some):
        mask(x, n, keys, value)
    got = call(x, scale=scale)
    for n, keys in enumerate(some):
        against(x, n, got, np.setdiff1d(np.arange(len(x["k"][n])), keys), scale, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("scale", SCALES)
def test_rows_whose_every_product_is_minus_infinity_are_empty(scale, d, dtype):
    x = make(d + 2, [1, 40, 700], 1, 2, 2, d, 16, dtype)
    for n, length in enumerate((1, 40, 700)):
        mask(x, n, range(length), worst("inf", scale, dtype))
    o, lse = call(x, scale=scale)
    assert not o.any() and torch.equal(lse, torch.full_like(lse, -float("inf")))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("scale", SCALES)
def test_rows_of_the_lowest_value_are_means(scale, d, dtype):
    """Every product rounds to the type's lowest value (what is added is less than half a step of it), so
    all weights are the same: those of queries of zeros."""
    lens = [1, 40, 700]
    x = make(d + 3, lens, 1, 2, 2, d, 16, dtype)
    value = worst("lowest", scale, dtype)
    for n, length in enumerate(lens):
        mask(x, n, range(length), value)
    o, lse = call(x, scale=scale)
    s = (d ** -0.5 if scale is None else scale) * value
    for n in range(len(lens)):
        r, b, _, _ = attention_ref(np.zeros_like(f64(x["q"][n])), f64(x["k"][n]), f64(x["v"][n]), 1.0, 0, dtype == BF16)
        check(f"o[{n}]", o[n], r, b, dtype)
        # the scale and its product are rounded; the logarithm is below half a step of it
        assert np.all(np.abs(f64(lse[n]) / s - 1) <= 3 * U)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("power,scale", [(p, s) for p in (40, 100) for s in (None, 0.1, -0.3, 1.0, 1e20)] + [(100, 1e-20)])
def test_one_key_takes_all_however_large_the_scores(power, scale, d, dtype):
    """Keys c e_0 with whole numbers c, a query 2^power e_0: the products are exact and differ by 2^power at
    least, scaled by 10^10 or more, so a row is the value of its best key."""
    s = d ** -0.5 if scale is None else scale
    lens = [1, 40, 700]
    x = make(d + power, lens, 1, 1, 2, d, 16, dtype)
    x["kp"].mul_(0.0)                            # what is not a number stays so
    x["q"].zero_()
    x["q"][..., 0] = 2.0 ** power
    rng = np.random.default_rng(power + d)
    best = []
    for n, length in enumerate(lens):
        c = rng.integers(-100, 100, length)
        best.append(int(rng.integers(0, length)))
        c[best[n]] = -101 if s < 0 else 101
        for j in range(length):
            x["kp"][x["table"][n, j // 16], :, j % 16, 0] = float(c[j])
    o, lse = call(x, scale=scale)
    score = 101 * 2.0 ** power * abs(s)
    for n, top in enumerate(best):
        assert torch.equal(o[n, 0], x["v"][n][top].cuda().expand_as(o[n, 0]))
        if score < 3e38:
            assert np.all(np.abs(f64(lse[n]) / score - 1) <= 3 * U)
