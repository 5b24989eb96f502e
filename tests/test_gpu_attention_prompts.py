"""Attention of hundreds and thousands of new tokens over the cache (prompts), of windows shorter than
those, and of short sequences behind wide page tables; chosen tokens against the 64-bit form."""
import numpy as np
import pytest
import torch

import gated_delta_rule_gdn_amd as g
from attention_common import attention_ref
from layer_common import check, f64
from test_gpu_paged_attention import call, compare, make

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g.lib()


def some(x, window=0, got=None):
    """The first, the last and a few other tokens of every sequence, each as the last of a shorter one."""
    o, lse = call(x, window=window) if got is None else got
    T, d = x["q"].shape[1], x["q"].shape[-1]
    rng = np.random.default_rng(T)
    for n, (k, v) in enumerate(zip(x["k"], x["v"])):
        L = len(k)
        for t in sorted({0, 1, T - 1, T // 2, max(T - L, 0), *rng.integers(0, T, 5).tolist()}):
            seen = L - T + t + 1
            if seen <= 0:
                assert not o[n, t].any() and torch.all(lse[n, t] == -float("inf"))
                continue
            r, b, rl, lb = attention_ref(f64(x["q"][n, t:t + 1]), f64(k[:seen]), f64(v[:seen]), d ** -0.5, window,
                                         x["q"].dtype == BF16)
            check(f"o[{n},{t}]", o[n, t:t + 1], r, b, x["q"].dtype)
            check(f"lse[{n},{t}]", lse[n, t:t + 1], rl, lb)
    return o, lse


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,hk,G,d,page,lens,window", [
    (300, 2, 4, 64, 16, [300, 511, 100, 0, 2000], 0),     # a prompt, one in pieces, padded ones
    (300, 2, 4, 128, 24, [300, 1000], 70),                # a window shorter than the prompt
    (1024, 1, 8, 128, 16, [1024], 0),                     # as many blocks of rows as run at once, and twice
    (1024, 2, 8, 128, 64, [1500], 0),
    (2048, 4, 4, 64, 16, [2048], 0),                      # more than run at once
    (700, 1, 3, 256, 100, [701, 900], 300)])
def test_many_new_tokens(T, hk, G, d, page, lens, window, dtype):
    some(make(T + d, lens, T, hk, G, d, page, dtype), window=window)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_value_in_a_prompt_stays_with_what_follows(bad, dtype):
    """The value of token 77 of 100: those before it have the bits they had."""
    x = make(7, [130], 100, 2, 2, 64, 16, dtype)
    want = call(x)
    at = 130 - 100 + 77
    x["vp"][x["table"][0, at // 16], 1, at % 16, 3] = bad
    o, lse = call(x)
    assert torch.equal(lse, want[1]) and torch.equal(o[:, :77], want[0][:, :77]) and torch.equal(o[:, :, :2], want[0][:, :, :2])
    assert not torch.isfinite(o[:, 77:, 2:, 3]).any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,window", [(1, 0), (1, 100), (3, 0), (3, 4000)])
def test_wide_tables(T, window, dtype):
    """A table of 262,144 places for sequences of up to 1,500."""
    compare(make(T + window, [0, 1, 700, 5, 33, 1500], T, 2, 3, 64, 16, dtype, extra=(1 << 14) - 94), window=window)


@pytest.mark.parametrize("N,hk", [(1024, 8), (4000, 1)])
def test_thousands_of_sequences_behind_wide_tables(N, hk):
    rng = np.random.default_rng(N)
    lens = [int(v) for v in rng.integers(0, 30, N)]
    lens[5], lens[N // 2], lens[N - 1] = 900, 2500, 1300
    compare(make(N, lens, 1, hk, 2, 64, 16, BF16, extra=500), only=[0, 4, 5, 6, 255, 256, N // 2, N - 2, N - 1])


@pytest.mark.parametrize("page", [257, 1000, 4096])
def test_large_pages(page):
    compare(make(page, [700, 5, 2 * page + 3], 2, 1, 4, 128, page, BF16))
