"""Attention of new tokens over a paged cache against the 64-bit form: lengths around every tile and
part, page sizes, heads, several new tokens, windows, masks that leave a row empty, garbage in
places that no token sees."""
import numpy as np
import pytest
import torch

import gated_delta_rule_gdn_amd as g
from attention_common import attention_ref
from layer_common import check, f64

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g.lib()


def make(seed, lens, T, hk, G, d, page, dtype, spare=2, std=2.0, garbage=float("nan"), extra=1):
    """A cache of shuffled pages; places behind a sequence's end and whole unused pages hold `garbage`,
    table entries behind its last page point nowhere."""
    gen = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pages, width = sum(need) + spare, max(need + [0]) + extra
    kp = torch.full((pages, hk, page, d), garbage)
    vp = torch.full((pages, hk, page, d), garbage)
    table = torch.full((len(lens), width), -7, dtype=torch.int32)
    order = torch.randperm(pages, generator=gen).tolist()
    ks, vs = [], []
    for i, n in enumerate(lens):
        k = torch.randn(n, hk, d, generator=gen).to(dtype)
        v = torch.randn(n, hk, d, generator=gen).to(dtype)
        for j in range(need[i]):
            pg = order.pop()
            table[i, j] = pg
            rows = slice(j * page, min(n, (j + 1) * page))
            kp[pg, :, :rows.stop - rows.start] = k[rows].transpose(0, 1).float()
            vp[pg, :, :rows.stop - rows.start] = v[rows].transpose(0, 1).float()
        ks.append(k)
        vs.append(v)
    q = (std * torch.randn(len(lens), T, hk * G, d, generator=gen)).to(dtype)
    return {"q": q.cuda(), "kp": kp.to(dtype).cuda(), "vp": vp.to(dtype).cuda(), "table": table.cuda(),
            "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"), "k": ks, "v": vs}


def call(x, **kw):
    return g.paged_attention_step(x["q"], x["kp"], x["vp"], x["table"], x["lens"], return_lse=True, **kw)


def compare(x, scale=None, window=0, only=None, got=None):
    o, lse = call(x, scale=scale, window=window) if got is None else got
    d = x["q"].shape[-1]
    for i in range(len(x["k"])) if only is None else only:
        r, b, rl, lb = attention_ref(f64(x["q"][i]), f64(x["k"][i]), f64(x["v"][i]), d ** -0.5 if scale is None else scale,
                                     window, x["q"].dtype == BF16)
        check(f"o[{i}]", o[i], r, b, x["q"].dtype)
        gl = f64(lse[i])
        empty = np.isinf(rl)
        assert np.all(gl[empty] == -np.inf) and not f64(o[i])[empty].any()
        check(f"lse[{i}]", np.where(empty, 0, gl), np.where(empty, 0, rl), lb)
    return o, lse


LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 511, 512, 513, 700]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_lengths(d, dtype):
    compare(make(d, LENS, 1, 2, 3, d, 16, dtype))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("page", [1, 3, 8, 16, 24, 32, 64, 100, 256])
def test_page_sizes(page, dtype):
    compare(make(page, [5, 77, 300, 0, 2 * page, page + 1], 1, 1, 4, 128, page, dtype))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,window", [(1, 0), (1, 37), (3, 0), (3, 150)])
@pytest.mark.parametrize("page", [4, 8, 12, 24, 40])
def test_pages_that_end_inside_a_tile(page, T, window, d, dtype):
    """Every other number of eights, and none: ends and windows that begin at every place of a page."""
    lens = [T - 1, page, 2 * page + 1, 130, 131, 135, 137, 141, 144, 500, 1029]
    compare(make(page * d + T, lens, T, 1, 8, d, page, dtype), window=window)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("hk,G", [(1, 1), (3, 1), (2, 8), (1, 16), (1, 17), (2, 32), (1, 40), (5, 2)])
def test_heads(hk, G, dtype):
    compare(make(hk * 50 + G, [130, 40, 601], 1, hk, G, 128, 32, dtype))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,G", [(2, 1), (4, 8), (5, 3), (8, 4), (3, 16), (40, 2)])
def test_new_tokens(T, G, d, dtype):
    """Among them sequences that have fewer tokens than are new: their first rows see nothing."""
    compare(make(T * 9 + G, [3, 1, 0, T, T + 1, 64, 333, 520], T, 2, G, d, 16, dtype))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [1, 4])
@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 100, 640, 100000])
def test_windows(window, T, dtype):
    x = make(window + T, [1, 40, 200, 900, 1300], T, 2, 2, 64, 16, dtype)
    compare(x, window=window)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,d,page", [(1, 64, 16), (3, 128, 24)])
@pytest.mark.parametrize("N,window", [(31, 500), (32, 500), (33, 150), (40, 1200), (40, 2500)])
def test_windows_of_sequences_for_every_cu(N, window, T, d, page, dtype):
    """Where every CU has a sequence and the window is short, no sequence is cut; next to that, and
    behind a longer window, they are."""
    rng = np.random.default_rng(N + window)
    lens = [int(n) for n in rng.integers(0, 1700, N - 3)] + [window, window + T, 2600]
    x = make(window + T + N, lens, T, 8, 1, d, page, dtype)
    compare(x, window=window, only=[0, 7, 19, N - 3, N - 2, N - 1])
    for i in (3, 11, N - 1):                    # alone they are cut
        y = {**x, "q": x["q"][i:i + 1], "table": x["table"][i:i + 1], "lens": x["lens"][i:i + 1],
             "k": x["k"][i:i + 1], "v": x["v"][i:i + 1]}
        compare(y, window=window)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_window_leaves_pages_behind(dtype):
    """Pages that lie before the window may be given away: their entries point nowhere, or at pages
    full of NaN."""
    x = make(3, [900, 1400], 2, 2, 2, 128, 16, dtype)
    want = call(x, window=300)
    x["table"][0, :37] = -1                     # places below 592 of 900 - 2 - 300 + 1 = 599
    x["table"][1, :68] = 10 ** 6                # below 1,088 of 1,099
    got = compare(x, window=300)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("hk,G,dtype", [(8, 4, BF16), (1, 2, F32), (2, 16, BF16), (1, 1, BF16)])
def test_one_long_sequence_is_cut_and_joined(hk, G, dtype):
    compare(make(4, [20011], 1, hk, G, 128, 64, dtype))


def test_long_and_short_together():
    compare(make(5, [9000, 1, 0, 513, 4097, 12, 0, 2600], 1, 2, 4, 128, 16, BF16))
    compare(make(6, [9000, 2, 0, 700], 3, 1, 6, 64, 32, F32))


def test_more_sequences_than_a_wave_has_lanes():
    rng = np.random.default_rng(7)
    for n in (64, 65, 200):
        lens = [int(v) for v in rng.integers(0, 60, n)]
        lens[n // 2] = 3000
        compare(make(n, lens, 1, 1, 2, 64, 16, BF16), only=[0, n // 2 - 1, n // 2, n // 2 + 1, n - 2, n - 1])


@pytest.mark.parametrize("n,hk,d", [(300, 1, 64), (257, 2, 128), (1500, 1, 64), (520, 4, 128)])
def test_hundreds_of_sequences(n, hk, d):
    """More of them than are looked at together, fewer and more than run at once, two long ones among
    them."""
    rng = np.random.default_rng(n)
    lens = [int(v) for v in rng.integers(0, 40, n)]
    lens[3], lens[n - 2] = 5000, 1300
    compare(make(n, lens, 1, hk, 2, d, 16, BF16), only=[0, 2, 3, 4, 63, 64, 255, 256, n - 3, n - 2, n - 1])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_garbage_behind_the_end_is_never_used(dtype):
    """NaN, infinities and the type's lowest value in the unused places give the same bits."""
    outs = []
    for garbage in (0.0, float("nan"), float("inf"), -float("inf"), torch.finfo(dtype).min):
        outs.append(call(make(8, [1, 33, 100, 700], 3, 2, 2, 128, 16, dtype, garbage=garbage)))
    for o, lse in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_values_that_are_not_finite_stay_with_the_tokens_that_see_them(bad, dtype):
    """The key or the value of new token 2 of 4: tokens 0 and 1 have the bits they had."""
    x = make(9, [50, 700], 4, 1, 3, 128, 16, dtype)
    want = call(x)
    for pool in ("kp", "vp"):
        y = dict(x)
        y[pool] = x[pool].clone()
        for i, n in enumerate((50, 700)):
            at = n - 4 + 2
            y[pool][x["table"][i, at // 16], 0, at % 16, 5] = bad
        o, lse = call(y)
        assert torch.equal(o[:, :2], want[0][:, :2]) and torch.equal(lse[:, :2], want[1][:, :2])
        if pool == "vp":
            assert not torch.isfinite(o[:, 2:, :, 5]).any()
            assert torch.equal(o[:, 2:, :, 6:], want[0][:, 2:, :, 6:]) and torch.equal(lse, want[1])
    # the same at the other end of a window: value of a place that token 0 sees alone
    want = call(x, window=40)
    y = dict(x, vp=x["vp"].clone())
    at = 700 - 4 - 40 + 1
    y["vp"][x["table"][1, at // 16], 0, at % 16, 5] = bad
    o, _ = call(y, window=40)
    assert torch.equal(o[0], want[0][0]) and torch.equal(o[1, 1:], want[0][1, 1:])
    assert not torch.isfinite(o[1, 0, :, 5]).any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 32), (128, 24), (256, 16)])
@pytest.mark.parametrize("N", [1, 34])
def test_a_value_that_is_not_finite_at_the_beginning_of_a_window(N, d, page, dtype):
    """Seen by token 0 of 3 alone, with several tiles behind it: the other tokens have the bits they had."""
    window = 700
    x = make(d + N, [1450] * N, 3, 8, 1, d, page, dtype)
    want = call(x, window=window)
    y = dict(x, vp=x["vp"].clone())
    at = 1450 - 3 - window + 1
    y["vp"][x["table"][N - 1, at // page], 3, at % page, d - 1] = float("nan")
    o, lse = call(y, window=window)
    assert torch.isnan(o[N - 1, 0, 3, d - 1])
    o[N - 1, 0, 3, d - 1] = want[0][N - 1, 0, 3, d - 1]
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_large_and_small_scores(dtype):
    """Scores of hundreds (one key takes all), differences far below the type's range, scales of zero
    and below."""
    x = make(10, [1, 90, 600], 1, 2, 2, 128, 16, dtype, std=40.0)
    compare(x, scale=1.0)
    for scale in (0.0, -0.3, 1e-30):
        compare(x, scale=scale)


def test_masked_keys_of_minus_infinity():
    """A caller's own mask: keys whose products are -inf take no part; if all are, the row is empty."""
    x = make(11, [40], 1, 1, 1, 64, 16, F32)
    x["q"][..., 0] = 1.0
    for j in range(5, 40):
        x["kp"][x["table"][0, j // 16], 0, j % 16, 0] = -float("inf")
    x["k"][0], x["v"][0] = x["k"][0][:5], x["v"][0][:5]
    compare(x)
    for j in range(5):
        x["kp"][x["table"][0, 0], 0, j, 0] = -float("inf")
    o, lse = call(x)
    assert not o.any() and torch.equal(lse, torch.full_like(lse, -float("inf")))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_shared_pages(dtype):
    """Forked sequences read the same pages: the same bits for the same query."""
    x = make(12, [500, 500, 500], 1, 2, 4, 128, 16, dtype)
    x["table"][1:] = x["table"][0]
    x["q"][1:] = x["q"][0]
    o, lse = call(x)
    assert torch.equal(o[1], o[0]) and torch.equal(o[2], o[0]) and torch.equal(lse[1], lse[0])
    compare(x, only=[0], got=(o, lse))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("pad,shift", [(16, 8), (5, 0), (3, 1)])
def test_slices_of_queries(pad, shift, dtype):
    x = make(13, [70, 200], 2, 2, 2, 64, 16, dtype)
    wide = torch.randn(2, 2, 4 * 64 + pad).to(dtype).cuda()
    view = wide[..., shift:shift + 256].unflatten(-1, (4, 64))
    view.copy_(x["q"])
    want = call(x)
    x["q"] = view
    assert all(torch.equal(a, b) for a, b in zip(call(x), want))


def test_wrong_tables_and_lengths_stay_inside():
    """Entries outside the pool and lengths outside the table are held inside: wrong results at worst,
    no access outside (checked by guard pages that hold NaN only in memory next to the pools)."""
    x = make(14, [100, 300], 1, 1, 2, 64, 16, BF16, garbage=0.0)
    x["table"][0, 2], x["table"][0, 3], x["table"][1, 7] = -5, 10 ** 9, 2 ** 31 - 1
    x["lens"][1] = 2 ** 31 - 1
    guard = torch.full((3, *x["kp"].shape), float("nan"), dtype=BF16, device="cuda")
    guard[1].copy_(x["kp"])
    x["kp"] = guard[1]
    o, lse = call(x)
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    x["lens"][:] = torch.tensor([-3, -2 ** 31], dtype=torch.int32)
    o, lse = call(x)
    assert not o.any() and torch.equal(lse, torch.full_like(lse, -float("inf")))


def test_nothing_cached():
    x = make(15, [0, 0], 2, 1, 2, 64, 16, F32, spare=0, extra=0)
    assert x["kp"].shape[0] == 0 and x["table"].shape[1] == 0
    o, lse = call(x)
    assert not o.any() and torch.equal(lse, torch.full_like(lse, -float("inf")))
    e = g.paged_attention_step(x["q"][:0], x["kp"], x["vp"], x["table"][:0], x["lens"][:0])
    assert e.shape == (0, 2, 2, 64)


def test_far_into_a_large_pool():
    """Rows whose elements lie beyond 2^32."""
    pages, hk, page, d = 1100, 16, 1024, 256
    kp = torch.zeros(pages, hk, page, d, dtype=BF16, device="cuda")
    vp = torch.zeros(pages, hk, page, d, dtype=BF16, device="cuda")
    small = make(16, [1500], 1, hk, 2, d, page, BF16)
    want = call(small)
    used = small["table"][0, :2].long()
    for pool, src in ((kp, small["kp"]), (vp, small["vp"])):
        pool[[pages - 1, pages - 2]] = src[used]
    big = dict(small, kp=kp, vp=vp, table=torch.tensor([[pages - 1, pages - 2, 0]], dtype=torch.int32, device="cuda"))
    assert all(torch.equal(a, b) for a, b in zip(call(big), want))


def test_same_bits_at_every_call_and_with_any_workspace():
    x = make(17, [5000, 30, 1200], 2, 2, 4, 128, 16, BF16)
    need = g.paged_attention_step_workspace_bytes(3, 2, 8, 2, 128, 16, x["table"].shape[1], BF16)
    a = call(x)
    for fill in (0, 255):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        assert all(torch.equal(p, q) for p, q in zip(call(x, workspace=ws), a))


def test_refusals():
    x = make(18, [600], 1, 2, 2, 64, 16, BF16)
    bad = dict(x, kp=x["kp"].float())
    with pytest.raises(TypeError):
        call(bad)
    with pytest.raises(ValueError):
        call(dict(x, vp=x["vp"][:, :, :8].contiguous()))
    with pytest.raises(ValueError):
        call(dict(x, kp=x["kp"].transpose(1, 2)))
    with pytest.raises(TypeError):
        call(dict(x, lens=x["lens"].long()))
    with pytest.raises(g.GDN2Error):
        call(x, window=-1)
    with pytest.raises(g.GDN2Error):
        call(dict(x, q=x["q"][:, :, :3].contiguous()))
    with pytest.raises(g.GDN2Error):
        call(x, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
