"""The paged cache with infinities and NaN on the GPU: what append stores for them,
and what attention makes of a visible token that holds them."""
import numpy as np
import pytest
import torch

from tests import kv_checks as C
from tests import kv_reference as R
from tests.test_gpu_kv_paged import BF16, F16, check_attention, i32, problem, q, to_gpu, values  # noqa: F401
from tests.test_kv_checks import not_numbers

pytestmark = pytest.mark.gpu
BITS = [2, 3, 4, 5, 6, 8]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("b", BITS)
def test_append_stores_the_array_quantisers_codes(q, D, b):  # noqa: F811
    """Codes and scales of qgemm_kv_quantize bit for bit, infinities and NaN among the values."""
    rng = np.random.default_rng(10 * D + b)
    heads, n = 2, 40
    s = problem(rng, [n], [n], heads, D, b, b, 64)
    cache, batch = to_gpu(q, s, heads)
    k, v = (not_numbers(rng, n * heads, D).reshape(n, heads, D) for _ in range(2))
    kd, vd = torch.as_tensor(k).cuda(), torch.as_tensor(v).cuda()
    q.qgemm_kv_append(kd, vd, cache, batch)
    s.append(k, v)
    assert np.array_equal(cache.pages.view(torch.uint8).cpu().numpy(), s.pages)
    codes = torch.empty(n, heads, D // 32, b, dtype=torch.int32, device="cuda")
    scales = torch.empty(n, heads, D // 32, dtype=F16, device="cuda")
    for x in (k, v):
        q.qgemm_kv_quantize(torch.as_tensor(x).cuda(), b, codes, scales)
        words = codes.cpu().numpy().view(np.uint8).reshape(n * heads, D // 32, 4 * b)
        got = np.unpackbits(words, axis=-1, bitorder="little").reshape(n * heads, D, b)
        want, want_s = R.codes_of(x.reshape(-1, D), b)
        assert np.array_equal((got * (1 << np.arange(b))).sum(-1), want)
        assert np.array_equal(scales.cpu().view(torch.int16).numpy().view(np.uint16).reshape(want_s.shape), want_s)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("b", BITS)
def test_append_of_sums_that_overflow(q, D, b):  # noqa: F811
    """Finite bf16 vectors whose rotation overflows: NaN elements take the zero point, their neighbours' codes stand."""
    rng = np.random.default_rng(20 * D + b)
    heads, n = 2, 19
    s = problem(rng, [n], [n], heads, D, b, b, 32)
    cache, batch = to_gpu(q, s, heads)
    k, v = (C.overflowing(rng, n * heads, D).reshape(n, heads, D) for _ in range(2))
    k[3], v[5] = rng.integers(-8, 9, (heads, D)), rng.integers(-8, 9, (heads, D))      # ordinary tokens between them
    q.qgemm_kv_append(*(torch.as_tensor(x).to(BF16).cuda() for x in (k, v)), cache, batch)
    for x, key in ((k, True), (v, False)):
        codes, scales = C.quantised(x.reshape(-1, D), b)
        for i in range(n):
            p, tile, slot = s.place(0, i)
            for h in range(heads):
                R.put_token(s.pages[p, h, tile], slot, codes[i * heads + h], scales[i * heads + h], D, b, b, key)
    assert np.array_equal(cache.pages.view(torch.uint8).cpu().numpy(), s.pages)


def spoil(s, seq, pos, key, scale):
    """Give a token an infinite or NaN scale in every head and group, codes at the zero point as append leaves them."""
    p, tile, slot = s.place(seq, pos)
    b = s.kb if key else s.vb
    for h in range(s.pages.shape[1]):
        R.put_token(s.pages[p, h, tile], slot, np.full(s.D, 1 << (b - 1)), np.full(s.D // 32, scale, np.uint16), s.D,
                    s.kb, s.vb, key)


@pytest.mark.parametrize("D,kb,vb", [(64, 4, 4), (64, 8, 8), (64, 6, 3), (128, 4, 4), (128, 3, 5), (256, 5, 3), (256, 8, 4)])
def test_rows_that_see_an_infinite_key_are_nan(q, D, kb, vb):  # noqa: F811
    """k' of an infinite scale is H (0 x inf) / D = NaN: whatever sign the rounding of its zero sums has, no row that
    sees the token is finite, and rows that do not see it are as without it."""
    rng = np.random.default_rng(7 * D + kb)
    heads, G = 2, 8
    lens, news, bad = [101, 99, 200, 64], [2, 1, 3, 1], [(0, 10), (1, 98), (2, 198)]
    s = problem(rng, lens, news, heads, D, kb, vb, 64)
    for seq, pos in bad:
        spoil(s, seq, pos, True, 0x7c00)
    cache, batch = to_gpu(q, s, heads)
    qs = values(rng, (7, heads * G, D), F16)
    out, lse = torch.empty(7, heads * G, D, dtype=F16, device="cuda"), torch.empty(7, heads * G, device="cuda")
    q.qgemm_kv_attend(torch.as_tensor(qs).to(F16).cuda(), cache, batch, out, q.kv_workspace(cache, heads * G), lse=lse)
    sees = np.array([True, True, True, False, True, True, False])
    assert torch.isnan(out[torch.as_tensor(sees)]).all() and torch.isnan(lse[torch.as_tensor(sees)]).all()
    with np.errstate(invalid="ignore"):
        ref = s.attend(qs, heads, D ** -0.5)
    keep = ~sees
    check_attention(out.double().cpu().numpy()[keep], lse.double().cpu().numpy()[keep], tuple(r[keep] for r in ref), F16,
                    D, 200)


def test_an_appended_infinity_reaches_the_rows_that_see_it(q):  # noqa: F811
    """Append and attend together: one element of one head's key is infinite."""
    rng = np.random.default_rng(6)
    heads, G, D, n = 3, 8, 64, 40
    cache = q.KVCache.zeros(4, 32, heads, D, 4, 4)
    k, v = (torch.as_tensor(values(rng, (n, heads, D), F16)).to(F16).cuda() for _ in range(2))
    k[20, 1, 7] = -float("inf")
    table, lens = i32([[3, 1]]), i32([n])
    q.qgemm_kv_append(k, v, cache, q.KVBatch(table, lens, i32([0, n])))
    qs = torch.as_tensor(values(rng, (n, heads * G, D), F16)).to(F16).cuda()
    out, lse = torch.empty_like(qs), torch.empty(n, heads * G, device="cuda")
    q.qgemm_kv_attend(qs, cache, q.KVBatch(table, lens, i32([0, n])), out, q.kv_workspace(cache, heads * G), lse=lse)
    nan = torch.isnan(out)
    assert nan[20:, G:2 * G].all() and torch.isnan(lse[20:, G:2 * G]).all()
    nan[20:, G:2 * G] = False
    assert not nan.any() and torch.isfinite(lse[:20]).all()


@pytest.mark.parametrize("D,b", [(64, 4), (128, 4), (128, 8), (128, 5), (256, 3)])
@pytest.mark.parametrize("scale", [0x7e00, 0x7c00])
def test_a_vanished_weight_does_not_hide_a_value_that_is_no_number(q, D, b, scale):  # noqa: F811
    """A visible token whose weight is below fp32's range still makes its rows NaN (0 x NaN), in tiles seen whole and
    in those at the row's end alike; a token that no row sees does not."""
    rng = np.random.default_rng(D + b)
    heads, G = 2, 8
    lens, news = [100, 100, 100, 100], [1, 1, 1, 2]
    s = problem(rng, lens, news, heads, D, b, b, 64)
    spoil(s, 0, 40, False, scale)            # a tile seen whole
    spoil(s, 1, 97, False, scale)            # the tile of the row's end
    spoil(s, 3, 99, False, scale)            # the second of two rows sees it
    cache, batch = to_gpu(q, s, heads)
    qs = values(rng, (5, heads * G, D), F16)
    out, lse = torch.empty(5, heads * G, D, dtype=F16, device="cuda"), torch.empty(5, heads * G, device="cuda")
    factor = 60.0                            # scores hundreds apart: all weights but a few are zero
    q.qgemm_kv_attend(torch.as_tensor(qs).to(F16).cuda(), cache, batch, out, q.kv_workspace(cache, heads * G),
                      scale=factor, lse=lse)
    nan = torch.isnan(out).all(-1).cpu().numpy()
    assert nan[[0, 1, 4]].all()
    assert torch.isfinite(out[[2, 3]]).all() and torch.isfinite(lse[[2, 3]]).all()


@pytest.mark.parametrize("D,b", [(64, 8), (128, 8), (256, 8)])
@pytest.mark.parametrize("scale", [0x7c00, 0x7bff])
def test_hidden_values_cost_the_visible_ones_no_bits(q, D, b, scale):  # noqa: F811
    """Small values next to one of infinite or largest scale, in the same tile, that the window hides: the weights keep
    the bits that the small ones need. An infinite one that only the last of three rows sees spoils that row alone."""
    rng = np.random.default_rng(D + scale)
    heads, G = 2, 4
    lens, news, window = [200, 150, 93], [1, 1, 3], 40
    s = problem(rng, lens, news, heads, D, b, b, 64, fill="none")
    C.centred(rng, s, heads)
    sv = R.parts(D, b, b)[3]
    part = s.pages[..., sv:sv + 2 * D].view(np.float16)
    part[...] = (part.astype(np.float64) * 2.0 ** -9).astype(np.float16)
    spoil(s, 1, 109, False, scale)           # the row at 149 sees 110 on
    spoil(s, 2, 92, False, 0x7c00)           # the last row alone
    spoil(s, 2, 33, False, scale)            # before every row's window
    spoil(s, 0, 159, False, scale)           # the row at 199 sees 160 on
    cache, batch = to_gpu(q, s, heads)
    qs = values(rng, (5, heads * G, D), F16, spread=0.1)
    out, lse = torch.empty(5, heads * G, D, dtype=F16, device="cuda"), torch.empty(5, heads * G, device="cuda")
    factor = 0.2 * D ** -0.5
    q.qgemm_kv_attend(torch.as_tensor(qs).to(F16).cuda(), cache, batch, out, q.kv_workspace(cache, heads * G),
                      scale=factor, window=window, lse=lse)
    assert not torch.isfinite(out[4]).any()
    with np.errstate(invalid="ignore"):
        r = C.attend_terms(s, qs, heads, factor, window)
    keep = slice(0, 4)
    r = {k: v[keep] for k, v in r.items()}
    got = out.double().cpu().numpy()[keep]
    # scales of 2^-15 count as 2^-13, so the largest product may be 2^8: twice the bound's share of small ones
    assert C.output_excess(got, r, torch.finfo(F16).eps, D, 2 * window, 8) <= 1
