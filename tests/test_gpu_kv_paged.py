"""The paged KV cache on the GPU against the layout's definition and 64-bit
attention (tests/kv_reference.py): append byte for byte over whole pages,
gather and attend within bounds that count their roundings, at ragged lengths,
empty rows, odd widths, strided operands and unused slots full of NaN."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from tests import kv_reference as R

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
U32 = 2.0 ** -24        # half a step of fp32, relative


@pytest.fixture(scope="module")
def q():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import mixed_bitwidth_weight_b200 as lib
    lib.qgemm_device_error(clear=True)
    yield lib
    torch.cuda.synchronize()
    assert lib.qgemm_device_error(clear=True) == 0


def i32(a):
    return torch.as_tensor(np.asarray(a, dtype=np.int32), device="cuda")


def values(rng, shape, dtype, spread=0.5):
    """fp16-exact values (bf16's grid for bf16), with a spread over heads and one outlier channel."""
    x = rng.standard_normal(shape) * np.exp(spread * rng.standard_normal((1, shape[1], 1)))
    x[..., rng.integers(shape[-1])] *= 10
    x = np.where(np.abs(x) < 2.0 ** -6, 0.0, x)        # every value exact in fp16 and bf16
    return torch.as_tensor(x).to(dtype).double().numpy()


def problem(rng, lens, news, heads, D, kb, vb, page, fill="tokens"):
    """Sequences over random pages; slots behind a sequence's end get NaN scales and any codes."""
    need = [max(1, -(-l // page)) for l in lens]
    P = sum(need) + 2
    rb = R.record_bytes(D, kb, vb)
    pages = rng.integers(0, 256, (P, heads, page // 32, rb), dtype=np.uint8)
    c = R.parts(D, kb, vb)
    for at in (c[1], c[3]):
        s = np.abs(rng.standard_normal((P, heads, page // 32, D))).astype(np.float16) * np.float16(0.7)
        pages[..., at:at + 2 * D] = s.view(np.uint8)
    order = rng.permutation(P)
    table = np.full((len(lens), max(need) + 1), 0x7fffffff, np.int32)     # entries past a sequence are garbage
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    s = R.Sequences(pages, table, lens, news, page, D, kb, vb)
    if fill == "tokens":
        for b, l in enumerate(lens):
            for pos in range(max(l, 0), need[b] * page):
                p, tile, slot = s.place(b, pos)
                for key, off in ((True, c[1]), (False, c[3])):
                    places = R.scale_places(D, key)[slot]
                    pages[p, :, tile, off:off + 2 * D].view(np.uint16)[:, places] = rng.choice([0x7e00, 0x7c00, 0xfe01])
    return s


def to_gpu(q, s, heads):
    pages = torch.as_tensor(s.pages.copy(), device="cuda").view(torch.int32)
    cache = q.KVCache(pages, s.page, heads, s.D, s.kb, s.vb)
    table = i32(s.table)
    return cache, q.KVBatch(table, i32(s.lens), i32(s.cu))


APPEND = [
    # lens, news, heads, D, kb, vb, page, dtype
    ([5, 40, 0, 64, 33], [5, 3, 0, 64, 1], 2, 128, 4, 4, 32, F16),
    ([5, 40, 7, 64, 33], [0, 33, 7, 2, 31], 3, 64, 3, 5, 64, BF16),
    ([1], [1], 1, 256, 2, 8, 32, F16),
    ([100, 2, 0], [70, 2, 1], 2, 256, 5, 3, 128, BF16),          # a padded sequence: one row, no token
    ([65, 3], [65, 5], 2, 64, 8, 2, 32, F16),                     # two rows before position 0
    ([37, 38], [37, 1], 5, 128, 6, 6, 256, BF16),
]


@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append_writes_its_bytes_and_no_others(q, case):
    lens, news, heads, D, kb, vb, page, dtype = APPEND[case]
    rng = np.random.default_rng(case)
    s = problem(rng, lens, news, heads, D, kb, vb, page)
    cache, batch = to_gpu(q, s, heads)
    T = int(s.cu[-1])
    rows = T + 3                                                   # padding rows behind the last sequence
    k, v = (values(rng, (rows, heads, D), dtype) for _ in range(2))
    # strided views of one fused array
    fused = torch.as_tensor(np.concatenate([k, v, k], axis=1)).to(dtype).cuda()
    q.qgemm_kv_append(fused[:, :heads], fused[:, heads:2 * heads], cache, batch)
    s.append(k[:T].astype(np.float16), v[:T].astype(np.float16))
    torch.cuda.synchronize()
    got = cache.pages.view(torch.uint8).cpu().numpy()
    assert np.array_equal(got, s.pages)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kb", [2, 3, 4, 5, 6, 8])
def test_append_and_gather_every_width(q, D, kb):
    """Each width for K with another for V: codes as qgemm_kv_quantize gives, read back as the oracle's values."""
    vb = {2: 6, 3: 2, 4: 8, 5: 4, 6: 3, 8: 5}[kb]
    rng = np.random.default_rng(100 * D + kb)
    heads, n = 3, 45
    s = problem(rng, [n], [n], heads, D, kb, vb, 32)
    cache, batch = to_gpu(q, s, heads)
    for dtype in (F16, BF16):
        k, v = (values(rng, (n, heads, D), dtype) for _ in range(2))
        kd, vd = (torch.as_tensor(a).to(dtype).cuda() for a in (k, v))
        q.qgemm_kv_append(kd, vd, cache, batch)
        ko, vo = torch.empty_like(kd), torch.empty_like(vd)
        q.qgemm_kv_gather(cache, batch, ko, vo)
        for src, got, b, key in ((k, ko, kb, True), (v, vo, vb, False)):
            codes, scales = R.codes_of(src.astype(np.float16).reshape(-1, D), b)
            u = (codes - 2.0 ** (b - 1)) * np.repeat(scales.view(np.float16).astype(np.float64), 32, axis=-1)
            check_rotated_back(got.double().cpu().numpy().reshape(-1, D), u, dtype)


@pytest.mark.parametrize("b", [2, 3, 4, 5, 6, 8])
def test_append_scales_from_zero_to_infinity(q, b):
    """Token i's values lie about 2^(i - 26): scales of 0, subnormal and normal ones, and infinity, byte for byte."""
    rng = np.random.default_rng(40 + b)
    heads, n, D = 2, 42, 128
    s = problem(rng, [n], [n], heads, D, b, b, 64)
    cache, batch = to_gpu(q, s, heads)
    size = 2.0 ** (np.arange(n) - 26.0)[:, None, None]
    k, v = (np.clip(rng.uniform(-1, 1, (n, heads, D)) * size, -65504, 65504).astype(np.float16) for _ in range(2))
    k[7] = 0
    v[-1, :, ::2], v[-1, :, 1::2] = 65504, -65504                  # one rotated value of 128 x 65504, the others 0
    with np.errstate(over="ignore", invalid="ignore"):
        s.append(k, v)
        kinds = R.codes_of(np.concatenate([k, v]).reshape(-1, D), b)[1].view(np.float16).astype(np.float64)
    assert (kinds == 0).any() and ((kinds > 0) & (kinds < 2.0 ** -14)).any() and np.isinf(kinds).any()
    q.qgemm_kv_append(torch.as_tensor(k).cuda(), torch.as_tensor(v).cuda(), cache, batch)
    assert np.array_equal(cache.pages.view(torch.uint8).cpu().numpy(), s.pages)


def check_rotated_back(got, u, dtype):
    """v = H u / D: each of log2 D single-precision stages rounds by at most U32 of sums no larger than
    sum |u|, and the result is rounded once to dtype (fp16's step is 2^-24 below 2^-14)."""
    D = u.shape[-1]
    want = u @ R.hadamard(D) / D
    slack = np.abs(u).sum(-1, keepdims=True) / D * math.log2(D) * U32 * 1.01
    tol = np.abs(want) * torch.finfo(dtype).eps / 2 * 1.01 + slack * 1.01 + 2.0 ** -25
    assert (np.abs(got - want) <= tol).all()


def test_append_matches_the_array_quantiser(q):
    """The same vectors through qgemm_kv_quantize give the same codes and scales (128 dims, 4 bits)."""
    rng = np.random.default_rng(5)
    k = values(rng, (64, 4, 128), F16)
    kd = torch.as_tensor(k).to(F16).cuda()
    cache = q.KVCache.zeros(2, 32, 4, 128, 4, 4)
    batch = q.KVBatch(i32([[1, 0]]), i32([64]), i32([0, 64]))
    q.qgemm_kv_append(kd, kd, cache, batch)
    back, arr = torch.empty_like(kd), torch.empty_like(kd)
    q.qgemm_kv_gather(cache, batch, torch.empty_like(kd), back)
    codes = torch.empty(64, 4, 4, 4, dtype=torch.int32, device="cuda")
    scales = torch.empty(64, 4, 4, dtype=F16, device="cuda")
    q.qgemm_kv_quantize(kd, 4, codes, scales)
    q.qgemm_kv_dequantize(codes, scales, 4, arr)
    assert (back - arr).abs().max().item() <= 2.0 ** -10 * arr.abs().max().item()


GATHER = [
    ([5, 40, 0, 64, 33], [5, 3, 0, 64, 1], 2, 128, 4, 4, 32, F16),
    ([200, 1, 0], [200, 1, 2], 3, 64, 3, 6, 64, BF16),
    ([129, 31], [100, 31], 1, 256, 8, 2, 128, F16),
    ([1000], [1000], 2, 128, 5, 3, 256, BF16),
]


@pytest.mark.parametrize("case", range(len(GATHER)))
def test_gather(q, case):
    lens, news, heads, D, kb, vb, page, dtype = GATHER[case]
    rng = np.random.default_rng(50 + case)
    s = problem(rng, lens, news, heads, D, kb, vb, page)
    cache, batch = to_gpu(q, s, heads)
    T = int(s.cu[-1])
    # written into strided views: [heads, rows, D] seen as [rows, heads, D]; padding rows keep what they hold
    outs = [torch.full((heads, T + 2, D), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    q.qgemm_kv_gather(cache, batch, outs[0].transpose(0, 1), outs[1].transpose(0, 1))
    torch.cuda.synchronize()
    for o, key in zip(outs, (True, False)):
        got = o.double().cpu().numpy()
        assert (got[:, T:] == 7.0).all()
        for b, (l, n) in enumerate(zip(lens, news)):
            skip = max(0, n - l)
            assert (got[:, s.cu[b]:s.cu[b] + skip] == 7.0).all()
            for h in range(heads):
                u = s.context(b, h, key)[l - n + skip:]
                check_rotated_back(got[h, s.cu[b] + skip:s.cu[b + 1]], u, dtype)


def check_attention(out, lse, ref, dtype, D, seen):
    """Bounds, with m = mass (sum of p |u_v| / D) and c = the largest sum of |terms| of a score:
    - a score: the query's two fp16 parts drop at most 2^-22 of each term, single-precision sums of D terms,
      group sums and the rotation another (D + 32) U32: ds = c (2^-22 + (D + 32) U32);
    - a weight: exp's relative error 2^-21 next to the score's, one rounding to fp16 (2^-11) and one of its
      product with the scale (2^-11): the numerator is off by (2^-10 + 2^-21 + ds + 2^-20) m, the sum of
      weights (never rounded) by 2^-21 + ds, so out by (2^-10 + 2 ds + 2^-18) m in all;
    - sums over `seen` tokens in single precision: seen U32 m at the very most, and matrix instructions keep
      two bits less than fp32's rounding: 4 seen U32 m;
    - weights below 2^-25 of the largest may vanish: seen 2^-25 m... counted in the same term;
    - out is rounded once."""
    o, e, mass, score = ref
    ds = score * (2.0 ** -22 + (D + 32) * U32) + 1e-30
    tol = mass * (2.0 ** -10 + 2 * ds + 2.0 ** -18 + 8 * seen * U32)
    tol = tol[..., None] * 1.01 + np.abs(o) * torch.finfo(dtype).eps / 2 * 1.01 + 2.0 ** -25
    assert np.isfinite(out).all()
    assert (np.abs(out - o) <= tol).all(), float((np.abs(out - o) / tol).max())
    if lse is not None:
        empty = np.isneginf(e)
        assert np.array_equal(np.isneginf(lse), empty)
        le = np.where(empty, 0, np.abs(np.where(empty, 0, lse) - np.where(empty, 0, e)))
        ltol = ds + 2.0 ** -20 + seen * U32 + 4 * U32 * np.abs(np.where(empty, 0, e))
        assert (le <= ltol).all(), float((le / ltol).max())


ATTEND = [
    # lens, news, kv heads, group, D, kb, vb, page, window, dtype
    ([1], [1], 1, 1, 128, 4, 4, 32, 0, F16),
    ([0, 1, 31, 32, 33, 63, 64, 65, 300], [1] * 9, 2, 8, 128, 4, 4, 64, 0, BF16),
    ([0, 0, 2, 40], [0, 2, 5, 3], 2, 3, 64, 3, 2, 32, 0, F16),
    ([700, 5, 129], [5, 5, 1], 1, 6, 256, 5, 3, 128, 0, BF16),
    ([513, 40], [1, 1], 3, 12, 64, 8, 8, 256, 0, F16),
    ([513, 40, 1200], [2, 8, 1], 2, 8, 128, 6, 5, 64, 100, F16),
    ([513, 64, 3], [3, 1, 3], 2, 4, 128, 2, 6, 32, 1, BF16),
    ([2000], [1], 2, 16, 128, 8, 4, 64, 33, F16),
    ([3000], [1], 1, 7, 256, 4, 8, 64, 0, F16),
    ([97, 97], [97, 50], 2, 2, 64, 4, 4, 32, 0, F16),             # whole prompts as queries
    ([1500, 1], [1, 1], 1, 40, 128, 3, 3, 64, 0, F16),
]


@pytest.mark.parametrize("case", range(len(ATTEND)))
@pytest.mark.parametrize("with_lse", [True, False])
def test_attend(q, case, with_lse):
    lens, news, heads, G, D, kb, vb, page, window, dtype = ATTEND[case]
    rng = np.random.default_rng(900 + case)
    s = problem(rng, lens, news, heads, D, kb, vb, page)
    cache, batch = to_gpu(q, s, heads)
    T, Hq = int(s.cu[-1]), heads * G
    qs = values(rng, (T + 2, Hq, D), dtype, spread=0.2)
    qd = torch.as_tensor(np.concatenate([qs, qs[:, :1]], axis=1)).to(dtype).cuda()[:, :Hq]
    out = torch.full((T + 2, Hq, D), 5.0, dtype=dtype, device="cuda")
    lse = torch.full((T + 2, Hq), 5.0, device="cuda") if with_lse else None
    ws = q.kv_workspace(cache, Hq)
    scale = 0.6 / math.sqrt(D)
    q.qgemm_kv_attend(qd, cache, batch, out, ws, scale=scale, window=window, lse=lse)
    torch.cuda.synchronize()
    assert int(ws.sum()) >= 0
    assert (out[T:] == 5.0).all() and (lse is None or (lse[T:] == 5.0).all())
    ref = s.attend(qs[:T], heads, scale, window)
    check_attention(out[:T].double().cpu().numpy(), None if lse is None else lse[:T].double().cpu().numpy(), ref, dtype,
                    D, max(lens))


@pytest.mark.parametrize("D,kb,vb", [(64, 4, 4), (128, 3, 8), (256, 8, 2)])
def test_attend_long_uneven_batch(q, D, kb, vb):
    """More work than one pass of the GPU's warps holds: many sequences, several pages each, every length."""
    rng = np.random.default_rng(D)
    lens = [int(x) for x in rng.integers(0, 900, 40)]
    news = [int(x) for x in rng.integers(0, 4, 40)]
    heads, G = 2, 5
    s = problem(rng, lens, news, heads, D, kb, vb, 64)
    cache, batch = to_gpu(q, s, heads)
    T = int(s.cu[-1])
    qs = values(rng, (T, heads * G, D), F16, spread=0.2)
    out = torch.empty(T, heads * G, D, dtype=F16, device="cuda")
    lse = torch.empty(T, heads * G, device="cuda")
    ws = q.kv_workspace(cache, heads * G)
    qd = torch.as_tensor(qs).to(F16).cuda()
    ref = s.attend(qs, heads, D ** -0.5)
    firsts = None
    for _ in range(3):                                             # the workspace comes back clean, results repeat
        out.fill_(3.0)
        q.qgemm_kv_attend(qd, cache, batch, out, ws, lse=lse)
        check_attention(out.double().cpu().numpy(), lse.double().cpu().numpy(), ref, F16, D, max(lens))
        if firsts is None:
            firsts = out.clone(), lse.clone()
        assert torch.equal(out, firsts[0]) and torch.equal(lse, firsts[1])


def test_long_sequence_split(q):
    """One long sequence, so that its length is split over the whole GPU and joined."""
    rng = np.random.default_rng(77)
    heads, G, D = 1, 8, 128
    s = problem(rng, [20011], [1], heads, D, 4, 4, 256)
    cache, batch = to_gpu(q, s, heads)
    qs = values(rng, (1, G, D), BF16, spread=0.1)
    out = torch.empty(1, G, D, dtype=BF16, device="cuda")
    lse = torch.empty(1, G, device="cuda")
    ws = q.kv_workspace(cache, G)
    for scale in (D ** -0.5, 0.0, -0.05, 2.0):
        q.qgemm_kv_attend(torch.as_tensor(qs).to(BF16).cuda(), cache, batch, out, ws, scale=scale, lse=lse)
        ref = s.attend(qs, heads, scale)
        check_attention(out.double().cpu().numpy(), lse.double().cpu().numpy(), ref, BF16, D, 20011)


def test_many_short_and_empty_sequences(q):
    """More sequences than a CTA has threads, most of them without new rows, some without tokens."""
    rng = np.random.default_rng(21)
    B, heads, G, D = 900, 2, 3, 64
    lens = [int(x) for x in rng.integers(0, 50, B)]
    news = [int(x) for x in (rng.random(B) < 0.15) * rng.integers(1, 3, B)]
    s = problem(rng, lens, news, heads, D, 4, 4, 32)
    cache, batch = to_gpu(q, s, heads)
    T = int(s.cu[-1])
    k, v = (values(rng, (T, heads, D), F16) for _ in range(2))
    q.qgemm_kv_append(*(torch.as_tensor(a).to(F16).cuda() for a in (k, v)), cache, batch)
    s.append(k.astype(np.float16), v.astype(np.float16))
    assert np.array_equal(cache.pages.view(torch.uint8).cpu().numpy(), s.pages)
    qs = values(rng, (T, heads * G, D), F16)
    out, lse = torch.empty(T, heads * G, D, dtype=F16, device="cuda"), torch.empty(T, heads * G, device="cuda")
    q.qgemm_kv_attend(torch.as_tensor(qs).to(F16).cuda(), cache, batch, out, q.kv_workspace(cache, heads * G), lse=lse)
    check_attention(out.double().cpu().numpy(), lse.double().cpu().numpy(), s.attend(qs, heads, D ** -0.5), F16, D, 50)
    ko, vo = torch.empty(T, heads, D, dtype=F16, device="cuda"), torch.empty(T, heads, D, dtype=F16, device="cuda")
    q.qgemm_kv_gather(cache, batch, ko, vo)
    for b in range(B):
        for i in range(max(0, news[b] - lens[b]), news[b]):
            u = s.context(b, 1, True)[lens[b] - news[b] + i]
            check_rotated_back(ko[s.cu[b] + i, 1].double().cpu().numpy()[None], u[None], F16)


def test_pages_past_four_gigabytes(q):
    """Offsets in the pool beyond 32 bits: a sequence's pages at its end."""
    rng = np.random.default_rng(22)
    heads, G, D, page, n = 8, 4, 128, 512, 1100
    words = q.qgemm_kv_page_words(heads, D, 8, 8, page)
    P = (5 << 30) // (4 * words)
    cache = q.KVCache(torch.zeros(P, words, dtype=torch.int32, device="cuda"), page, heads, D, 8, 8)
    batch = q.KVBatch(i32([[P - 1, 0, P - 2]]), i32([n]), i32([0, n]))
    k, v = (torch.as_tensor(values(rng, (n, heads, D), F16)).to(F16).cuda() for _ in range(2))
    q.qgemm_kv_append(k, v, cache, batch)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    q.qgemm_kv_gather(cache, batch, ko, vo)
    # 8 bits: within half a step of the group's scale in the rotated domain, sqrt(D) of them at most back
    for x, y in ((k, ko), (v, vo)):
        err = (x.double() - y.double()).norm(dim=-1)
        step = x.double().norm(dim=-1) * math.sqrt(D) / 127     # a scale is max |u| / 127 <= |H x| / 127
        assert (err <= step * math.sqrt(D) / 2 / math.sqrt(D) * 1.05 + 1e-3).all()
    small = q.KVCache.zeros(3, page, heads, D, 8, 8)            # the same tokens near the start
    near = q.KVBatch(i32([[2, 0, 1]]), i32([n]), i32([0, n]))
    q.qgemm_kv_append(k, v, small, near)
    qd = torch.as_tensor(values(rng, (1, heads * G, D), F16)).to(F16).cuda()
    outs = []
    for c, table in ((cache, [[P - 1, 0, P - 2]]), (small, [[2, 0, 1]])):
        o = torch.empty(1, heads * G, D, dtype=F16, device="cuda")
        q.qgemm_kv_attend(qd, c, q.KVBatch(i32(table), i32([n]), i32([0, 1])), o, q.kv_workspace(c, heads * G))
        outs.append(o)
    assert torch.equal(*outs)


def test_strided_and_expanded_operands(q):
    """out as [heads, rows, D] seen from the side, one query expanded over all rows, a large page."""
    rng = np.random.default_rng(23)
    heads, G, D, page = 2, 4, 128, 1024
    lens, news = [1500, 70], [3, 2]
    s = problem(rng, lens, news, heads, D, 4, 4, page)
    cache, batch = to_gpu(q, s, heads)
    qs = values(rng, (1, heads * G, D), BF16)
    qd = torch.as_tensor(qs).to(BF16).cuda().expand(5, -1, -1)
    out = torch.empty(heads * G, 5, D, dtype=BF16, device="cuda")
    lse = torch.empty(5, heads * G, device="cuda")
    q.qgemm_kv_attend(qd, cache, batch, out.transpose(0, 1), q.kv_workspace(cache, heads * G), lse=lse,
                      window=(1 << 31) - 1)
    ref = s.attend(np.repeat(qs, 5, axis=0), heads, D ** -0.5)
    check_attention(out.transpose(0, 1).double().cpu().numpy(), lse.double().cpu().numpy(), ref, BF16, D, 1500)


def test_tiny_and_huge_values(q):
    """Values near the ends of the types' ranges: scales of V far below and above 1, scores that differ by a lot."""
    rng = np.random.default_rng(24)
    heads, G, D = 2, 8, 128
    for exponent in (-13, -6, 8):
        s = problem(rng, [300, 33], [1, 1], heads, D, 4, 4, 64)
        c = R.parts(D, 4, 4)
        sc = s.pages[..., c[3]:c[3] + 2 * D].view(np.float16)
        finite = np.isfinite(sc)
        sc[finite] = (sc[finite].astype(np.float64) * 2.0 ** exponent).astype(np.float16)
        cache, batch = to_gpu(q, s, heads)
        qs = values(rng, (2, heads * G, D), BF16) * 2.0 ** -20
        out, lse = torch.empty(2, heads * G, D, dtype=BF16, device="cuda"), torch.empty(2, heads * G, device="cuda")
        scale = 2.0 ** 20 * D ** -0.5
        q.qgemm_kv_attend(torch.as_tensor(qs).to(BF16).cuda(), cache, batch, out, q.kv_workspace(cache, heads * G),
                          scale=scale, lse=lse)
        o, e, mass, score = s.attend(qs, heads, scale)
        got = out.double().cpu().numpy()
        # weight times scale is fp16: below 2^-14 in steps of 2^-24 next to weights of 2^10 and more, so each of
        # the 300 tokens may add 2^-35 of a code of 8 to the relative terms of check_attention
        extra = 300 * 2.0 ** -35 * 8 * math.sqrt(D)
        ds = score * (2.0 ** -22 + (D + 32) * U32)
        tol = (mass * (2.0 ** -10 + 2 * ds + 2.0 ** -18 + 8 * 300 * U32))[..., None] * 1.01
        tol = tol + np.abs(o) * torch.finfo(BF16).eps / 2 * 1.01 + extra
        assert (np.abs(got - o) <= tol).all(), float((np.abs(got - o) / tol).max())


def test_decoding_loop(q):
    """A prompt written in uneven chunks, then tokens one by one with a captured append + attend that is replayed
    as the lengths grow across pages: every step against 64 bits."""
    rng = np.random.default_rng(11)
    heads, G, D, kb, vb, page = 2, 4, 128, 4, 5, 32
    total = [50, 9]
    s = problem(rng, total, [0, 0], heads, D, kb, vb, page, fill="none")
    cache, _ = to_gpu(q, s, heads)
    table, lens, cu = i32(s.table), i32([0, 0]), i32([0, 0, 0])
    batch = q.KVBatch(table, lens, cu)
    k, v = (values(rng, (59, heads, D), F16) for _ in range(2))
    kd, vd = (torch.as_tensor(a).to(F16).cuda() for a in (k, v))
    ws = q.kv_workspace(cache, heads * G)

    def step(lens_now, news, rows):
        s.lens, s.news = lens_now, news
        s.cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        lens.copy_(i32(lens_now))
        cu.copy_(i32(s.cu))
        s.append(k[rows].astype(np.float16), v[rows].astype(np.float16))

    rows = np.concatenate([np.arange(0, 29), np.arange(50, 52)])
    step([29, 2], [29, 2], rows)
    q.qgemm_kv_append(kd[rows], vd[rows], cache, batch)
    kin, vin = (torch.empty(2, heads, D, dtype=F16, device="cuda") for _ in range(2))
    qin = torch.empty(2, heads * G, D, dtype=F16, device="cuda")
    out, lse = torch.empty_like(qin), torch.empty(2, heads * G, device="cuda")
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, b = 29, 2
    first = True
    while a < 50:
        rows = np.array([a, 50 + b])
        news = [1, 1] if b < 9 else [1, 0]
        rows = rows[:sum(news)]
        a, b = a + 1, b + news[1]
        step([a, b], news, rows)
        n = len(rows)
        kin[:n], vin[:n] = kd[rows], vd[rows]
        qs = values(rng, (2, heads * G, D), F16)
        qin.copy_(torch.as_tensor(qs).to(F16))
        if first:
            torch.cuda.synchronize()
            with torch.cuda.graph(graph, stream=side):
                q.qgemm_kv_append(kin, vin, cache, batch)
                q.qgemm_kv_attend(qin, cache, batch, out, ws, lse=lse)
            first = False
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(cache.pages.view(torch.uint8).cpu().numpy(), s.pages)
        check_attention(out[:n].double().cpu().numpy(), lse[:n].double().cpu().numpy(),
                        s.attend(qs[:n], heads, D ** -0.5), F16, D, 50)
    assert a == 50 and b == 9


FIRST_IN_CAPTURE = """
import torch
import mixed_bitwidth_weight_b200 as q
i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
g = torch.Generator(device="cuda").manual_seed(3)
cache = q.KVCache.zeros(4, 64, 2, 128, 4, 4)
batch = q.KVBatch(i32([[2, 0, 3]]), i32([150]), i32([0, 150]))
one = q.KVBatch(i32([[2, 0, 3]]), i32([150]), i32([0, 1]))
k, v = (torch.randn(150, 2, 128, generator=g, device="cuda").half() for _ in range(2))
x = torch.randn(1, 8, 128, generator=g, device="cuda").half()
out, eager, ws = torch.zeros_like(x), torch.zeros_like(x), q.kv_workspace(cache, 8)
kb, vb = torch.zeros_like(k), torch.zeros_like(v)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    q.qgemm_kv_append(k, v, cache, batch)
    q.qgemm_kv_gather(cache, batch, kb, vb)
    q.qgemm_kv_attend(x, cache, one, out, ws)
graph.replay()
torch.cuda.synchronize()
q.qgemm_kv_attend(x, cache, one, eager, ws)
assert torch.equal(out, eager) and out.abs().sum() > 0
assert (kb - k).abs().max() < 1.0 and (vb - v).abs().max() < 1.0
assert q.qgemm_device_error() == 0
print("captured first")
"""


def test_first_calls_of_a_process_inside_a_capture():
    """No call has to come before a capture: a fresh process's first ones are captured, then replayed."""
    r = subprocess.run([sys.executable, "-c", FIRST_IN_CAPTURE], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


def test_two_streams_with_their_own_workspaces(q):
    rng = np.random.default_rng(12)
    heads, G, D = 2, 8, 128
    s = problem(rng, [3000, 700], [1, 1], heads, D, 4, 4, 64)
    cache, batch = to_gpu(q, s, heads)
    qs = values(rng, (2, heads * G, D), F16)
    qd = torch.as_tensor(qs).to(F16).cuda()
    streams = [torch.cuda.Stream() for _ in range(2)]
    bufs = [(torch.empty_like(qd), torch.empty(2, heads * G, device="cuda"), q.kv_workspace(cache, heads * G))
            for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, (o, l, w) in zip(streams, bufs):
            q.qgemm_kv_attend(qd, cache, batch, o, w, lse=l, stream=st)
    torch.cuda.synchronize()
    ref = s.attend(qs, heads, D ** -0.5)
    for o, l, _ in bufs:
        check_attention(o.double().cpu().numpy(), l.double().cpu().numpy(), ref, F16, D, 3000)


def test_not_a_number_stays_in_its_row(q):
    """A NaN query makes its own row NaN, a NaN scale of a visible token the rows that see it; others are untouched."""
    rng = np.random.default_rng(13)
    heads, G, D = 2, 4, 128
    s = problem(rng, [200, 90], [1, 1], heads, D, 4, 4, 64)
    c = R.parts(D, 4, 4)
    p, tile, slot = s.place(1, 40)
    s.pages[p, 1, tile, c[3]:c[3] + 2 * D].view(np.uint16)[R.scale_places(D, False)[slot]] = 0x7e00
    cache, batch = to_gpu(q, s, heads)
    qs = values(rng, (2, heads * G, D), F16)
    qd = torch.as_tensor(qs).to(F16).cuda()
    qd[0, 2, 5] = float("nan")
    out, lse = torch.empty_like(qd), torch.empty(2, heads * G, device="cuda")
    q.qgemm_kv_attend(qd, cache, batch, out, q.kv_workspace(cache, heads * G), lse=lse)
    o, e = out.double().cpu().numpy(), lse.double().cpu().numpy()
    bad = np.zeros((2, heads * G), bool)
    bad[0, 2] = True
    bad[1, G:] = True
    assert np.isnan(o[bad]).all() and np.isnan(e[0, 2])
    ref = s.attend(qs, heads, D ** -0.5)
    keep = ~bad
    check_attention(o[keep][None], e[keep][None], tuple(r[keep][None] for r in ref), F16, D, 200)
    # a NaN token behind a row's position, or before its window, does not reach it
    s = problem(rng, [200], [3], heads, D, 4, 4, 64)
    for pos, part in ((199, c[3]), (199, c[1]), (150, c[3])):
        p, tile, slot = s.place(0, pos)
        key = part == c[1]
        s.pages[p, :, tile, part:part + 2 * D].view(np.uint16)[:, R.scale_places(D, key)[slot]] = 0x7e00
    cache, batch = to_gpu(q, s, heads)
    qs = values(rng, (3, heads * G, D), F16)
    out, lse = torch.empty(3, heads * G, D, dtype=F16, device="cuda"), torch.empty(3, heads * G, device="cuda")
    q.qgemm_kv_attend(torch.as_tensor(qs).to(F16).cuda(), cache, batch, out, q.kv_workspace(cache, heads * G), lse=lse,
                      window=40)
    with np.errstate(invalid="ignore"):
        ref = s.attend(qs, heads, D ** -0.5, 40)
    check_attention(out[:2].double().cpu().numpy(), lse[:2].double().cpu().numpy(), tuple(r[:2] for r in ref), F16, D,
                    200)
    assert torch.isnan(out[2]).all() and torch.isnan(lse[2]).all()


def test_positions_without_a_page_are_refused(q):
    """A table entry outside the pool: the error word says so, the call neither reads nor writes there, and the
    other sequences' results stand."""
    rng = np.random.default_rng(14)
    heads, G, D, page = 2, 4, 64, 32
    s = problem(rng, [70, 40, 64], [2, 1, 3], heads, D, 4, 4, page, fill="none")
    good = s.table.copy()
    before = s.pages.copy()
    s.table[0, 2] = -1                                             # where sequence 0's new tokens belong
    s.table[2, 0] = len(s.pages)                                   # the first page of sequence 2
    cache, batch = to_gpu(q, s, heads)
    k = values(rng, (6, heads, D), F16)
    kd = torch.as_tensor(k).to(F16).cuda()
    q.qgemm_kv_append(kd, kd, cache, batch)
    assert q.qgemm_device_error(clear=True) == q.DEV_BAD_PAGE
    s.table = good
    s.append(k.astype(np.float16), k.astype(np.float16))
    for pos in (68, 69):                                           # what append left out
        p, tile, slot = s.place(0, pos)
        s.pages[p, :, tile] = before[p, :, tile]
    assert np.array_equal(cache.pages.view(torch.uint8).cpu().numpy(), s.pages)
    qs = values(rng, (6, heads * G, D), F16)
    qd = torch.as_tensor(qs).to(F16).cuda()
    out, lse = torch.empty_like(qd), torch.empty(6, heads * G, device="cuda")
    q.qgemm_kv_attend(qd, cache, batch, out, q.kv_workspace(cache, heads * G), lse=lse)
    assert q.qgemm_device_error(clear=True) == q.DEV_BAD_PAGE
    ref = s.attend(qs, heads, D ** -0.5)
    check_attention(out[2:3].double().cpu().numpy(), lse[2:3].double().cpu().numpy(), tuple(r[2:3] for r in ref), F16, D,
                    70)
    # a sequence longer than its row of the table
    batch = q.KVBatch(i32(s.table[1:2, :1]), i32([40]), i32([0, 1]))
    q.qgemm_kv_append(kd[:1], kd[:1], cache, batch)
    assert q.qgemm_device_error(clear=True) == q.DEV_BAD_PAGE
    ko = torch.full_like(kd[:1], 9.0)
    q.qgemm_kv_gather(cache, batch, ko, ko.clone())
    assert q.qgemm_device_error(clear=True) == q.DEV_BAD_PAGE
    assert (ko == 9.0).all()


def test_no_sequences_or_rows(q):
    cache = q.KVCache.zeros(1, 32, 2, 64, 4, 4)
    empty = q.KVBatch(torch.zeros(0, 3, dtype=torch.int32, device="cuda"), i32([]), i32([0]))
    k = torch.zeros(0, 2, 64, dtype=F16, device="cuda")
    q.qgemm_kv_append(k, k, cache, empty)
    out = torch.full((3, 4, 64), 2.0, dtype=F16, device="cuda")
    q.qgemm_kv_attend(out.clone(), cache, empty, out, q.kv_workspace(cache, 4))
    torch.cuda.synchronize()
    assert (out == 2.0).all()


def test_binding_refusals(q):
    cache = q.KVCache.zeros(2, 32, 2, 64, 4, 4)
    batch = q.KVBatch(i32([[0, 1]]), i32([3]), i32([0, 1]))
    k = torch.zeros(1, 2, 64, dtype=F16, device="cuda")
    ws = q.kv_workspace(cache, 4)
    qq, out = torch.zeros(1, 4, 64, dtype=F16, device="cuda"), torch.zeros(1, 4, 64, dtype=F16, device="cuda")
    for bad in (k[:, :1], k[0], torch.zeros(1, 2, 128, dtype=F16, device="cuda")):
        with pytest.raises(ValueError):
            q.qgemm_kv_append(bad, k, cache, batch)
    with pytest.raises(ValueError):
        q.qgemm_kv_append(k, torch.zeros(2, 2, 64, dtype=F16, device="cuda"), cache, batch)
    with pytest.raises(TypeError):
        q.qgemm_kv_append(k.float(), k.float(), cache, batch)
    with pytest.raises(TypeError):
        q.qgemm_kv_append(k, k.bfloat16(), cache, batch)
    with pytest.raises(TypeError):
        q.qgemm_kv_append(k.cpu(), k.cpu(), cache, batch)
    with pytest.raises(ValueError):
        q.qgemm_kv_append(torch.zeros(1, 2, 128, dtype=F16, device="cuda")[..., ::2], k, cache, batch)
    with pytest.raises(ValueError):
        q.qgemm_kv_attend(qq[:, :3], cache, batch, out[:, :3], ws)
    with pytest.raises(TypeError):
        q.qgemm_kv_attend(qq, cache, batch, out.bfloat16(), ws)
    with pytest.raises(ValueError):
        q.qgemm_kv_attend(qq, cache, batch, torch.zeros(2, 4, 64, dtype=F16, device="cuda"), ws)
    with pytest.raises(ValueError):
        q.qgemm_kv_attend(qq, cache, batch, out, ws, lse=torch.zeros(1, 3, device="cuda"))
    with pytest.raises(q.QGemmError):
        q.qgemm_kv_attend(qq, cache, batch, out, ws[:16 - 8])
    with pytest.raises(q.QGemmError):
        q.qgemm_kv_attend(qq, cache, batch, out, ws, scale=float("inf"))
    with pytest.raises(q.QGemmError):
        q.qgemm_kv_gather(cache, batch, k.expand(1, 2, 64)[:, :1].expand(1, 2, 64), k)
    with pytest.raises(ValueError):
        q.kv_workspace(cache, 3)
    with pytest.raises(TypeError):
        q.KVBatch(i32([[0, 1]]).long(), i32([3]), i32([0, 1]))
    torch.cuda.synchronize()
