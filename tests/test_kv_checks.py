"""The paged cache's checks on the CPU: the quantiser's steps against the oracle for
inputs that are not numbers, whole records, and attention outputs that went wrong
in ways that a bound per element lets pass."""
import numpy as np
import pytest

from tests import kv_checks as C
from tests import kv_reference as R

BITS = [2, 3, 4, 5, 6, 8]


def not_numbers(rng, n, D):
    v = rng.standard_normal((n, D)).astype(np.float16)
    v[0, 3], v[1, D - 1], v[2, 0] = np.inf, -np.inf, np.nan
    v[3, ::7], v[4, 5], v[4, 6] = 65504, np.inf, np.nan
    v[5], v[6] = np.inf, 65504
    return v


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("b", BITS)
def test_quantiser_steps_are_the_oracles(D, b):
    v = not_numbers(np.random.default_rng(D + b), 12, D)
    codes, scales = C.quantised(v.astype(np.float32), b)
    want, want_s = R.codes_of(v, b)
    assert np.array_equal(codes, want) and np.array_equal(scales, want_s)
    assert (codes[[0, 1, 2, 4, 5]] == 1 << (b - 1)).all()           # nothing but zero points


@pytest.mark.parametrize("D", [64, 128, 256])
def test_overflowing_vectors_keep_normal_groups(D):
    v = C.overflowing(np.random.default_rng(D), 5, D)
    u = C.rotated(v).reshape(5, D // 32, 32)
    assert np.isnan(u).any(-1).all() and not np.isinf(u).any()
    codes, scales = C.quantised(v, 4)
    s = scales.view(np.float16).astype(np.float64)
    assert (s >= 2.0 ** -14).all() and np.isfinite(s).all()
    assert (codes.reshape(u.shape)[np.isnan(u)] == 8).all() and (codes.reshape(u.shape)[~np.isnan(u)] != 8).any()


@pytest.mark.parametrize("D,kb,vb", [(64, 3, 8), (64, 2, 5), (128, 4, 3), (128, 5, 6), (256, 8, 2), (256, 6, 4)])
def test_whole_records(D, kb, vb):
    rng = np.random.default_rng(D + kb)
    pages = rng.integers(0, 256, (2, 3, 2, R.record_bytes(D, kb, vb)), dtype=np.uint8)
    for key, b in ((True, kb), (False, vb)):
        codes = rng.integers(0, 1 << b, (2, 3, 2, 32, D), dtype=np.uint8)
        scales = rng.standard_normal((2, 3, 2, 32, D // 32)).astype(np.float16)
        C.put_part(pages, codes, scales, D, kb, vb, key)
        want = (codes - 2.0 ** (b - 1)) * np.repeat(scales.astype(np.float64), 32, axis=-1)
        assert np.array_equal(R.record_values(pages, D, kb, vb, key), want)


def sequences(rng, lens, heads, D, kb, vb, page=64):
    need = [-(-l // page) for l in lens]
    pages = np.zeros((sum(need), heads, page // 32, R.record_bytes(D, kb, vb)), np.uint8)
    table = np.zeros((len(lens), max(need)), np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = np.arange(at, at + n)
        at += n
    s = R.Sequences(pages, table, lens, [1] * len(lens), page, D, kb, vb)
    C.centred(rng, s, heads)
    return s


def rounded(s, q, heads, scale, twice):
    """Attention with weights times scales (and, if `twice`, weights before them) rounded to fp16."""
    T, Hq, D = q.shape
    G, H, out = Hq // heads, R.hadamard(D), np.zeros(q.shape)
    sv = R.parts(D, s.kb, s.vb)[3]
    for b, l in enumerate(s.lens):
        for h in range(heads):
            hq = slice(h * G, h * G + G)
            k, v = s.context(b, h, True), s.context(b, h, False)
            tiles, per = np.arange(-(-l // 32)), s.page // 32
            rec = s.pages[s.table[b, tiles // per], h, tiles % per]
            sc = np.ascontiguousarray(rec[..., sv:sv + 2 * D]).view(np.float16)[..., R.scale_places(D, False)]
            sc = np.repeat(sc.reshape(-1, D // 32)[:l].astype(np.float64), 32, axis=-1)
            x = q[b, hq] @ H @ k.T * (scale / D)
            w = np.exp(x - x.max(-1, keepdims=True)) * 2.0 ** 9
            p = w.astype(np.float16).astype(np.float64) if twice else w
            ws = (p[:, :, None] * sc).astype(np.float16).astype(np.float64)
            out[b, hq] = np.einsum("gtd,td->gd", ws, v / sc) @ H / (D * w.sum(-1, keepdims=True))
    return out.astype(np.float16).astype(np.float64)


def test_wrong_outputs_are_told_from_rounded_ones():
    rng = np.random.default_rng(3)
    lens, heads, G, D = [3000, 2500], 2, 4, 128
    s = sequences(rng, lens, heads, D, 4, 4)
    q = rng.standard_normal((2, heads * G, D))
    args = (heads, 0.3 * D ** -0.5)
    r = C.attend_terms(s, q, *args)
    ref = s.attend(q, *args)
    assert np.allclose(r["out"], ref[0], rtol=1e-12, atol=1e-14) and np.allclose(r["lse"], ref[1], rtol=1e-12)
    measure = lambda out: C.output_excess(out, r, 2.0 ** -10, D, 3000, 188)  # noqa: E731
    once, twice = (rounded(s, q, *args, t) for t in (False, True))
    assert measure(once) < 0.5 and measure(twice) < 1
    assert C.rounding_share(once, r) < 0.75 < C.rounding_share(twice, r)

    def mutant(change):
        m = R.Sequences(s.pages.copy(), s.table, s.lens, s.news, s.page, D, 4, 4)
        change(m.pages, R.parts(D, 4, 4)[2])
        return m.attend(q, *args)[0]

    def lost(pages, v):             # the first 640 tokens of sequence 0 count in the sum of weights alone
        pages[:10, ..., v + 4 * D * 4:] = 0

    def one_tile(pages, v):
        pages[20, :, 1, v + 4 * D * 4:] = 0

    def swapped(pages, v):          # V of pages 3 and 4 in each other's place
        pages[[3, 4], ..., v:] = pages[[4, 3], ..., v:]

    def heads_swapped(pages, v):
        pages[:, [0, 1], :, v:] = pages[:, [1, 0], :, v:]

    for change in (lost, one_tile, swapped, heads_swapped):
        assert measure(mutant(change)) > 1, change.__name__
    small = np.where(np.abs(once) < 0.2 * np.abs(once).max(), 0, once)
    for out in (small, np.zeros_like(once), np.roll(once, 1, axis=-1), once * 1.02):
        assert measure(out) > 1
