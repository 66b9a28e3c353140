"""Attention over the paged cache for every head size and pair of widths, and the
norm of its error where a length is split over warps and CTAs (tests/kv_checks.py)."""
import numpy as np
import pytest
import torch

from tests import kv_checks as C
from tests.test_gpu_kv_paged import BF16, F16, check_attention, problem, q, values  # noqa: F401
from tests.test_gpu_kv_wide import attend

pytestmark = pytest.mark.gpu
BITS = [2, 3, 4, 5, 6, 8]


@pytest.mark.parametrize("vb", BITS)
@pytest.mark.parametrize("kb", BITS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attend_every_pair_of_widths(q, D, kb, vb):  # noqa: F811
    rng = np.random.default_rng(1000 * D + 10 * kb + vb)
    lens, news, heads, G = [331, 70, 33, 1], [1, 3, 1, 1], 2, 4
    s = problem(rng, lens, news, heads, D, kb, vb, 32, fill="none")
    C.centred(rng, s, heads)
    qs = values(rng, (6, heads * G, D), F16, spread=0.2)
    scale = 0.5 * D ** -0.5
    out, lse = attend(q, s, heads, G, qs, F16, scale)
    check_attention(out, lse, s.attend(qs, heads, scale), F16, D, 331)
    assert C.output_excess(out, C.attend_terms(s, qs, heads, scale), torch.finfo(F16).eps, D, 331, 22) <= 1


SPLIT = [
    # lens, kv heads, group, D, kb, vb, page, window, dtype, chain
    ([20011], 1, 8, 128, 4, 4, 256, 0, F16, 64),                  # one length over the whole GPU
    ([20011], 1, 8, 256, 8, 8, 256, 0, F16, 64),
    ([9000], 2, 3, 256, 4, 4, 64, 0, BF16, 64),
    ([15000, 7], 1, 8, 64, 3, 6, 128, 0, BF16, 64),
    ([3000, 2500, 1, 700], 2, 4, 128, 8, 8, 64, 0, F16, 190),     # items of some warps each
    ([4000, 900], 2, 8, 128, 6, 4, 64, 700, F16, 48),
]


@pytest.mark.parametrize("case", range(len(SPLIT)))
def test_no_piece_of_a_split_length_is_lost(q, case):  # noqa: F811
    lens, heads, G, D, kb, vb, page, window, dtype, chain = SPLIT[case]
    rng = np.random.default_rng(300 + case)
    s = problem(rng, lens, [1] * len(lens), heads, D, kb, vb, page, fill="none")
    C.centred(rng, s, heads)
    qs = values(rng, (len(lens), heads * G, D), dtype, spread=0.1)
    scale = 0.2 * D ** -0.5
    out, lse = attend(q, s, heads, G, qs, dtype, scale, window)
    check_attention(out, lse, s.attend(qs, heads, scale, window), dtype, D, max(lens))
    r = C.attend_terms(s, qs, heads, scale, window)
    assert C.output_excess(out, r, torch.finfo(dtype).eps, D, max(lens), chain) <= 1


@pytest.mark.parametrize("D,vb", [(64, 8), (128, 4), (256, 3)])
def test_weights_are_rounded_once(q, D, vb):  # noqa: F811
    """The mean square of the error is that of one fp16 rounding of weight times scale, not of two."""
    rng = np.random.default_rng(D)
    lens, heads, G = [1500, 1200, 900, 1100], 4, 4
    s = problem(rng, lens, [1] * 4, heads, D, 8, vb, 64, fill="none")
    C.centred(rng, s, heads)
    qs = values(rng, (4, heads * G, D), F16, spread=0.1)
    scale = 0.3 * D ** -0.5
    out, _ = attend(q, s, heads, G, qs, F16, scale)
    assert C.rounding_share(out, C.attend_terms(s, qs, heads, scale)) < 0.75
