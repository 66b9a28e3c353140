"""The paged cache with infinities and NaN on the GPU: what append stores for them."""
import numpy as np
import pytest
import torch

from tests import kv_checks as C
from tests import kv_reference as R
from tests.test_gpu_kv_paged import BF16, F16, problem, q, to_gpu  # noqa: F401
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
