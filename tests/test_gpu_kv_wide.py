"""Attention over the widest records of the paged cache: 8-bit keys and values of 256
dims, 17408 bytes for 32 tokens of a head."""
import numpy as np
import pytest
import torch

from tests.test_gpu_kv_paged import BF16, F16, check_attention, problem, q, to_gpu, values  # noqa: F401

pytestmark = pytest.mark.gpu


def attend(q, s, heads, G, qs, dtype, scale, window=0):  # noqa: F811
    cache, batch = to_gpu(q, s, heads)
    T = int(s.cu[-1])
    out = torch.empty(T, heads * G, s.D, dtype=dtype, device="cuda")
    lse = torch.empty(T, heads * G, device="cuda")
    ws = q.kv_workspace(cache, heads * G)
    qd = torch.as_tensor(qs).to(dtype).cuda()
    q.qgemm_kv_attend(qd, cache, batch, out, ws, scale=scale, window=window, lse=lse)
    first = out.clone(), lse.clone()
    out.fill_(3.0)
    q.qgemm_kv_attend(qd, cache, batch, out, ws, scale=scale, window=window, lse=lse)
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


@pytest.mark.parametrize("lens", [[1], [0, 31, 33, 64], [513], [20011]])
def test_wide_records(q, lens):  # noqa: F811
    rng = np.random.default_rng(sum(lens))
    heads, G, D, news = 1, 7, 256, [min(max(l, 1), 2) for l in lens]
    s = problem(rng, lens, news, heads, D, 8, 8, 64)
    qs = values(rng, (sum(news), heads * G, D), F16, spread=0.2)
    out, lse = attend(q, s, heads, G, qs, F16, 0.5 * D ** -0.5)
    check_attention(out, lse, s.attend(qs, heads, 0.5 * D ** -0.5), F16, D, max(lens))


def test_uneven_batch_of_wide_records(q):  # noqa: F811
    """8-bit keys and values of 256 dims: more sequences than fit one pass, several tokens each, a window."""
    rng = np.random.default_rng(8)
    lens = [int(x) for x in rng.integers(0, 900, 40)]
    news = [int(x) for x in rng.integers(0, 4, 40)]
    heads, G, D = 2, 5, 256
    for fill, window in (("tokens", 0), ("tokens", 130)):
        s = problem(rng, lens, news, heads, D, 8, 8, 64, fill=fill)
        qs = values(rng, (int(s.cu[-1]), heads * G, D), BF16, spread=0.2)
        out, lse = attend(q, s, heads, G, qs, BF16, D ** -0.5, window)
        check_attention(out, lse, s.attend(qs, heads, D ** -0.5, window), BF16, D, 900)
