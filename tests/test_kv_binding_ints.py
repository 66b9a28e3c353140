"""Whole numbers that do not fit the C interface's 32 bits are refused by the
binding of the paged KV cache; they would be cut to their low 32 bits."""
import ctypes
from types import SimpleNamespace

import pytest
import torch

import mixed_bitwidth_weight_b200 as q

WRAP = 1 << 32


@pytest.mark.parametrize("at", range(5))
@pytest.mark.parametrize("by", [WRAP, -WRAP])
def test_page_geometry(at, by):
    good = [2, 128, 4, 4, 64]
    assert q.qgemm_kv_page_words(*good) > 0
    bad = list(good)
    bad[at] += by
    with pytest.raises(ValueError):
        q.qgemm_kv_page_words(*bad)
    with pytest.raises(ValueError):
        q.KVCache.zeros(1, bad[4], bad[0], bad[1], bad[2], bad[3], device="cpu")


def test_workspace_heads():
    c = q._CacheStruct(0x7f0000000000, 4, 64, 2, 128, 4, 4)
    with pytest.raises(ValueError):
        q.kv_workspace(SimpleNamespace(_ref=ctypes.byref(c), kv_heads=2, device_index=0), WRAP + 8)


@pytest.mark.gpu
def test_window_and_rows():
    cache = q.KVCache.zeros(2, 32, 2, 64, 4, 4)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    batch = q.KVBatch(i32([[0, 1]]), i32([40]), i32([0, 1]))
    x = torch.zeros(1, 4, 64, dtype=torch.float16, device="cuda")
    ws = q.kv_workspace(cache, 4)
    for window in (WRAP + 5, WRAP, 1 << 31, -WRAP):
        with pytest.raises(ValueError):
            q.qgemm_kv_attend(x, cache, batch, torch.empty_like(x), ws, window=window)
    k = x[:, :2].expand(WRAP + 1, 2, 64)
    with pytest.raises(ValueError):
        q.qgemm_kv_append(k, k, cache, batch)
    q.qgemm_kv_attend(x, cache, batch, torch.empty_like(x), ws, window=(1 << 31) - 1)
    torch.cuda.synchronize()
    assert q.qgemm_device_error(clear=True) == 0
