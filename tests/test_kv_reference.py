"""The paged cache's layout on the CPU: every code and scale of a record has a
place of its own, together they fill the record, and tokens put into a record
come back as the oracle's values."""
import numpy as np
import pytest

from tests import kv_reference as R
import mixed_bitwidth_weight_b200 as q
import oracle

BITS = [2, 3, 4, 5, 6, 8]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("b", BITS)
@pytest.mark.parametrize("key", [True, False])
def test_codes_tile_their_part(D, b, key):
    lo, hi, sh = R._code_bytes(D, b, key)
    used = np.zeros(4 * D * b * 8, int)
    for i in range(b):
        bit = sh + i
        np.add.at(used, np.where(bit < 8, lo, hi) * 8 + bit % 8, 1)
    assert (used == 1).all()
    assert sorted(R.scale_places(D, key).ravel()) == list(range(D))
    # a token's bytes are its own: no byte holds codes of two tokens
    owner = np.full(4 * D * b, -1)
    for t in range(R.TILE):
        mine = np.unique(np.concatenate([lo[t], np.where(sh[t] + b > 8, hi[t], lo[t])]))
        assert (owner[mine] == -1).all()
        owner[mine] = t
    assert (owner >= 0).all()


@pytest.mark.parametrize("D,kb,vb", [(64, 3, 8), (64, 2, 5), (128, 4, 3), (128, 5, 6), (256, 8, 2)])
def test_tokens_come_back(D, kb, vb):
    rng = np.random.default_rng(D + kb)
    v = rng.standard_normal((R.TILE, D)).astype(np.float16)
    rec = np.full(R.record_bytes(D, kb, vb), 0xa5, np.uint8)
    for key, b in ((True, kb), (False, vb)):
        codes, scales = R.codes_of(v, b)
        for t in range(R.TILE):
            R.put_token(rec, t, codes[t], scales[t], D, kb, vb, key)
    for key, b in ((True, kb), (False, vb)):
        x = R.record_values(rec, D, kb, vb, key) @ R.hadamard(D) / D
        words, scales = oracle.kv_quantize(v, b)
        back = oracle.kv_dequantize(words, scales, D, b).view(np.float16)
        assert np.abs(x - back).max() <= np.abs(back).max() * 2.0 ** -10


@pytest.mark.parametrize("D", [64, 128, 256])
def test_page_words(D):
    assert q.qgemm_kv_page_words(3, D, 4, 5, 64) == 3 * 2 * R.record_bytes(D, 4, 5) // 4
    for bad in ((0, D, 4, 4, 64), (1, 96, 4, 4, 64), (1, D, 4, 4, 48), (1, D, 4, 4, 16), (1, D, 4, 4, 8192),
                (1025, D, 4, 4, 64)):
        with pytest.raises(q.QGemmError) as e:
            q.qgemm_kv_page_words(*bad)
        assert e.value.status == -2
    for bits in ((1, 4), (4, 7), (0, 0), (9, 4)):
        with pytest.raises(q.QGemmError) as e:
            q.qgemm_kv_page_words(1, D, *bits, 64)
        assert e.value.status == -3
