"""The paged KV cache in numpy, from the layout's definition in include/qgemm.h:
where each code and scale of a token lies in its record, and attention over
what a record stands for in 64 bits."""
import numpy as np

import oracle

TILE = 32


def record_bytes(D, kb, vb):
    return 4 * D * (kb + vb + 1)


def parts(D, kb, vb):
    """Byte offsets of K codes, K scales, V codes, V scales."""
    return 0, 4 * D * kb, 4 * D * kb + 2 * D, 4 * D * (kb + vb) + 2 * D


def code_bits(D, b, key):
    """[32, D]: first bit of each (token slot, dim)'s code in its code part."""
    t, d = np.arange(TILE)[:, None], np.arange(D)[None, :]
    if key:
        stream, unit, i = 4 * (t % 8) + d % 32 // 8, (t // 8) * (D // 32) + d // 32, d % 8 + 0 * t
        slot = np.array([0, 1, 4, 5, 2, 3, 6, 7])[i] if b >= 5 else i
    else:
        stream = 4 * (d % 32 // 4) + t // 2 % 4
        unit = (2 * (t // 8) + t % 2) * (D // 64) + d // 64
        slot = 4 * (d // 32 % 2) + d % 4 + 0 * t
    bit = unit * 8 * b + slot * b                       # in the stream
    C = next(c for c in (16, 8, 4) if D * b // 16 % c == 0)
    byte = bit // 8
    return ((byte // C * 32 + stream) * C + byte % C) * 8 + bit % 8, C


def scale_places(D, key):
    """[32, D / 32]: index of each (token slot, group)'s scale in its scale part."""
    t, g, G = np.arange(TILE)[:, None], np.arange(D // 32)[None, :], D // 32
    if key:
        return (t % 8 * 4 + t // 8) * G + g
    return ((t // 2 % 4 * G + g) * 4 + t // 8) * 2 + t % 2


def _code_bytes(D, b, key):
    """[32, D] and [32, D]: the byte of a code's first bit and the byte of its
    last one (codes of one unit run through its bytes, which stay in one chunk
    or go on in the stream's next)."""
    first, C = code_bits(D, b, key)
    t, d = np.arange(TILE)[:, None], np.arange(D)[None, :]
    byte = first // 8
    in_chunk = byte % C
    nxt = np.where(in_chunk + 1 < C, byte + 1, byte - in_chunk + 32 * C)
    return byte, nxt, first % 8


def put_token(rec, slot, codes, scales, D, kb, vb, key):
    """Store one token's codes [D] and fp16-bit scales [D / 32] in a record (uint8)."""
    b, (ck, sk, cv, sv) = (kb if key else vb), parts(D, kb, vb)
    lo, hi, sh = _code_bytes(D, b, key)
    at = ck if key else cv
    for d in range(D):
        word = int(rec[at + lo[slot, d]])
        two = sh[slot, d] + b > 8
        if two:
            word |= int(rec[at + hi[slot, d]]) << 8
        word = (word & ~(((1 << b) - 1) << int(sh[slot, d]))) | int(codes[d]) << int(sh[slot, d])
        rec[at + lo[slot, d]] = word & 0xff
        if two:
            rec[at + hi[slot, d]] = word >> 8
    rec[(sk if key else sv):][:2 * D].view(np.uint16)[scale_places(D, key)[slot]] = scales


def record_values(rec, D, kb, vb, key):
    """Rotated values of records [..., bytes] -> float64 [..., 32, D]."""
    b, (ck, sk, cv, sv) = (kb if key else vb), parts(D, kb, vb)
    lo, hi, sh = _code_bytes(D, b, key)
    at = ck if key else cv
    two = sh + b > 8
    hi = np.where(two, hi, lo)
    word = rec[..., at + lo].astype(np.int64) | rec[..., at + hi].astype(np.int64) << 8
    code = (word >> sh) & ((1 << b) - 1)
    so = sk if key else sv
    s = np.ascontiguousarray(rec[..., so:so + 2 * D]).view(np.float16)[..., scale_places(D, key)]
    return (code - 2.0 ** (b - 1)) * np.repeat(s.astype(np.float64), 32, axis=-1)


def hadamard(D):
    i = np.arange(D)
    ones = np.vectorize(lambda v: bin(v).count("1") & 1)
    return 1.0 - 2.0 * ones(i[:, None] & i[None, :])


def codes_of(v, b):
    """The oracle's codes uint8 [n, D] and scales (fp16 bits) [n, D / 32] of fp16 vectors [n, D]."""
    words, scales = oracle.kv_quantize(np.ascontiguousarray(v), b)
    n, D = v.shape
    bits = np.unpackbits(np.ascontiguousarray(words).reshape(n, D // 32, b).view(np.uint8).reshape(n, D // 32, 4 * b),
                         axis=-1, bitorder="little").reshape(n, D, b)
    return (bits * (1 << np.arange(b))).sum(-1).astype(np.uint8), scales


class Sequences:
    """Block table and lengths on the host; pages as uint8 [P, heads, tiles, bytes]."""

    def __init__(self, pages, table, lens, news, page, D, kb, vb):
        self.pages, self.table, self.lens, self.news = pages, table, list(lens), list(news)
        self.page, self.D, self.kb, self.vb = page, D, kb, vb
        self.cu = np.concatenate([[0], np.cumsum(self.news)]).astype(np.int32)

    def place(self, b, pos):
        return self.table[b, pos // self.page], pos % self.page // TILE, pos % TILE

    def append(self, k, v):
        """k, v fp16 [rows, heads, D]: what qgemm_kv_append leaves in the pages."""
        T, H, D = k.shape
        kc, ks = codes_of(k.reshape(T * H, D), self.kb)
        vc, vs = codes_of(v.reshape(T * H, D), self.vb)
        for b, (l, n) in enumerate(zip(self.lens, self.news)):
            for i in range(n):
                pos, row = l - n + i, self.cu[b] + i
                if pos < 0:
                    continue
                p, tile, slot = self.place(b, pos)
                for h in range(H):
                    rec = self.pages[p, h, tile]
                    put_token(rec, slot, kc[row * H + h], ks[row * H + h], D, self.kb, self.vb, True)
                    put_token(rec, slot, vc[row * H + h], vs[row * H + h], D, self.kb, self.vb, False)

    def context(self, b, head, key, length=None):
        """Rotated values of sequence b's first tokens, float64 [length, D]."""
        length = self.lens[b] if length is None else length
        if length <= 0:
            return np.zeros((0, self.D))
        tiles = np.arange(-(-length // TILE))
        per = self.page // TILE
        rec = self.pages[self.table[b, tiles // per], head, tiles % per]
        return record_values(rec, self.D, self.kb, self.vb, key).reshape(-1, self.D)[:length]

    def attend(self, q, heads, scale, window=0):
        """q float64 [rows, q_heads, D] -> out, lse, and per output the bounds
        `mass` = sum_t p_t sum_d |u_v| / D (what relative errors of the weights
        scale with) and `score` = the largest scale / D sum_d |Hq| |u_k|."""
        T, Hq, D = q.shape
        G, H = Hq // heads, hadamard(D)
        out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
        mass, score = np.zeros((T, Hq)), np.zeros((T, Hq))
        for b, (l, n) in enumerate(zip(self.lens, self.news)):
            for h in range(heads):
                k, v = self.context(b, h, True), self.context(b, h, False)
                for i in range(n):
                    pos = l - n + i
                    lo = max(0, pos - window + 1) if window else 0
                    if pos < 0:
                        continue
                    row = self.cu[b] + i
                    hq = slice(h * G, h * G + G)
                    u = q[row, hq] @ H
                    kk, vv = k[lo:pos + 1], v[lo:pos + 1]
                    s = u @ kk.T * (scale / D)
                    m = s.max(-1, keepdims=True)
                    p = np.exp(s - m)
                    tot = p.sum(-1, keepdims=True)
                    out[row, hq] = (p / tot) @ vv @ H / D
                    lse[row, hq] = (m + np.log(tot))[:, 0]
                    mass[row, hq] = (p / tot) @ np.abs(vv).sum(-1) / D
                    score[row, hq] = (np.abs(u) @ np.abs(kk).T).max(-1) * abs(scale) / D
        return out, lse, mass, score
