"""Sharper checks of the paged KV cache: the quantiser's steps in numpy for every
input (infinities, NaN, sums that overflow), whole records from codes and scales,
and a bound on the norm of an attention output's error that a lost or misplaced
piece of V cannot meet."""
import math

import numpy as np

from tests import kv_reference as R

U32 = 2.0 ** -24        # half a step of fp32, relative
U16 = 2.0 ** -11        # of fp16


def rotated(v):
    """H_D v in single precision, strides 1, 2, ..., D / 2, each sum rounded."""
    u = np.array(v, np.float32)
    D, st = u.shape[-1], 1
    with np.errstate(over="ignore", invalid="ignore"):
        while st < D:
            x = u.reshape(*u.shape[:-1], D // (2 * st), 2, st)
            u = np.stack([x[..., 0, :] + x[..., 1, :], x[..., 0, :] - x[..., 1, :]], axis=-2).reshape(u.shape)
            st *= 2
    return u


def quantised(v, b):
    """Codes uint8 [n, D] and scales (fp16 bits) [n, D / 32] of vectors [n, D] in single precision. What is not a
    number has no size and the zero point's code."""
    u = rotated(v)
    n, D = u.shape
    z = 2 ** (b - 1)
    g = u.reshape(n, D // 32, 32)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        s = (np.where(np.isnan(g), 0, np.abs(g)).max(-1) / np.float32(z - 1)).astype(np.float16)
        s32 = s.astype(np.float32)
        inv = np.where(s32 == 0, np.float32(0), np.float32(1) / s32)
        r = np.rint(g * inv[..., None])
    code = np.where(np.isnan(r), 0, np.clip(r, -z, z - 1)) + z
    return code.reshape(n, D).astype(np.uint8), s.view(np.uint16)


def overflowing(rng, n, D):
    """Finite vectors on bf16's grid [n, D] whose rotation in single precision makes NaN of some elements of every
    group and leaves the others of ordinary size: four elements of 1e38 in each half of a group sum past the
    type's end, the halves' infinities meet as inf - inf in one group and as -inf + inf in the next."""
    x = np.rint(rng.standard_normal((n, D)) * 8) * 0.25
    big = float(np.float32(2.0 ** 126))
    for g in range(D // 32):
        x[:, 32 * g:32 * g + 4] = big
        x[:, 32 * g + 16:32 * g + 20] = big if g % 2 == 0 else -big
    return x


def pack_part(codes, b, key):
    """Codes [..., 32, D] -> the bytes [..., 4 D b] of a record's code part."""
    D = codes.shape[-1]
    lo, hi, sh = R._code_bytes(D, b, key)
    bits = np.zeros(codes.shape[:-2] + (4 * D * b * 8,), np.uint8)
    for i in range(b):
        bit = sh + i
        bits[..., np.where(bit < 8, lo * 8 + bit, hi * 8 + bit - 8)] = codes >> i & 1
    return np.packbits(bits, axis=-1, bitorder="little")


def put_part(pages, codes, scales, D, kb, vb, key):
    """Codes [P, heads, tiles, 32, D] and scales fp16 [P, heads, tiles, 32, D / 32] into the records of pages."""
    ck, sk, cv, sv = R.parts(D, kb, vb)
    b, c, s = (kb, ck, sk) if key else (vb, cv, sv)
    pages[..., c:c + 4 * D * b] = pack_part(codes, b, key)
    part = np.empty(scales.shape[:-2] + (D,), np.float16)
    part[..., R.scale_places(D, key)] = scales
    pages[..., s:s + 2 * D] = part.view(np.uint8)


def centred(rng, s, heads):
    """Zero-mean codes (1 .. 2^b - 1) and scales of ordinary size in all of s's pages."""
    P, _, tiles, _ = s.pages.shape
    for key, b in ((True, s.kb), (False, s.vb)):
        codes = rng.integers(1, 1 << b, (P, heads, tiles, R.TILE, s.D), dtype=np.uint8)
        scales = (0.7 / (1 << (b - 2)) * np.exp(0.3 * rng.standard_normal((P, heads, tiles, R.TILE, s.D // 32))))
        put_part(s.pages, codes, scales.astype(np.float16), s.D, s.kb, s.vb, key)


def attend_terms(s, q, heads, scale, window=0):
    """64-bit attention with what bounds its error: out, lse, `mass` = sum_t p_t |u_t|_2 / sqrt(D), `spread` =
    sqrt(sum_t p_t^2 |u_t|_2^2 / D), `score` = the largest scale / D sum_d |Hq| |u_k|, `top` = the largest |u_v|."""
    T, Hq, D = q.shape
    G, H = Hq // heads, R.hadamard(D)
    r = dict(out=np.zeros((T, Hq, D)), lse=np.full((T, Hq), -np.inf))
    for name in ("mass", "spread", "score", "top"):
        r[name] = np.zeros((T, Hq))
    for b, (l, n) in enumerate(zip(s.lens, s.news)):
        for h in range(heads):
            if n == 0 or l <= 0:
                continue
            k, v = s.context(b, h, True), s.context(b, h, False)
            for i in range(n):
                pos, row, hq = l - n + i, s.cu[b] + i, slice(h * G, h * G + G)
                if pos < 0:
                    continue
                lo = max(0, pos - window + 1) if window else 0
                u, kk, vv = q[row, hq] @ H, k[lo:pos + 1], v[lo:pos + 1]
                x = u @ kk.T * (scale / D)
                m = x.max(-1, keepdims=True)
                p = np.exp(x - m)
                tot = p.sum(-1, keepdims=True)
                p = p / tot
                size = np.sqrt((vv * vv).sum(-1) / D)
                r["out"][row, hq] = p @ vv @ H / D
                r["lse"][row, hq] = (m + np.log(tot))[:, 0]
                r["mass"][row, hq] = p @ size
                r["spread"][row, hq] = np.sqrt(p ** 2 @ size ** 2)
                r["score"][row, hq] = (np.abs(u) @ np.abs(kk).T).max(-1) * abs(scale) / D
                r["top"][row, hq] = np.abs(vv).max()
    return r


def output_tolerance(r, eps, D, seen, chain):
    """Bound on |out - exact|_2 of every row and head (|H x|_2 = sqrt(D) |x|_2 throughout):
    - weight times scale is rounded once to fp16, by at most U16 of its size, each (token, group) by itself. The
      roundings are spread over the half step, a third of its square on average, and independent of the codes'
      signs: the error's mean square is U16^2 / 3 spread^2, from hundreds of terms; six times its root bounds it.
      Few tokens do not average, but then spread is mass and six times the root is 3.4 times the most they can be;
    - a weight's relative error: the score's, ds (as in the lse), and 2^-19 for its exponential, in numerator and
      sum: 2 (ds + 2^-19) mass;
    - single-precision sums: `chain` additions one after the other on matrix instructions, which keep two bits less
      than fp32: chain 4 U32 mass; the joins add 2 x 160 fused multiply-adds at most, but of parts of mass that sum
      to it: 32 U32 mass covers ten levels of them;
    - products below 2^-14 are rounded in steps of 2^-24 next to a largest one of at least 2^10 / 2: seen 2^-34 top;
    - out is rounded once: eps / 2 of each element, and 2^-25 sqrt(D) where fp16's steps stop shrinking."""
    ds = r["score"] * (2.0 ** -22 + (D + 32) * U32)
    norm = np.sqrt((r["out"] ** 2).sum(-1))
    return (6 * U16 / math.sqrt(3) * r["spread"] + (2 * (ds + 2.0 ** -19) + (4 * chain + 32) * U32) * r["mass"]
            + seen * 2.0 ** -34 * r["top"] + eps / 2 * norm + 2.0 ** -25 * math.sqrt(D))


def output_excess(out, r, eps, D, seen, chain):
    """Largest error in units of its bound: more than 1 is wrong."""
    err = np.sqrt(((out - r["out"]) ** 2).sum(-1))
    return float(np.max(err / output_tolerance(r, eps, D, seen, chain))) if err.size else 0.0


def rounding_share(out, r):
    """Mean square of what the rounding of weight times scale to fp16 leaves in fp16 outputs, in units of
    U16^2 / 3 spread^2, the output's own rounding taken off. One rounding of products whose mantissas m spread over
    octaves gives the mean of 1 / m^2 under 1 / (m ln 2) on [1, 2): 3 / (8 ln 2) = 0.54. Two give 1.08. Over
    thousands of elements the mean is within a few percent of that; 0.75 parts the two."""
    o = r["out"]
    err = ((out - o) ** 2).sum(-1) - ((o.astype(np.float16).astype(np.float64) - o) ** 2).sum(-1)
    return float((err / (U16 ** 2 / 3 * r["spread"] ** 2)).mean())
