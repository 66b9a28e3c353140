// Reading tokens back from the paged KV cache: v' = H_D ((q - z) s) / D.
//
// One warp per (record of 32 tokens, head, K or V), 16 tokens at a time.  The
// rotation inside a group of 32 dims is a matrix product with the Hadamard
// matrix's +-1 on m16n8k16: the codes' bits are the A operand as they are masked
// out of their words (subnormal fp16, see kv_attend.cuh), every product and sum
// is a whole number below 2^14 times 2^-24, so this part is exact; -z appears in
// the sum over a group's constant column only, where the accumulator starts at
// -32 z.  Then the group's scale, the butterflies between groups (within a
// lane) in fp32, and one rounding.  The columns are dealt to lanes so that a
// lane ends with 8 neighbouring dims of a token: 16-byte stores.  V's streams
// pair two tokens of one dim; movmatrix turns each 8 x 8 block into rows of tokens.
// Butterflies by shuffles would cost 64 of them per 8 tokens (4 cycles each, 1900
// cycles a record of 128 dims against about 1000).  45223 tokens of 8 heads of 128 at 4
// bits in 58 us (237 MB, 4.1 TB/s; a warp per vector took 330 us).  Bound by the latency of the
// loads: 14 warps an SM (109 registers a thread) issue on 46% of the cycles, and waiting for
// memory is the largest stall (2.8 of 7.5 warp cycles an instruction); no pipe is above 31%.
#pragma once

#include "kv_attend.cuh"

namespace qg {

// B operand of k step s and column tile nt: half e pairs fields i = 2 s + e of dims
// d = 8 j + i and d + 4 with column n = 8 (r / 2) + 2 nt + r % 2 (lane 4 r + j).  The
// entry's sign is the parity of d & n = [j & r / 2] + [i & 2 nt] + [i & r % 2], the
// dim 4 further adds nt / 2; its size undoes the field's place (see Fld: at 4 bits even
// fields take H_d - H_{d+1} / 16).
template <int B>
QG_DEV uint32_t had_operand(int i, int nt, uint32_t lane_sign, bool odd) {
    const uint32_t lo = __builtin_popcount(i & (2 * nt)) & 1, hi = lo ^ (nt >> 1);
    const uint32_t sign = (lo << 15 | hi << 31) ^ lane_sign ^ ((i & 1) && odd ? 0x80008000u : 0u);
    const uint32_t one = (uint32_t)(15 - Fld<B>::at(i % Fld<B>::N)) << 10;  // fp16 2^-at
    const uint32_t size = B == 4 && !(i & 1) ? (odd ? 0x3c40u : 0x3b80u) : one;  // 17/16 or 15/16
    return (size * 0x10001u) ^ sign;
}

template <int D, int B, bool KEY>
QG_DEV void gather_part(const uint8_t* part, const KvBlock& blk, int tile_pos, int64_t row0, uint16_t* out,
                        int64_t row_stride, bool bf16, int lane) {
    constexpr int G = D / 32, NW = D * B / 64, UT = D / 64 * 8 * B;
    const int j = lane & 3, r = lane >> 2;
    uint32_t hb[2][4][2];
    const uint32_t lane_sign = (__popc(j & (r >> 1)) & 1) ? 0x80008000u : 0u;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) hb[s][nt][e] = had_operand<B>(2 * s + e, nt, lane_sign, r & 1);
    const float zero = j == 0 ? -32.f * (float)(1 << (B - 1)) * 5.9604644775390625e-8f : 0.f;
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
        const int p_lo = tile_pos + 16 * half;
        if (p_lo + 16 <= blk.first || p_lo >= blk.end) continue;
        uint32_t w[NW];
        load_words<D, B>(part, half, lane, w);
        const __half* sc = reinterpret_cast<const __half*>(part + 4 * D * B);
        float c[G][4][4];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            uint32_t a[2][4];
            if constexpr (KEY) {
                k_fragment<D, B>(w, g, 0, a[0]);
                k_fragment<D, B>(w, g, 1, a[1]);
            } else {
                const int unit = (g >> 1) * 8 * B + (g & 1) * 4 * B;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int t0 = (2 * k) * UT + unit, t1 = (2 * k + 1) * UT + unit;
                    uint32_t f[4];
                    if constexpr (B <= 4) {
                        const uint32_t x = halves_from(w, t0, t1, 4 * B);
                        f[0] = field<B, 0>(x);
                        f[1] = field<B, 1>(x);
                        f[2] = field<B, 2 % Fld<B>::N>(x);
                        f[3] = field<B, 3 % Fld<B>::N>(x);
                    } else {
                        const uint32_t x = halves_from(w, t0, t1, 2 * B), y = halves_from(w, t0 + 2 * B, t1 + 2 * B, 2 * B);
                        f[0] = field<B, 0>(x);
                        f[1] = field<B, 1>(x);
                        f[2] = field<B, 0>(y);
                        f[3] = field<B, 1>(y);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) a[i >> 1][2 * (i & 1) + k] = movm_trans(f[i]);
                }
            }
            const int t = 16 * half + r;
            const float s0 = __half2float(sc[kv_scale_at<D, KEY>(t, g)]) * 16777216.f;
            const float s1 = __half2float(sc[kv_scale_at<D, KEY>(t + 8, g)]) * 16777216.f;
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
                float (&x)[4] = c[g][nt];
                x[0] = x[2] = nt == 0 ? zero : 0.f;
                x[1] = x[3] = 0.f;
                mma_f16(x, a[0][0], a[0][1], a[0][2], a[0][3], hb[0][nt][0], hb[0][nt][1]);
                mma_f16(x, a[1][0], a[1][1], a[1][2], a[1][3], hb[1][nt][0], hb[1][nt][1]);
                x[0] *= s0;
                x[1] *= s0;
                x[2] *= s1;
                x[3] *= s1;
            }
        }
#pragma unroll
        for (int st = 1; st < G; st <<= 1)
#pragma unroll
            for (int g = 0; g < G; ++g)
                if (!(g & st))
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float u = c[g][i >> 2][i & 3], v = c[g + st][i >> 2][i & 3];
                        c[g][i >> 2][i & 3] = u + v;
                        c[g + st][i >> 2][i & 3] = u - v;
                    }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int pos = p_lo + 8 * k + r;
            if (pos < blk.first || pos >= blk.end) continue;
            uint16_t* p = out + (row0 + pos) * row_stride + 8 * j;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                uint32_t o[4];
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    const float u = c[g][nt][2 * k] * (1.f / (float)D), v = c[g][nt][2 * k + 1] * (1.f / (float)D);
                    if (bf16) {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(u, v);
                        o[nt] = *reinterpret_cast<const uint32_t*>(&h);
                    } else {
                        o[nt] = h2_bits(__floats2half2_rn(u, v));
                    }
                }
                *reinterpret_cast<uint4*>(p + 32 * g) = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
    }
}

template <int D>
__global__ void __launch_bounds__(32 * kKvWarps) kv_gather_kernel(KvPages pg, KvBatch bt, KvRows k, KvRows v, int bf16) {
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * kKvWarps + (threadIdx.x >> 5);
    const bool key = (item & 1) == 0;
    const int64_t bh = item >> 1, number = bh / pg.heads;
    const int head = (int)(bh - number * pg.heads);
    KvBlock blk;
    if (number >= (int64_t)bt.rows / kTileTokens + 2ll * bt.num_seqs || !kv_block<kTileTokens>(bt, (int)number, lane, blk))
        return;
    const uint8_t* rec = kv_record(pg, bt, blk.b, blk.first, head, kv_record_bytes<D>(pg.kb, pg.vb));
    if (!rec) return;
    const int tile_pos = blk.first & ~(kTileTokens - 1);
    const KvRows& dst = key ? k : v;
    uint16_t* out = reinterpret_cast<uint16_t*>(dst.p) + head * dst.head;
    const int64_t row0 = (int64_t)blk.row0 - blk.pos0;
    const uint8_t* part = key ? rec : rec + 4 * D * pg.kb + 2 * D;
    switch (key ? pg.kb : pg.vb) {
#define QG_GATHER(B)                                                                              \
    case B:                                                                                       \
        if (key)                                                                                  \
            gather_part<D, B, true>(part, blk, tile_pos, row0, out, dst.row, bf16 != 0, lane);    \
        else                                                                                      \
            gather_part<D, B, false>(part, blk, tile_pos, row0, out, dst.row, bf16 != 0, lane);   \
        break;
        QG_GATHER(2)
        QG_GATHER(3)
        QG_GATHER(4)
        QG_GATHER(5)
        QG_GATHER(6)
        QG_GATHER(8)
#undef QG_GATHER
    }
}

}  // namespace qg
