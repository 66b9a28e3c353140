// Paged quantised KV cache: write new tokens into pages, read tokens back, and
// attention of new tokens over the pages.
//
// A sequence's tokens live in pages named by its row of the block table; a page
// holds page_size tokens of every KV head, as one record per head and 32 tokens
// (a tile).  The codes and scales are those of kv_cache.cuh: u = H_D v, groups
// of 32 with one fp16 scale s, code q, u ~ (q - 2^(b-1)) s.
//
// Record of 4 D (kb + vb + 1) bytes: K codes, K scales, V codes, V scales.
// Codes are 32 lane streams, one per lane of the warp that multiplies the tile
// (lane 4 r + j holds what the matrix instruction's A fragment wants of its
// row r), in units of 8 codes = b bytes, little-endian, slot i at bits
// [b i, b i + b):
//   K  token 8 tt + r, dim 32 g + 8 j + i: lane 4 r + j, unit tt G + g; slots
//      hold i = 0..7 (b <= 4) or i = 0,1,4,5,2,3,6,7 (b >= 5), G = D / 32;
//   V  token 8 tt + 2 j + u, dim 64 h + 32 e + 4 r + i: lane 4 r + j, unit
//      (2 tt + u) D/64 + h, slot 4 e + i.
// A unit belongs to one token, so tokens are written with plain byte stores,
// whatever the width.  Streams are stored in chunks of C bytes (the largest of
// 16, 8, 4 that divides half a stream, D b / 16), chunk c of lane l at
// (32 c + l) C: a warp reads its chunks with one conflict-free access each.
// Scales: K [r][tt][g], V [j][g][tt][u].
#pragma once

#include <cuda_bf16.h>

#include "kv_cache.cuh"

namespace qg {

constexpr int kTileTokens = 32;

struct KvPages {
    uint8_t* base;
    int64_t num_pages;
    int64_t page_bytes;  // of all heads
    int32_t page_size, heads, kb, vb;
};

struct KvBatch {
    const int32_t* table;
    int64_t table_stride;
    const int32_t* lens;
    const int32_t* cu;
    int32_t num_seqs, max_pages, rows;
};

// a [rows][heads][D] operand with any row and head stride (elements)
struct KvRows {
    uint8_t* p;
    int64_t row, head;
};

template <int D>
QG_DEV int kv_record_bytes(int kb, int vb) {
    return 4 * D * (kb + vb + 1);
}

// log2 of a stream's chunk size
template <int D>
QG_DEV int kv_chunk_log2(int b) {
    const int half = D / 16 * b;
    return (half & 15) == 0 ? 4 : (half & 7) == 0 ? 3 : 2;
}

// byte y of lane l's stream, from the start of the record's code part
QG_DEV int kv_stream_at(int lane, int y, int clog) {
    return ((((y >> clog) << 5) + lane) << clog) + (y & ((1 << clog) - 1));
}

template <bool BF16>
QG_DEV float kv_to_float(uint16_t v) {
    if constexpr (BF16) return __uint_as_float((uint32_t)v << 16);
    return __half2float(__ushort_as_half(v));
}
template <bool BF16>
QG_DEV uint16_t kv_from_float(float v) {
    if constexpr (BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(v));
    return __half_as_ushort(__float2half_rn(v));
}

// Record of (sequence b, position pos, head), or null (with the error word set)
// when the table has no valid page for it.
QG_DEV uint8_t* kv_record(const KvPages& pg, const KvBatch& bt, int b, int pos, int head, int rec_bytes) {
    const int pi = pos / pg.page_size, in = pos - pi * pg.page_size;
    const int page = pi < bt.max_pages ? bt.table[b * bt.table_stride + pi] : -1;
    if (page < 0 || page >= pg.num_pages) {
        set_dev_error(QGEMM_DEV_BAD_PAGE);
        return nullptr;
    }
    const int tiles = pg.page_size / kTileTokens;
    return pg.base + page * pg.page_bytes + (int64_t)(head * tiles + in / kTileTokens) * rec_bytes;
}

// place of token slot t's scale of group g in the record's scale part (halves)
template <int D, bool KEY>
QG_DEV int kv_scale_at(int t, int g) {
    constexpr int G = D / 32;
    if constexpr (KEY) return ((t & 7) * 4 + (t >> 3)) * G + g;
    return ((((t >> 1) & 3) * G + g) * 4 + (t >> 3)) * 2 + (t & 1);
}

// slot i of a K unit of 5 bits and more holds dim kv_wide(i) of the eight (its own inverse)
QG_DEV constexpr int kv_wide(int i) { return (i & 4) ? ((i & 2) ? i : i - 2) : ((i & 2) ? i + 2 : i); }

// ---------------------------------------------------- blocks of a batch's rows
// The new tokens of a sequence are cut where their positions are multiples of N
// (8 or 32).  Sequence b's blocks are numbered from cu[b] / N + 2 b on: with n
// rows it has at most (n - 2) / N + 2 of them, so numbers never meet, no sum over
// the sequences is needed, and rows / N + 2 num_seqs numbers are enough.
struct KvBlock {
    int b, row0, pos0, first, end;  // sequence; its first row and that row's position; positions [first, end) of the block
};

template <int N>
QG_DEV bool kv_block(const KvBatch& bt, int number, int lane, KvBlock& k) {
    int lo = 0, n = bt.num_seqs;
    while (n > 1) {  // the last sequence whose first number is <= number, 32 at a time
        const int step = (n + 31) / 32, i = lane * step;
        const bool le = i < n && max(bt.cu[lo + i], 0) / N + 2 * (lo + i) <= number;
        const int m = max(31 - __clz(__ballot_sync(0xffffffffu, le)), 0);
        lo += m * step;
        n = min(step, n - m * step);
    }
    const int c0 = bt.cu[lo], c1 = bt.cu[lo + 1], at = number - (max(c0, 0) / N + 2 * lo);
    if (c0 < 0 || at < 0) return false;
    k.b = lo;
    k.row0 = c0;
    k.pos0 = bt.lens[lo] - c1 + c0;
    const int rows = min(c1, bt.rows) - c0;  // rows that the operands have
    if (rows <= 0) return false;
    const int64_t start = (int64_t)(max(k.pos0, 0) / N + at) * N, end = (int64_t)k.pos0 + rows;
    if (start >= end || start > 0x7fffff00) return false;
    k.first = max((int)start, k.pos0);
    k.end = (int)(end < start + N ? end : start + N);
    return true;
}

// ------------------------------------------------------------------- append
// One warp per (8 positions, head, K or V); four lanes a token, lane 4 t + j
// with dims 32 g + 8 j + i: it is also the token's lane of the K stream, and
// holds the V streams' rows 2 j and 2 j + 1.  Butterflies in the order strides
// 1, 2, ..., D / 2 (8 and 16 between the four lanes), each rounded to nearest:
// the codes of kv_quant_kernel, bit for bit.  Codes are packed in registers and
// stored in the widest pieces that a token owns (16 bytes of K, 8 of V at 128
// dims and 4 bits; eight neighbouring tokens fill whole sectors).
// Bound by instructions, not by HBM: 32768 tokens of 8 heads of 128 at 4 bits 70 us in fp16 and 71
// in bf16, 172 MB read and written (2.4 TB/s).  956 instructions a warp (8 tokens of one head's K or
// V), 372 of them fp32 additions; the schedulers issue on 78% of the cycles.

// bits [at, at + b) of a bit string in 32-bit words, `at` constant after unrolling
template <int NW>
QG_DEV void put_bits(uint32_t (&w)[NW], int at, int b, uint32_t v) {
    w[at >> 5] |= v << (at & 31);
    if ((at & 31) + b > 32) w[(at >> 5) + 1] |= v >> (32 - (at & 31));
}

// store a token's PB bytes (words w) at byte y0 of stream `lane`
template <int PB, int C, int NW>
QG_DEV void put_stream(uint8_t* part, int lane, int y0, const uint32_t (&w)[NW]) {
    constexpr int V = (PB % 16 == 0 && C == 16) ? 16 : (PB % 8 == 0 && C >= 8) ? 8 : PB % 4 == 0 ? 4 : PB % 2 == 0 ? 2 : 1;
    constexpr int clog = C == 16 ? 4 : C == 8 ? 3 : 2;
#pragma unroll
    for (int y = 0; y < PB; y += V) {
        uint8_t* p = part + kv_stream_at(lane, y0 + y, clog);
        if constexpr (V == 16) *reinterpret_cast<uint4*>(p) = make_uint4(w[y / 4], w[y / 4 + 1], w[y / 4 + 2], w[y / 4 + 3]);
        if constexpr (V == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[y / 4], w[y / 4 + 1]);
        if constexpr (V == 4) *reinterpret_cast<uint32_t*>(p) = w[y / 4];
        if constexpr (V == 2) *reinterpret_cast<uint16_t*>(p) = (uint16_t)(w[y / 4] >> (8 * (y % 4)));
        if constexpr (V == 1) *p = (uint8_t)(w[y / 4] >> (8 * (y % 4)));
    }
}

template <int D, int B, bool KEY, bool BF16>
QG_DEV void put_token(uint8_t* part, int t, int lane, bool mine, float (&x)[D / 32][8]) {
    constexpr int G = D / 32, z = 1 << (B - 1);
    constexpr int half = D * B / 16, C = half % 16 == 0 ? 16 : half % 8 == 0 ? 8 : 4;
    const int j = lane & 3, tt = t >> 3;
    constexpr int N = B == 2 ? 8 : B <= 5 ? 4 : 2;  // codes whose bits a float holds exactly
    __half sh[G];
    float code[G][8];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[g][i]));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        sh[g] = __float2half_rn(__fdiv_rn(amax, (float)(z - 1)));
        const float s = __half2float(sh[g]);
        const float inv = s == 0.f ? 0.f : __frcp_rn(s);  // the zero point everywhere where s is 0
#pragma unroll
        for (int i = 0; i < 8; ++i) code[g][i] = __fmul_rn(x[g][i], inv);
        // A normal scale is at least (1 - 2^-11) max / (z - 1): |u / s| <= (z - 1) (1 + 2^-10) rounds to
        // z - 1 at most.  Others are clamped (before rounding: the bounds are whole, so it is the same), and
        // what is not a number (an infinite value over an infinite scale too) takes the zero point.
        if (!(s >= 6.103515625e-5f && s <= 65504.f))
#pragma unroll
            for (int i = 0; i < 8; ++i)
                code[g][i] = isnan(code[g][i]) ? 0.f : fminf(fmaxf(code[g][i], (float)(-z)), (float)(z - 1));
        // rounded to nearest even by adding 1.5 2^23; from here whole numbers 0 .. 2 z - 1
#pragma unroll
        for (int i = 0; i < 8; ++i) code[g][i] = __fsub_rn(__fadd_rn(code[g][i], 12582912.f + (float)z), 12582912.f);
    }
    // N codes as one number, by exact fused multiply-adds
    constexpr int NJ = 8 * G / N;
    float num[NJ];
    auto at = [&](int n) -> float& {  // the lane's n-th code in the order of its units' slots
        if constexpr (KEY) return code[n >> 3][B >= 5 ? kv_wide(n & 7) : n & 7];
        const int e = n / (4 * G), h = n / 8 % (G / 2), i = n & 7;
        return code[2 * h + (i >> 2)][4 * e + (i & 3)];
    };
    auto join = [&] {
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < NJ; ++n) {
            float v = at(n * N + N - 1);
#pragma unroll
            for (int i = N - 2; i >= 0; --i) v = fmaf(v, (float)(1 << B), at(n * N + i));
            num[n] = v;
            if constexpr (BF16) sum += v;
        }
        return sum;
    };
    // Sums of bf16 values may overflow and leave NaN in a group of normal scale (fp16's cannot, and an infinite or
    // NaN input leaves no number in any group).  It shows in the numbers' sum (32768 bf16 tokens of 8 heads of 128
    // at 4 bits: +1.5%, 256 dims +6%, 64 dims and fp16 no change).
    if (isnan(join())) {
#pragma unroll
        for (int n = 0; n < 8 * G; ++n) at(n) = isnan(at(n)) ? (float)z : at(n);
        join();
    }
    auto bits = [](float v) { return __float_as_uint(v + 8388608.f) & 0x7fffffu; };  // of 2^23 + v
    if (!mine) return;
    if constexpr (KEY) {
        constexpr int PB = G * B;  // the lane's units of all groups
        uint32_t w[(PB + 3) / 4 + 1] = {};
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int i = 0; i < 8; i += N) put_bits(w, (g * 8 + i) * B, N * B, bits(num[(g * 8 + i) / N]));
        put_stream<PB, C>(part, lane, tt * PB, w);
    } else {
        constexpr int PB = D / 64 * B;
        const int u = t & 1, jt = (t >> 1) & 3;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            uint32_t w[(PB + 3) / 4 + 1] = {};
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
#pragma unroll
                for (int i = 0; i < 8; i += N)
                    put_bits(w, (h * 8 + i) * B, N * B, bits(num[(e * 4 * G + h * 8 + i) / N]));
            put_stream<PB, C>(part, 4 * (2 * j + e) + jt, (2 * tt + u) * PB, w);
        }
    }
    __half* sc = reinterpret_cast<__half*>(part + 4 * D * B);
#pragma unroll
    for (int g = 0; g < G; ++g)
        if ((g & 3) == j) sc[kv_scale_at<D, KEY>(t, g)] = sh[g];
}

template <int D, bool BF16>
__global__ void __launch_bounds__(32 * kKvWarps) kv_append_kernel(KvPages pg, KvBatch bt, KvRows k, KvRows v) {
    constexpr int G = D / 32;
    const int lane = threadIdx.x & 31, j = lane & 3;
    // K and V of one head are neighbours, heads of one block of rows too
    const int64_t item = (int64_t)blockIdx.x * kKvWarps + (threadIdx.x >> 5);
    const bool key = (item & 1) == 0;
    const int64_t bh = item >> 1, number = bh / pg.heads;
    const int head = (int)(bh - number * pg.heads);
    KvBlock blk;
    if (number >= (int64_t)bt.rows / 8 + 2ll * bt.num_seqs || !kv_block<8>(bt, (int)number, lane, blk)) return;
    const int pos = (blk.first & ~7) + (lane >> 2);
    const bool mine = pos >= blk.first && pos < blk.end;
    uint8_t* rec = kv_record(pg, bt, blk.b, blk.first, head, kv_record_bytes<D>(pg.kb, pg.vb));
    if (!rec) return;
    const KvRows& src = key ? k : v;
    const int64_t row = blk.row0 + (mine ? pos : blk.first) - blk.pos0;
    const uint16_t* p = reinterpret_cast<const uint16_t*>(src.p) + row * src.row + head * src.head + 8 * j;
    float x[G][8];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(p + 32 * g));
        const uint32_t q[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[g][i] = kv_to_float<BF16>((uint16_t)((i & 1) ? q[i / 2] >> 16 : q[i / 2] & 0xffffu));
    }
#pragma unroll
    for (int st = 1; st < D; st <<= 1)
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (st < 8) {
                    if (i & st) continue;
                    const float a = x[g][i], c = x[g][i | (st & 7)];
                    x[g][i] = __fadd_rn(a, c);
                    x[g][i | (st & 7)] = __fsub_rn(a, c);
                } else if (st < 32) {
                    const float o = __shfl_xor_sync(0xffffffffu, x[g][i], st / 8);
                    x[g][i] = (lane & (st / 8)) ? __fsub_rn(o, x[g][i]) : __fadd_rn(x[g][i], o);
                } else {
                    if (g & (st / 32)) continue;
                    const float a = x[g][i], c = x[(g | (st / 32)) % G][i];
                    x[g][i] = __fadd_rn(a, c);
                    x[(g | (st / 32)) % G][i] = __fsub_rn(a, c);
                }
            }
    const int t = pos & (kTileTokens - 1);
    if (key) {
        switch (pg.kb) {
            case 2: put_token<D, 2, true, BF16>(rec, t, lane, mine, x); break;
            case 3: put_token<D, 3, true, BF16>(rec, t, lane, mine, x); break;
            case 4: put_token<D, 4, true, BF16>(rec, t, lane, mine, x); break;
            case 5: put_token<D, 5, true, BF16>(rec, t, lane, mine, x); break;
            case 6: put_token<D, 6, true, BF16>(rec, t, lane, mine, x); break;
            default: put_token<D, 8, true, BF16>(rec, t, lane, mine, x); break;
        }
    } else {
        uint8_t* part = rec + 4 * D * pg.kb + 2 * D;
        switch (pg.vb) {
            case 2: put_token<D, 2, false, BF16>(part, t, lane, mine, x); break;
            case 3: put_token<D, 3, false, BF16>(part, t, lane, mine, x); break;
            case 4: put_token<D, 4, false, BF16>(part, t, lane, mine, x); break;
            case 5: put_token<D, 5, false, BF16>(part, t, lane, mine, x); break;
            case 6: put_token<D, 6, false, BF16>(part, t, lane, mine, x); break;
            default: put_token<D, 8, false, BF16>(part, t, lane, mine, x); break;
        }
    }
}

}  // namespace qg
