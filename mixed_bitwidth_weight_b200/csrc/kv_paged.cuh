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

// Sequence of row t (the last b with cu[b] <= t), found by the whole warp 32
// entries at a time; -1 behind the last sequence's rows.
QG_DEV int kv_find_seq(const int32_t* cu, int num_seqs, int t, int lane) {
    int lo = 0, n = num_seqs + 1;  // the answer's entry is the last of cu[lo, lo + n) that is <= t
    if (t < cu[0]) return -1;
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int i = lane * step;
        const bool le = i < n && cu[lo + i] <= t;
        const int k = 31 - __clz(__ballot_sync(0xffffffffu, le));
        if (k < 0) return -1;
        lo += k * step;
        n = min(step, n - k * step);
    }
    return lo < num_seqs ? lo : -1;
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

// Lane, unit and first dims of unit n (0 .. D/8 - 1) of a token in slot t of
// its tile: K unit n = 4 g + j, V unit n = 8 h + r.
template <int D, bool KEY>
QG_DEV void kv_unit(int n, int t, int& lane, int& unit, int& d0, int& d1) {
    if constexpr (KEY) {
        const int g = n >> 2, j = n & 3;
        lane = 4 * (t & 7) + j;
        unit = (t >> 3) * (D / 32) + g;
        d0 = 32 * g + 8 * j;
        d1 = d0 + 4;
    } else {
        const int h = n >> 3, r = n & 7;
        lane = 4 * r + ((t >> 1) & 3);
        unit = ((t >> 3) * 2 + (t & 1)) * (D / 64) + h;
        d0 = 64 * h + 4 * r;
        d1 = d0 + 32;
    }
}

// place of token slot t's scale of group g in the record's scale part (halves)
template <int D, bool KEY>
QG_DEV int kv_scale_at(int t, int g) {
    constexpr int G = D / 32;
    if constexpr (KEY) return ((t & 7) * 4 + (t >> 3)) * G + g;
    return ((((t >> 1) & 3) * G + g) * 4 + (t >> 3)) * 2 + (t & 1);
}

// slot i of a K unit of 5 bits and more holds dim kv_wide(i) of the eight (its own inverse)
QG_DEV int kv_wide(int i) { return (i & 4) ? ((i & 2) ? i : i - 2) : ((i & 2) ? i + 2 : i); }

// ------------------------------------------------------------------- append
// One warp per (row, head, K or V): rotate, quantise (the steps of
// kv_quant_kernel, so the same codes bit for bit) and store the token's units.
template <int D, bool BF16>
__global__ void __launch_bounds__(32 * kKvWarps) kv_append_kernel(KvPages pg, KvBatch bt, KvRows k, KvRows v) {
    constexpr int E = D / 32, G = 32 / E;
    __shared__ uint8_t sh_codes[kKvWarps][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t item = (int64_t)blockIdx.x * kKvWarps + warp;
    const bool key = (item & 1) == 0;
    const int64_t th = item >> 1;
    const int row = (int)(th / pg.heads), head = (int)(th - (int64_t)row * pg.heads);
    if (row >= bt.rows) return;
    const int b = kv_find_seq(bt.cu, bt.num_seqs, row, lane);
    if (b < 0) return;
    const int pos = bt.lens[b] - bt.cu[b + 1] + row;
    if (pos < 0) return;
    const int rb = kv_record_bytes<D>(pg.kb, pg.vb);
    uint8_t* rec = kv_record(pg, bt, b, pos, head, rb);
    if (!rec) return;
    const KvRows& src = key ? k : v;
    const uint16_t* p = reinterpret_cast<const uint16_t*>(src.p) + row * src.row + head * src.head + E * lane;
    float x[E];
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = kv_to_float<BF16>(p[i]);
    fwht_warp<E>(x, lane);
    const int bits = key ? pg.kb : pg.vb, z = 1 << (bits - 1);
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
    for (int o = 1; o < G; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const __half sh = __float2half_rn(__fdiv_rn(amax, (float)(z - 1)));
    const float s = __half2float(sh);
    const float inv = (s == 0.f) ? 0.f : __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < E; ++i) {
        float tq = rintf(__fmul_rn(x[i], inv));
        if (tq != tq) tq = 0.f;
        tq = fminf(fmaxf(tq, (float)(-z)), (float)(z - 1));
        sh_codes[warp][E * lane + i] = (uint8_t)((int)tq + z);
    }
    __syncwarp();
    const int t = pos & (kTileTokens - 1);
    uint8_t* part = key ? rec : rec + 4 * D * pg.kb + 2 * D;
    if (lane < D / 8) {
        int l, unit, d0, d1;
        if (key)
            kv_unit<D, true>(lane, t, l, unit, d0, d1);
        else
            kv_unit<D, false>(lane, t, l, unit, d0, d1);
        uint64_t w = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int m = (key && bits >= 5) ? kv_wide(i) : i;
            const int d = (m < 4 ? d0 + m : d1 + m - 4);
            w |= (uint64_t)sh_codes[warp][d] << (i * bits);
        }
        const int clog = kv_chunk_log2<D>(bits);
        for (int i = 0; i < bits; ++i) part[kv_stream_at(l, unit * bits + i, clog)] = (uint8_t)(w >> (8 * i));
    }
    if (lane % G == 0) {
        const int g = lane / G;
        __half* sc = reinterpret_cast<__half*>(part + 4 * D * bits);
        sc[key ? kv_scale_at<D, true>(t, g) : kv_scale_at<D, false>(t, g)] = sh;
    }
}

// Rotated values of token slot t: this lane's E dims E lane .. E lane + E - 1.
// sh: D bytes of the warp's own.
template <int D, bool KEY>
QG_DEV void kv_load_token(const uint8_t* rec, int t, int kb, int vb, uint8_t* sh, int lane, float (&x)[D / 32]) {
    constexpr int E = D / 32;
    const int bits = KEY ? kb : vb, z = 1 << (bits - 1);
    const uint8_t* part = KEY ? rec : rec + 4 * D * kb + 2 * D;
    __syncwarp();
    if (lane < D / 8) {
        int l, unit, d0, d1;
        kv_unit<D, KEY>(lane, t, l, unit, d0, d1);
        const int clog = kv_chunk_log2<D>(bits);
        uint64_t w = 0;
        for (int i = 0; i < bits; ++i) w |= (uint64_t)part[kv_stream_at(l, unit * bits + i, clog)] << (8 * i);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int m = (KEY && bits >= 5) ? kv_wide(i) : i;
            sh[m < 4 ? d0 + m : d1 + m - 4] = (uint8_t)((w >> (i * bits)) & ((1u << bits) - 1u));
        }
    }
    __syncwarp();
    const __half* sc = reinterpret_cast<const __half*>(part + 4 * D * bits);
    const float s = __half2float(sc[kv_scale_at<D, KEY>(t, E * lane / 32)]);
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = __fmul_rn((float)((int)sh[E * lane + i] - z), s);  // exact
}

// ------------------------------------------------------------------- gather
// One warp per (row, head, K or V): v' = H_D u' / D.
template <int D, bool BF16>
__global__ void __launch_bounds__(32 * kKvWarps) kv_gather_kernel(KvPages pg, KvBatch bt, KvRows k, KvRows v) {
    constexpr int E = D / 32;
    __shared__ uint8_t sh_codes[kKvWarps][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t item = (int64_t)blockIdx.x * kKvWarps + warp;
    const bool key = (item & 1) == 0;
    const int64_t th = item >> 1;
    const int row = (int)(th / pg.heads), head = (int)(th - (int64_t)row * pg.heads);
    if (row >= bt.rows) return;
    const int b = kv_find_seq(bt.cu, bt.num_seqs, row, lane);
    if (b < 0) return;
    const int pos = bt.lens[b] - bt.cu[b + 1] + row;
    if (pos < 0) return;
    const uint8_t* rec = kv_record(pg, bt, b, pos, head, kv_record_bytes<D>(pg.kb, pg.vb));
    if (!rec) return;
    float x[E];
    const int t = pos & (kTileTokens - 1);
    if (key)
        kv_load_token<D, true>(rec, t, pg.kb, pg.vb, sh_codes[warp], lane, x);
    else
        kv_load_token<D, false>(rec, t, pg.kb, pg.vb, sh_codes[warp], lane, x);
    fwht_warp<E>(x, lane);
    const KvRows& dst = key ? k : v;
    uint16_t* p = reinterpret_cast<uint16_t*>(dst.p) + row * dst.row + head * dst.head + E * lane;
#pragma unroll
    for (int i = 0; i < E; ++i) p[i] = kv_from_float<BF16>(__fmul_rn(x[i], 1.f / (float)D));
}

}  // namespace qg
