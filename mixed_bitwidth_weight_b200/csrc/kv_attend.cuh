// Attention of new tokens over the paged, quantised KV cache (layout in
// kv_paged.cuh), without expanding it.
//
//   out_n = sum_t p_tn v'_t / sum_t p_tn,  p_tn = exp(scale q_n . k'_t),
//   k' = H u_k / D, v' = H u_v / D, u = (c - z) s_g, z = 2^(b-1), H H = D I.
// H is symmetric, so q . k' = (H q) . u_k / D and sum_t p v' = H (sum_t p u_v) / D:
// each query row is rotated once, each output row once, and the cache's codes
// meet the matrix instructions as they are.
//
// Scores, per group g of 32 dims: sum_d (Hq)_d (c - z) on m16n8k16 with the
// codes as the A operand (16 tokens), 8 query rows as B.  A code's bits, masked
// out of its word, ARE an fp16 number: the subnormal c 2^-24 (or, i bits further
// up where it lies, c 2^(i-24); the query carries 2^-i).  So a pair of codes costs one
// AND, and up to 5 bits one exact multiplication more (kNorm).  The accumulators start
// at -z sum_d (Hq)_d instead of 0, and the token's scale multiplies the group's sum in
// fp32.  The rotated query is held as two fp16 parts (22 bits, scaled by the row's power
// of two), each times the exact codes.
// Output: A = codes of V (16 dims x 16 tokens), c - z by one exact fused
// multiply-add a pair (starting at -z sum p would lose the sum of many tokens to
// cancellation), B = p s_g.  p, s and their product are fp32, the product is
// rounded once to fp16 (2^-12 on average; rounding p first cost a third more error
// and saved 4% of the time), the sum of weights is not rounded.  p is scaled so that the
// products stay below 2^15 and weights keep 11 bits down to 2^-24 of the largest.
// The products turn from [token][row] to the B operand's [row][token] by movmatrix.
//
// The legacy matrix instruction, because its operands are registers: a code is
// masked into place and multiplied without a store.  tcgen05 would need every
// expanded tile written to tensor or shared memory first (the V tile transposed),
// and 8 query rows fill 1/16 of its M.
//
// What bounds it: instructions, not HBM, below 8 bits.  A tile of 32 tokens of 128
// dims at 4 bits takes 663 instructions of a warp: 48 mma, 106 logic, 128 fp16 arithmetic
// and 32 conversions, 56 byte permutes, 74 fp32.  Measured on the four
// schedulers, m16n8k16 takes 8.4 cycles, integer and fp16 instructions 2 each, and
// they overlap little (one with four ANDs and four fp16 adds: 17.7 cycles of 24.4):
// 340 cycles a tile and SM against the 205 that its 4608 bytes take from HBM.
// 8 heads x 128, 64 query heads: 4/4 bits, 524288 tokens 176 us (3.4 TB/s, 53% of measured
// HBM); 8/8 bits, 262144 tokens 99 us (5.8 TB/s, 89%).
//
// Work: the (sequence, head, 8 rows, 32-token tile) space is cut into equal runs per
// CTA and per warp, whatever the lengths (all read on the device).  Every 8 rows walk all tiles
// that any new row of their sequence sees, and unpack them again.  A warp walks its
// run with a ring of bulk copies (one record each; a separate feeding warp was slower,
// per-lane asynchronous copies too); what it has of an item is joined in shared memory
// per CTA, and across CTAs by the last one to arrive, in a fixed order, so results
// repeat bit for bit.  Eight warps of up to 255 registers: twelve of 168 gained 4% on
// long sequences and lost 15% on short ones, except at 64 dims.  Scan, seek, first copies
// and join are about 8 us whatever the length.  At 256 dims join slots and query areas
// leave a ring of one record a warp for 30 of the 36 pairs of widths (more where they sum
// to 6 bits or fewer), so a warp's copies and its arithmetic do not overlap, and ptxas
// spills: 96 to 128 bytes of stack a thread.
#pragma once

#include "kv_paged.cuh"

namespace qg {

struct KvAttend {
    KvPages pg;
    KvBatch bt;
    KvRows q, out;
    float* lse;  // [rows][q_heads] or null
    int32_t q_heads, group, window, bf16;
    int32_t stages, ring_bytes;  // of a warp's ring
    float scale;
    unsigned int* tickets;  // [CTAs], zero between calls
    float* partial;         // [CTAs][2] slots
};

constexpr int kAttMaxStages = 8;
constexpr int kAttLowest = -14;       // V scales below 2^-13 count as if they were that
constexpr float kAttNone = -3.4e38f;  // the weights' offset before any token: below every finite score

// KB, VB as in the kernel: known widths, or 0.
template <int D, int KB = 0, int VB = 0>
struct AttCfg {
    static constexpr int W = D <= 64 ? 12 : 8;   // warps: 168 registers a thread with 12, 255 with 8
    static constexpr int T = 32 * W;
    static constexpr int G = D / 32;
    static constexpr int RB = 8;                      // query rows of an item: the N of the matrix instruction
    static constexpr int OS = D + 4;                  // row stride of a slot: conflict-free float4 stores
    static constexpr int SlotFloats = RB * OS + 2 * RB;
    static constexpr int SlotBytes = SlotFloats * 4;
    static constexpr int GSlot = RB * D + 2 * RB;     // floats of a global slot
    // an item's rotated query: [g][hi, lo][lane] 16 bytes, then zq [g][8], f [8];
    // QN of them are shared by the CTA's warps.  256 dims at 8/8 bits leave room for 2: a ring of one
    // record of 17408 bytes for each of eight warps (65536 tokens x 8 heads 78.5 us, 3.6 TB/s; seven
    // warps beside 4 areas 85)
    static constexpr int QN = D <= 128 ? 6 : KB + VB == 16 ? 2 : 4;
    static constexpr int QZero = G * 256, QFactor = QZero + G * 8;
    static constexpr int QFloats = QFactor + 8, QBytes = QFloats * 4;
    // shared memory: slots, query areas, barriers, fragments, prefix sums, rings
    static constexpr int QAt = W * SlotBytes;
    static constexpr int BarAt = (QAt + QN * QBytes + 15) / 16 * 16;
    static constexpr int FragAt = BarAt + W * 8 * 8;
    static constexpr int PrefixAt = FragAt + 2 * W * 24;
    static constexpr int RingAt = (PrefixAt + T * 8 + 127) / 128 * 128;
    static_assert(W * SlotBytes >= QN * RB * D * 2, "the query rows of QN items pass through the slots");
    // the join's weights and row buffer lie over the query areas
    static constexpr int MaxCtas = 160;
    static_assert(QN * QBytes >= (RB * MaxCtas + RB * D + 2 * RB * 2 * W) * 4, "join buffers");
    static constexpr int MaxShared = 226 * 1024;  // 227 KB a CTA, some of it static
    static constexpr int RingRoom = (MaxShared - RingAt) / W / 128 * 128;
    static constexpr int WidestRecord = 4 * D * (KB > 0 ? KB + VB + 1 : 8 + 6 + 1);  // 8/8 is always known
    static_assert(RingRoom >= WidestRecord && RingRoom >= SlotBytes, "a ring holds a record of any width, or a slot");
};

// a slot's fragment: tiles [a, b) of the item whose first tile is number `item`
struct AttFrag {
    long long item;
    int row0, rows, head, tiles;  // the item's rows: `rows` from row0 x group on, of KV head `head`; tiles 0: no fragment
};
static_assert(sizeof(AttFrag) == 24 && kAttMaxStages == 8, "the shared-memory layout");

QG_DEV void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// the first of a chain
QG_DEV void mma_f16_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1,
                         const float (&c)[4]) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

QG_DEV uint32_t movm_trans(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

QG_DEV void cp_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
QG_DEV void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

QG_DEV float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
QG_DEV uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
QG_DEV __half2 bits_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }

// ------------------------------------------------------------ code extraction
// Fields of one 32-bit word: its low half holds n codes of one row, its high
// half the n codes that pair with them (n = 4 for b <= 4, else 2).  Field i is
// used where it lies when it ends below bit 10 (a subnormal's mantissa), else
// the word is shifted down first.  At 4 bits the odd fields keep the code below
// them, c_i + 16 c_{i+1}, which saves a shift per word: the query's even entries
// take q_i - q_{i+1} / 16 for it, and the output's odd rows (O_i + 16 O_{i+1})
// are parted at the end, both linear.
template <int B>
struct Fld {
    static constexpr int N = B <= 4 ? 4 : 2;
    static constexpr int pre(int i) { return B * i + B <= 10 ? 0 : (B == 4 ? 8 : B * i); }
    static constexpr int at(int i) { return B * i - pre(i); }  // the value is c 2^(at - 24)
    static constexpr uint32_t mask(int i) {
        return (B == 4 && (i & 1) ? 0xffu : ((1u << B) - 1u) << at(i)) * 0x10001u;
    }
    // -z in the field's place times 2^10, as a pair of normal fp16 numbers
    static constexpr uint32_t minus_zero(int i) {
        const uint32_t v = B == 4 && (i & 1) ? 0x88u : (1u << (B - 1)) << at(i);
        int e = 0;
        while ((v >> e) > 1) ++e;
        return (0x8000u | (uint32_t)(e + 1) << 10 | (v - (1u << e)) << (10 - e)) * 0x10001u;
    }
};

template <int B, int I>
QG_DEV uint32_t field(uint32_t x) {
    if constexpr (B == 4 && I == 3) return __byte_perm(x, 0, 0x4341);  // the upper byte of each half
    if constexpr (B == 4 && I == 2) return __byte_perm(x, 0, 0x4341) & Fld<B>::mask(I);
    if constexpr (B == 8 && I == 1) return __byte_perm(x, 0, 0x4341);
    if constexpr (Fld<B>::pre(I) == 0) return x & Fld<B>::mask(I);
    return (x >> Fld<B>::pre(I)) & Fld<B>::mask(I);
}

// shift a run-time width's field i carries (for the query and the output)
QG_DEV int field_at(int b, int i) {
    i = b <= 4 ? i : (i & 1);
    if (b * i + b <= 10) return b * i;
    return b == 4 ? b * i - 8 : 0;
}

// a register whose low bits are the stream's from bit `pos` on (pos constant after unrolling)
template <int NW>
QG_DEV uint32_t bits_from(const uint32_t (&w)[NW], int pos, int need) {
    const int i = pos >> 5, o = pos & 31;
    if (o == 0) return w[i];
    if (o + need <= 32) return w[i] >> o;
    return __funnelshift_r(w[i], w[i + 1], o);
}

// (low half: bits from p0; high half: bits from p1); the fields' masks drop the rest
template <int NW>
QG_DEV uint32_t halves_from(const uint32_t (&w)[NW], int p0, int p1, int need) {
    uint32_t a, b;
    int ya, yb;
    if ((p0 & 7) == 0 && (p0 & 31) + 16 <= 32) {
        a = w[p0 >> 5];
        ya = (p0 & 31) >> 3;
    } else {
        a = bits_from(w, p0, need);
        ya = 0;
    }
    if ((p1 & 7) == 0 && (p1 & 31) + 16 <= 32) {
        b = w[p1 >> 5];
        yb = (p1 & 31) >> 3;
    } else {
        b = bits_from(w, p1, need);
        yb = 0;
    }
    return __byte_perm(a, b, ya | (ya + 1) << 4 | (yb + 4) << 8 | (yb + 5) << 12);
}

// K: the low and high four (b <= 4) or two codes of a unit part, side by side
template <int B, int NW>
QG_DEV uint32_t k_word(const uint32_t (&w)[NW], int pos) {
    if constexpr (B == 4 || B == 8) {
        return w[pos >> 5];
    } else if constexpr (B == 2) {
        const int y = (pos & 31) >> 3;
        return __byte_perm(w[pos >> 5], 0, y | y << 4 | (y + 1) << 8 | (y + 1) << 12);
    } else {
        constexpr int gap = B == 3 ? 12 : 2 * B;
        const uint32_t t = bits_from(w, pos, 2 * gap);
        return (t & 0xffffu) | ((t << (16 - gap)) & 0xffff0000u);
    }
}

// half a tile's words of this lane's stream
template <int D, int B>
QG_DEV void load_words(const uint8_t* part, int half, int lane, uint32_t (&w)[D * B / 64]) {
    constexpr int NW = D * B / 64;
    constexpr int V = NW % 4 == 0 ? 4 : NW % 2 == 0 ? 2 : 1;
#pragma unroll
    for (int c = 0; c < NW / V; ++c) {
        const uint8_t* p = part + ((half * (NW / V) + c) * 32 + lane) * (4 * V);
        if constexpr (V == 4) {
            const uint4 u = *reinterpret_cast<const uint4*>(p);
            w[4 * c] = u.x;
            w[4 * c + 1] = u.y;
            w[4 * c + 2] = u.z;
            w[4 * c + 3] = u.w;
        } else if constexpr (V == 2) {
            const uint2 u = *reinterpret_cast<const uint2*>(p);
            w[2 * c] = u.x;
            w[2 * c + 1] = u.y;
        } else {
            w[c] = *reinterpret_cast<const uint32_t*>(p);
        }
    }
}

// ------------------------------------------------------------------- scores
// The query rows of an item in the B operand's layout: hi and lo parts, per
// group and k step two registers, and -z 2^-24 times their sums.
template <int D>
struct AttQ {
    uint32_t hi[D / 32][4], lo[D / 32][4];
    float zq[D / 32][4];  // an accumulator's four: rows r and r + 8 start alike
    float f[2];  // factor of a score, log2 units
    // the accumulators' C operand is four consecutive registers: without the moves that the compiler
    // cannot see through it keeps two and copies them before each use (which it is left to do where
    // the registers for four are not there)
    QG_DEV void set_zero(int g, float x, float y) {
        zq[g][0] = zq[g][2] = x;
        zq[g][1] = zq[g][3] = y;
        if constexpr (D <= 128) {
            asm volatile("mov.b32 %0, %1;" : "=f"(zq[g][2]) : "f"(x));
            asm volatile("mov.b32 %0, %1;" : "=f"(zq[g][3]) : "f"(y));
        }
    }
};

// A registers of one k step (0, 1) of group g: rows tokens 8 tt + r (word x0's) and 8 (tt + 1) + r (x1's)
template <int D, int B>
QG_DEV void k_fragment(const uint32_t (&w)[D * B / 64], int g, int step, uint32_t (&a)[4]) {
    const int p0 = g * 8 * B, p1 = (D / 32 + g) * 8 * B;  // units of the two tokens
    if constexpr (B <= 4) {
        const uint32_t x0 = k_word<B>(w, p0), x1 = k_word<B>(w, p1);
        if (step == 0) {
            a[0] = field<B, 0>(x0);
            a[1] = field<B, 0>(x1);
            a[2] = field<B, 1>(x0);
            a[3] = field<B, 1>(x1);
        } else {
            a[0] = field<B, 2 % Fld<B>::N>(x0);
            a[1] = field<B, 2 % Fld<B>::N>(x1);
            a[2] = field<B, 3 % Fld<B>::N>(x0);
            a[3] = field<B, 3 % Fld<B>::N>(x1);
        }
    } else {
        const uint32_t x0 = k_word<B>(w, p0 + 4 * B * step), x1 = k_word<B>(w, p1 + 4 * B * step);
        a[0] = field<B, 0>(x0);
        a[1] = field<B, 0>(x1);
        a[2] = field<B, 1>(x0);
        a[3] = field<B, 1>(x1);
    }
}

// Scores of a tile, s[half][c].  The four dependent matrix instructions of a
// group are issued a step at a time over all groups, so that eight chains (four
// with 64 dims) hide each other's latency.
// The matrix instruction aligns products by their operands' exponents, and a subnormal's
// is that of 2^-14 whatever its leading zeros: codes of b bits would lose up to 10 - b of
// the sum's 24 bits, 5e-6 of a score's size at 2 to 4 bits.  Up to 5 bits they are
// therefore made normal numbers, times 2^10, by one exact multiplication a pair (3e-7,
// and 2% of the time); the query's
// factors know (att_row_scale).
template <int B>
constexpr bool kNorm = B <= 5;

template <int D, int B>
QG_DEV void scores_tile(const uint8_t* rec, int lane, const AttQ<D>& q, float (&s)[2][4]) {
    constexpr int G = D / 32, NW = D * B / 64, HB = D == 256 || (D == 128 && B <= 4) ? 1 : 2;  // halves at a time, as measured
#pragma unroll
    for (int h0 = 0; h0 < 2; h0 += HB) {
        uint32_t w[HB][NW], sc[HB][G];
        float c[HB][G][4];
#pragma unroll
        for (int h = 0; h < HB; ++h) {
            load_words<D, B>(rec, h0 + h, lane, w[h]);
            // scales of tokens 16 half + r and + 8, groups in pairs
            const uint8_t* p = rec + 4 * D * B + (((lane >> 2) * 4 + 2 * (h0 + h)) * G) * 2;
            if constexpr (G == 2) {
                const uint2 u = *reinterpret_cast<const uint2*>(p);
                sc[h][0] = u.x;
                sc[h][1] = u.y;
            } else {
#pragma unroll
                for (int i = 0; i < G; i += 4) {
                    const uint4 u = *reinterpret_cast<const uint4*>(p + 4 * i);
                    sc[h][i] = u.x;
                    sc[h][i + 1] = u.y;
                    sc[h][i + 2] = u.z;
                    sc[h][i + 3] = u.w;
                }
            }
        }
#pragma unroll
        for (int step = 0; step < 2; ++step) {
            uint32_t a[HB][G][4];
#pragma unroll
            for (int h = 0; h < HB; ++h)
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    uint32_t(&x)[4] = a[h][g];
                    k_fragment<D, B>(w[h], g, step, x);
                    if constexpr (kNorm<B>)
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[i] = h2_bits(__hmul2(bits_h2(x[i]), bits_h2(0x64006400u)));
                    if (step == 0)
                        mma_f16_from(c[h][g], x[0], x[1], x[2], x[3], q.hi[g][0], q.hi[g][1], q.zq[g]);
                    else
                        mma_f16(c[h][g], x[0], x[1], x[2], x[3], q.hi[g][2], q.hi[g][3]);
                }
#pragma unroll
            for (int h = 0; h < HB; ++h)
#pragma unroll
                for (int g = 0; g < G; ++g)
                    mma_f16(c[h][g], a[h][g][0], a[h][g][1], a[h][g][2], a[h][g][3], q.lo[g][2 * step],
                            q.lo[g][2 * step + 1]);
        }
#pragma unroll
        for (int h = 0; h < HB; ++h)
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const __half2 u0 = bits_h2(sc[h][g / 2]), u1 = bits_h2(sc[h][G / 2 + g / 2]);
                const float s0 = (g & 1) ? __high2float(u0) : __low2float(u0);
                const float s1 = (g & 1) ? __high2float(u1) : __low2float(u1);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float si = i < 2 ? s0 : s1, ci = c[h][g][i];
                    s[h0 + h][i] = g == 0 ? ci * si : fmaf(ci, si, s[h0 + h][i]);
                }
            }
    }
}

// a value of the call's type, fp16 or bf16
QG_DEV float att_in(const KvAttend& a, uint16_t v) { return a.bf16 ? kv_to_float<true>(v) : kv_to_float<false>(v); }
QG_DEV uint16_t att_out(const KvAttend& a, float v) { return a.bf16 ? kv_from_float<true>(v) : kv_from_float<false>(v); }

// A rotated row's power-of-two scale (largest magnitude into [2^14, 2^15), so that
// both fp16 parts keep their bits; the score scale's sign goes with it), -z 2^-24,
// and the factor that turns a score into log2 units.  The factor is positive, so
// masked scores stay -inf and maxima can be taken before it.
struct AttRowScale {
    float up, zero, f;
};
template <int D>
QG_DEV AttRowScale att_row_scale(const KvAttend& a, float amax) {
    int e = (int)(__float_as_uint(amax) >> 23) - 127;  // 128 for infinity: no scaling then
    e = e >= 128 ? 14 : max(e, -100);
    AttRowScale r;
    r.up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
    if (a.scale < 0.f) r.up = -r.up;
    const float unit = a.pg.kb <= 5 ? 6.103515625e-5f : 5.9604644775390625e-8f;  // 2^-14 or 2^-24, see kNorm
    r.zero = -(float)(1 << (a.pg.kb - 1)) * unit;
    r.f = fmaxf(fabsf(a.scale) * (1.4426950408889634f / (float)D) / unit *
                    __uint_as_float((uint32_t)(127 - 14 + e) << 23),
                1e-30f);
    return r;
}

// Rotate query row n (of 8), a warp to a row, split it into its two
// parts and put them where the B operand's lanes read them (row n's dims
// 32 g + 8 j + i are lane 4 n + j's, pair i % 4, half i / 4).  p: the row in shared memory.
template <int D>
QG_DEV void rotate_query(const KvAttend& a, const uint16_t* p, float* area, int n, int lane) {
    using C = AttCfg<D>;
    constexpr int E = D / 32;
    float x[E];
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = att_in(a, p[E * lane + i]);
    fwht_warp<E>(x, lane);
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const AttRowScale rs = att_row_scale<D>(a, amax);
    uint16_t* out = reinterpret_cast<uint16_t*>(area);
    float sum = 0.f;
    const int g = E * lane / 32;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int d = E * lane + i, pair = d & 3;
        const float v = x[i] * rs.up;
        float vd = v * __uint_as_float((uint32_t)(127 - field_at(a.pg.kb, pair)) << 23);
        if (a.pg.kb == 4 && !(i & 1)) vd = fmaf(x[(i + 1) % E] * rs.up, -0.0625f, vd);
        const __half hi = __float2half_rn(vd), lo = __float2half_rn(vd - __half2float(hi));
        const int at = (((g * 2) * 32 + 4 * n + ((d & 31) >> 3)) * 4 + pair) * 2 + ((d >> 2) & 1);
        out[at] = __half_as_ushort(hi);
        out[at + 32 * 8] = __half_as_ushort(lo);
        sum += v;
    }
#pragma unroll
    for (int o = 1; o < 32 / E; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane % (32 / E) == 0) area[C::QZero + g * 8 + n] = rs.zero * sum;
    if (lane == 0) area[C::QFactor + n] = rs.f;
}

// The same for all rows of an item by one warp for itself, straight into the B
// operand's registers: lane 4 n + j rotates its share of row n, strides 1, 2, 4 and
// 32 .. within the lane, 8 and 16 between the four lanes of the row.
template <int D>
QG_DEV void rotate_queries(const KvAttend& a, int row0, int rows, int r_base, int head, int lane, AttQ<D>& q) {
    constexpr int G = D / 32;
    const int r = r_base + (lane >> 2);
    float x[G][8];
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[g][i] = 0.f;
    if (r < rows) {
        const int tok = r / a.group, hq = head * a.group + (r - tok * a.group);
        const uint16_t* p = reinterpret_cast<const uint16_t*>(a.q.p) + (row0 + tok) * a.q.row + hq * a.q.head;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const uint4 u = __ldg(reinterpret_cast<const uint4*>(p + 32 * g + 8 * (lane & 3)));
            const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[g][i] = att_in(a, (uint16_t)((i & 1) ? v[i / 2] >> 16 : v[i / 2] & 0xffff));
        }
    }
    float amax = 0.f;
#pragma unroll
    for (int st = 1; st < D; st <<= 1)
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (st < 8) {
                    if (i & st) continue;
                    const float u = x[g][i], v = x[g][i | (st & 7)];
                    x[g][i] = u + v;
                    x[g][i | (st & 7)] = u - v;
                } else if (st < 32) {
                    const float o = __shfl_xor_sync(0xffffffffu, x[g][i], st / 8);
                    x[g][i] = (lane & (st / 8)) ? o - x[g][i] : x[g][i] + o;
                } else {
                    if (g & (st / 32)) continue;
                    const float u = x[g][i], v = x[(g | (st / 32)) % G][i];
                    x[g][i] = u + v;
                    x[(g | (st / 32)) % G][i] = u - v;
                }
            }
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[g][i]));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const AttRowScale rs = att_row_scale<D>(a, amax);
    const int src = (lane & 3) * 8;  // lane of row 2 j
#pragma unroll
    for (int g = 0; g < G; ++g) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float u = x[g][i] * rs.up, v = x[g][i + 4] * rs.up;
            const float dn = __uint_as_float((uint32_t)(127 - field_at(a.pg.kb, i)) << 23);
            float ud = u * dn, vd = v * dn;
            if (a.pg.kb == 4 && !(i & 1)) {
                ud = fmaf(x[g][(i + 1) & 3] * rs.up, -0.0625f, ud);
                vd = fmaf(x[g][4 + ((i + 1) & 3)] * rs.up, -0.0625f, vd);
            }
            const __half2 hi = __floats2half2_rn(ud, vd);
            q.hi[g][i] = h2_bits(hi);
            q.lo[g][i] = h2_bits(__floats2half2_rn(ud - __low2float(hi), vd - __high2float(hi)));
            sum += u + v;
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        sum *= rs.zero;
        q.set_zero(g, __shfl_sync(0xffffffffu, sum, src), __shfl_sync(0xffffffffu, sum, src + 4));
    }
    q.f[0] = __shfl_sync(0xffffffffu, rs.f, src);
    q.f[1] = __shfl_sync(0xffffffffu, rs.f, src + 4);
}

template <int D>
QG_DEV void load_queries(const float* area, int lane, AttQ<D>& q) {
    using C = AttCfg<D>;
    constexpr int G = D / 32;
    const uint4* f = reinterpret_cast<const uint4*>(area);
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const uint4 h = f[(g * 2) * 32 + lane], l = f[(g * 2 + 1) * 32 + lane];
        q.hi[g][0] = h.x, q.hi[g][1] = h.y, q.hi[g][2] = h.z, q.hi[g][3] = h.w;
        q.lo[g][0] = l.x, q.lo[g][1] = l.y, q.lo[g][2] = l.z, q.lo[g][3] = l.w;
        const float2 z = *reinterpret_cast<const float2*>(area + C::QZero + g * 8 + 2 * (lane & 3));
        q.set_zero(g, z.x, z.y);
    }
    const float2 v = *reinterpret_cast<const float2*>(area + C::QFactor + 2 * (lane & 3));
    q.f[0] = v.x;
    q.f[1] = v.y;
}

// ------------------------------------------------------------------- output
// A registers of half a tile's V codes, (c - z) 2^-14 in units of their fields, one exact
// fused multiply-add a pair (which also makes them normal numbers, see kNorm): f[g][k][i]
// holds field i of group g's dims for tokens 16 half + 8 k + 2 j + {0, 1}.
template <int D, int B>
QG_DEV void v_fields(const uint8_t* part, int half, int lane, uint32_t (&f)[D / 32][2][4]) {
    constexpr int G = D / 32, NW = D * B / 64, UT = D / 64 * 8 * B;  // UT: bits of a token's units
    uint32_t w[NW];
    load_words<D, B>(part, half, lane, w);
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int unit = (g >> 1) * 8 * B + (g & 1) * 4 * B;  // this group's four codes in a token's units
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int t0 = (2 * k) * UT + unit, t1 = (2 * k + 1) * UT + unit;
            if constexpr (B <= 4) {
                const uint32_t x = halves_from(w, t0, t1, 4 * B);
                f[g][k][0] = field<B, 0>(x);
                f[g][k][1] = field<B, 1>(x);
                f[g][k][2] = field<B, 2 % Fld<B>::N>(x);
                f[g][k][3] = field<B, 3 % Fld<B>::N>(x);
            } else {
                const uint32_t x = halves_from(w, t0, t1, 2 * B), y = halves_from(w, t0 + 2 * B, t1 + 2 * B, 2 * B);
                f[g][k][0] = field<B, 0>(x);
                f[g][k][1] = field<B, 1>(x);
                f[g][k][2] = field<B, 0>(y);
                f[g][k][3] = field<B, 1>(y);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f[g][k][i] = h2_bits(__hfma2(bits_h2(f[g][k][i]), bits_h2(0x64006400u),
                                             bits_h2(Fld<B>::minus_zero(i % Fld<B>::N))));
        }
    }
}

// acc += (codes of V) x (weights times scales): half a tile.  w[c]: the weight of
// token 16 half + 8 (c / 2) + r for row 2 j + c % 2.  The product with the
// group's scale is taken in fp32 and rounded once, to the fp16 of the B operand;
// movmatrix turns it from [token][row] to [row][token].  hidden: bit 4 half + c of a
// (token, row) that the mask leaves out, whatever its scale holds; a visible token's NaN
// counts however small its weight.
template <int D, bool Masked>
QG_DEV void v_product(const uint8_t* scales, int half, int lane, const uint32_t (&f)[D / 32][2][4],
                      const float (&w)[4], uint32_t hidden, float (&acc)[D / 16][4]) {
    constexpr int G = D / 32;
    const int r = lane >> 2;
    const uint32_t pick = (r & 1) ? 0x7632u : 0x5410u;  // u of token 8 tt + r
    scales += ((r >> 1) * G * 8 + 4 * half) * 2;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const uint2 su = *reinterpret_cast<const uint2*>(scales + g * 16);
        const __half2 sh = bits_h2(__byte_perm(su.x, su.y, pick));
        const float s0 = __low2float(sh), s1 = __high2float(sh);
        float b[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            b[c] = w[c] * (c < 2 ? s0 : s1);
            if constexpr (Masked) b[c] = hidden >> (4 * half + c) & 1 ? 0.f : b[c];
        }
        const uint32_t b0 = movm_trans(h2_bits(__floats2half2_rn(b[0], b[1])));
        const uint32_t b1 = movm_trans(h2_bits(__floats2half2_rn(b[2], b[3])));
        mma_f16(acc[2 * g], f[g][0][0], f[g][0][1], f[g][1][0], f[g][1][1], b0, b1);
        mma_f16(acc[2 * g + 1], f[g][0][2], f[g][0][3], f[g][1][2], f[g][1][3], b0, b1);
    }
}

template <int D, int B, bool Masked>
QG_DEV void output_tile(const uint8_t* part, int lane, const float (&w)[2][4], uint32_t hidden, float (&acc)[D / 16][4]) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        uint32_t f[D / 32][2][4];
        v_fields<D, B>(part, half, lane, f);
        v_product<D, Masked>(part + 4 * D * B, half, lane, f, w[half], hidden, acc);
    }
}

// largest V scale among this lane's share of the tile's, up to token slot `last` (slots behind
// the last visible token may hold anything)
template <int D>
QG_DEV __half2 v_scale_max(const uint8_t* part, int vb, int lane, int last) {
    constexpr int G = D / 32, N = D / 64;  // words of a lane, [j][g][tt] in all
    const uint32_t* w = reinterpret_cast<const uint32_t*>(part + 4 * D * vb) + N * lane;
    __half2 m = bits_h2(0);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        uint32_t u = w[i];
        if (last < kTileTokens - 1) {
            const int at = N * lane + i, t = 8 * (at & 3) + 2 * (at / (4 * G));
            u &= t + 1 <= last ? 0xffffffffu : t <= last ? 0xffffu : 0u;
        }
        m = __hmax2(m, bits_h2(u));
    }
    return m;
}

// The largest that weights have to fit, among slots first to last: a hidden one shall not cost the
// visible ones their bits, and an infinite one makes its rows NaN whatever the weights.
template <int D>
QG_DEV float v_scale_fit(const uint8_t* part, int vb, int lane, int first, int last) {
    constexpr int G = D / 32, N = D / 64;
    const __half* s = reinterpret_cast<const __half*>(part + 4 * D * vb) + 2 * N * lane;
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 2 * N; ++i) {
        const int at = N * lane + i / 2, t = 8 * (at & 3) + 2 * (at / (4 * G)) + (i & 1);
        const float v = __half2float(s[i]);
        if (t >= first && t <= last && v < INFINITY) m = fmaxf(m, v);
    }
    return m;
}

// ------------------------------------------------------------------- the run
// What a sequence gives: n query rows (x group) in nrb blocks over `tiles` tiles
// from tile t0 on.  An item has one tile at least, so that empty rows are written.
struct AttSeq {
    int row0, n, len, pos0, t0, tiles, nrb;  // pos0: the first row's position
};

template <int RB>
QG_DEV AttSeq att_seq(const KvAttend& a, int b) {
    AttSeq s;
    s.row0 = max(a.bt.cu[b], 0);
    const int end = a.bt.cu[b + 1];
    s.n = min(end, a.bt.rows) - s.row0;
    s.len = a.bt.lens[b];
    s.pos0 = s.len - end + s.row0;
    s.t0 = 0;
    s.tiles = 1;
    s.nrb = 0;
    if (s.n <= 0) return s;
    s.nrb = (int)(((int64_t)s.n * a.group + RB - 1) / RB);
    if (s.len <= 0) return s;
    const int64_t first = a.window > 0 ? (int64_t)s.pos0 - a.window + 1 : 0;
    s.t0 = (int)(first > 0 ? first / kTileTokens : 0);
    s.tiles = (int)(((int64_t)s.len + kTileTokens - 1) / kTileTokens) - s.t0;
    return s;
}

QG_DEV long long div_ll(long long a, int b) {
    return (a >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

struct AttCursor {
    int b, h, rb, tile;
    AttSeq s;
};

// where tile number `at` of the call lies; prefix: tiles before each thread's chunk of sequences
template <int RB>
QG_DEV void att_seek(const KvAttend& a, const long long* prefix, int nthreads, int chunk, long long at, AttCursor& c) {
    int lo = 0, hi = min(nthreads, (a.bt.num_seqs + chunk - 1) / chunk);  // the last entry <= at is in [lo, hi)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] <= at)
            lo = mid;
        else
            hi = mid;
    }
    long long rem = at - prefix[lo];
    c.b = lo * chunk;
    for (;; ++c.b) {
        c.s = att_seq<RB>(a, c.b);
        const long long work = (long long)c.s.nrb * a.pg.heads * c.s.tiles;
        if (rem < work || c.b + 1 >= a.bt.num_seqs) break;
        rem -= work;
    }
    const long long item = div_ll(rem, c.s.tiles);
    c.tile = (int)(rem - item * c.s.tiles);
    c.h = (int)div_ll(item, max(c.s.nrb, 1));
    c.rb = (int)(item - (long long)c.h * c.s.nrb);
}

// the next tile, number `at` of the call, if there is one (`more`); sequences without
// rows are passed over by a new search
template <int RB>
QG_DEV void att_next(const KvAttend& a, const long long* prefix, int nthreads, int chunk, AttCursor& c, bool more,
                     long long at) {
    if (++c.tile < c.s.tiles) return;
    c.tile = 0;
    if (++c.rb < c.s.nrb) return;
    c.rb = 0;
    if (++c.h < a.pg.heads) return;
    c.h = 0;
    if (!more || c.b + 1 >= a.bt.num_seqs) return;
    ++c.b;
    c.s = att_seq<RB>(a, c.b);
    if (c.s.nrb == 0) att_seek<RB>(a, prefix, nthreads, chunk, at, c);
}

// rotate back, divide and store one row held by a warp (E consecutive dims a lane);
// at: the row's number, (query row) x group + (head of the group)
template <int D>
QG_DEV void store_row(const KvAttend& a, float (&o)[D / 32], float m, float l, int at, int head, int lane) {
    constexpr int E = D / 32;
    fwht_warp<E>(o, lane);
    const int row = at / a.group, hq = head * a.group + (at - row * a.group);
    const float inv = l == 0.f ? 0.f : 1.f / (l * (float)D);
    uint16_t v[E];
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = att_out(a, o[i] * inv);
    uint16_t* p = reinterpret_cast<uint16_t*>(a.out.p) + (int64_t)row * a.out.row + hq * a.out.head + E * lane;
    if constexpr (E == 2) {
        *reinterpret_cast<uint32_t*>(p) = v[0] | (uint32_t)v[1] << 16;
    } else {
#pragma unroll
        for (int i = 0; i < E; i += 4)
            *reinterpret_cast<uint2*>(p + i) = make_uint2(v[i] | (uint32_t)v[i + 1] << 16, v[i + 2] | (uint32_t)v[i + 3] << 16);
    }
    if (a.lse && lane == 0) a.lse[(int64_t)row * a.q_heads + hq] = (m + log2f(l)) * 0.6931471805599453f;
}

// KB, VB: the widths, or 0 where they are read from `a`.  Known widths make a tile's
// work one run of instructions that hides the softmax's latency behind the codes' masks;
// they are built for 4/4 and 8/8.  Known against read, us (8 KV heads, 64 query heads; one long
// sequence, and 64 of 200 to 4096 tokens):
//   64 dims, 524288 tokens: 4/4 111 / 114, 50 / 52; 8/8 107 / 117, 55 / 60;
//   128 dims, 262144 tokens: 4/4 98 / 107, 76 / 86; 8/8 100 / 109, 78 / 92;
//   256 dims, 131072 tokens: 4/4 112 / 119, 140 / 161.
template <int D, int KB, int VB>
__global__ void __launch_bounds__(AttCfg<D, KB, VB>::T, 1) kv_attend_kernel(KvAttend a) {
    if constexpr (KB > 0) {
        a.pg.kb = KB;
        a.pg.vb = VB;
    }
    using C = AttCfg<D, KB, VB>;
    constexpr int W = C::W, G = C::G, RB = C::RB, E = D / 32, T = C::T;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ long long sh_total[W];
    __shared__ uint32_t sh_items[W];
    __shared__ int sh_last[2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rec_bytes = kv_record_bytes<D>(a.pg.kb, a.pg.vb), k_bytes = 4 * D * a.pg.kb + 2 * D;
    float* slots = reinterpret_cast<float*>(smem);
    float* areas = reinterpret_cast<float*>(smem + C::QAt);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BarAt) + warp * kAttMaxStages;
    AttFrag* frags = reinterpret_cast<AttFrag*>(smem + C::FragAt);
    long long* prefix = reinterpret_cast<long long*>(smem + C::PrefixAt);
    uint8_t* rings = smem + C::RingAt;
    uint8_t* ring = rings + warp * a.ring_bytes;

    // ---- the call's work, this CTA's and each warp's share
    const int chunk = (a.bt.num_seqs + T - 1) / T;
    long long mine = 0, mine_items = 0;
    for (int b = threadIdx.x * chunk; b < min((int)(threadIdx.x + 1) * chunk, a.bt.num_seqs); ++b) {
        const AttSeq s = att_seq<RB>(a, b);
        mine += (long long)s.nrb * a.pg.heads * s.tiles;
        mine_items += (long long)s.nrb * a.pg.heads;
    }
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
    }
    // (items are only averaged over: a count that saturates does)
    const uint32_t warp_items = __reduce_add_sync(0xffffffffu, (uint32_t)min(mine_items, 1ll << 21));
    if (lane == 31) {
        sh_total[warp] = inc;
        sh_items[warp] = warp_items;
    }
    if (lane < kAttMaxStages) mbar_init(&full[lane], 1);
    if (threadIdx.x < 2 * W) frags[threadIdx.x].tiles = 0;
    fence_mbar_init();
    __syncthreads();
    long long before = 0, total = 0, total_items = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        if (w < warp) before += sh_total[w];
        total += sh_total[w];
        total_items += sh_items[w];
    }
    prefix[threadIdx.x] = before + inc - mine;
    __syncthreads();
    // An average item's tiles a CTA at least, up to 16 of them: a join across CTAs costs more
    // than two tiles a warp
    const long long share =
        max(div_ll(total + gridDim.x - 1, gridDim.x), min(div_ll(total + total_items - 1, max((int)total_items, 1)), 16ll));
    const long long cta0 = min(share * blockIdx.x, total), cta1 = min(cta0 + share, total);
    if (cta0 >= cta1) return;
    // warp w's first tile: shares differ by one at most
    const int cta_tiles = (int)(cta1 - cta0);
    const long long w0 = cta0 + (cta_tiles / W) * warp + min(warp, cta_tiles % W);
    int count = cta_tiles / W + (warp < cta_tiles % W ? 1 : 0);
    const long long w_end = w0 + count;

    // ---- Walk the CTA's first items.  Where it has no more than QN all warps share their
    // rotated queries: each warp fetches some of the rows here, ahead of the cache's tiles,
    // and rotates them once those are on their way.
    uint16_t* raw = reinterpret_cast<uint16_t*>(smem);  // [item][RB][D], over the slots
    auto fetch_row = [&](const AttSeq& s, int head, int rb, int r, uint16_t* dst) {
        r += rb * RB;
        const uint16_t* p = nullptr;
        if (r < s.n * a.group) {
            const int tok = s.n == 1 ? 0 : r / a.group, hq = head * a.group + (r - tok * a.group);
            p = reinterpret_cast<const uint16_t*>(a.q.p) + (s.row0 + tok) * a.q.row + hq * a.q.head;
        }
        for (int i = lane * 8; i < D; i += 256) {  // 16 bytes a lane
            if (p)
                cp_async16(dst + i, p + i);
            else
                *reinterpret_cast<uint4*>(dst + i) = make_uint4(0, 0, 0, 0);
        }
    };
    // The warp's own place first: the first entries of its block table are on their way meanwhile.
    const int lps = 31 - __clz(a.pg.page_size / kTileTokens);  // log2 tiles per page
    AttCursor pc{}, cc;                                        // the place of the copies, the place of the sums
    int page_base = 0, page_b = -1, page_id = 0;               // lane i: page page_base + i of sequence page_b
    auto load_pages = [&](int pi) {
        page_b = pc.b;
        page_base = pi;
        const int i = pi + lane;
        page_id = i < a.bt.max_pages && ((int64_t)i << lps) * kTileTokens < pc.s.len
                      ? a.bt.table[pc.b * a.bt.table_stride + i]
                      : -1;
    };
    if (count > 0) {
        att_seek<RB>(a, prefix, T, chunk, w0, pc);
        load_pages((pc.s.t0 + pc.tile) >> lps);
    }
    cc = pc;
    int my_item = 0, items = 0;
    {
        AttCursor c;
        att_seek<RB>(a, prefix, T, chunk, cta0, c);
        long long at = cta0 - c.tile;
        for (; items <= C::QN && at < cta1; ++items) {
            if (items < C::QN)
                for (int r = (warp + W - items * RB % W) % W; r < RB; r += W)
                    fetch_row(c.s, c.h, c.rb, r, raw + (items * RB + r) * D);
            if (w0 >= at) my_item = items;
            at += c.s.tiles;
            c.tile = c.s.tiles - 1;
            att_next<RB>(a, prefix, T, chunk, c, at < cta1, at);
        }
    }
    const bool shared_q = items <= C::QN;

    // ---- The ring: whole records, each warp its own.
    int left = count, page_left = 0;                           // tiles of the run, of the page, still to copy
    uint32_t bad = 0;                                          // stages whose tile has no page
    bool dead = false, has = false;
    const uint8_t* src = nullptr;
    auto issue = [&](int s) {
        if (page_left == 0) {
            const int t = pc.s.t0 + pc.tile, pi = t >> lps, in = t & ((1 << lps) - 1);
            if (page_b != pc.b || (uint32_t)(pi - page_base) >= 32u) load_pages(pi);
            const int page = __shfl_sync(0xffffffffu, page_id, pi - page_base);
            has = (uint32_t)page < (uint32_t)a.pg.num_pages && pc.s.len > 0;
            if (!has && pc.s.len > 0 && lane == 0) set_dev_error(QGEMM_DEV_BAD_PAGE);
            src = a.pg.base + page * a.pg.page_bytes + (int64_t)((pc.h << lps) + in) * rec_bytes;
            page_left = min((1 << lps) - in, pc.s.tiles - pc.tile);
        }
        bad = (bad & ~(1u << s)) | (has ? 0u : 1u << s);
        if (lane == 0) {
            if (has && !dead) {
                mbar_arrive_expect_tx(&full[s], rec_bytes);
                bulk_g2s(ring + s * rec_bytes, src, rec_bytes, &full[s]);
            } else {
                mbar_arrive(&full[s]);
            }
        }
        src += rec_bytes;
        --left;
        ++pc.tile;
        if (--page_left == 0 && pc.tile == pc.s.tiles) {
            --pc.tile;
            att_next<RB>(a, prefix, T, chunk, pc, left > 0, w_end - left);
        }
    };
    for (int i = 0; i < a.stages && left > 0; ++i) issue(i);

    // ---- rotated queries: rows of the CTA's items dealt out to the warps
    cp_async_wait_all();
    __syncwarp();
    if (shared_q)
        for (int i = 0; i < items; ++i)
            for (int r = (warp + W - i * RB % W) % W; r < RB; r += W)
                rotate_query<D>(a, raw + (i * RB + r) * D, areas + i * C::QFloats, r, lane);
    __syncthreads();

    // ---- one warp's run, item by item
    AttQ<D> q;
    float acc[2 * G][4], mo[2], l[2];  // weights are 2^(x - mo)
    int stage = 0, parity = 0, rec_at = 0;
    const int j = lane & 3, r8 = lane >> 2;
    for (long long at = w0; count > 0;) {
        const AttSeq& cs = cc.s;
        const int n_tiles = min(count, cs.tiles - cc.tile);  // of this item, here
        const int rows = cs.n * a.group, r_base = cc.rb * RB;
        if (shared_q)
            load_queries<D>(areas + my_item * C::QFloats, lane, q);
        else
            rotate_queries<D>(a, cs.row0, rows, r_base, cc.h, lane, q);
        ++my_item;
        const int lo_pos = cs.pos0 + r_base / a.group;
        const int hi_pos = cs.pos0 + (min(r_base + RB, rows) - 1) / a.group;
        // tiles [u0, u1) of these are seen whole by every row
        const int t_base = (cs.t0 + cc.tile) * kTileTokens;
        const int u1 = (lo_pos + 1 - t_base) >> 5, u0 = a.window > 0 ? ((hi_pos - a.window - t_base) >> 5) + 1 : 0;
        int qpos[2], ve = kAttLowest;  // ve: exponent of the largest V scale seen
        float limit[2];       // a score may reach this before mo moves
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            qpos[c] = cs.pos0 + (r_base + 2 * j + c) / a.group;
            mo[c] = limit[c] = kAttNone;
            l[c] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 2 * G; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[i][c] = 0.f;
#pragma unroll 1
        for (int it = 0; it < n_tiles; ++it) {
            if (!mbar_try_wait(&full[stage], parity) && !dead && !mbar_wait(&full[stage], parity)) dead = true;
            // (given up: no copy is issued any more and nothing is waited for; the run goes on over
            // whatever the ring holds, and the error word says so)
            float s[2][4];
            const uint8_t* rec = ring + rec_at;
            const uint8_t* vpart = rec + k_bytes;
            if constexpr (KB > 0) {
                scores_tile<D, KB>(rec, lane, q, s);
            } else {
                switch (a.pg.kb) {
#define QG_SCORES(B)                        \
    case B:                                 \
        scores_tile<D, B>(rec, lane, q, s); \
        break;
                    QG_SCORES(2)
                    QG_SCORES(3)
                    QG_SCORES(4)
                    QG_SCORES(5)
                    QG_SCORES(6)
                    QG_SCORES(8)
#undef QG_SCORES
                }
            }
            // a tile without a page shows nothing
            const bool none = bad >> stage & 1;
            const bool masked = it < u0 || it >= u1 || none;
            int last = kTileTokens;  // last slot that any row sees
            uint32_t hidden = 0;
            // A score of a visible token is -inf only where its scale is infinite: the sum it meets is 0 where
            // append left zero points, give or take a rounding, and 0 x inf is not a number.  (Left at -inf it
            // would drop the token without a trace; +inf makes the row NaN by itself.)
            const float nan = __uint_as_float(0x7fc00000u);
            if (masked) {
                const int t_first = t_base + it * kTileTokens;
                last = none ? -1 : hi_pos - t_first;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int t = t_first + 16 * h + 8 * (c >> 1) + r8, pos = qpos[c & 1];
                        if (t > pos || none || (a.window > 0 && t <= pos - a.window)) {
                            s[h][c] = -INFINITY;
                            hidden |= 1u << (4 * h + c);
                        } else if (s[h][c] == -INFINITY) {
                            s[h][c] = nan;
                        }
                    }
            }
            // Weights are 2^(x - mo): at most 2^(10 - ve) when mo is set, and it is moved when one
            // would pass 2^(14 - ve), so that weight times scale (below 2^(ve + 1)) fits fp16.
            // (The weights are computed before it is known, again if it has to be moved, and after the rare
            // infinite score of a tile seen whole, which takes the same branch: 1% in all, 2% in one of its own.)
            float w[2][4];
            auto weigh = [&] {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        w[h][c] = ex2(fmaf(s[h][c], q.f[c & 1], -mo[c & 1]));
            };
            weigh();
            float tm[2];
            bool over = false;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                tm[c] = q.f[c] * fmaxf(fmaxf(s[0][c], s[0][c + 2]), fmaxf(s[1][c], s[1][c + 2]));
                over |= tm[c] > limit[c];
            }
            const __half2 vmax = v_scale_max<D>(vpart, a.pg.vb, lane, last);
            over |= !__hblt2(vmax, bits_h2((uint32_t)(16 + ve) * 0x04000400u));  // 2^(ve + 1), infinity for 15
            const float lo = fminf(fminf(fminf(s[0][0], s[0][1]), fminf(s[0][2], s[0][3])),
                                   fminf(fminf(s[1][0], s[1][1]), fminf(s[1][2], s[1][3])));
            over |= !masked && lo == -INFINITY;
            if (__any_sync(0xffffffffu, over)) {
                if (!masked)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int c = 0; c < 4; ++c) s[h][c] = s[h][c] == -INFINITY ? nan : s[h][c];
                const int first = a.window > 0 ? lo_pos - a.window + 1 - t_base - it * kTileTokens : 0;
                float t = v_scale_fit<D>(vpart, a.pg.vb, lane, first, last);
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
                const int vn = min(max((int)(__float_as_uint(t) >> 23) - 127, ve), 15);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    t = tm[c];
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
                    const float mn = fmaxf(mo[c] + (float)(vn - ve), t - (float)(10 - vn));
                    const float k = mo[c] == mn ? 1.f : ex2(mo[c] - mn);
                    mo[c] = mn;
                    limit[c] = mn + (float)(14 - vn);
                    l[c] *= k;
#pragma unroll
                    for (int i = 0; i < 2 * G; ++i) {
                        acc[i][c] *= k;
                        acc[i][c + 2] *= k;
                    }
                }
                ve = vn;
                weigh();
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                l[0] += w[h][0] + w[h][2];
                l[1] += w[h][1] + w[h][3];
            }
            if constexpr (VB > 0) {
                if (masked)
                    output_tile<D, VB, true>(vpart, lane, w, hidden, acc);
                else
                    output_tile<D, VB, false>(vpart, lane, w, 0, acc);
            } else {
                switch (a.pg.vb) {
#define QG_OUTPUT(B)                                               \
    case B:                                                        \
        if (masked)                                                \
            output_tile<D, B, true>(vpart, lane, w, hidden, acc);  \
        else                                                       \
            output_tile<D, B, false>(vpart, lane, w, 0, acc);      \
        break;
                    QG_OUTPUT(2)
                    QG_OUTPUT(3)
                    QG_OUTPUT(4)
                    QG_OUTPUT(5)
                    QG_OUTPUT(6)
                    QG_OUTPUT(8)
#undef QG_OUTPUT
                }
            }
            __syncwarp();
            if (left > 0) issue(stage);
            rec_at += rec_bytes;
            if (++stage == a.stages) {
                stage = rec_at = 0;
                parity ^= 1;
            }
        }
        // this warp's part of the item is done: its slot, in the sums' own units
        const bool frag_head = cc.tile == 0;
        // (one that began before this warp is its first, and may leave copies in flight;
        // one that goes on behind it is its last, and finds the ring drained)
        float* slot = frag_head ? reinterpret_cast<float*>(ring) : slots + warp * C::SlotFloats;
        AttFrag& fr = frags[warp * 2 + (frag_head ? 1 : 0)];
#pragma unroll
        for (int i = 0; i < 2 * G; ++i)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float &u = acc[i][c], &v = acc[i][c + 2];  // fields 2 (i % 2) and the next
                u *= __uint_as_float((uint32_t)(127 + 14 - field_at(a.pg.vb, 2 * (i & 1))) << 23);
                v *= __uint_as_float((uint32_t)(127 + 14 - field_at(a.pg.vb, 2 * (i & 1) + 1)) << 23);
                if (a.pg.vb == 4) v -= u * 0.0625f;
            }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) l[c] += __shfl_xor_sync(0xffffffffu, l[c], o);
        }
        if (frag_head && cc.tile + n_tiles == cs.tiles) {
            // the whole item: rotate back in this layout (dim 32 g + 4 r + i) and store
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float x[G][4];
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[g][i] = acc[2 * g + (i >> 1)][(i & 1) * 2 + c];
#pragma unroll
                for (int g = 0; g < G; ++g) {
#pragma unroll
                    for (int st = 1; st < 4; st <<= 1)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (!(i & st)) {
                                const float u = x[g][i], v = x[g][i + st];
                                x[g][i] = u + v;
                                x[g][i + st] = u - v;
                            }
#pragma unroll
                    for (int ls = 4; ls < 32; ls <<= 1)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float o = __shfl_xor_sync(0xffffffffu, x[g][i], ls);
                            x[g][i] = (lane & ls) ? o - x[g][i] : x[g][i] + o;
                        }
                }
#pragma unroll
                for (int st = 1; st < G; st <<= 1)
#pragma unroll
                    for (int g = 0; g < G; ++g)
                        if (!(g & st))
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float u = x[g][i], v = x[g + st][i];
                                x[g][i] = u + v;
                                x[g + st][i] = u - v;
                            }
                const int r = r_base + 2 * j + c;
                if (r < rows) {
                    const int tok = r / a.group, hq = cc.h * a.group + (r - tok * a.group);
                    const float inv = l[c] == 0.f ? 0.f : 1.f / (l[c] * (float)D);
                    uint16_t* o = reinterpret_cast<uint16_t*>(a.out.p) + (cs.row0 + tok) * a.out.row +
                                  hq * a.out.head + 4 * r8;
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        uint16_t v[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[i] = att_out(a, x[g][i] * inv);
                        *reinterpret_cast<uint2*>(o + 32 * g) =
                            make_uint2(v[0] | (uint32_t)v[1] << 16, v[2] | (uint32_t)v[3] << 16);
                    }
                    if (a.lse && r8 == 0)
                        a.lse[(int64_t)(cs.row0 + tok) * a.q_heads + hq] =
                            (mo[c] + log2f(l[c])) * 0.6931471805599453f;
                }
            }
        } else {
            __syncwarp();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int r = 2 * j + c;
#pragma unroll
                for (int g = 0; g < G; ++g)
                    *reinterpret_cast<float4*>(slot + r * C::OS + 32 * g + 4 * r8) =
                        make_float4(acc[2 * g][c], acc[2 * g][c + 2], acc[2 * g + 1][c],
                                    acc[2 * g + 1][c + 2]);
                if (r8 == 0) {
                    slot[RB * C::OS + r] = mo[c];
                    slot[RB * C::OS + RB + r] = l[c];
                }
            }
            if (lane == 0) {
                // the item's first tile as a number of the call
                fr.item = at - cc.tile;
                fr.row0 = cs.row0 * a.group + r_base;
                fr.rows = min(RB, rows - r_base);
                fr.head = cc.h;
                fr.tiles = cs.tiles;
            }
        }
        at += n_tiles;
        count -= n_tiles;
        cc.tile = cs.tiles - 1;
        att_next<RB>(a, prefix, T, chunk, cc, count > 0, at);
    }
    if (dead)  // what is still in flight into this warp's ring
        for (int i = 0; i < a.stages; ++i) mbar_wait(&full[i], parity ^ (i < stage ? 1 : 0));
    __syncthreads();

    // ---- join: fragments lie in order (warp, slot); those of one item are neighbours
    float* weights = areas;                          // [RB][MaxCtas]
    float* rowbuf = areas + RB * C::MaxCtas;         // [RB][D]
    float* stats = rowbuf + RB * D;                  // [RB][2 W] maxima, then sums, by the group's first fragment
    constexpr int Vecs = RB * D / 4;                 // float4s of an item's rows
    auto slot_of = [&](int k) {
        return (k & 1) ? reinterpret_cast<float*>(rings + (k >> 1) * a.ring_bytes) : slots + (k >> 1) * C::SlotFloats;
    };
    // lane k < 2 W: fragment k, the first and the last of its group
    const AttFrag fr = frags[min(lane, 2 * W - 1)];
    const bool active = lane < 2 * W && fr.tiles > 0;
    const uint32_t act = __ballot_sync(0xffffffffu, active);
    if (act == 0) return;
    const uint32_t below = act & ((1u << lane) - 1u);
    const int prev = below ? 31 - __clz(below) : 0;
    const long long prev_item = __shfl_sync(0xffffffffu, fr.item, prev);
    const uint32_t heads = __ballot_sync(0xffffffffu, active && (below == 0 || prev_item != fr.item));
    const uint32_t upto = heads & ((2u << lane) - 1u), above = heads & ~((2u << lane) - 1u);
    const int gfirst = upto ? 31 - __clz(upto) : 0, gend = above ? __ffs(above) - 1 : 2 * W;
    const bool whole = fr.item >= cta0 && fr.item + fr.tiles <= cta1;
    for (int r = warp; r < RB; r += W) {
        const float* sl = slot_of(active ? lane : gfirst);
        const float ms = active ? sl[RB * C::OS + r] : -INFINITY, ls = active ? sl[RB * C::OS + RB + r] : 0.f;
        float mx = ms;
#pragma unroll
        for (int o = 1; o < 2 * W; o <<= 1) {
            const float v = __shfl_up_sync(0xffffffffu, mx, o);
            if (lane - o >= gfirst) mx = fmaxf(mx, v);
        }
        mx = __shfl_sync(0xffffffffu, mx, gend - 1);
        const float w = !active ? 0.f : ms == mx ? 1.f : ex2(ms - mx);
        float lt = active ? w * ls : 0.f;
#pragma unroll
        for (int o = 1; o < 2 * W; o <<= 1) {
            const float v = __shfl_up_sync(0xffffffffu, lt, o);
            if (lane - o >= gfirst) lt += v;
        }
        if (lane < 2 * W) weights[r * C::MaxCtas + lane] = w;
        lt = __shfl_sync(0xffffffffu, lt, gend - 1);
        if (heads >> lane & 1) {
            stats[r * 2 * W + lane] = mx;
            stats[(RB + r) * 2 * W + lane] = lt;
            if (!whole) {
                float* gslot = a.partial + ((size_t)blockIdx.x * 2 + (fr.item < cta0 ? 0 : 1)) * C::GSlot;
                gslot[RB * D + r] = mx;
                gslot[RB * D + RB + r] = lt;
            }
        }
    }
    __syncthreads();
    // each group's sum of weighted fragments into its first one (element by element the same thread's), or out
    const uint32_t wholes = __ballot_sync(0xffffffffu, whole) & heads;
    for (uint32_t hs = heads; hs; hs &= hs - 1) {
        const int f = __ffs(hs) - 1, e = __shfl_sync(0xffffffffu, gend, f);
        const long long item = __shfl_sync(0xffffffffu, fr.item, f);
        float* dst = a.partial + ((size_t)blockIdx.x * 2 + (item < cta0 ? 0 : 1)) * C::GSlot;
        for (int i = threadIdx.x; i < Vecs; i += T) {
            const int r = i / (D / 4), at = r * C::OS + (i % (D / 4)) * 4;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (uint32_t ks = act & ~((1u << f) - 1u) & (uint32_t)((1ull << e) - 1u); ks; ks &= ks - 1) {
                const int k = __ffs(ks) - 1;
                const float w = weights[r * C::MaxCtas + k];
                const float4 v = *reinterpret_cast<const float4*>(slot_of(k) + at);
                o.x = fmaf(w, v.x, o.x);
                o.y = fmaf(w, v.y, o.y);
                o.z = fmaf(w, v.z, o.z);
                o.w = fmaf(w, v.w, o.w);
            }
            if (wholes >> f & 1)
                *reinterpret_cast<float4*>(slot_of(f) + at) = o;
            else
                *reinterpret_cast<float4*>(dst + 4 * i) = o;
        }
    }
    if (wholes != heads) __threadfence();
    __syncthreads();
    // a group that goes on in other CTAs: its last CTA to get here joins them (at most two
    // groups a CTA; the ticket is that of the item's first CTA)
    if (warp == 0 && (heads >> lane & 1) && !whole) {
        const int c0 = (int)(fr.item / share), c1 = (int)((fr.item + fr.tiles - 1) / share);
        const bool last = atomicAdd(&a.tickets[c0], 1u) == (unsigned)(c1 - c0);
        if (last) a.tickets[c0] = 0;
        __threadfence();
        sh_last[fr.item < cta0 ? 0 : 1] = last;
    }
    for (int i = warp; i < __popc(wholes) * RB; i += W) {
        const int f = __fns(wholes, 0, i / RB + 1), r = i % RB;
        const AttFrag& g = frags[f];
        if (r >= g.rows) continue;
        float o[E];
#pragma unroll
        for (int k = 0; k < E; ++k) o[k] = slot_of(f)[r * C::OS + E * lane + k];
        store_row<D>(a, o, stats[r * 2 * W + f], stats[(RB + r) * 2 * W + f], g.row0 + r, g.head, lane);
    }
    if (wholes == heads) return;
    __syncthreads();
    for (uint32_t hs = heads & ~wholes; hs; hs &= hs - 1) {
        const AttFrag g = frags[__ffs(hs) - 1];
        if (!sh_last[g.item < cta0 ? 0 : 1]) continue;
        const int c0 = (int)(g.item / share), c1 = (int)((g.item + g.tiles - 1) / share);
        auto part_of = [&](int k) { return a.partial + ((size_t)k * 2 + (k == c0 ? 1 : 0)) * C::GSlot; };
        __syncthreads();
        for (int r = warp; r < RB; r += W) {
            float ms[C::MaxCtas / 32], ls[C::MaxCtas / 32], mx = -INFINITY, lt = 0.f;
#pragma unroll
            for (int i = 0; i < C::MaxCtas / 32; ++i) {
                const int k = c0 + lane + 32 * i;
                ms[i] = k <= c1 ? __ldcg(part_of(k) + RB * D + r) : -INFINITY;
                ls[i] = k <= c1 ? __ldcg(part_of(k) + RB * D + RB + r) : 0.f;
                mx = fmaxf(mx, ms[i]);
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
#pragma unroll
            for (int i = 0; i < C::MaxCtas / 32; ++i) {
                const int k = c0 + lane + 32 * i;
                if (k > c1) continue;
                const float w = ms[i] == mx ? 1.f : ex2(ms[i] - mx);
                lt = fmaf(w, ls[i], lt);
                weights[r * C::MaxCtas + k - c0] = w;
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) lt += __shfl_xor_sync(0xffffffffu, lt, o);
            if (lane == 0) {
                stats[r * 2 * W] = mx;
                stats[(RB + r) * 2 * W] = lt;
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < Vecs; i += T) {
            const int r = i / (D / 4);
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
            for (int k = c0; k <= c1; ++k) {
                const float w = weights[r * C::MaxCtas + k - c0];
                const float4 v = __ldcg(reinterpret_cast<const float4*>(part_of(k)) + i);
                o.x = fmaf(w, v.x, o.x);
                o.y = fmaf(w, v.y, o.y);
                o.z = fmaf(w, v.z, o.z);
                o.w = fmaf(w, v.w, o.w);
            }
            *reinterpret_cast<float4*>(rowbuf + 4 * i) = o;
        }
        __syncthreads();
        for (int r = warp; r < g.rows; r += W) {
            float o[E];
#pragma unroll
            for (int k = 0; k < E; ++k) o[k] = rowbuf[r * D + E * lane + k];
            store_row<D>(a, o, stats[r * 2 * W], stats[(RB + r) * 2 * W], g.row0 + r, g.head, lane);
        }
    }
}

}  // namespace qg
