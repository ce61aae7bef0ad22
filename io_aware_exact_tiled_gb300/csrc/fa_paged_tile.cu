// Attention over the paged 8-bit cache for requests with many query rows
// (prompts and pieces of prompts): tcgen05 products on tiles of 128 rows.
//
// Same computation as fa_paged_split.cuh. With hundreds of rows for each cached key
// the time is that of the two products, 4 n len d flops for each query head.
// Measured against 1,871 TFLOP/s of bf16 products: d = 128, two requests of
// about 2,000 new tokens behind 15,000 to 16,384, 32 query heads, 789 us = 1,345
// TFLOP/s (the chain of S, softmax and P V of two row tiles: the tensor pipe is
// active 57 % of the time); d = 64, eight prompts of 314 to 1,967 tokens, 16
// heads, 98 us = 255 TFLOP/s (a unit's start and end, and three times the
// products' time for the softmax).
//
// Work: a unit is (request, key head, pair of row tiles); a row is (new token,
// query head of the group), token-major, so that a tile of 128 rows sees
// nearly the same keys in all of them. The units' key tiles (128 keys, only
// those that some row sees) form one line that is cut into equal quotas for
// the persistent CTAs, as in the split-key kernel; the rows of a unit that was
// cut are merged by whoever finishes last. Each unit takes kPtUnitCost more
// places on the line than it has tiles: what its start and end cost.
//
// A CTA holds two row tiles so that each V tile is converted once for 256
// rows. Warps:
//   0      copies K and V tiles by TMA, E4M3 as they lie, and their block scales
//          (units of one row tile: without the scales)
//   1, 2   issue the products of row tile 0, 1
//   3      allocates TMEM (units of one row tile: then fetches the block scales)
//   4-7    softmax of row tile 0: thread = row
//   8-11   softmax of row tile 1
//   12-15  convert V to f16: thread = key
//
// S = Q K^T runs on 8-bit operands: each row of Q, divided by a power of two,
// is the sum of two numbers, in E5M2 (three of bfloat16's eight bits) and E4M3
// (the other five, one of them by its sign). Both hold an element exactly down
// to 2^-13 of the row's largest (E4M3 ends there); a row with more than an eighth
// of its elements below that, or that leaves out more than 2^-20 of its largest,
// summed over its elements, makes its row tile wide: then Q is three numbers in
// E5M2, exact down to 2^-23 and within 2^-31 of the largest below. Two 8-bit
// products cost what one f16 product costs, and K needs no conversion and half
// the shared memory; three cost half as much again. Measured, rows of normal
// values and the same with a channel 4,096 times larger: pieces of prompts 789
// and 891 us at d = 128, 690 and 714 at d = 64; prompts 152 and 211, 97 and 125
// us (a wide row is split twice).
// O += P V runs on f16: V's numbers convert exactly, P keeps 11 bits.
// Block scales: ks multiplies the exponent's slope and log2(vs) is added to
// the exponent, so P holds 2^(s - mu) vs; mu follows the largest of these
// products, and P's rounding is relative to it whatever the scales are. The
// row sum takes vs out again, for each group of 16 keys (the smallest block).
#include <math_constants.h>

#include "fa_common.cuh"
#include "fa_paged.h"
#include "tmap.h"

namespace fa {

constexpr float kPtLn2 = 0.69314718055994530942f;
constexpr float kPtRescale = 8.0f;  // log2 units
constexpr float kPtOffset = 6.0f;   // log2 of the factor on P before its rounding to f16
constexpr float kPtSpan = 60.0f;    // log2 of the largest ratio of V's block scales that is kept apart
// key tiles' time that a unit's Q, first S and output take (eight prompts of 256
// to 1,999 tokens, 16 heads: d = 64 105 us with 1, 94 with 6, 99 with 12; d = 128
// 177, 160 with 6, 155 with 8 and with 12)
template <int D>
constexpr int kPtUnitCost = paged_tile_cost(D);
constexpr int kPtScaleSlots = 8;
constexpr uint32_t kFmtE5M2 = 1;  // kind::f8f6f4 operand format code
constexpr int kPtNanSlots = 4;
constexpr int kPtAhead = 8;  // tiles whose block ids and scales are on their way or in use

template <int D, bool ONE>
struct PtCfg {
    // K stages, and stages of V as it lies in the cache (d = 128, where the third
    // part of Q takes their room: 795 us for pieces of prompts with three and two
    // stages and Q's two parts alone, 793 with these; units of one row tile have
    // one Q there)
    static constexpr int KS = D == 128 ? (ONE ? 3 : 2) : 6;
    static constexpr int RS = D == 128 ? (ONE ? 3 : 1) : 4;
    // Barriers that tell of K's arrival, tile u's being u % KB. A wait by parity
    // tells two rounds of a barrier apart but not three, so whoever waits for a
    // tile has to know that the one before with its barrier has landed. ONE: a
    // product warp knows that of every other tile, its own.
    static constexpr int KB = ONE && KS % 2 ? 2 * KS : KS;
    static_assert(!ONE || KB % 2 == 0, "barriers of K of units of one row tile");
    static constexpr int VS = 2;                  // stages of converted V
    static constexpr int NREG = D / 64;           // 128-byte-wide regions of an f16 row
    // the three parts of a row tile's Q: rows of 128 bytes, d = 64: the first
    // two parts side by side, the third in rows of its own
    static constexpr int Q_BYTES = D == 128 ? 49152 : 32768;
    __host__ __device__ static constexpr int q_part(int part) {
        return D == 128 ? part * 16384 : part == 2 ? 16384 : part * 64;
    }
    static constexpr int K_BYTES = 128 * D;
    static constexpr int V_BYTES = 128 * D * 2;
    // one Q for both groups of softmax warps, where there is no room for two
    static constexpr bool ONE_Q = ONE && D == 128;
    static constexpr int Q_OFF = 0;
    static constexpr int K_OFF = Q_OFF + (ONE_Q ? 1 : 2) * Q_BYTES;
    static constexpr int R_OFF = K_OFF + KS * K_BYTES;
    static constexpr int V_OFF = R_OFF + RS * K_BYTES;
    static constexpr int SC_OFF = V_OFF + VS * V_BYTES;       // float [slots][24]: ks, log2 vs, 1 / vs of 8 groups
    static constexpr int NAN_OFF = SC_OFF + kPtScaleSlots * 96;  // u64 [slots][D]: {tag, first key with a NaN value}
    static constexpr int AHEAD_OFF = NAN_OFF + kPtNanSlots * D * 8;  // ONE: int ids [2][kPtAhead][8], ..
    static constexpr int BAR_OFF = AHEAD_OFF + (ONE ? kPtAhead * 128 : 0);  // .. float {ks, vs} [kPtAhead][8]
    static constexpr int USED = BAR_OFF + 512;
    static constexpr int SMEM = USED + 1024;
    // TMEM: S of row tile i and half h of the keys at 128 i + 64 h, O at 256 +
    // 128 i. P of a half: d = 64 behind O, d = 128 (no room) over its S.
    static constexpr int COL_S = 0, COL_O = 256;
    static constexpr bool P_OVER_S = D == 128;
    static constexpr int COL_P = P_OVER_S ? COL_S : COL_O + 64, P_STRIDE = P_OVER_S ? 64 : 32;
    // S = Q K^T of a part of Q in E5M2 or E4M3, and K in E4M3
    __host__ __device__ static constexpr uint32_t id_s(bool e5m2) {
        return idesc_make(128, 64, kFmtE4M3, false, false) | (e5m2 ? kFmtE5M2 << 7 : 0u);
    }
    static constexpr uint32_t ID_PV = idesc_make(128, D, 0 /* f16 */, false, true);
    static_assert(SMEM <= 232448 - 2048, "shared memory");
};

struct PtParams {
    const uint16_t* q;
    const float *k_scale, *v_scale;
    uint16_t* o;
    float* lse;
    const int32_t *cu_seqlens, *cache_len, *block_table;
    int B, Hq, Hkv, G, total, max_new, max_blocks, num_blocks, bs_log2;
    float scale_log2;
    int causal;
    int split_rows;  // requests of no more rows are the split-key kernel's
    FastDiv by_g;    // division by G
    int *status, *counters;
    int max_units;
    float *pm, *pl, *po;
    PagedJoin join;  // a pass of a call with shared prefixes
};

__device__ __forceinline__ void named_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// The tag of piece `seg` in the list of NaN values: later pieces' are smaller,
// and none is that of an entry nobody has written.
__device__ __forceinline__ uint32_t pt_nan_tag(int seg) { return ~static_cast<uint32_t>(seg + 1); }
// Whether `v` holds in all `threads` threads that meet at the barrier.
__device__ __forceinline__ bool named_all(int id, int threads, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %3, 0;\n\tbar.red.and.pred p, %1, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(threads), "r"(static_cast<uint32_t>(v))
        : "memory");
    return r != 0;
}
__device__ __forceinline__ uint32_t pt_e5m2x2_from_f16x2(uint32_t x) {
    uint16_t r;
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(x));
    return r;
}
// An E5M2 number is the upper byte of the f16 number of the same value.
__device__ __forceinline__ uint32_t pt_f16x2_from_e5m2x2(uint32_t x) { return __byte_perm(x, 0u, 0x1404); }
__device__ __forceinline__ uint32_t pt_e4m3x2_from_f16x2(uint32_t x) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ uint32_t pt_add_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// 1 or 0 for each half of |a| < b.
__device__ __forceinline__ uint32_t pt_below_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("{\n\t.reg .b32 t;\n\tabs.f16x2 t, %1;\n\tset.lt.f16x2.f16x2 %0, t, %2;\n\t}" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Two bf16 numbers times f, as an f16 pair.
__device__ __forceinline__ uint32_t pt_scaled_f16x2(uint32_t v, float f) {
    return pack_f16x2(__uint_as_float(v << 16) * f, __uint_as_float(v & 0xFFFF0000u) * f);
}
// Sum of the two halves of an f16 pair.
__device__ __forceinline__ float pt_sum_f16x2(uint32_t x) {
    float r, t;
    asm("{\n\t.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(r), "=f"(t)
        : "r"(x));
    return r + t;
}
__device__ __forceinline__ uint32_t pt_sub_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Bounded wait of a whole warp, in few instructions (the five roles' loops
// compete for the instruction cache). False after FA_WAIT_LIMIT_NS or once
// the CTA is aborting; the role then leaves its loop and reports (pt_gave_up).
__device__ __forceinline__ bool pt_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    uint64_t t0 = 0;
    for (uint32_t it = 1; !__all_sync(0xffffffffu, mbar_try_wait(bar, parity)); ++it) {
        if ((it & 255u) == 0) {
            if (it == 256u) t0 = globaltimer_ns();
            if (*abort_flag || globaltimer_ns() - t0 > FA_WAIT_LIMIT_NS) return false;
        }
    }
    return true;
}
__device__ __forceinline__ void pt_gave_up(volatile int* abort_flag, int* status, int role) {
    if (!*abort_flag) {
        *abort_flag = 1;
        atomicCAS(status, 0, FA_DEV_TIMEOUT | (role << 8));
    }
}
// A value that all lanes of a warp share.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ uint64_t sdesc_sw64(uint32_t saddr, uint32_t sbo) {
    return (sdesc_sw128(saddr, 16, sbo) & ~(7ull << 61)) | (4ull << 61);
}

// Q's row r, times f, as parts whose sum it is, into a row tile's buffer: two
// (E5M2, E4M3), or in a wide row tile three (E5M2 each). Returns how many
// elements are below 2^-2, the only ones that two parts may not hold exactly.
template <int D, bool WIDE>
__device__ __forceinline__ float pt_split_q(const uint4 (&x)[D / 8], float f, uint8_t* qb, int r) {
    using C = PtCfg<D, false>;
    uint32_t small = 0u;  // f16 pair
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
        const uint32_t w[8] = {x[2 * j].x,     x[2 * j].y,     x[2 * j].z,     x[2 * j].w,
                               x[2 * j + 1].x, x[2 * j + 1].y, x[2 * j + 1].z, x[2 * j + 1].w};
        uint32_t part[3][4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            uint32_t b[3][2];
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                // exact in f16 down to 2^-24
                uint32_t a = pt_scaled_f16x2(w[2 * y + z], f);
                if constexpr (!WIDE) small = pt_add_f16x2(small, pt_below_f16x2(a, 0x34003400u));
                b[0][z] = pt_e5m2x2_from_f16x2(a);
                a = pt_sub_f16x2(a, pt_f16x2_from_e5m2x2(b[0][z]));
                if constexpr (WIDE) {
                    b[1][z] = pt_e5m2x2_from_f16x2(a);
                    b[2][z] = pt_e5m2x2_from_f16x2(pt_sub_f16x2(a, pt_f16x2_from_e5m2x2(b[1][z])));
                } else {
                    b[1][z] = pt_e4m3x2_from_f16x2(a);
                }
            }
#pragma unroll
            for (int k = 0; k < (WIDE ? 3 : 2); ++k) part[k][y] = __byte_perm(b[k][0], b[k][1], 0x5410);
        }
#pragma unroll
        for (int k = 0; k < (WIDE ? 3 : 2); ++k) {
            const int c = D == 64 && k == 1 ? j + 4 : j;  // 16-byte piece of the row
            const int at = (D == 128 || k == 2 ? C::q_part(k) : 0) + r * 128 + ((c ^ (r & 7)) << 4);
            sts128(smem_u32(qb + at), part[k][0], part[k][1], part[k][2], part[k][3]);
        }
    }
    return pt_sum_f16x2(small);
}

// Whether two parts hold a row of Q, times f: what they leave out is 2^-9 at
// most, summed over the elements, and no more than an eighth of these is small
// (where a few large elements stand above the others, all may hang on those).
template <int D>
__device__ __noinline__ bool pt_two_parts_hold(const uint16_t* row, float f) {
    float left = 0.f;
    int small = 0;
#pragma unroll 4
    for (int j = 0; j < D / 8; ++j) {
        const uint4 x = reinterpret_cast<const uint4*>(row)[j];
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const uint32_t a = pt_scaled_f16x2(w[y], f);
            const uint32_t b = pt_sub_f16x2(a, pt_f16x2_from_e5m2x2(pt_e5m2x2_from_f16x2(a)));
            const uint32_t lo = w[y] & 0x7FFFu, hi = (w[y] >> 16) & 0x7FFFu;
            const uint32_t less = pt_below_f16x2(a, 0x34003400u);  // 1 is 0x3C00
            small += (lo && (less & 0xFFFFu)) + (hi && (less >> 16));
            left += pt_sum_f16x2(pt_sub_f16x2(b, f16x2_from_e4m3x2(pt_e4m3x2_from_f16x2(b))) & 0x7FFF7FFFu);
        }
    }
    return left <= 0x1p-9f && small <= D / 8;
}

// A function of its own: few row tiles take it, and the roles' loops compete
// for the instruction cache.
template <int D>
__device__ __noinline__ void pt_split_q_wide(const uint16_t* row, float f, uint8_t* qb, int r) {
    uint4 x[D / 8];
#pragma unroll
    for (int j = 0; j < D / 8; ++j) x[j] = row ? reinterpret_cast<const uint4*>(row)[j] : make_uint4(0u, 0u, 0u, 0u);
    pt_split_q<D, true>(x, f, qb, r);
}

struct PtWide {
    static constexpr bool value = true;
};
struct PtNarrow {
    static constexpr bool value = false;
};

struct PtReq {
    int b, n, len, tok0;
    int npair;        // pairs of row tiles
    long long tiles;  // key tiles of all pairs of one key head, each with its unit's cost
};
struct PtSeg {
    PtReq r;
    int hk, pair;
    int ntile;        // key tiles of the unit
    int c0, c1;       // this piece's tiles
    long long line0;  // position of the unit's first tile on the line (its cost lies in front of it)
    int unit;         // index of the unit among all
};

// Keys that new token `tok` of a request sees.
__device__ __forceinline__ int pt_visible(const PtParams& p, const PtReq& r, int tok) {
    return p.causal ? min(max(r.len - r.n + tok + 1, 0), r.len) : r.len;
}
// Key tiles that the rows of a unit (RT of them) need (at least one, so that
// rows that see nothing get their zero output).
template <int RT>
__device__ __forceinline__ int pt_tiles(const PtParams& p, const PtReq& r, int pair) {
    const int last = min(pair * RT + RT - 1, r.n * p.G - 1);
    return max(1, (pt_visible(p, r, p.by_g.div(last)) + 127) >> 7);
}
template <int D, bool PFX, int RT>
__device__ __forceinline__ void pt_request(const PtParams& p, int b, PtReq& r) {
    int i0 = b, i1 = b + 1;
    if constexpr (PFX) paged_members(p.join, i0, i1);
    const int t0 = min(max(p.cu_seqlens[i0], 0), p.total), t1 = min(max(p.cu_seqlens[i1], t0), p.total);
    r.b = b;
    r.tok0 = t0;
    r.n = min(t1 - t0, p.max_new);
    if (static_cast<long long>(r.n) * p.G <= p.split_rows) r.n = 0;
    r.len = min(max(p.cache_len[b], 0), p.max_blocks << p.bs_log2);
    r.npair = static_cast<int>((static_cast<long long>(r.n) * p.G + RT - 1) / RT);
    r.tiles = 0;
    for (int i = 0; i < r.npair; ++i) r.tiles += pt_tiles<RT>(p, r, i) + kPtUnitCost<D>;
}

// ONE (a prefix's rows, which see all its keys): a unit is one row tile, and the
// two softmax groups and product warps, "row tiles" i below, take every other of
// its key tiles: with few rows the time is the chain of S, softmax and P V, and
// two chains hide one another (64 rows behind 262,001 tokens, d = 128: 228 us a
// call with units of two row tiles, 173 so; six groups of 32 to 172 rows, d = 64:
// 83 and 79). What bounds it is the softmax warps' chain: a half tile takes one
// 1,980 cycles, with 38 % of the issue slots used.
template <int D, bool PFX, bool ONE>
__global__ void __launch_bounds__(512, 1)
    fa_paged_tile_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const __grid_constant__ PtParams p) {
    using C = PtCfg<D, ONE>;
    // rows of a unit; from one key tile of a row tile to its next
    constexpr int RT = ONE ? 128 : 256, STEP = ONE ? 2 : 1;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ long long scan_w[16], scan_u[16], scan_o[PFX ? 16 : 1];
    __shared__ long long start_line;
    __shared__ int start_b, start_units, abort_s, last_s[2], nan_piece[kPtNanSlots], wide_s[2];
    __shared__ uint32_t tmem_slot;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if constexpr (PFX) paged_let_next();

    // ---- the line of key tiles: total length, and the request at this CTA's start
    const int per = (p.B + 511) / 512;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    long long mw = 0, mu = 0;
    for (int b = b0; b < b1; ++b) {
        PtReq r;
        pt_request<D, PFX, RT>(p, b, r);
        mu += static_cast<long long>(r.npair) * p.Hkv;
        mw += r.tiles * p.Hkv;
        if constexpr (PFX) {
            if (p.join.first && blockIdx.x == 0) {  // the prefixes' pass has no other kernel that would report these
                int i0 = b, i1 = b + 1;
                const bool good = paged_members(p.join, i0, i1) && p.cache_len[b] == r.len;
                if (!good) atomicCAS(p.status, 0, FA_DEV_INVALID | (100 << 8));
            }
        }
    }
    long long iw = mw, iu = mu;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, iw, off), c = __shfl_up_sync(0xffffffffu, iu, off);
        if (lane >= off) {
            iw += a;
            iu += c;
        }
    }
    if (lane == 31) {
        scan_w[warp] = iw;
        scan_u[warp] = iu;
    }
    if constexpr (PFX) {
        if (p.join.other_len) {  // places of the split-key kernel's line
            long long other = 0;
            for (int b = tid; b < p.join.other_n; b += 512)
                if (p.join.other_cu[b + 1] > p.join.other_cu[b])
                    other += max(1, (min(max(p.join.other_len[b], 0), p.join.other_cap) + 31) >> 5) + p.join.other_cost;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) other += __shfl_xor_sync(0xffffffffu, other, off);
            if (lane == 0) scan_o[warp] = other * p.Hkv;
        }
    }
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::BAR_OFF);
    uint64_t* q_full = bars;                   // [2] Q parts of a row tile stored
    uint64_t* s_full = q_full + 2;             // [2][2] S of a row tile and half of the keys ready
    uint64_t* p_full = s_full + 4;             // [2][2] its P stored, O rescaled
    uint64_t* pv_done = p_full + 4;            // [2][2] its P V done
    uint64_t* drain = pv_done + 4;             // [2]
    uint64_t* nan_full = drain + 2;            // [4] a piece's V has been looked over
    uint64_t* nan_empty = nan_full + kPtNanSlots;  // [4] both row tiles' softmax warps are through with that piece
    uint64_t* sc_full = nan_empty + kPtNanSlots;   // [8] scales stored
    [[maybe_unused]] uint64_t* asked = sc_full + kPtScaleSlots;  // ONE: [8] K of a tile requested
    uint64_t* k_full = sc_full + (ONE ? 2 : 1) * kPtScaleSlots;  // [KB]
    uint64_t* k_empty = k_full + C::KB;        // [KS] both row tiles' S done
    uint64_t* r_full = k_empty + C::KS;        // [RS] V landed
    uint64_t* r_empty = r_full + C::RS;        // [RS] V read
    uint64_t* v_full = r_empty + C::RS;        // [VS] V converted
    uint64_t* v_empty = v_full + C::VS;        // [VS] both row tiles' P V done
    if (tid == 0) {
        abort_s = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 128);
            mbar_init(&drain[i], 1);
            for (int h = 0; h < 2; ++h) {
                mbar_init(&s_full[2 * i + h], 1);
                mbar_init(&p_full[2 * i + h], 128);
                mbar_init(&pv_done[2 * i + h], 1);
            }
        }
        for (int i = 0; i < kPtNanSlots; ++i) {
            mbar_init(&nan_full[i], 128);
            mbar_init(&nan_empty[i], 256);
        }
        for (int i = 0; i < kPtScaleSlots; ++i) {
            mbar_init(&sc_full[i], 1);
            if (ONE) mbar_init(&asked[i], 1);
        }
        for (int i = 0; i < C::KB; ++i) mbar_init(&k_full[i], 1);
        for (int i = 0; i < C::KS; ++i) mbar_init(&k_empty[i], ONE ? 1 : 2);
        for (int i = 0; i < C::RS; ++i) {
            mbar_init(&r_full[i], 1);
            mbar_init(&r_empty[i], 128);
        }
        for (int i = 0; i < C::VS; ++i) {
            mbar_init(&v_full[i], 128);
            mbar_init(&v_empty[i], ONE ? 1 : 2);
        }
        fence_barrier_init();
    }
    // NaN values that only some rows see: for each column the piece's tag
    // (a later piece's entry replaces an earlier one's) and the first key;
    // and the piece that noted one last. A piece's slot is used again four
    // pieces on, once all softmax warps have said that they are through with it
    // (nan_empty): a row tile without rows, or whose rows see none of a piece's
    // keys, has no products that would hold the conversion of V back for them.
    // So nan_full is at most one phase ahead of those that wait for it.
    unsigned long long* nan_first = reinterpret_cast<unsigned long long*>(sm + C::NAN_OFF);
    for (int i = tid; i < kPtNanSlots * D; i += 512) nan_first[i] = ~0ull;
    if (tid < kPtNanSlots) nan_piece[tid] = -1;
    __syncthreads();
    long long W = 0, U = 0, bw = 0, bu = 0;
    for (int w = 0; w < 16; ++w) {
        if (w < warp) {
            bw += scan_w[w];
            bu += scan_u[w];
        }
        W += scan_w[w];
        U += scan_u[w];
    }
    // CTAs that work: all, or where the requests' own pass runs beside this one its share
    int ctas = kPagedCtas;
    if constexpr (PFX) {
        if (p.join.other_len) {
            long long other = 0;
            for (int w = 0; w < 16; ++w) other += scan_o[w];
            ctas = paged_share(p.join, W, other);
        }
    }
    const long long quota = max((W + ctas - 1) / ctas, 2ll);
    const long long x0 = quota * blockIdx.x, x1 = min(x0 + quota, W);
    if (U > p.max_units || x0 >= x1) {  // uniform over the CTA, before any TMEM use
        // (too many units: overlapping offsets, which the split-key kernel reports)
        if constexpr (PFX) paged_wait_before();
        return;
    }
    bw += iw - mw;
    bu += iu - mu;
    if (x0 >= bw && x0 < bw + mw) {
        for (int b = b0; b < b1; ++b) {
            PtReq r;
            pt_request<D, PFX, RT>(p, b, r);
            if (x0 < bw + r.tiles * p.Hkv) {
                start_b = b;
                start_line = bw;
                start_units = static_cast<int>(bu);
                break;
            }
            bw += r.tiles * p.Hkv;
            bu += static_cast<long long>(r.npair) * p.Hkv;
        }
    }
    if (warp == 3) {
        tmem_alloc(&tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_slot;

    // Every role walks the same pieces.
    long long rline = start_line;
    int runits = start_units;
    auto find = [&](PtSeg& s, long long x) {  // the piece that starts at x, in the current request or a later one
        while (x >= rline + s.r.tiles * p.Hkv) {
            rline += s.r.tiles * p.Hkv;
            runits += s.r.npair * p.Hkv;
            pt_request<D, PFX, RT>(p, s.r.b + 1, s.r);
        }
        const long long off = x - rline;
        s.hk = static_cast<int>(div_short(off, s.r.tiles));
        long long rest = off - s.hk * s.r.tiles;
        s.pair = 0;
        for (;;) {
            s.ntile = pt_tiles<RT>(p, s.r, s.pair);
            if (rest < s.ntile + kPtUnitCost<D>) break;
            rest -= s.ntile + kPtUnitCost<D>;
            ++s.pair;
        }
        s.line0 = x - rest + kPtUnitCost<D>;
        s.c0 = max(static_cast<int>(rest) - kPtUnitCost<D>, 0);
        s.c1 = static_cast<int>(min(static_cast<long long>(s.ntile), x1 - s.line0));
        s.unit = runits + s.hk * s.r.npair + s.pair;
    };
    auto next = [&](PtSeg& s) -> bool {  // false if what is left is no tile, or only the cost in front of one
        const long long x = s.line0 + s.c1;
        if (x >= x1) return false;
        if (s.pair + 1 < s.r.npair) {  // the usual step: the next pair of the same head
            ++s.pair;
            ++s.unit;
            s.ntile = pt_tiles<RT>(p, s.r, s.pair);
            s.c0 = 0;
            s.line0 = x + kPtUnitCost<D>;
            s.c1 = static_cast<int>(min(static_cast<long long>(s.ntile), x1 - s.line0));
        } else {
            find(s, x);
        }
        return s.c1 > 0;
    };
    // key tiles that row tile i of a piece takes part in: [c0, end)
    auto half_end = [&](const PtSeg& s, int i) {
        if (ONE) return s.c1;
        const int rows = s.r.n * p.G, base = s.pair * RT + i * 128;
        if (base >= rows) return s.c0;
        const int last = min(base + 127, rows - 1);
        return max(s.c0, min(s.c1, (pt_visible(p, s.r, p.by_g.div(last)) + 127) >> 7));
    };
    auto wait_warp = [&](uint64_t* bar, uint32_t parity) { return pt_wait(bar, parity, &abort_s); };
    PtSeg s;
    pt_request<D, PFX, RT>(p, start_b, s.r);
    find(s, x0);
    const bool any = s.c1 > s.c0;  // uniform over the CTA: not only the cost in front of a tile

    if (!any) {
        // nothing but TMEM to give back
    } else if (warp < 4) {
        regs_dec<96>();
        // (In this order, and in this form: the roles' code shares the instruction
        // cache. With the loaders first, told apart by a plain condition, prompts of
        // 9,322 tokens over 8,192 keys, d = 64, took 443 us, 430 so; six groups of
        // drafts 82 and 79; pieces of prompts at d = 128 778 and 773.)
        if (warp == 1 || warp == 2) {
            // ------------------------------------------------------ products of row tile i
            // A key tile's two halves of 64 keys have S columns of their own:
            // while the softmax warps work on one half, P V and the next
            // tile's S of the other half run. One issuer for each row tile: a
            // half's wait, twelve products and two commits take a warp about
            // 450 cycles to issue, which one warp for both could not hide.
            const int i = warp - 1;
            const uint32_t leader = elect_one_sync();
            const uint64_t dQ = sdesc_sw128(smem_u32(sm + C::Q_OFF) + (C::ONE_Q ? 0 : i * C::Q_BYTES), 16, 1024);
            const uint64_t dK = D == 128 ? sdesc_sw128(smem_u32(sm + C::K_OFF), 16, 1024)
                                         : sdesc_sw64(smem_u32(sm + C::K_OFF), 512);
            const uint64_t dV = sdesc_sw128(smem_u32(sm + C::V_OFF), 16384, 1024);
            const uint32_t tm0 = uniform(tm) + i * 128;
            int u = 0, nseg = 0, np = 0;  // tiles walked, pieces with work, tiles of P multiplied
            bool ok = true;
            // The tiles [c0, c1) of a piece, of which row tile i takes part in
            // those up to `end`; one loop for each form of Q, so that neither
            // tests it between its products.
            // (ONE: every other tile.)
            if constexpr (ONE) {
                auto walk = [&](auto form, int c0, int c1, int end) {
                    constexpr bool kWide = decltype(form)::value;
                    const int first = c0 + i;
                    u += first - c0;
                    for (int t = first; t < c1 + STEP; t += STEP, u += STEP) {
                        const int st = u % C::KS, kb = u % C::KB, vs = (u - STEP) % C::VS;
                        const bool now = t < c1, before = t > first;  // a tile of K, and one of V, of this row tile's
                        const uint64_t vd = sdesc_advance(dV, vs * C::V_BYTES), kd = sdesc_advance(dK, st * C::K_BYTES);
                        if (now && !(ok = wait_warp(&k_full[kb], (u / C::KB) & 1))) break;
                        if (before && !(ok = wait_warp(&v_full[vs], ((u - STEP) / C::VS) & 1))) break;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t tS = tm0 + C::COL_S + h * 64, tO = tm0 + C::COL_O;
                            const uint32_t tP = tm0 + C::COL_P + h * C::P_STRIDE;
                            if (before && t - STEP < end) {
                                if (!(ok = wait_warp(&p_full[2 * i + h], np & 1))) break;
                                tc_fence_after();
                                const uint32_t more = !(t - STEP == first && h == 0);
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    umma_ts<false>(leader, tO, tP + kk * 8, sdesc_advance(vd, h * 8192 + kk * 2048),
                                                   C::ID_PV, kk > 0 ? 1u : more);
                                umma_commit(leader, &pv_done[2 * i + h]);
                            }
                            if (t < end) {
                                // Only products with the same accumulator are bound to
                                // the order of their issue: where S takes P's place,
                                // P V has to be done.
                                if (C::P_OVER_S && before && !(ok = wait_warp(&pv_done[2 * i + h], np & 1))) break;
                                tc_fence_after();
#pragma unroll
                                for (int part = 0; part < (kWide ? 3 : 2); ++part)
#pragma unroll
                                    for (int kk = 0; kk < D / 32; ++kk)
                                        umma_ss_f8(leader, tS, sdesc_advance(dQ, C::q_part(part) + kk * 32),
                                                   sdesc_advance(kd, h * (C::K_BYTES / 2) + kk * 32),
                                                   C::id_s(kWide || part == 0), part || kk ? 1u : 0u);
                                umma_commit(leader, &s_full[2 * i + h]);
                            }
                        }
                        if (!ok) break;
                        // this row tile has read K of tile t and V of the one before
                        if (now) umma_commit(leader, &k_empty[st]);
                        if (before) umma_commit(leader, &v_empty[vs]);
                        np += before && t - STEP < end;
                    }
                };
                int upos = 0;  // tiles of the pieces before
                do {
                    // warp-uniform in the compiler's eyes too, so that descriptors and
                    // TMEM addresses stay in uniform registers
                    const int c0 = uniform(s.c0), c1 = uniform(s.c1), end = uniform(half_end(s, i));
                    const bool some = end > c0 + i;
                    u = upos;
                    if (some && !(ok = wait_warp(&q_full[i], nseg & 1))) break;
                    if (some && uniform(wide_s[i])) walk(PtWide{}, c0, c1, end);
                    else walk(PtNarrow{}, c0, c1, end);
                    if (!ok) break;
                    nseg += some;
                    upos += c1 - c0;
                } while (__any_sync(0xffffffffu, next(s)));
            } else {
                auto walk = [&](auto form, int c0, int c1, int end) {
                    constexpr bool kWide = decltype(form)::value;
                    for (int t = c0; t <= c1; ++t, ++u) {
                        const int st = u % C::KS, vs = (u - 1) % C::VS;
                        const uint64_t vd = sdesc_advance(dV, vs * C::V_BYTES), kd = sdesc_advance(dK, st * C::K_BYTES);
                        if (t < c1 && !(ok = wait_warp(&k_full[st], (u / C::KS) & 1))) break;
                        if (t > c0 && !(ok = wait_warp(&v_full[vs], ((u - 1) / C::VS) & 1))) break;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t tS = tm0 + C::COL_S + h * 64, tO = tm0 + C::COL_O;
                            const uint32_t tP = tm0 + C::COL_P + h * C::P_STRIDE;
                            if (t > c0 && t <= end) {
                                if (!(ok = wait_warp(&p_full[2 * i + h], np & 1))) break;
                                tc_fence_after();
                                const uint32_t more = !(t - 1 == c0 && h == 0);
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    umma_ts<false>(leader, tO, tP + kk * 8, sdesc_advance(vd, h * 8192 + kk * 2048),
                                                   C::ID_PV, kk > 0 ? 1u : more);
                                umma_commit(leader, &pv_done[2 * i + h]);
                            }
                            if (t < end) {
                                // Only products with the same accumulator are bound to
                                // the order of their issue: where S takes P's place,
                                // P V has to be done.
                                if (C::P_OVER_S && t > c0 && !(ok = wait_warp(&pv_done[2 * i + h], np & 1))) break;
                                tc_fence_after();
#pragma unroll
                                for (int part = 0; part < (kWide ? 3 : 2); ++part)
#pragma unroll
                                    for (int kk = 0; kk < D / 32; ++kk)
                                        umma_ss_f8(leader, tS, sdesc_advance(dQ, C::q_part(part) + kk * 32),
                                                   sdesc_advance(kd, h * (C::K_BYTES / 2) + kk * 32),
                                                   C::id_s(kWide || part == 0), part || kk ? 1u : 0u);
                                umma_commit(leader, &s_full[2 * i + h]);
                            }
                        }
                        if (!ok) break;
                        // this row tile has read K of tile t and V of tile t - 1
                        if (t < c1) umma_commit(leader, &k_empty[st]);
                        if (t > c0) umma_commit(leader, &v_empty[vs]);
                        np += t > c0 && t <= end;
                    }
                    --u;  // the last round had no tile of its own
                };
                do {
                    // warp-uniform in the compiler's eyes too, so that descriptors and
                    // TMEM addresses stay in uniform registers
                    const int c0 = uniform(s.c0), c1 = uniform(s.c1), end = uniform(half_end(s, i));
                    if (end > c0 && !(ok = wait_warp(&q_full[i], nseg & 1))) break;
                    if (end > c0 && uniform(wide_s[i])) walk(PtWide{}, c0, c1, end);
                    else walk(PtNarrow{}, c0, c1, end);
                    if (!ok) break;
                    nseg += end > c0;
                } while (__any_sync(0xffffffffu, next(s)));
            }
            if (!ok) pt_gave_up(&abort_s, p.status, 96);
            // every MMA issued so far must be complete before TMEM is released
            umma_commit(leader, &drain[i]);
            mbar_wait_teardown(&drain[i], 0, 200000000ull);
        } else if (warp == 0 || ONE) {
            if constexpr (ONE) {
                // A tile's loads depend on one another (block id, then scales and
                // copies): ids come four tiles ahead and scales two, by asynchronous
                // copies of a lane for each group of 16 keys. One warp requests the
                // copies and another sees to the scales: together they took a warp
                // 2,370 cycles a tile, which is what a prefix of few rows then took
                // (64 rows behind 262,001 tokens: the kernel 190 us, 168 so). With two row
                // tiles a tile takes longer than that.
                const int bs = 1 << p.bs_log2, box = min(bs, 128);
                int* ahead = reinterpret_cast<int*>(sm + C::AHEAD_OFF) + (warp == 0 ? 0 : 8 * kPtAhead);
                auto has = [&](int t) { return lane < 8 && t < s.c1 && t * 128 + lane * 16 < s.r.len; };
                auto id_at = [&](int t) { return ahead + (t % kPtAhead) * 8 + lane; };  // lanes 0..7
                auto fetch_id = [&](int t) {
                    if (has(t))
                        cp_async4(id_at(t), &p.block_table[static_cast<size_t>(s.r.b) * p.max_blocks +
                                                           ((t * 128 + lane * 16) >> p.bs_log2)]);
                };
                auto is_block = [&](int id) { return id >= 0 && id < p.num_blocks; };
                auto row_of = [&](int id, int t) {
                    return static_cast<int>(((static_cast<long long>(id) * p.Hkv + s.hk) << p.bs_log2) +
                                            ((t * 128 + lane * 16) & (bs - 1)));
                };
                // the first lane of each box of min(block, 128) rows requests it
                const bool asks = lane < 8 && lane % (box >> 4) == 0;
                if (warp == 0) {
                    // ------------------------------------------------------ K and V tiles
                    int u = 0, klast = -1;
                    bool ok = true;
                    do {
#pragma unroll 1
                        for (int t = 0; t < 4; ++t) {
                            fetch_id(s.c0 + t);
                            cp_async_commit();
                        }
                        for (int t = s.c0; ok && t < s.c1; ++t, ++u) {
                            const int st = u % C::KS, kb = u % C::KB, rs = u % C::RS;
                            cp_async_wait<3>();
                            int id = has(t) ? *id_at(t) : 0;
                            if (!is_block(id)) {
                                atomicCAS(p.status, 0, FA_DEV_INVALID | (94 << 8));
                                id = 0;
                            }
                            fetch_id(t + 4);
                            cp_async_commit();
                            const int row = row_of(id, t);
                            if (!(ok = wait_warp(&k_empty[st], ((u / C::KS) & 1) ^ 1))) break;
                            if (lane == 0) {
                                mbar_arrive(&asked[u % kPtScaleSlots]);
                                mbar_arrive_expect_tx(&k_full[kb], C::K_BYTES);
                            }
                            __syncwarp();
                            if (asks)
                                tma_load_2d(sm + C::K_OFF + st * C::K_BYTES + lane * 16 * D, &tmK, 0, row, &k_full[kb]);
                            if (!(ok = wait_warp(&r_empty[rs], ((u / C::RS) & 1) ^ 1))) {
                                klast = u + 1;
                                break;
                            }
                            if (lane == 0) mbar_arrive_expect_tx(&r_full[rs], C::K_BYTES);
                            __syncwarp();
                            if (asks)
                                tma_load_2d(sm + C::R_OFF + rs * C::K_BYTES + lane * 16 * D, &tmV, 0, row, &r_full[rs]);
                        }
                        cp_async_wait<0>();
                    } while (ok && next(s));
                    if (!ok) pt_gave_up(&abort_s, p.status, 95);
                    // let every copy in flight land before the CTA can exit
                    if (lane == 0) {
                        const int nk = max(u, klast);
                        for (int i = 0; i < C::KB && i < nk; ++i) {
                            const int last = i + ((nk - 1 - i) / C::KB) * C::KB;
                            mbar_wait_teardown(&k_full[i], (last / C::KB) & 1, 200000000ull);
                        }
                        for (int i = 0; i < C::RS && i < u; ++i) {
                            const int last = i + ((u - 1 - i) / C::RS) * C::RS;
                            mbar_wait_teardown(&r_full[i], (last / C::RS) & 1, 200000000ull);
                        }
                    }
                } else {
                    // ------------------------------------------------------ scales
                    // A slot is written once K of its tile has been requested: the tile
                    // eight before it, whose slot it was, is then through its softmax.
                    float* raw = reinterpret_cast<float*>(ahead + 8 * kPtAhead);  // {ks, vs} [kPtAhead][8]
                    float* sc = reinterpret_cast<float*>(sm + C::SC_OFF);
                    auto fetch_scales = [&](int t) {
                        if (!has(t)) return;
                        const int id = *id_at(t);
                        if (!is_block(id)) return;
                        const size_t x = static_cast<size_t>(id) * p.Hkv + s.hk;
                        cp_async4(raw + ((t % kPtAhead) * 8 + lane) * 2, &p.k_scale[x]);
                        cp_async4(raw + ((t % kPtAhead) * 8 + lane) * 2 + 1, &p.v_scale[x]);
                    };
                    int u = 0;
                    bool ok = true;
                    do {
                        float vref = 0.f;  // largest V scale met so far in this piece
#pragma unroll 1
                        for (int t = 0; t < 4; ++t) fetch_id(s.c0 + t);
                        cp_async_commit();
                        cp_async_wait<0>();
                        fetch_scales(s.c0);
                        cp_async_commit();
                        fetch_scales(s.c0 + 1);
                        cp_async_commit();
                        for (int t = s.c0; ok && t < s.c1; ++t, ++u) {
                            cp_async_wait<1>();
                            float ks = 0.f, vs = 0.f;
                            if (has(t) && is_block(*id_at(t))) {
                                ks = raw[((t % kPtAhead) * 8 + lane) * 2];
                                vs = raw[((t % kPtAhead) * 8 + lane) * 2 + 1];
                            }
                            fetch_scales(t + 2);
                            fetch_id(t + 4);
                            cp_async_commit();
                            float top = vs;
#pragma unroll
                            for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                            vref = fmaxf(vref, top);
                            // groups whose scale is below 2^-60 of the largest (blocks of
                            // zeros have 2^-126) count as if it were that
                            const float lv = fmaxf(fmaxf(log2f(vs), log2f(vref) - kPtSpan), -100.f), il = exp2f(-lv);
                            const int slot = u % kPtScaleSlots;
                            if (!(ok = wait_warp(&asked[slot], (u / kPtScaleSlots) & 1))) break;
                            if (lane < 8) {
                                sc[slot * 24 + lane] = ks;
                                sc[slot * 24 + 8 + lane] = lv;
                                sc[slot * 24 + 16 + lane] = il;
                            }
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&sc_full[slot]);
                        }
                        cp_async_wait<0>();
                    } while (ok && next(s));
                    if (!ok) pt_gave_up(&abort_s, p.status, 99);
                }
            } else {
                // ------------------------------------------------------ K and V tiles and scales
                const int bs = 1 << p.bs_log2, box = min(bs, 128);
                int u = 0, klast = -1;
                bool ok = true;
                float* sc = reinterpret_cast<float*>(sm + C::SC_OFF);
                do {
                    float vref = 0.f;  // largest V scale met so far in this piece
                    for (int t = s.c0; ok && t < s.c1; ++t, ++u) {
                        const int st = u % C::KS, slot = u % kPtScaleSlots;
                        // lane i < 8: the group of 16 keys from 16 i on
                        int id = 0;
                        float ks = 0.f, vs = 0.f;
                        const int key = t * 128 + lane * 16;
                        if (lane < 8 && key < s.r.len) {
                            id = p.block_table[static_cast<size_t>(s.r.b) * p.max_blocks + (key >> p.bs_log2)];
                            if (id < 0 || id >= p.num_blocks) {
                                atomicCAS(p.status, 0, FA_DEV_INVALID | (94 << 8));
                                id = 0;
                            } else {
                                ks = p.k_scale[static_cast<size_t>(id) * p.Hkv + s.hk];
                                vs = p.v_scale[static_cast<size_t>(id) * p.Hkv + s.hk];
                            }
                        }
                        if (!(ok = wait_warp(&k_empty[st], ((u / C::KS) & 1) ^ 1))) break;
                        if (lane == 0) mbar_arrive_expect_tx(&k_full[st], C::K_BYTES);
                        __syncwarp();
                        // the first lane of each box of min(block, 128) rows requests it
                        const bool asks = lane < 8 && lane % (box >> 4) == 0;
                        const int row = static_cast<int>(((static_cast<long long>(id) * p.Hkv + s.hk) << p.bs_log2) +
                                                         ((t * 128 + lane * 16) & (bs - 1)));
                        if (asks)
                            tma_load_2d(sm + C::K_OFF + st * C::K_BYTES + lane * 16 * D, &tmK, 0, row, &k_full[st]);
                        float top = vs;
#pragma unroll
                        for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                        vref = fmaxf(vref, top);
                        if (lane < 8) {
                            // groups whose scale is below 2^-60 of the largest (blocks of
                            // zeros have 2^-126) count as if it were that
                            const float lv = fmaxf(fmaxf(log2f(vs), log2f(vref) - kPtSpan), -100.f);
                            sc[slot * 24 + lane] = ks;
                            sc[slot * 24 + 8 + lane] = lv;
                            sc[slot * 24 + 16 + lane] = exp2f(-lv);
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sc_full[slot]);
                        const int rs = u % C::RS;
                        if (!(ok = wait_warp(&r_empty[rs], ((u / C::RS) & 1) ^ 1))) {
                            klast = u + 1;
                            break;
                        }
                        if (lane == 0) mbar_arrive_expect_tx(&r_full[rs], C::K_BYTES);
                        __syncwarp();
                        if (asks)
                            tma_load_2d(sm + C::R_OFF + rs * C::K_BYTES + lane * 16 * D, &tmV, 0, row, &r_full[rs]);
                    }
                } while (ok && next(s));
                if (!ok) pt_gave_up(&abort_s, p.status, 95);
                // let every copy in flight land before the CTA can exit
                if (lane == 0) {
                    const int nk = max(u, klast);
                    for (int i = 0; i < C::KS && i < nk; ++i) {
                        const int last = i + ((nk - 1 - i) / C::KS) * C::KS;
                        mbar_wait_teardown(&k_full[i], (last / C::KS) & 1, 200000000ull);
                    }
                    for (int i = 0; i < C::RS && i < u; ++i) {
                        const int last = i + ((u - 1 - i) / C::RS) * C::RS;
                        mbar_wait_teardown(&r_full[i], (last / C::RS) & 1, 200000000ull);
                    }
                }
            }
        }
    } else if (warp < 12) {
        // ---------------------------------------------------------- softmax of row tile i
        regs_inc<152>();
        const int i = (warp - 4) >> 2, wq = warp & 3, r = wq * 32 + lane;
        const uint32_t tl = tm + (static_cast<uint32_t>(wq * 32) << 16);
        const uint32_t tS = tl + C::COL_S + i * 128, tO = tl + C::COL_O + i * 128, tP = tl + C::COL_P + i * 128;
        uint8_t* qb = sm + C::Q_OFF + (C::ONE_Q ? 0 : i * C::Q_BYTES);
        int u = 0, ns = 0, seg = 0;  // tiles walked, halves of them multiplied, pieces
        bool ok = true;
        do {
            const int end = half_end(s, i);
            const int rows = s.r.n * p.G, base = s.pair * RT + (ONE ? 0 : i * 128);
            const int row = base + (ONE && rows - base <= 64 ? r & 63 : r);
            const bool row_ok = row < rows;
            // ONE, at most 64 rows: lanes 64 .. 127 have the same rows, and take the
            // second half of each tile's keys, lanes 0 .. 63 the first
            const bool twice = ONE && rows - base <= 64;
            const int tok = row_ok ? p.by_g.div(row) : 0, hq = s.hk * p.G + (row_ok ? row - tok * p.G : 0);
            const int limit = row_ok ? pt_visible(p, s.r, tok) : 0;
            const size_t qrow = (static_cast<size_t>(s.r.tok0 + tok) * p.Hq + hq) * D;
            float rc = 0.f, mu = -CUDART_INF_F, l = 0.f;
            const int first = ONE ? s.c0 + i : s.c0;  // key tile
            if (end > first) {
                // ---- Q: the row's power of two, then its parts
                uint4 x[D / 8];
#pragma unroll
                for (int j = 0; j < D / 8; ++j)
                    x[j] = row_ok ? reinterpret_cast<const uint4*>(p.q + qrow)[j] : make_uint4(0u, 0u, 0u, 0u);
                uint32_t m2 = 0;  // bf16 bits, ordered like the magnitudes, both halves of a word at once
#pragma unroll
                for (int j = 0; j < D / 8; ++j)
                    m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(x[j].x & 0x7FFF7FFFu, x[j].y & 0x7FFF7FFFu),
                                               __vmaxu2(x[j].z & 0x7FFF7FFFu, x[j].w & 0x7FFF7FFFu)));
                const uint32_t top = max(m2 & 0xFFFFu, m2 >> 16);
                const bool wild = top >= 0x7F80u;  // an infinity or a NaN
                // largest magnitude to [2^11, 2^12), two parts: what is not below
                // 2^-2 is exact, what is leaves out 2^-10 at most
                const int e0 = top >> 7 && !wild ? static_cast<int>(top >> 7) - 138 : 0;
                int e = min(max(e0, -120), 120);
                const float f = exp2i(-e);
                // ONE_Q: row tile 0's warps write Q for both, and where both take
                // part (a piece of one key tile is row tile 0's alone) neither has
                // its products started before it is whole. (At d = 64 each has its
                // own: six groups of drafts 85 us a call with one Q, 82 so.)
                const bool writes = !C::ONE_Q || i == 0, both = C::ONE_Q && s.c1 - s.c0 > 1;
                bool fits = true;
                if (writes) {
                    // a row of few small elements leaves out little for certain
                    // (zeros count as small here)
                    const bool few = pt_split_q<D, false>(x, f, qb, r) <= 2.f || top == 0 || wild;
                    fits = few || pt_two_parts_hold<D>(p.q + qrow, f);
                }
                if (C::ONE_Q) fence_proxy_async_smem();
                __syncwarp();
                const bool wide = !(both ? named_all(3, 256, fits) : named_all(1 + i, 128, fits));
                if (wide) {  // [2^14, 2^15), three
                    e = min(max(e0 - 3, -120), 120);
                    if (writes) pt_split_q_wide<D>(row_ok ? p.q + qrow : nullptr, exp2i(-e), qb, r);
                    if (both) {
                        fence_proxy_async_smem();
                        named_sync(3, 256);
                    }
                }
                if (r == 0) wide_s[i] = wide;
                rc = wild ? CUDART_NAN_F : p.scale_log2 * exp2i(e);  // such a row has no finite result
                fence_proxy_async_smem();
                mbar_arrive(&q_full[i]);
            }
            // rows that the first row's keys bound: tiles below need no mask
            const int vis_min = pt_visible(p, s.r, p.by_g.div(min(base, rows - 1)));
#pragma unroll 1
            for (int th = 2 * first; th < 2 * end; th += (th & 1) ? 2 * STEP - 1 : 1) {
                const int t = th >> 1, h = th & 1;  // key tile and half of it
                const int us = u + (t - s.c0), slot = us % kPtScaleSlots;
                if (h == 0 && !(ok = wait_warp(&sc_full[slot], (us / kPtScaleSlots) & 1))) break;
                if (!(ok = wait_warp(&s_full[2 * i + h], (ns >> 1) & 1))) break;
                tc_fence_after();
                if constexpr (ONE) {
                    if (twice && (r >> 6) != h) {  // the other lanes' keys (uniform over the warp)
                        uint32_t zero[32];
#pragma unroll
                        for (int k = 0; k < 32; ++k) zero[k] = 0u;
                        tmem_st32(tP + h * C::P_STRIDE, zero);
                        tmem_st_wait();
                        tc_fence_before();
                        mbar_arrive(&p_full[2 * i + h]);
                        ++ns;
                        continue;
                    }
                }
                const uint32_t tSh = tS + h * 64;
                uint32_t sr[2][32];
                tmem_ld32(tSh, sr[0]);
                tmem_ld32(tSh + 32, sr[1]);
                const float4* sc4 = reinterpret_cast<const float4*>(sm + C::SC_OFF + slot * 96) + h;
                const float4 ks4 = sc4[0], lv4 = sc4[2], il4 = sc4[4];
                float c2[4] = {ks4.x * rc, ks4.y * rc, ks4.z * rc, ks4.w * rc};
                const float lv[4] = {lv4.x, lv4.y, lv4.z, lv4.w}, il[4] = {il4.x, il4.y, il4.z, il4.w};
                tmem_ld_wait(sr[0]);
                tmem_ld_wait(sr[1]);
                if (t * 128 + h * 64 + 64 > vis_min) {
                    const int lim = limit - t * 128 - h * 64;
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (c * 32 + k >= lim) sr[c][k] = __float_as_uint(-CUDART_INF_F);
                }
                float m_new = mu;
#pragma unroll
                for (int gr = 0; gr < 4; ++gr) {
                    const uint32_t* v = &sr[gr >> 1][(gr & 1) * 16];
                    float a = -CUDART_INF_F, b = -CUDART_INF_F;
#pragma unroll
                    for (int k = 0; k < 16; k += 4) {
                        a = fmax3(a, __uint_as_float(v[k]), __uint_as_float(v[k + 1]));
                        b = fmax3(b, __uint_as_float(v[k + 2]), __uint_as_float(v[k + 3]));
                    }
                    a = fmaxf(a, b);
                    // a slope of zero (a block of zeros) would turn masked scores into NaN
                    c2[gr] = c2[gr] < 1e-37f || a == -CUDART_INF_F ? 1e-37f : c2[gr];
                    m_new = fmaxf(m_new, fmaf(a, c2[gr], lv[gr]));
                }
                const bool resc = m_new - mu > kPtRescale;
                float alpha = 1.f;
                if (resc) {
                    alpha = ex2_approx(mu - m_new);
                    mu = m_new;
                    l *= alpha;
                }
                const float sub = mu == -CUDART_INF_F ? 0.f : mu - kPtOffset;
                uint32_t pk[32];
#pragma unroll
                for (int gr = 0; gr < 4; ++gr) {
                    const float add = lv[gr] - sub;
                    const uint64_t cc = f2_make(c2[gr], c2[gr]), aa = f2_make(add, add);
                    uint64_t sum = 0ull;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint32_t* v = &sr[gr >> 1][(gr & 1) * 16 + 2 * k];
                        float y0, y1;
                        f2_split(f2_fma(f2_make(__uint_as_float(v[0]), __uint_as_float(v[1])), cc, aa), y0, y1);
                        const float e0 = ex2_approx(y0), e1 = ex2_approx(y1);
                        pk[gr * 8 + k] = pack_f16x2(e0, e1);
                        sum = f2_add(sum, f2_make(e0, e1));
                    }
                    float a, b;
                    f2_split(sum, a, b);
                    l = fmaf(a + b, il[gr], l);
                }
                tmem_st32(tP + h * C::P_STRIDE, pk);
                if (__any_sync(0xffffffffu, resc) && th > 2 * first) {
                    // O of the halves so far is final once the last one's P V
                    // is (the ones before it were issued ahead of this S; the
                    // next one waits for this half's P)
                    if (!(ok = wait_warp(&pv_done[2 * i + (h ^ 1)], ((ns - 1) >> 1) & 1))) break;
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t ov[32];
                        tmem_ld32(tO + c * 32, ov);
                        tmem_ld_wait(ov);
#pragma unroll
                        for (int k = 0; k < 32; ++k) ov[k] = __float_as_uint(__uint_as_float(ov[k]) * alpha);
                        tmem_st32(tO + c * 32, ov);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                if (!FA_DROP_THIS_ARRIVE(ns == 0)) mbar_arrive(&p_full[2 * i + h]);
                ++ns;
            }
            u += s.c1 - s.c0;
            // ---------------------------------------------------- the piece's rows
            if (ok && end > first) ok = wait_warp(&pv_done[2 * i + 1], ((ns - 1) >> 1) & 1);
            if (ok) ok = wait_warp(&nan_full[seg % kPtNanSlots], (seg / kPtNanSlots) & 1);
            // the row tile's warps leave together, so that none waits for the others below
            // (ONE: of both row tiles, for the same reason)
            if (!(ok = ONE ? named_all(3, 256, ok) : named_all(1 + i, 128, ok))) break;
            if (base >= rows) {  // no rows: nothing to write or to merge, in no piece of the unit
                mbar_arrive(&nan_empty[seg % kPtNanSlots]);
                ++seg;
                continue;
            }
            tc_fence_after();
            const unsigned long long* nf = nan_first + (seg % kPtNanSlots) * D;
            const uint32_t nan_tag = pt_nan_tag(seg);
            const bool nan_seen = nan_piece[seg % kPtNanSlots] == seg;
            ++seg;
            const bool whole = s.c0 == 0 && s.c1 == s.ntile;
            // (ONE: the parts of a whole unit lie in a third slot, until row tile 0 joins them)
            const int slot = ONE && whole ? 2 * kPagedCtas + static_cast<int>(blockIdx.x)
                                          : 2 * static_cast<int>(blockIdx.x) + (s.line0 <= x0 ? 0 : 1);
            const bool leave = ONE || !whole;
            float inv = leave ? 1.f : l == 0.f ? 0.f : 1.f / l;
            // PFX: weight of the prefix, if there is one, in the row's output, and L
            [[maybe_unused]] float before = -1.f, lse_all = 0.f;
            [[maybe_unused]] const size_t orow = qrow / D;
            auto row_weights = [&](float M, float L, float& own) {
                lse_all = L == 0.f ? -CUDART_INF_F : (M - kPtOffset + log2f(L)) * kPtLn2;
                if (p.join.leaves) {
                    if (row_ok) p.join.ml[orow] = paged_leave(M, L);
                } else if (row_ok && paged_joins(p.join, s.r.b)) {
                    const PagedWeights w = paged_weights(M, L, paged_left(p.join, orow));
                    own = w.own;
                    before = w.prefix;
                    lse_all = w.lse;
                }
            };
            // columns c .. c + 7 of the row, normalised
            auto put_row = [&](int c, float (&v)[8]) {
                float4* at = reinterpret_cast<float4*>(p.join.o + qrow + c);
                if (p.join.leaves) {
                    at[0] = make_float4(v[0], v[1], v[2], v[3]);
                    at[1] = make_float4(v[4], v[5], v[6], v[7]);
                    return;
                }
                if (!(before < 0.f)) {
                    const float4 x = __ldcg(at), y = __ldcg(at + 1);
                    v[0] = fmaf(before, x.x, v[0]);
                    v[1] = fmaf(before, x.y, v[1]);
                    v[2] = fmaf(before, x.z, v[2]);
                    v[3] = fmaf(before, x.w, v[3]);
                    v[4] = fmaf(before, y.x, v[4]);
                    v[5] = fmaf(before, y.y, v[5]);
                    v[6] = fmaf(before, y.z, v[6]);
                    v[7] = fmaf(before, y.w, v[7]);
                }
                *reinterpret_cast<uint4*>(p.o + qrow + c) =
                    make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                               pack_bf16x2(v[6], v[7]));
            };
            if constexpr (PFX) {
                if (!p.join.leaves) paged_wait_before();
                if (!leave) row_weights(mu, l, inv);
            }
            // partial outputs lie as [d / 4][128 rows] float4, coalesced over the rows
            float4* po = reinterpret_cast<float4*>(p.po) + (static_cast<size_t>(2 * slot + i) * (D / 4)) * 128 + r;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t ov[32];
                if (end > first) {
                    tmem_ld32(tO + c * 32, ov);
                    tmem_ld_wait(ov);
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) ov[k] = 0u;
                }
                if (nan_seen) {
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (static_cast<uint32_t>(nf[c * 32 + k] >> 32) == nan_tag &&
                            static_cast<int>(nf[c * 32 + k] & 0xFFFFFFFFu) < limit)
                            ov[k] = __float_as_uint(CUDART_NAN_F);
                }
                if (!leave) {
                    if constexpr (PFX) {
                        if (row_ok) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                float v[8];
#pragma unroll
                                for (int y = 0; y < 8; ++y) v[y] = __uint_as_float(ov[8 * k + y]) * inv;
                                put_row(c * 32 + k * 8, v);
                            }
                        }
                    } else if (row_ok) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint4 w;
                            w.x = pack_bf16x2(__uint_as_float(ov[8 * k + 0]) * inv, __uint_as_float(ov[8 * k + 1]) * inv);
                            w.y = pack_bf16x2(__uint_as_float(ov[8 * k + 2]) * inv, __uint_as_float(ov[8 * k + 3]) * inv);
                            w.z = pack_bf16x2(__uint_as_float(ov[8 * k + 4]) * inv, __uint_as_float(ov[8 * k + 5]) * inv);
                            w.w = pack_bf16x2(__uint_as_float(ov[8 * k + 6]) * inv, __uint_as_float(ov[8 * k + 7]) * inv);
                            reinterpret_cast<uint4*>(p.o + qrow + c * 32)[k] = w;
                        }
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        po[(c * 8 + k) * 128] =
                            make_float4(__uint_as_float(ov[4 * k]), __uint_as_float(ov[4 * k + 1]),
                                        __uint_as_float(ov[4 * k + 2]), __uint_as_float(ov[4 * k + 3]));
                }
            }
            tc_fence_before();  // O has been read: the next piece's products may overwrite it
            mbar_arrive(&nan_empty[(seg - 1) % kPtNanSlots]);
            const float lse_off = kPtOffset;
            if (!leave) {
                if constexpr (PFX) {
                    if (row_ok && !p.join.leaves) p.lse[static_cast<size_t>(hq) * p.total + s.r.tok0 + tok] = lse_all;
                } else if (row_ok)
                    p.lse[static_cast<size_t>(hq) * p.total + s.r.tok0 + tok] =
                        l == 0.f ? -CUDART_INF_F : (mu - lse_off + log2f(l)) * kPtLn2;
            } else {
                p.pm[slot * kPagedTileRows + i * 128 + r] = mu;
                p.pl[slot * kPagedTileRows + i * 128 + r] = l;
                // pieces of a unit lie in consecutive CTAs; whoever finishes last
                // merges them in order
                const int f = static_cast<int>(div_short(s.line0, quota));
                const int e = static_cast<int>(div_short(s.line0 + s.ntile - 1, quota));
                if constexpr (ONE) {
                    if (whole) {
                        // the parts are read past L1: written that far before the barrier
                        __threadfence();
                        named_sync(3, 256);
                        if (i == 0 && row_ok && !(twice && r >= 64)) {
                            const int n = twice ? 4 : 2;  // parts: row tile k & 1, lanes 64 (k >> 1) + r
                            auto at = [&](int k) { return slot * kPagedTileRows + (k & 1) * 128 + 64 * (k >> 1) + r; };
                            float M = -CUDART_INF_F, L = 0.f, w[4];
                            for (int k = 0; k < n; ++k) M = fmaxf(M, __ldcg(&p.pm[at(k)]));
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                w[k] = 0.f;
                                if (k >= n) continue;
                                const float m = __ldcg(&p.pm[at(k)]);
                                w[k] = m == -CUDART_INF_F ? 0.f : ex2_approx(m - M);
                                L = fmaf(w[k], __ldcg(&p.pl[at(k)]), L);
                            }
                            float own = L == 0.f ? 0.f : 1.f / L;
                            row_weights(M, L, own);
                            for (int c = 0; c < D; c += 8) {
                                float v[8] = {};
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    if (k >= n) continue;
                                    const float4* src = reinterpret_cast<const float4*>(p.po) +
                                                        (static_cast<size_t>(2 * slot + (k & 1)) * (D / 4) + c / 4) * 128 +
                                                        64 * (k >> 1) + r;
                                    const float4 x = __ldcg(src), y = __ldcg(src + 128);
                                    v[0] = fmaf(w[k], x.x, v[0]);
                                    v[1] = fmaf(w[k], x.y, v[1]);
                                    v[2] = fmaf(w[k], x.z, v[2]);
                                    v[3] = fmaf(w[k], x.w, v[3]);
                                    v[4] = fmaf(w[k], y.x, v[4]);
                                    v[5] = fmaf(w[k], y.y, v[5]);
                                    v[6] = fmaf(w[k], y.z, v[6]);
                                    v[7] = fmaf(w[k], y.w, v[7]);
                                }
#pragma unroll
                                for (int y = 0; y < 8; ++y) v[y] *= own;
                                put_row(c, v);
                            }
                        }
                        continue;
                    }
                }
                if constexpr (PFX) {
                    if (p.join.cuts) {  // merged by a kernel of its own, over the whole GPU
                        if (r == 0 && i == 0 && s.c0 == 0)
                            p.join.cuts[slot] = {1, s.r.tok0, s.pair * RT, rows, s.hk, f, e, ONE ? (twice ? 4 : 2) : 1, s.line0, quota};
                        continue;
                    }
                }
                __threadfence();
                named_sync(1 + i, 128);
                if (r == 0) last_s[i] = atomicAdd(&p.counters[2 * s.unit + i], 1) == e - f;
                named_sync(1 + i, 128);
                if (last_s[i]) {
                    __threadfence();
                    auto piece = [&](int cta) { return 2 * cta + (s.line0 <= quota * cta ? 0 : 1); };
                    float M = -CUDART_INF_F, L = 0.f;
                    for (int cta = f; cta <= e; ++cta)
                        M = fmaxf(M, __ldcg(&p.pm[piece(cta) * kPagedTileRows + i * 128 + r]));
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        float4 acc[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                        L = 0.f;
                        for (int cta = f; cta <= e; ++cta) {
                            const int sl = piece(cta), at = sl * kPagedTileRows + i * 128 + r;
                            const float mc = __ldcg(&p.pm[at]);
                            const float w = mc == -CUDART_INF_F ? 0.f : ex2_approx(mc - M);
                            L = fmaf(w, __ldcg(&p.pl[at]), L);
                            const float4* src = reinterpret_cast<const float4*>(p.po) +
                                                (static_cast<size_t>(2 * sl + i) * (D / 4) + c * 8) * 128 + r;
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const float4 v = __ldcg(src + k * 128);
                                acc[k].x = fmaf(w, v.x, acc[k].x);
                                acc[k].y = fmaf(w, v.y, acc[k].y);
                                acc[k].z = fmaf(w, v.z, acc[k].z);
                                acc[k].w = fmaf(w, v.w, acc[k].w);
                            }
                        }
                        float iL = L == 0.f ? 0.f : 1.f / L;
                        if constexpr (PFX) {
                            row_weights(M, L, iL);
                            if (row_ok) {
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    float v[8] = {acc[2 * k].x * iL,     acc[2 * k].y * iL,     acc[2 * k].z * iL,
                                                  acc[2 * k].w * iL,     acc[2 * k + 1].x * iL, acc[2 * k + 1].y * iL,
                                                  acc[2 * k + 1].z * iL, acc[2 * k + 1].w * iL};
                                    put_row(c * 32 + k * 8, v);
                                }
                            }
                        } else if (row_ok) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                uint4 w;
                                w.x = pack_bf16x2(acc[2 * k].x * iL, acc[2 * k].y * iL);
                                w.y = pack_bf16x2(acc[2 * k].z * iL, acc[2 * k].w * iL);
                                w.z = pack_bf16x2(acc[2 * k + 1].x * iL, acc[2 * k + 1].y * iL);
                                w.w = pack_bf16x2(acc[2 * k + 1].z * iL, acc[2 * k + 1].w * iL);
                                reinterpret_cast<uint4*>(p.o + qrow + c * 32)[k] = w;
                            }
                        }
                    }
                    if constexpr (PFX) {
                        if (row_ok && !p.join.leaves) p.lse[static_cast<size_t>(hq) * p.total + s.r.tok0 + tok] = lse_all;
                    } else if (row_ok)
                        p.lse[static_cast<size_t>(hq) * p.total + s.r.tok0 + tok] =
                            L == 0.f ? -CUDART_INF_F : (M - lse_off + log2f(L)) * kPtLn2;
                }
            }
        } while (next(s));
        if (!ok) pt_gave_up(&abort_s, p.status, 97);
    } else {
        // ---------------------------------------------------------- V to f16, thread = key
        regs_dec<112>();
        const int r = (warp - 12) * 32 + lane;
        int u = 0, seg = 0;
        bool ok = true;
        do {
            const int rows = s.r.n * p.G;
            const int vis_min = pt_visible(p, s.r, p.by_g.div(s.pair * RT));
            const int vis_max = pt_visible(p, s.r, p.by_g.div(min(s.pair * RT + RT - 1, rows - 1)));
            unsigned long long* nf = nan_first + (seg % kPtNanSlots) * D;
            if (!(ok = wait_warp(&nan_empty[seg % kPtNanSlots], ((seg / kPtNanSlots) & 1) ^ 1))) break;
            for (int t = s.c0; t < s.c1; ++t, ++u) {
                const int vs = u % C::VS, rs = u % C::RS;
                ok = wait_warp(&r_full[rs], (u / C::RS) & 1);
                if (!ok) break;
                // row r as TMA swizzled it (d = 64: two bits of the row index
                // above its 64-byte pair)
                uint4 x[D / 16];
                const uint32_t rb = smem_u32(sm + C::R_OFF + rs * C::K_BYTES) + r * D;
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
                    x[j] = lds128_u4(rb + ((D == 128 ? j ^ (r & 7) : j ^ ((r >> 1) & 3)) << 4));
                ok = wait_warp(&v_empty[vs], ((u / C::VS) & 1) ^ 1);
                if (!ok) break;
                if (t * 128 + 128 > vis_min) {
                    // rows that no query sees count as zero; a NaN that only
                    // some see is noted and taken out, the softmax warps give
                    // it back to the rows that see it
                    const int key = t * 128 + r;
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            if (key >= vis_max) w[y] = 0u;
                            const uint32_t nb = ((w[y] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                            if (nb) {
                                nan_piece[seg % kPtNanSlots] = seg;
#pragma unroll
                                for (int z = 0; z < 4; ++z)
                                    if ((nb >> (8 * z)) & 0x80u) {
                                        atomicMin(&nf[j * 16 + y * 4 + z],
                                                  (static_cast<unsigned long long>(pt_nan_tag(seg)) << 32) |
                                                      static_cast<uint32_t>(key));
                                        w[y] &= ~(0xFFu << (8 * z));
                                    }
                            }
                        }
                        x[j] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                // row r of the [128 keys x 64 columns] swizzled regions
                uint8_t* vb = sm + C::V_OFF + vs * C::V_BYTES + r * 128;
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
                    uint32_t h[8];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        h[2 * y] = f16x2_from_e4m3x2(w[y]);
                        h[2 * y + 1] = f16x2_from_e4m3x2(w[y] >> 16);
                    }
                    uint8_t* reg = vb + (j >> 2) * 16384;
                    const int c = (j & 3) * 2;
                    sts128(smem_u32(reg + ((c ^ (r & 7)) << 4)), h[0], h[1], h[2], h[3]);
                    sts128(smem_u32(reg + (((c + 1) ^ (r & 7)) << 4)), h[4], h[5], h[6], h[7]);
                }
                // Only here, with every loaded value used, may the copy of a later
                // tile take the row's place: the arrival does not wait for loads
                // whose values are still on their way (released right behind the
                // loads, the row was overwritten under them about once in 10^4
                // tiles).
                mbar_arrive(&r_empty[rs]);
                fence_proxy_async_smem();
                mbar_arrive(&v_full[vs]);
            }
            if (!ok) break;
            mbar_arrive(&nan_full[seg % kPtNanSlots]);
            ++seg;
        } while (next(s));
        if (!ok) pt_gave_up(&abort_s, p.status, 98);
    }
    if constexpr (PFX) paged_wait_before();
    tc_fence_before();
    __syncthreads();
    if (warp == 3) {
        tc_fence_after();
        tmem_dealloc(tm, 512);
    }
}

// K or V as [num_blocks * Hkv * block_size rows, d] in boxes of a block (at most
// 128 rows), with the swizzle of its row length.
static bool make_tmap_rows(CUtensorMap* map, const void* base, uint64_t rows, int d, uint32_t box_rows) {
    EncodeTiledFn fn = encode_tiled_fn();
    if (!fn) return false;
    cuuint64_t gdim[2] = {static_cast<cuuint64_t>(d), rows};
    cuuint64_t gstride[1] = {static_cast<cuuint64_t>(d)};
    cuuint32_t box[2] = {static_cast<cuuint32_t>(d), box_rows};
    cuuint32_t estride[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), gdim, gstride, box, estride,
              CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool PFX, bool ONE = false>
static cudaError_t launch_tile(const PagedArgs& a, const PtParams& p, cudaStream_t stream) {
    using C = PtCfg<D, ONE>;
    CUtensorMap tk, tv;
    const uint64_t rows = static_cast<uint64_t>(a.num_blocks) * a.Hkv * a.block_size;
    const uint32_t box = a.block_size < 128 ? a.block_size : 128;
    if (!make_tmap_rows(&tk, a.k_cache, rows, D, box) || !make_tmap_rows(&tv, a.v_cache, rows, D, box))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = once_per_device(done, [] {
        return cudaFuncSetAttribute(fa_paged_tile_kernel<D, PFX, ONE>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at;
    const cudaLaunchConfig_t cfg = paged_config(512, C::SMEM, stream, PFX && a.chained, &at);
    return cudaLaunchKernelEx(&cfg, fa_paged_tile_kernel<D, PFX, ONE>, tk, tv, p);
}

cudaError_t launch_paged_tile(const PagedArgs& a, cudaStream_t stream) {
    PtParams p;
    p.q = static_cast<const uint16_t*>(a.q);
    p.k_scale = a.k_scale;
    p.v_scale = a.v_scale;
    p.o = static_cast<uint16_t*>(a.o);
    p.lse = a.lse;
    p.cu_seqlens = a.cu_seqlens;
    p.cache_len = a.cache_len;
    p.block_table = a.block_table;
    p.B = a.B;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.G = a.Hq / a.Hkv;
    p.by_g = make_fast_div(p.G);
    p.split_rows = a.split_rows;
    p.total = a.total;
    p.max_new = a.max_new;
    p.max_blocks = a.max_blocks;
    p.num_blocks = a.num_blocks;
    p.bs_log2 = 0;
    while ((1 << p.bs_log2) < a.block_size) ++p.bs_log2;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.causal = a.causal;
    p.status = a.status;
    p.counters = a.tile_counters;
    p.max_units = a.max_tile_units;
    p.pm = a.tile_pm;
    p.pl = a.tile_pl;
    p.po = a.tile_po;
    p.join = a.join;
    if (a.one_tile) return a.d == 64 ? launch_tile<64, true, true>(a, p, stream) : launch_tile<128, true, true>(a, p, stream);
    if (a.join.ml) return a.d == 64 ? launch_tile<64, true>(a, p, stream) : launch_tile<128, true>(a, p, stream);
    return a.d == 64 ? launch_tile<64, false>(a, p, stream) : launch_tile<128, false>(a, p, stream);
}

}  // namespace fa
