// Device side shared by the norm kernels: positions, angles and rows.
#pragma once

#include "fa_norm.h"
#include "sm103_ptx.cuh"

namespace fa {

// Angles are held as fractions of a turn in 64-bit fixed point: f / (2 pi)
// modulo 1 once for each frequency, then position * fraction modulo 2^64, which
// drops whole turns exactly. The fraction is within 2^-64 (either term's
// rounding is half of that at most), so that an angle is good to 2^-33 of a turn
// at any 32-bit position; 64-bit floating point would do as well, at a few
// results a cycle and SM. A negative frequency has the fraction of its opposite,
// negated: hi - floor(hi) is exact only where hi is not negative.
__device__ __forceinline__ uint64_t turn_fraction(double f) {
    constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;  // 1 / (2 pi)
    const double a = fabs(f), hi = a * kHi, lo = fma(a, kLo, fma(a, kHi, -hi));
    const uint64_t t = __double2ull_rn((hi - floor(hi)) * 0x1p64) + static_cast<uint64_t>(__double2ll_rn(lo * 0x1p64));
    return f < 0. ? 0ull - t : t;
}

// Cosine and sine of `a` turns: the nearest quarter turn, and the Taylor series
// of what is left, |x| <= pi / 4, up to x^11 (x^13 / 13! < 2^-36) and x^10
// (x^12 / 12! < 2^-33).
__device__ __forceinline__ void turn_cos_sin(uint64_t a, float& c, float& s) {
    const uint32_t i = static_cast<uint32_t>((a + 0x80000000ull) >> 32), quarter = (i + 0x20000000u) >> 30;
    const float r = static_cast<float>(static_cast<int>(i - (quarter << 30)));
    const float x = fmaf(r, 0x1.921fb6p+1f * 0x1p-31f, r * (-0x1.777a5cp-24f * 0x1p-31f)), x2 = x * x;
    float u = fmaf(x2, -1.f / 39916800.f, 1.f / 362880.f);
    u = fmaf(x2, u, -1.f / 5040.f);
    u = fmaf(x2, u, 1.f / 120.f);
    u = fmaf(x2, u, -1.f / 6.f);
    const float sn = fmaf(x * x2, u, x);
    float v = fmaf(x2, -1.f / 3628800.f, 1.f / 40320.f);
    v = fmaf(x2, v, -1.f / 720.f);
    v = fmaf(x2, v, 1.f / 24.f);
    v = fmaf(x2, v, -0.5f);
    const float cs = fmaf(x2, v, 1.f);
    const float p = quarter & 1 ? sn : cs, q = quarter & 1 ? cs : sn;
    c = (quarter + 1) & 2 ? -p : p;
    s = quarter & 2 ? -q : q;
}

// Last b in [0, B) with cu[b] <= t, found by the warp together.
__device__ __forceinline__ int warp_find(const int32_t* cu, int B, int t, int lane) {
    int lo = 0, n = B;
    while (n > 1) {
        const int step = (n + 31) >> 5, at = lane * step;
        const uint32_t in = __ballot_sync(0xffffffffu, at < n && cu[lo + at] <= t);
        const int k = in ? 31 - __clz(in) : 0;
        lo += k * step;
        n = min(step, n - k * step);
    }
    return lo;
}

// Position of token t of a packed batch whose sequence is b; arithmetic modulo 2^32.
__device__ __forceinline__ int packed_position(const NormArgs& p, int b, int t) {
    const uint32_t from = p.ends ? static_cast<uint32_t>(p.ends[b]) - static_cast<uint32_t>(p.cu_seqlens[b + 1])
                                 : 0u - static_cast<uint32_t>(p.cu_seqlens[b]);
    return static_cast<int>(from + static_cast<uint32_t>(t));
}

// A row of D elements lies in D / 16 lanes, sixteen elements each, as two chunks
// of eight that hold whole pairs of the rotation: neighbours (INTER), or element
// i in one chunk and element i + rot / 2 in the other.
template <int D, bool INTER>
struct NormLane {
    static constexpr int TPR = D / 16;          // lanes of a row
    static constexpr int RPW = 32 / TPR;        // rows of a warp
    static constexpr int OWN = 8 / RPW;         // angles that a lane computes of its eight
    int j, g;    // lane of its row, row of the warp
    int a, b;    // first elements of the two chunks
    __device__ __forceinline__ NormLane(int lane, int rot) : j(lane % TPR), g(lane / TPR) {
        const int np = rot >> 4;  // pairs of chunks that rotate
        if (INTER) {
            a = j * 8;
            b = (j + TPR) * 8;
        } else if (j < np) {
            a = j * 8;
            b = (j + np) * 8;
        } else {
            a = j * 16;
            b = a + 8;
        }
    }
    // index of the frequency of this lane's angle i (0..7); rot / 2 or more: none
    __device__ __forceinline__ int freq(int i) const {
        if (INTER) return i < 4 ? (a >> 1) + i : (b >> 1) + i - 4;
        return 8 * j + i;
    }
};

// Cosines and sines of a lane's eight angles, two to a word.
struct NormTurn {
    uint64_t c[4], s[4];
};

// Angles of a token that all rows of the warp share: each lane computes OWN of
// them, the rest come from the lanes of the other rows.
template <int D, bool INTER>
__device__ __forceinline__ void warp_turn(const NormLane<D, INTER>& ln, const uint64_t (&f)[NormLane<D, INTER>::OWN],
                                          int pos, NormTurn& t) {
    using L = NormLane<D, INTER>;
    float c[L::OWN], s[L::OWN], cc[8], ss[8];
#pragma unroll
    for (int i = 0; i < L::OWN; ++i) turn_cos_sin(static_cast<uint64_t>(static_cast<int64_t>(pos)) * f[i], c[i], s[i]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int from = (i / L::OWN) * L::TPR + ln.j;
        cc[i] = __shfl_sync(0xffffffffu, c[i % L::OWN], from);
        ss[i] = __shfl_sync(0xffffffffu, s[i % L::OWN], from);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        t.c[i] = f2_make(cc[2 * i], cc[2 * i + 1]);
        t.s[i] = f2_make(ss[2 * i], ss[2 * i + 1]);
    }
}

// A lane's sixteen elements, two to a word: the first elements u of its pairs in
// x[0..3], the second ones v in x[4..7].
typedef uint64_t NormVec[8];

__device__ __forceinline__ uint64_t f2_neg(uint64_t x) { return x ^ 0x8000000080000000ull; }
__device__ __forceinline__ uint64_t f2_all(float x) { return f2_make(x, x); }

// Rotated by +angle, or by -angle (BACK).
template <bool BACK>
__device__ __forceinline__ void rotate_row(NormVec& x, const NormTurn& t) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t s = BACK ? f2_neg(t.s[i]) : t.s[i], u = x[i], v = x[i + 4];
        x[i] = f2_fma(u, t.c[i], f2_neg(f2_mul(v, s)));
        x[i + 4] = f2_fma(u, s, f2_mul(v, t.c[i]));
    }
}

template <int TPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int off = 1; off < TPR; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}
// Sum over the row of the products of two lanes' elements.
template <int TPR>
__device__ __forceinline__ float row_dot(const NormVec& x, const NormVec& y) {
    uint64_t a = f2_mul(x[0], y[0]), b = f2_mul(x[1], y[1]);
#pragma unroll
    for (int i = 2; i < 8; i += 2) {
        a = f2_fma(x[i], y[i], a);
        b = f2_fma(x[i + 1], y[i + 1], b);
    }
    float lo, hi;
    f2_split(f2_add(a, b), lo, hi);
    return row_sum<TPR>(lo + hi);
}

// r with 1 / sqrt(mean x^2 + eps) = f r, x then being scaled by f: 1 but for a
// row whose squares leave fp32's range.
template <int D, int TPR>
__device__ __forceinline__ float row_rms(NormVec& x, float eps, float& f) {
    float ss = row_dot<TPR>(x, x);
    const bool big = ss > 1e38f;
    f = big ? 0x1p-70f : 1.f;
    if (__any_sync(0xffffffffu, big)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = f2_mul(x[i], f2_all(f));
        ss = row_dot<TPR>(x, x);
        eps = eps * f * f;
    }
    return rsqrtf(fmaf(ss, 1.f / D, eps));
}

// The raw words of a lane's two chunks.
template <typename T>
struct NormRaw {
    static constexpr int PIECES = sizeof(T);  // of 16 bytes
    uint4 w[PIECES];
    // first element of piece i
    __device__ __forceinline__ static int at(int i, int a, int b) {
        return sizeof(T) == 2 ? (i ? b : a) : (i < 2 ? a : b) + 4 * (i & 1);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void load(const T* row, int a, int b) {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) w[i] = *reinterpret_cast<const uint4*>(row + at(i, a, b));
    }
    __device__ __forceinline__ void store(T* row, int a, int b) const {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) *reinterpret_cast<uint4*>(row + at(i, a, b)) = w[i];
    }
    // Word i of eight (bf16) or sixteen (fp32).
    __device__ __forceinline__ uint32_t word(int i) const {
        const uint4& v = w[i >> 2];
        return (i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w;
    }
    template <bool INTER>
    __device__ __forceinline__ void get(NormVec& x) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 2) {
                if constexpr (INTER) {
                    const uint32_t p = word(2 * i), q = word(2 * i + 1);
                    x[i] = f2_make(__uint_as_float(p << 16), __uint_as_float(q << 16));
                    x[i + 4] = f2_make(__uint_as_float(p & 0xFFFF0000u), __uint_as_float(q & 0xFFFF0000u));
                } else {
                    x[i] = f2_from_bf16x2(word(i));
                    x[i + 4] = f2_from_bf16x2(word(i + 4));
                }
            } else {
                const int u = INTER ? 4 * i : 2 * i, v = INTER ? 4 * i + 1 : 8 + 2 * i, next = INTER ? 2 : 1;
                x[i] = f2_make(__uint_as_float(word(u)), __uint_as_float(word(u + next)));
                x[i + 4] = f2_make(__uint_as_float(word(v)), __uint_as_float(word(v + next)));
            }
        }
    }
    template <bool INTER>
    __device__ __forceinline__ void set(const NormVec& x) {
        uint32_t y[4 * PIECES];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float u0, u1, v0, v1;
            f2_split(x[i], u0, u1);
            f2_split(x[i + 4], v0, v1);
            if constexpr (sizeof(T) == 2) {
                y[INTER ? 2 * i : i] = INTER ? pack_bf16x2(u0, v0) : pack_bf16x2(u0, u1);
                y[INTER ? 2 * i + 1 : i + 4] = INTER ? pack_bf16x2(u1, v1) : pack_bf16x2(v0, v1);
            } else {
                const int u = INTER ? 4 * i : 2 * i, v = INTER ? 4 * i + 1 : 8 + 2 * i, next = INTER ? 2 : 1;
                y[u] = __float_as_uint(u0);
                y[u + next] = __float_as_uint(u1);
                y[v] = __float_as_uint(v0);
                y[v + next] = __float_as_uint(v1);
            }
        }
#pragma unroll
        for (int i = 0; i < PIECES; ++i) w[i] = make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
    }
};

template <typename T>
__device__ __forceinline__ float norm_weight(const T* w, int i) {
    if constexpr (sizeof(T) == 2) return __uint_as_float(static_cast<uint32_t>(w[i]) << 16);
    else return w[i];
}
// Where a row of weights in shared memory has element i: in the order of NormVec
// within each chunk of eight.
template <bool INTER>
__device__ __forceinline__ int norm_place(int i) {
    return INTER ? (i & ~7) | ((i & 1) << 2) | ((i >> 1) & 3) : i;
}
template <bool INTER>
__device__ __forceinline__ void lds_row(NormVec& y, const float* row, int a, int b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // INTER: u of a, u of b, v of a, v of b
        const int at = INTER ? (i & 1 ? b : a) + 4 * (i >> 1) : (i < 2 ? a : b) + 4 * (i & 1);
        const float4 v = *reinterpret_cast<const float4*>(row + at);
        y[2 * i] = f2_make(v.x, v.y);
        y[2 * i + 1] = f2_make(v.z, v.w);
    }
}

// One row of the forward: x / rms(x) * w (w null: x as it is), rotated.
template <int D, bool INTER>
__device__ __forceinline__ void norm_row(NormVec& x, const float* w, const NormLane<D, INTER>& ln, float eps,
                                         const NormTurn& t) {
    if (w) {
        float f;
        NormVec y;
        const float r = row_rms<D, NormLane<D, INTER>::TPR>(x, eps, f);
        lds_row<INTER>(y, w, ln.a, ln.b);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = f2_mul(f2_mul(x[i], f2_all(r)), y[i]);
    }
    rotate_row<false>(x, t);
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// Where a warp stands among its items: steps [pass, end) of token (b, n), one at
// least (parts <= np, which the callers see to).
struct NormCursor {
    long long it;
    int t, b, n, pass, end;
    __device__ __forceinline__ bool open(const NormArgs& p, long long items, int parts, int np) {
        if (it >= items) return false;
        t = static_cast<int>(parts == 1 ? it : div_short(it, parts));
        const int part = static_cast<int>(it - static_cast<long long>(t) * parts);
        b = p.cu_seqlens ? 0 : p.by_n.div(t);
        n = p.cu_seqlens ? t : t - b * p.N;
        pass = np * part / parts;
        end = np * (part + 1) / parts;
        return true;
    }
    // Position of the token; false if it is of no sequence.
    __device__ __forceinline__ bool position(const NormArgs& p, int lane, int& pos) const {
        if (p.cu_seqlens) {
            const int s = warp_find(p.cu_seqlens, p.B, t, lane);
            pos = packed_position(p, s, t);
            return t >= p.cu_seqlens[s] && t < p.cu_seqlens[s + 1];
        }
        pos = p.ends ? static_cast<int>(static_cast<uint32_t>(p.ends[b]) - static_cast<uint32_t>(p.N - n)) : n;
        return true;
    }
};

// A lane's frequencies: the OWN that it computes for its warp.
template <int D, bool INTER>
__device__ __forceinline__ void lane_turns(const NormLane<D, INTER>& ln, const uint64_t* turns, int rot,
                                           uint64_t (&f)[NormLane<D, INTER>::OWN]) {
    constexpr int OWN = NormLane<D, INTER>::OWN;
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
        const int at = ln.freq(ln.g * OWN + i);
        f[i] = at < rot / 2 ? turns[at] : 0ull;
    }
}

// Stages of a warp's ring in shared memory: the rows of a step each.
template <typename T>
constexpr int kNormStages = sizeof(T) == 2 ? 6 : 3;
template <typename T>
constexpr int kNormRing = kNormThreads / 32 * kNormStages<T> * NormRaw<T>::PIECES * 32 * 16;  // bytes

// Tokens' rows, RPW heads a step, first q's and then k's, for warp `w` of `nw`.
// Each lane copies its own pieces of the steps to come into shared memory and
// reads them back itself: no barriers.
template <typename T, int D, bool INTER>
__device__ __forceinline__ void norm_forward(const NormArgs& p, const uint64_t* turns, const float* weights,
                                             uint4* ring, int w, int nw, int parts, int warp, int lane) {
    using L = NormLane<D, INTER>;
    constexpr int S = kNormStages<T>, PIECES = NormRaw<T>::PIECES;
    const L ln(lane, p.rot);
    uint64_t f[L::OWN];
    lane_turns<D, INTER>(ln, turns, p.rot, f);
    ring += warp * S * PIECES * 32 + lane;
    const int pq = (p.Hq + L::RPW - 1) / L::RPW, np = pq + (p.Hkv + L::RPW - 1) / L::RPW;
    const float* wq = p.q_weight ? weights : nullptr;
    const float* wk = p.k_weight ? weights + D : nullptr;
    const long long items = static_cast<long long>(p.tokens) * parts;
    auto row = [&](const NormRows& q, const NormRows& k, const NormCursor& c, T*& at) {
        const bool is_k = c.pass >= pq;
        const int h = (is_k ? c.pass - pq : c.pass) * L::RPW + ln.g;
        const NormRows& r = is_k ? k : q;
        at = static_cast<T*>(r.data) + c.b * r.batch + h * r.head + c.n * r.token;
        return h < (is_k ? p.Hkv : p.Hq);
    };
    NormCursor in{w}, at{w};
    bool more = in.open(p, items, parts, np);
    int slot = 0, next = 0;
    auto issue = [&] {
        T* src;
        if (more) {
            if (row(p.q, p.k, in, src)) {
#pragma unroll
                for (int i = 0; i < PIECES; ++i)
                    cp_async16(ring + (next * PIECES + i) * 32, src + NormRaw<T>::at(i, ln.a, ln.b));
            }
            if (++in.pass == in.end) {
                in.it += nw;
                more = in.open(p, items, parts, np);
            }
        }
        cp_async_commit();
        next = next + 1 == S ? 0 : next + 1;
    };
#pragma unroll 1
    for (int i = 0; i < S - 1; ++i) issue();
    for (; at.open(p, items, parts, np); at.it += nw) {
        int pos;
        const bool there = at.position(p, lane, pos);
        NormTurn turn;
        warp_turn<D, INTER>(ln, f, pos, turn);
        for (; at.pass < at.end; ++at.pass) {
            cp_async_wait<S - 2>();
            NormRaw<T> raw;
#pragma unroll
            for (int i = 0; i < PIECES; ++i) raw.w[i] = ring[(slot * PIECES + i) * 32];
            slot = slot + 1 == S ? 0 : slot + 1;
            issue();  // into the slot of the step before this one
            NormVec x;
            raw.template get<INTER>(x);
            norm_row<D, INTER>(x, at.pass >= pq ? wk : wq, ln, p.eps, turn);
            raw.template set<INTER>(x);
            T* dst;
            if (row(p.q_out, p.k_out, at, dst) && there) raw.store(dst, ln.a, ln.b);
        }
    }
    cp_async_wait<0>();
}

// Fractions of a turn and the weights in fp32, into shared memory. The caller synchronises.
template <typename T, int D, bool INTER>
__device__ __forceinline__ void norm_tables(const NormArgs& p, uint64_t* turns, float* weights, int tid, int threads) {
    for (int i = tid; i < p.rot / 2; i += threads) turns[i] = turn_fraction(p.inv_freq[i]);
    for (int i = tid; i < 2 * D; i += threads) {
        const T* w = static_cast<const T*>(i < D ? p.q_weight : p.k_weight);
        if (w) weights[(i & ~(D - 1)) + norm_place<INTER>(i & (D - 1))] = norm_weight(w, i & (D - 1));
    }
}

}  // namespace fa
