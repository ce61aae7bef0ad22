// Device side shared by the norm kernels: positions, angles and rows.
#pragma once

#include "fa_norm.h"
#include "sm103_ptx.cuh"

namespace fa {

// Angles are held as fractions of a turn in 64-bit fixed point: f / (2 pi)
// modulo 1 once for each frequency, then position * fraction modulo 2^64, which
// drops whole turns exactly. The fraction's last place is 2^-64, so that an
// angle is good to 2^-33 of a turn at any 32-bit position; 64-bit floating
// point would do as well, at a few results a cycle and SM.
__device__ __forceinline__ uint64_t turn_fraction(double f) {
    constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;  // 1 / (2 pi)
    const double hi = f * kHi, lo = fma(f, kLo, fma(f, kHi, -hi));
    return __double2ull_rz((hi - floor(hi)) * 0x1p64) + static_cast<uint64_t>(__double2ll_rn(lo * 0x1p64));
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

struct NormTurn {
    float c[8], s[8];
};

// Angles of a token that all rows of the warp share: each lane computes OWN of
// them, the rest come from the lanes of the other rows.
template <int D, bool INTER>
__device__ __forceinline__ void warp_turn(const NormLane<D, INTER>& ln, const uint64_t (&f)[NormLane<D, INTER>::OWN],
                                          int pos, NormTurn& t) {
    using L = NormLane<D, INTER>;
    float c[L::OWN], s[L::OWN];
#pragma unroll
    for (int i = 0; i < L::OWN; ++i) turn_cos_sin(static_cast<uint64_t>(static_cast<int64_t>(pos)) * f[i], c[i], s[i]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int from = (i / L::OWN) * L::TPR + ln.j;
        t.c[i] = __shfl_sync(0xffffffffu, c[i % L::OWN], from);
        t.s[i] = __shfl_sync(0xffffffffu, s[i % L::OWN], from);
    }
}

// x[0..7]: chunk a, x[8..15]: chunk b. Rotated by +angle, or by -angle (BACK).
template <bool INTER, bool BACK>
__device__ __forceinline__ void rotate_row(float (&x)[16], const NormTurn& t) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int u = INTER ? 2 * i : i, v = INTER ? 2 * i + 1 : i + 8;
        const float s = BACK ? -t.s[i] : t.s[i], a = x[u], b = x[v];
        x[u] = fmaf(a, t.c[i], -(b * s));
        x[v] = fmaf(a, s, b * t.c[i]);
    }
}

template <int TPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int off = 1; off < TPR; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// r with 1 / sqrt(mean x^2 + eps) = f r, x then being scaled by f: 1 but for a
// row whose squares leave fp32's range.
template <int D, int TPR>
__device__ __forceinline__ float row_rms(float (&x)[16], float eps, float& f) {
    auto squares = [&] {
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            a = fmaf(x[i], x[i], a);
            b = fmaf(x[i + 8], x[i + 8], b);
        }
        return row_sum<TPR>(a + b);
    };
    float ss = squares();
    const bool big = ss > 1e38f;
    f = big ? 0x1p-70f : 1.f;
    if (__any_sync(0xffffffffu, big)) {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] *= f;
        ss = squares();
    }
    return rsqrtf(fmaf(ss, 1.f / D, eps * f * f));
}

// The raw words of a lane's two chunks.
template <typename T>
struct NormRaw;
template <>
struct NormRaw<uint16_t> {
    uint4 w[2];
    __device__ __forceinline__ void zero() { w[0] = w[1] = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void load(const uint16_t* row, int a, int b) {
        w[0] = *reinterpret_cast<const uint4*>(row + a);
        w[1] = *reinterpret_cast<const uint4*>(row + b);
    }
    __device__ __forceinline__ void get(float (&x)[16]) const {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const uint32_t v[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[8 * c + 2 * i] = __uint_as_float(v[i] << 16);
                x[8 * c + 2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
            }
        }
    }
    __device__ __forceinline__ void set(const float (&x)[16]) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
            w[c] = make_uint4(pack_bf16x2(x[8 * c], x[8 * c + 1]), pack_bf16x2(x[8 * c + 2], x[8 * c + 3]),
                              pack_bf16x2(x[8 * c + 4], x[8 * c + 5]), pack_bf16x2(x[8 * c + 6], x[8 * c + 7]));
    }
    __device__ __forceinline__ void store(uint16_t* row, int a, int b) const {
        *reinterpret_cast<uint4*>(row + a) = w[0];
        *reinterpret_cast<uint4*>(row + b) = w[1];
    }
};
template <>
struct NormRaw<float> {
    float4 w[4];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __device__ __forceinline__ void load(const float* row, int a, int b) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(row + (i < 2 ? a : b) + 4 * (i & 1));
    }
    __device__ __forceinline__ void get(float (&x)[16]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[4 * i] = w[i].x;
            x[4 * i + 1] = w[i].y;
            x[4 * i + 2] = w[i].z;
            x[4 * i + 3] = w[i].w;
        }
    }
    __device__ __forceinline__ void set(const float (&x)[16]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    }
    __device__ __forceinline__ void store(float* row, int a, int b) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<float4*>(row + (i < 2 ? a : b) + 4 * (i & 1)) = w[i];
    }
};

template <typename T>
__device__ __forceinline__ float norm_weight(const T* w, int i) {
    if constexpr (sizeof(T) == 2) return __uint_as_float(static_cast<uint32_t>(w[i]) << 16);
    else return w[i];
}

// Eight floats at a and eight at b of a row of D floats in shared memory.
__device__ __forceinline__ void lds_row(float (&y)[16], const float* row, int a, int b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 v = *reinterpret_cast<const float4*>(row + (i < 2 ? a : b) + 4 * (i & 1));
        y[4 * i] = v.x;
        y[4 * i + 1] = v.y;
        y[4 * i + 2] = v.z;
        y[4 * i + 3] = v.w;
    }
}

// One row of the forward: x / rms(x) * w (w null: x as it is), rotated.
template <int D, bool INTER>
__device__ __forceinline__ void norm_row(float (&x)[16], const float* w, const NormLane<D, INTER>& ln, float eps,
                                         const NormTurn& t) {
    if (w) {
        float f, y[16];
        const float r = row_rms<D, NormLane<D, INTER>::TPR>(x, eps, f);
        lds_row(y, w, ln.a, ln.b);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = x[i] * r * y[i];
    }
    rotate_row<INTER, false>(x, t);
}

// Tokens' rows [pass * RPW, + RPW) of q and then of k, for warp `w` of `nw`.
template <typename T, int D, bool INTER>
__device__ __forceinline__ void norm_forward(const NormArgs& p, const uint64_t* turns, const float* weights, int w,
                                             int nw, int parts, int lane) {
    using L = NormLane<D, INTER>;
    const L ln(lane, p.rot);
    uint64_t f[L::OWN];
#pragma unroll
    for (int i = 0; i < L::OWN; ++i) {
        const int at = ln.freq(ln.g * L::OWN + i);
        f[i] = at < p.rot / 2 ? turns[at] : 0ull;
    }
    const int pq = (p.Hq + L::RPW - 1) / L::RPW, pk = (p.Hkv + L::RPW - 1) / L::RPW, np = pq + pk;
    const float* wq = p.q_weight ? weights : nullptr;
    const float* wk = p.k_weight ? weights + D : nullptr;
    const long long items = static_cast<long long>(p.tokens) * parts;
    for (long long it = w; it < items; it += nw) {
        const int t = static_cast<int>(parts == 1 ? it : div_short(it, parts));
        const int part = static_cast<int>(it - static_cast<long long>(t) * parts);
        int b = 0, n = t, pos;
        if (p.cu_seqlens) {
            const int s = warp_find(p.cu_seqlens, p.B, t, lane);
            if (t < p.cu_seqlens[s] || t >= p.cu_seqlens[s + 1]) continue;  // of no sequence: left as it is
            pos = packed_position(p, s, t);
        } else {
            b = p.by_n.div(t);
            n = pos = t - b * p.N;
            if (p.ends) pos = static_cast<int>(static_cast<uint32_t>(p.ends[b]) - static_cast<uint32_t>(p.N - n));
        }
        const int p0 = np * part / parts, p1 = np * (part + 1) / parts;
        auto row = [&](const NormRows& q, const NormRows& k, int pass, T*& at) {
            const bool is_k = pass >= pq;
            const int h = (is_k ? pass - pq : pass) * L::RPW + ln.g;
            const NormRows& r = is_k ? k : q;
            at = static_cast<T*>(r.data) + b * r.batch + h * r.head + n * r.token;
            return h < (is_k ? p.Hkv : p.Hq);
        };
        NormRaw<T> next;
        T* at;
        next.zero();
        if (row(p.q, p.k, p0, at)) next.load(at, ln.a, ln.b);
        NormTurn turn;
        warp_turn<D, INTER>(ln, f, pos, turn);
        for (int pass = p0; pass < p1; ++pass) {
            NormRaw<T> raw = next;
            next.zero();
            if (pass + 1 < p1 && row(p.q, p.k, pass + 1, at)) next.load(at, ln.a, ln.b);
            float x[16];
            raw.get(x);
            norm_row<D, INTER>(x, pass >= pq ? wk : wq, ln, p.eps, turn);
            raw.set(x);
            if (row(p.q_out, p.k_out, pass, at)) raw.store(at, ln.a, ln.b);
        }
    }
}

// Fractions of a turn and the weights in fp32, into shared memory. The caller synchronises.
template <typename T, int D>
__device__ __forceinline__ void norm_tables(const NormArgs& p, uint64_t* turns, float* weights, int tid, int threads) {
    for (int i = tid; i < p.rot / 2; i += threads) turns[i] = turn_fraction(p.inv_freq[i]);
    for (int i = tid; i < 2 * D; i += threads) {
        const T* w = static_cast<const T*>(i < D ? p.q_weight : p.k_weight);
        if (w) weights[i] = norm_weight(w, i < D ? i : i - D);
    }
}

}  // namespace fa
