// Norm of queries and keys for each head with the position's rotation in the
// same pass, and its gradient.
//
// Forward, for a head x of d elements at position s:
//   y = x / sqrt(mean(x^2) + eps) * w,    z = R(s) y,
// R turning the pair (y_u, y_v) of frequency i by s f_i. Backward, with dz:
//   u = R(s)^T dz,  xh = x r,  r = 1 / sqrt(mean(x^2) + eps),
//   dw = sum of u xh over all rows,   dx = r (u w - xh mean(u w xh)).
//
// Bound: the heads' bytes, once in and once out. Measured, [2, 16 + 16, 16384,
// 128] bf16: forward 98 us = 5,480 GB/s (81 % of a copy's rate; 70 % of the issue
// slots are used), gradient 139 + 4 us = 5,800 GB/s, with 32 + 8 heads 126 and 172;
// fp32 252 and 408 us = 4,265 and 3,950 GB/s; one token of 16 requests, 32 + 8
// heads: 6.4 us in a graph, of which a launch alone takes 2.
//
// A warp takes one token at a time: four (d = 128) or eight heads in a step,
// sixteen elements a lane, so that the token's angles are computed once for all
// its heads. What has to be hidden is the latency of HBM: each lane's pieces come
// through a ring of asynchronous copies, five steps ahead (loaded a step ahead
// into registers: 135 us forward, 224 gradient). Arithmetic is in fp32 pairs.
// Pointers kept from step to step instead of formed anew cost registers: 112 us
// with four CTAs on an SM, 99 with three and eight stages. The gradient
// takes q and then k, so that one set of sixteen sums for the weights stays in
// registers; CTAs leave their sums to a second kernel, which adds them in order.
#include <type_traits>

#include "fa_norm.cuh"

namespace fa {

template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kNormThreads, sizeof(T) == 2 ? 4 : 3)
    fa_norm_kernel(const __grid_constant__ NormArgs p, int parts) {
    extern __shared__ __align__(16) uint4 ring[];
    __shared__ uint64_t turns[D / 2];
    __shared__ __align__(16) float weights[2 * D];
    const int tid = threadIdx.x;
    norm_tables<T, D, INTER>(p, turns, weights, tid, kNormThreads);
    __syncthreads();
    norm_forward<T, D, INTER>(p, turns, weights, ring, blockIdx.x * (kNormThreads / 32) + (tid >> 5),
                              gridDim.x * (kNormThreads / 32), parts, tid >> 5, tid & 31);
}

template <typename T>
constexpr int kBwdStages = sizeof(T) == 2 ? 5 : 3;
template <typename T>
constexpr int kBwdRing = kNormThreads / 32 * kBwdStages<T> * 2 * NormRaw<T>::PIECES * 32 * 16;

template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kNormThreads, 2) fa_norm_bwd_kernel(const __grid_constant__ NormArgs p, int most) {
    using L = NormLane<D, INTER>;
    constexpr int WARPS = kNormThreads / 32, S = kBwdStages<T>, PIECES = NormRaw<T>::PIECES;
    extern __shared__ __align__(16) uint4 rings[];
    __shared__ uint64_t turns[D / 2];
    __shared__ __align__(16) float weights[2 * D];
    __shared__ __align__(16) float sums[WARPS][D];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    norm_tables<T, D, INTER>(p, turns, weights, tid, kNormThreads);
    if (blockIdx.x == 0 && tid == 0) *p.status = 0;
    __syncthreads();
    const L ln(lane, p.rot);
    uint64_t f[L::OWN];
    lane_turns<D, INTER>(ln, turns, p.rot, f);
    uint4* ring = rings + warp * S * 2 * PIECES * 32 + lane;
    const int w = blockIdx.x * WARPS + warp, nw = gridDim.x * WARPS;
    for (int ten = 0; ten < 2; ++ten) {  // q, then k: one set of sums in registers
        const NormRows rx = ten ? p.k : p.q, ru = ten ? p.k_out : p.q_out, rd = ten ? p.dk : p.dq;
        const int H = ten ? p.Hkv : p.Hq, np = (H + L::RPW - 1) / L::RPW;
        // of this tensor's own steps: an item without one would stop the ring's
        // cursor, which moves on behind an item's last step
        const int parts = min(most, np);
        const long long items = static_cast<long long>(p.tokens) * parts;
        const bool has_w = ten ? p.k_weight : p.q_weight;
        auto row = [&](const NormRows& r, const NormCursor& c) {
            return static_cast<T*>(r.data) + c.b * r.batch + (c.pass * L::RPW + ln.g) * r.head + c.n * r.token;
        };
        NormVec acc = {};
        NormCursor in{w}, at{w};
        bool more = in.open(p, items, parts, np);
        int slot = 0, next = 0;
        auto issue = [&] {
            if (more) {
                if (in.pass * L::RPW + ln.g < H) {
                    const T* u = row(ru, in);
#pragma unroll
                    for (int i = 0; i < PIECES; ++i)
                        cp_async16(ring + (next * 2 * PIECES + i) * 32, u + NormRaw<T>::at(i, ln.a, ln.b));
                    if (has_w) {
                        const T* x = row(rx, in);
#pragma unroll
                        for (int i = 0; i < PIECES; ++i)
                            cp_async16(ring + ((next * 2 + 1) * PIECES + i) * 32, x + NormRaw<T>::at(i, ln.a, ln.b));
                    }
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
                const bool mine = there && at.pass * L::RPW + ln.g < H;
                NormRaw<T> raw;
                NormVec u, x;
                raw.zero();
                if (mine && has_w) {
#pragma unroll
                    for (int i = 0; i < PIECES; ++i) raw.w[i] = ring[((slot * 2 + 1) * PIECES + i) * 32];
                }
                raw.template get<INTER>(x);
                raw.zero();
                if (mine) {
#pragma unroll
                    for (int i = 0; i < PIECES; ++i) raw.w[i] = ring[(slot * 2 * PIECES + i) * 32];
                }
                raw.template get<INTER>(u);
                slot = slot + 1 == S ? 0 : slot + 1;
                issue();  // into the slot of the step before this one
                rotate_row<true>(u, turn);
                if (has_w) {
                    float sc;
                    NormVec y;
                    const float r = row_rms<D, L::TPR>(x, p.eps, sc);
                    lds_row<INTER>(y, weights + ten * D, ln.a, ln.b);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        x[i] = f2_mul(x[i], f2_all(r));
                        acc[i] = f2_fma(u[i], x[i], acc[i]);
                        u[i] = f2_mul(u[i], y[i]);
                    }
                    const float dot = row_dot<L::TPR>(u, x) * (-1.f / D), rs = r * sc;
#pragma unroll
                    for (int i = 0; i < 8; ++i) u[i] = f2_mul(f2_fma(f2_all(dot), x[i], u[i]), f2_all(rs));
                }
                raw.template set<INTER>(u);
                if (mine) raw.store(row(rd, at), ln.a, ln.b);
            }
        }
        cp_async_wait<0>();
        if (!has_w) continue;
        // this CTA's sums, in a fixed order
        float a[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) f2_split(acc[i], a[2 * i], a[2 * i + 1]);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
#pragma unroll
            for (int off = L::TPR; off < 32; off <<= 1) a[i] += __shfl_xor_sync(0xffffffffu, a[i], off);
            // element of u (i < 8) or v of pair i & 7
            const int k = i & 7;
            const int e = INTER ? (k < 4 ? ln.a : ln.b) + 2 * (k & 3) + (i >> 3) : (i < 8 ? ln.a : ln.b) + k;
            if (ln.g == 0) sums[warp][e] = a[i];
        }
        __syncthreads();
        if (tid < D) {
            float x = 0.f;
#pragma unroll
            for (int i = 0; i < WARPS; ++i) x += sums[i][tid];
            p.partial[(static_cast<size_t>(blockIdx.x) * 2 + ten) * D + tid] = x;
        }
        __syncthreads();
    }
}

// Sums of the CTAs' partial gradients of the weights: 32 columns a CTA.
__global__ void __launch_bounds__(1024) fa_norm_bwd_sum_kernel(const __grid_constant__ NormArgs p, int ctas) {
    __shared__ float part[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int at = blockIdx.x * 32 + lane, ten = at >= p.d;
    float* out = ten ? p.dk_weight : p.dq_weight;
    if (!out) return;  // uniform over the CTA: d is a multiple of 32
    float x = 0.f;
    for (int c = warp; c < ctas; c += 32) x += p.partial[static_cast<size_t>(c) * 2 * p.d + at];
    part[warp][lane] = x;
    __syncthreads();
    x = part[lane][warp];  // column `warp`, a lane for each part
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    if (lane == 0) out[blockIdx.x * 32 + warp - (ten ? p.d : 0)] = x;
}

// Parts that a token's heads are cut into, so that few tokens use many warps.
static int norm_parts(const NormArgs& a, int warps, int passes) {
    const int want = (warps + a.tokens - 1) / a.tokens;
    return want < 1 ? 1 : want > passes ? passes : want;
}
static int passes_of(int heads, int d) { return (heads * (d / 16) + 31) / 32; }

template <typename T, int D, bool INTER>
static cudaError_t launch_fwd(const NormArgs& a, cudaStream_t stream) {
    const int most = 152 * (sizeof(T) == 2 ? 4 : 3), warps = kNormThreads / 32;
    const int parts = norm_parts(a, most * warps, passes_of(a.Hq, D) + passes_of(a.Hkv, D));
    const long long ctas = (static_cast<long long>(a.tokens) * parts + warps - 1) / warps;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = once_per_device(done, [] {
        return cudaFuncSetAttribute(fa_norm_kernel<T, D, INTER>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kNormRing<T>);
    });
    if (e != cudaSuccess) return e;
    fa_norm_kernel<T, D, INTER>
        <<<static_cast<unsigned>(ctas < most ? ctas : most), kNormThreads, kNormRing<T>, stream>>>(a, parts);
    return cudaGetLastError();
}

template <typename T, int D, bool INTER>
static cudaError_t launch_bwd(const NormArgs& a, cudaStream_t stream, int* nlaunch) {
    const int warps = kNormThreads / 32, parts = norm_parts(a, kNormBwdCtas * warps, passes_of(a.Hq, D));
    const long long want = (static_cast<long long>(a.tokens) * parts + warps - 1) / warps;
    const int ctas = static_cast<int>(want < kNormBwdCtas ? want : kNormBwdCtas);
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = once_per_device(done, [] {
        return cudaFuncSetAttribute(fa_norm_bwd_kernel<T, D, INTER>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kBwdRing<T>);
    });
    if (e != cudaSuccess) return e;
    fa_norm_bwd_kernel<T, D, INTER><<<ctas, kNormThreads, kBwdRing<T>, stream>>>(a, parts);
    *nlaunch = 1;
    if (a.q_weight || a.k_weight) {
        fa_norm_bwd_sum_kernel<<<2 * D / 32, 1024, 0, stream>>>(a, ctas);
        *nlaunch = 2;
    }
    return cudaGetLastError();
}

template <typename F>
static void dispatch(const NormArgs& a, F&& f) {
    auto typed = [&](auto t) {
        using T = decltype(t);
        if (a.d == 64) a.interleaved ? f(t, std::integral_constant<int, 64>{}, std::true_type{})
                                     : f(t, std::integral_constant<int, 64>{}, std::false_type{});
        else a.interleaved ? f(t, std::integral_constant<int, 128>{}, std::true_type{})
                           : f(t, std::integral_constant<int, 128>{}, std::false_type{});
    };
    if (a.fp32) typed(float{});
    else typed(uint16_t{});
}

cudaError_t launch_norm(const NormArgs& a, cudaStream_t stream, int* nlaunch) {
    cudaError_t e = cudaSuccess;
    *nlaunch = 1;
    dispatch(a, [&](auto t, auto d, auto inter) {
        e = launch_fwd<decltype(t), decltype(d)::value, decltype(inter)::value>(a, stream);
    });
    return e;
}

cudaError_t launch_norm_bwd(const NormArgs& a, cudaStream_t stream, int* nlaunch) {
    cudaError_t e = cudaSuccess;
    dispatch(a, [&](auto t, auto d, auto inter) {
        e = launch_bwd<decltype(t), decltype(d)::value, decltype(inter)::value>(a, stream, nlaunch);
    });
    return e;
}

}  // namespace fa
