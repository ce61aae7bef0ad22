// Norm of queries and keys for each head with the position's rotation in the
// same pass, and its gradient.
//
// Forward, for a head x of d elements at position s:
//   y = x / sqrt(mean(x^2) + eps) * w,    z = R(s) y,
// R turning the pair (y_u, y_v) of frequency i by s f_i. Backward, with dz:
//   u = R(s)^T dz,  xh = x r,  r = 1 / sqrt(mean(x^2) + eps),
//   dw = sum of u xh over all rows,   dx = r (u w - xh mean(u w xh)).
//
// Bound: the heads' bytes, once in and once out.
//
// A warp takes one token at a time: four (d = 128) or eight heads in a step,
// sixteen elements a lane, so that the token's angles are computed once for all
// its heads.
#include <type_traits>

#include "fa_norm.cuh"

namespace fa {

template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kNormThreads) fa_norm_kernel(const __grid_constant__ NormArgs p, int parts) {
    __shared__ uint64_t turns[D / 2];
    __shared__ __align__(16) float weights[2 * D];
    const int tid = threadIdx.x;
    norm_tables<T, D>(p, turns, weights, tid, kNormThreads);
    __syncthreads();
    norm_forward<T, D, INTER>(p, turns, weights, blockIdx.x * (kNormThreads / 32) + (tid >> 5),
                              gridDim.x * (kNormThreads / 32), parts, tid & 31);
}

template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kNormThreads) fa_norm_bwd_kernel(const __grid_constant__ NormArgs p, int parts) {
    using L = NormLane<D, INTER>;
    constexpr int WARPS = kNormThreads / 32;
    __shared__ uint64_t turns[D / 2];
    __shared__ __align__(16) float weights[2 * D];
    __shared__ __align__(16) float sums[WARPS][D];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    norm_tables<T, D>(p, turns, weights, tid, kNormThreads);
    if (blockIdx.x == 0 && tid == 0) *p.status = 0;
    __syncthreads();
    const L ln(lane, p.rot);
    uint64_t f[L::OWN];
#pragma unroll
    for (int i = 0; i < L::OWN; ++i) {
        const int at = ln.freq(ln.g * L::OWN + i);
        f[i] = at < p.rot / 2 ? turns[at] : 0ull;
    }
    const long long items = static_cast<long long>(p.tokens) * parts;
    for (int ten = 0; ten < 2; ++ten) {  // q, then k: one set of sums in registers
        const NormRows rx = ten ? p.k : p.q, ru = ten ? p.k_out : p.q_out, rd = ten ? p.dk : p.dq;
        const int H = ten ? p.Hkv : p.Hq, np = (H + L::RPW - 1) / L::RPW;
        const bool has_w = ten ? p.k_weight : p.q_weight;
        float acc[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = 0.f;
        for (long long it = blockIdx.x * WARPS + warp; it < items; it += gridDim.x * WARPS) {
            const int t = static_cast<int>(parts == 1 ? it : div_short(it, parts));
            const int part = static_cast<int>(it - static_cast<long long>(t) * parts);
            int b = 0, n = t, pos;
            if (p.cu_seqlens) {
                const int s = warp_find(p.cu_seqlens, p.B, t, lane);
                if (t < p.cu_seqlens[s] || t >= p.cu_seqlens[s + 1]) continue;
                pos = packed_position(p, s, t);
            } else {
                b = p.by_n.div(t);
                n = pos = t - b * p.N;
                if (p.ends) pos = static_cast<int>(static_cast<uint32_t>(p.ends[b]) - static_cast<uint32_t>(p.N - n));
            }
            const int p0 = np * part / parts, p1 = np * (part + 1) / parts;
            const T* x_at = static_cast<const T*>(rx.data) + b * rx.batch + n * rx.token;
            const T* u_at = static_cast<const T*>(ru.data) + b * ru.batch + n * ru.token;
            T* d_at = static_cast<T*>(rd.data) + b * rd.batch + n * rd.token;
            NormRaw<T> next_u, next_x;
            auto load = [&](int pass) {
                next_u.zero();
                next_x.zero();
                const int h = pass * L::RPW + ln.g;
                if (pass < p1 && h < H) {
                    next_u.load(u_at + h * ru.head, ln.a, ln.b);
                    if (has_w) next_x.load(x_at + h * rx.head, ln.a, ln.b);
                }
            };
            load(p0);
            NormTurn turn;
            warp_turn<D, INTER>(ln, f, pos, turn);
            for (int pass = p0; pass < p1; ++pass) {
                NormRaw<T> raw = next_u;
                float u[16], x[16];
                raw.get(u);
                next_x.get(x);
                load(pass + 1);
                rotate_row<INTER, true>(u, turn);
                if (has_w) {
                    float sc, y[16];
                    const float r = row_rms<D, L::TPR>(x, p.eps, sc);
                    lds_row(y, weights + ten * D, ln.a, ln.b);
                    float dot = 0.f;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        x[i] *= r;
                        acc[i] = fmaf(u[i], x[i], acc[i]);
                        u[i] *= y[i];
                        dot = fmaf(u[i], x[i], dot);
                    }
                    dot = row_sum<L::TPR>(dot) * (1.f / D);
                    const float rs = r * sc;
#pragma unroll
                    for (int i = 0; i < 16; ++i) u[i] = rs * fmaf(-dot, x[i], u[i]);
                }
                raw.set(u);
                const int h = pass * L::RPW + ln.g;
                if (h < H) raw.store(d_at + h * rd.head, ln.a, ln.b);
            }
        }
        if (!has_w) continue;
        // this CTA's sums, in a fixed order
#pragma unroll
        for (int i = 0; i < 16; ++i)
#pragma unroll
            for (int off = L::TPR; off < 32; off <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], off);
        if (ln.g == 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) sums[warp][(i < 8 ? ln.a : ln.b) + (i & 7)] = acc[i];
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
static void launch_fwd(const NormArgs& a, cudaStream_t stream) {
    const int most = 152 * 4, parts = norm_parts(a, most * 8, passes_of(a.Hq, D) + passes_of(a.Hkv, D));
    const long long ctas = (static_cast<long long>(a.tokens) * parts + 7) / 8;
    fa_norm_kernel<T, D, INTER><<<static_cast<unsigned>(ctas < most ? ctas : most), kNormThreads, 0, stream>>>(a, parts);
}

template <typename T, int D, bool INTER>
static int launch_bwd(const NormArgs& a, cudaStream_t stream) {
    const int parts = norm_parts(a, kNormBwdCtas * 8, passes_of(a.Hq, D));
    const long long want = (static_cast<long long>(a.tokens) * parts + 7) / 8;
    const int ctas = static_cast<int>(want < kNormBwdCtas ? want : kNormBwdCtas);
    fa_norm_bwd_kernel<T, D, INTER><<<ctas, kNormThreads, 0, stream>>>(a, parts);
    if (!a.q_weight && !a.k_weight) return 1;
    fa_norm_bwd_sum_kernel<<<2 * D / 32, 1024, 0, stream>>>(a, ctas);
    return 2;
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
    dispatch(a, [&](auto t, auto d, auto inter) {
        launch_fwd<decltype(t), decltype(d)::value, decltype(inter)::value>(a, stream);
    });
    *nlaunch = 1;
    return cudaGetLastError();
}

cudaError_t launch_norm_bwd(const NormArgs& a, cudaStream_t stream, int* nlaunch) {
    dispatch(a, [&](auto t, auto d, auto inter) {
        *nlaunch = launch_bwd<decltype(t), decltype(d)::value, decltype(inter)::value>(a, stream);
    });
    return cudaGetLastError();
}

}  // namespace fa
