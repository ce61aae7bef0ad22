// Attention over the paged 8-bit cache for a batch whose requests share prefixes.
//
// Two passes of the kernels of fa_paged_split.cuh and fa_paged_tile.cu. In the
// first, a group of requests is one request whose new tokens are all of theirs
// and whose keys are the prefix, so that a prefix is read once for all rows that
// share it; it leaves each row's maximum and sum and its output, normalised, in
// fp32. The second is each request over its own tokens, and joins the two. The
// kernels are chained: one starts on the SMs that the one before leaves idle.
#include <math_constants.h>

#include "fa_paged_split.cuh"

namespace fa {

// Pieces of the prefixes' units that the row-tile kernel cut between CTAs. One
// long prefix has few units with a piece in every other CTA, so this takes all
// SMs (where whoever finished last merged, prefixes of 32,768 tokens and 256 rows
// took MERGE_FIG us longer): a CTA has 128 rows and 8 or 16 of their columns.
constexpr int kMergeCtas = 2 * kPagedCtas;

template <int D>
__global__ void __launch_bounds__(256) fa_paged_merge_kernel(const __grid_constant__ PagedArgs a) {
    constexpr int COLS = 2, PARTS = D / 4 / (2 * COLS);  // float4 columns of a thread; CTAs of a row tile
    __shared__ int list[2 * kPagedCtas], n_s;
    const int tid = threadIdx.x, r = tid & 127, G = a.Hq / a.Hkv;
    paged_let_next();
    paged_wait_before();
    if (tid < 32) {  // the units that were cut, in the same order in every CTA
        constexpr int PER = (2 * kPagedCtas + 31) / 32;
        bool is[PER];
        int n = 0;
#pragma unroll
        for (int k = 0; k < PER; ++k)
            is[k] = k * 32 + tid < 2 * kPagedCtas && __ldcg(&a.join.cuts[k * 32 + tid].valid);
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const uint32_t in = __ballot_sync(0xffffffffu, is[k]);
            if (is[k]) list[n + __popc(in & ((1u << tid) - 1u))] = k * 32 + tid;
            n += __popc(in);
        }
        if (tid == 0) n_s = n;
    }
    __syncthreads();
    const int items = n_s * 2 * PARTS;
    for (int it = blockIdx.x; it < items; it += kMergeCtas) {
        const PagedCut& cut = a.join.cuts[list[it / (2 * PARTS)]];
        const int i = it / PARTS & 1, c0 = ((it % PARTS) * 2 + (tid >> 7)) * COLS;
        const int parts = cut.parts, shift = parts >> 1, first = cut.first;  // log2 of parts
        const int row = cut.row0 + (parts > 1 ? 0 : i * 128) + r;
        const int n = (cut.last - first + 1) * parts;  // pieces' parts
        if (row >= cut.rows || (parts > 1 && i) || (parts == 4 && r >= 64)) continue;
        // part k: its half slot, times 128 and with the lane
        auto at = [&](int k) {
            const int slot = 2 * cut.piece(first + (k >> shift));
            return (parts == 1 ? slot + i : slot + (k & 1)) * 128 + (parts == 4 ? 32 * (k & 2) : 0) + r;
        };
        float M = -CUDART_INF_F;
#pragma unroll 8
        for (int k = 0; k < n; ++k) M = fmaxf(M, __ldcg(&a.tile_pm[at(k)]));
        float4 acc[COLS];
#pragma unroll
        for (int y = 0; y < COLS; ++y) acc[y] = make_float4(0.f, 0.f, 0.f, 0.f);
        float L = 0.f;
#pragma unroll 8
        for (int k = 0; k < n; ++k) {
            const int x = at(k);
            const float m = __ldcg(&a.tile_pm[x]), w = m == -CUDART_INF_F ? 0.f : ex2_approx(m - M);
            L = fmaf(w, __ldcg(&a.tile_pl[x]), L);
            const float4* src = reinterpret_cast<const float4*>(a.tile_po) +
                                (static_cast<size_t>(x >> 7) * (D / 4) + c0) * 128 + (x & 127);
#pragma unroll
            for (int y = 0; y < COLS; ++y) {
                const float4 v = __ldcg(src + y * 128);
                acc[y].x = fmaf(w, v.x, acc[y].x);
                acc[y].y = fmaf(w, v.y, acc[y].y);
                acc[y].z = fmaf(w, v.z, acc[y].z);
                acc[y].w = fmaf(w, v.w, acc[y].w);
            }
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;
        const int tok = row / G;
        const size_t orow = static_cast<size_t>(cut.tok0 + tok) * a.Hq + cut.hk * G + row - tok * G;
        if (c0 == 0) a.join.ml[orow] = make_float2(M, L);
#pragma unroll
        for (int k = 0; k < COLS; ++k)
            reinterpret_cast<float4*>(a.join.o + orow * D)[c0 + k] =
                make_float4(acc[k].x * inv, acc[k].y * inv, acc[k].z * inv, acc[k].w * inv);
    }
}

cudaError_t launch_fwd_paged_prefix(const PagedArgs& prefix, const PagedArgs& own, cudaStream_t stream, int* nlaunch) {
    *nlaunch = 0;
    cudaError_t e = cudaSuccess;
    if (own.ev_begin) cudaEventRecord(own.ev_begin, stream);
    for (PagedArgs a : {prefix, own}) {
        const bool tiles = paged_has_tiles(a.max_new, a.Hq / a.Hkv, a.d);
        if (e == cudaSuccess && a.split_rows > 0) {
            a.chained = *nlaunch > 0;
            e = launch_split<true>(a, stream);
            ++*nlaunch;
        }
        if (e == cudaSuccess && tiles) {
            a.chained = *nlaunch > 0;
            e = launch_paged_tile(a, stream);
            ++*nlaunch;
        }
        if (e == cudaSuccess && tiles && a.join.first) {
            cudaLaunchAttribute at;
            cudaLaunchConfig_t cfg = paged_config(256, 0, stream, true, &at);
            cfg.gridDim = dim3(kMergeCtas);
            e = a.d == 64 ? cudaLaunchKernelEx(&cfg, fa_paged_merge_kernel<64>, a)
                          : cudaLaunchKernelEx(&cfg, fa_paged_merge_kernel<128>, a);
            ++*nlaunch;
        }
    }
    if (own.ev_end) cudaEventRecord(own.ev_end, stream);
    return e;
}

}  // namespace fa
