// Attention over the paged 8-bit cache for a batch whose requests share prefixes.
//
// Two passes of the kernels of fa_paged_split.cuh and fa_paged_tile.cu. In one, a
// group of requests is one request whose new tokens are all of theirs and whose
// keys are the prefix, so that a prefix is read once for all rows that share it;
// it leaves each row's maximum and sum and its output, normalised, in fp32. The
// other is each request over its own tokens. Softmax over both sets of keys is
// then their sum with weights from maxima and sums (paged_weights).
//
// The kernels are chained: one starts on the SMs that the one before leaves idle.
// Where the prefixes are the row-tile kernel's and the own tokens the split-key
// kernel's (decoding), both work at once on parts of the GPU that the lengths set
// (paged_share), and a merge joins them. Elsewhere the prefixes' pass comes
// first and the other one joins what it left as it writes its rows.
//
// Bound: the cache's bytes, each prefix once; with many rows the products, in fact
// the softmax. Measured (d = 128, 32 + 8 heads): 64 requests behind 32,768 tokens
// with 2,066 of their own on average 122 us (339 MB: 50); 16 behind 262,001 173 us
// (544 MB: 80; the softmax warps, below); 4 of 30 tokens behind 1,000 27 us, a chain
// of latencies: scan 5, first chunk 4, merge of the warps 3, own pass and joining
// 8. Eight prompts of 9,322 tokens together behind 8,192, 16 heads: 558 us at d =
// 64 (175), 714 at d = 128 (350).
#include <math_constants.h>

#include "fa_paged_split.cuh"

namespace fa {

// Pieces of the prefixes' units that the row-tile kernel cut between CTAs. One
// long prefix has few units with a piece in every other CTA, so this takes all
// SMs: a CTA has 128 rows (a lane of the row tile for a thread) and 8 of their
// columns, in four groups that take every fourth piece each. (256 rows behind
// 32,768 tokens: 6 us; merged by whoever finished last 27, by two groups of
// columns that take all pieces 16.)
constexpr int kMergeCtas = 2 * kPagedCtas, kMergeGroups = 4, kMergeThreads = 128 * kMergeGroups;

template <int D>
__global__ void __launch_bounds__(kMergeThreads)
    fa_paged_merge_kernel(const __grid_constant__ PagedArgs a, const __grid_constant__ PagedJoin own) {
    constexpr int COLS = 2, CUTS = D / 4 / COLS;  // float4 columns of a thread; CTAs of a row tile
    __shared__ int list[2 * kPagedCtas], n_s;
    __shared__ float2 ml_s[kMergeGroups][128];
    __shared__ float4 o_s[kMergeGroups][COLS][128];
    const int tid = threadIdx.x, r = tid & 127, g = tid >> 7, G = a.Hq / a.Hkv;
    paged_let_next();
    paged_wait_before();
    if (tid < 32) {  // the units that were cut, in the same order in every CTA
        constexpr int PER = (2 * kPagedCtas + 31) / 32;
        uint32_t is = 0;
        int n = 0;
#pragma unroll
        for (int k = 0; k < PER; ++k)
            if (k * 32 + tid < 2 * kPagedCtas && __ldcg(&a.join.cuts[k * 32 + tid].valid)) is |= 1u << k;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const uint32_t in = __ballot_sync(0xffffffffu, is >> k & 1u);
            if (is >> k & 1u) list[n + __popc(in & ((1u << tid) - 1u))] = k * 32 + tid;
            n += __popc(in);
        }
        if (tid == 0) n_s = n;
    }
    __syncthreads();
    // Four columns of a row's output, and L, from the prefix's maximum, sum and
    // output and what the other pass left; a row of no request has none.
    auto finish = [&](size_t row, int tok, int hq, float2 ml, int c, float4 x) {
        const float2 b = __ldcg(&own.ml[row]);
        if (!(__float_as_uint(b.y) >> 31)) return;
        const PagedWeights w = paged_weights(b.x, -b.y, ml);
        const float4 y = __ldcg(reinterpret_cast<const float4*>(own.o + row * D) + c);
        const float u = w.own * -b.y, v = w.prefix;
        auto mix = [&](float p, float q) { return fmaf(u, q, v * p); };
        reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + row * D)[c] =
            make_uint2(pack_bf16x2(mix(x.x, y.x), mix(x.y, y.y)), pack_bf16x2(mix(x.z, y.z), mix(x.w, y.w)));
        if (c == 0) a.lse[static_cast<size_t>(hq) * a.total + tok] = w.lse;
    };
    const int items = n_s * 2 * CUTS;
    for (int it = blockIdx.x; it < items; it += kMergeCtas) {
        const PagedCut& cut = a.join.cuts[list[it / (2 * CUTS)]];
        const int i = it / CUTS & 1, c0 = it % CUTS * COLS, parts = cut.parts, first = cut.first;
        if (parts > 1 && i) continue;  // both row tiles at once
        const int per = parts > 1 ? 2 : 1, n = (cut.last - first + 1) * per;  // parts of this lane in a piece; of all
        auto at = [&](int k) {  // half slot
            return 2 * cut.piece(per > 1 ? first + (k >> 1) : first + k) + (per > 1 ? k & 1 : i);
        };
        float M = -CUDART_INF_F, L = 0.f;
#pragma unroll 8
        for (int k = g; k < n; k += kMergeGroups) M = fmaxf(M, __ldcg(&a.tile_pm[at(k) * 128 + r]));
        float4 acc[COLS];
#pragma unroll
        for (int y = 0; y < COLS; ++y) acc[y] = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](float w, const float4& v, float4& x) {
            x.x = fmaf(w, v.x, x.x);
            x.y = fmaf(w, v.y, x.y);
            x.z = fmaf(w, v.z, x.z);
            x.w = fmaf(w, v.w, x.w);
        };
#pragma unroll 8
        for (int k = g; k < n; k += kMergeGroups) {
            const int x = at(k);
            const float m = __ldcg(&a.tile_pm[x * 128 + r]), w = m == -CUDART_INF_F ? 0.f : ex2_approx(m - M);
            L = fmaf(w, __ldcg(&a.tile_pl[x * 128 + r]), L);
            const float4* src = reinterpret_cast<const float4*>(a.tile_po) +
                                (static_cast<size_t>(x) * (D / 4) + c0) * 128 + r;
#pragma unroll
            for (int y = 0; y < COLS; ++y) add(w, __ldcg(src + y * 128), acc[y]);
        }
        ml_s[g][r] = make_float2(M, L);
#pragma unroll
        for (int y = 0; y < COLS; ++y) o_s[g][y][r] = acc[y];
        __syncthreads();
        // the groups' parts, of both lanes of a row where it has two
        const int row = cut.row0 + (parts > 1 ? 0 : i * 128) + r, lanes = parts == 4 ? 2 : 1;
        if (g < COLS && row < cut.rows && (lanes == 1 || r < 64)) {
            M = -CUDART_INF_F;
            L = 0.f;
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = 0; k < kMergeGroups * lanes; ++k) M = fmaxf(M, ml_s[k & 3][(k >> 2) * 64 + r].x);
            for (int k = 0; k < kMergeGroups * lanes; ++k) {
                const float2 b = ml_s[k & 3][(k >> 2) * 64 + r];
                const float w = b.x == -CUDART_INF_F ? 0.f : ex2_approx(b.x - M);
                L = fmaf(w, b.y, L);
                add(w, o_s[k & 3][g][(k >> 2) * 64 + r], sum);
            }
            const float inv = L == 0.f ? 0.f : 1.f / L;
            const int tok = row / G;
            const size_t orow = static_cast<size_t>(cut.tok0 + tok) * a.Hq + cut.hk * G + row - tok * G;
            sum = make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv);
            if (own.ml) {
                finish(orow, cut.tok0 + tok, cut.hk * G + row - tok * G, make_float2(M, L), c0 + g, sum);
            } else {
                if (c0 + g == 0) a.join.ml[orow] = paged_leave(M, L);
                reinterpret_cast<float4*>(a.join.o + orow * D)[c0 + g] = sum;
            }
        }
        __syncthreads();
    }
    if (!own.ml) return;
    // rows of units that were not cut: D / 4 threads a row
    const int rows = a.total * a.Hq;
    for (int row = blockIdx.x * (kMergeThreads / (D / 4)) + tid / (D / 4); row < rows;
         row += kMergeCtas * (kMergeThreads / (D / 4))) {
        const float2 b = __ldcg(&a.join.ml[row]);
        if (!(__float_as_uint(b.y) >> 31)) continue;
        const int tok = row / a.Hq, c = tid % (D / 4);
        finish(row, tok, row - tok * a.Hq, make_float2(b.x, -b.y), c,
               __ldcg(reinterpret_cast<const float4*>(a.join.o + static_cast<size_t>(row) * D) + c));
    }
}

static cudaError_t launch_merge(const PagedArgs& prefix, const PagedJoin& own, cudaStream_t stream) {
    cudaLaunchAttribute at;
    cudaLaunchConfig_t cfg = paged_config(kMergeThreads, 0, stream, true, &at);
    cfg.gridDim = dim3(kMergeCtas);
    return prefix.d == 64 ? cudaLaunchKernelEx(&cfg, fa_paged_merge_kernel<64>, prefix, own)
                          : cudaLaunchKernelEx(&cfg, fa_paged_merge_kernel<128>, prefix, own);
}

cudaError_t launch_fwd_paged_prefix(const PagedArgs& prefix, const PagedArgs& own, cudaStream_t stream, int* nlaunch) {
    const int group = own.Hq / own.Hkv;
    const bool pre_tiles = paged_has_tiles(prefix.max_new, group, prefix.d);
    const bool own_tiles = paged_has_tiles(own.max_new, group, own.d);
    *nlaunch = 0;
    cudaError_t e = cudaSuccess;
    auto run = [&](const PagedArgs& a, cudaError_t (*launch)(const PagedArgs&, cudaStream_t)) {
        if (e != cudaSuccess) return;
        PagedArgs x = a;
        x.chained = *nlaunch > 0;
        e = launch(x, stream);
        ++*nlaunch;
    };
    if (own.ev_begin) cudaEventRecord(own.ev_begin, stream);
    run(prefix, pre_tiles ? launch_paged_tile : launch_split<true>);
    if (own.join.leaves) {  // both at once, then the merge
        run(own, launch_split<true>);
        if (e == cudaSuccess) e = launch_merge(prefix, own.join, stream);
        ++*nlaunch;
    } else {
        if (pre_tiles && prefix.join.cuts) {
            if (e == cudaSuccess) e = launch_merge(prefix, PagedJoin{}, stream);
            ++*nlaunch;
        }
        if (own_tiles) run(own, launch_paged_tile);  // first: the longer of the two
        run(own, launch_split<true>);
    }
    if (own.ev_end) cudaEventRecord(own.ev_end, stream);
    return e;
}

}  // namespace fa
