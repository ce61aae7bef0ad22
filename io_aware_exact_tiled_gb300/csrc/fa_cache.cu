// The paged 8-bit key/value cache: block plan and quantising append.
#include <math_constants.h>

#include "fa_paged.h"
#include "sm103_ptx.cuh"

namespace fa {

__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

// --------------------------------------------------------------------------
// plan
// --------------------------------------------------------------------------
// Request b has len tokens in had = ceil(len / bs) blocks and brings n more:
// it needs ceil((len + n) / bs) - had blocks. With the inclusive prefix sum
// of the needs, a request is served iff it needs none or its sum is within
// the free count; its blocks are then ring entries head + (exclusive sum) ..,
// so every block id, slot and table entry follows from prefix sums alone, in
// parallel and in the order of the requests.
//
// One cluster: every CTA scans all requests (they are few, and come from L2)
// into its own shared memory, then takes its share of the tokens. The scan is
// the only reader of cache_len and free_state, so after the cluster barrier
// CTA 0 may write their new values, in place if the caller wants that.
struct PlanSum {
    long long tok, need, freed;
};

__device__ __forceinline__ PlanSum plan_add(PlanSum a, PlanSum b) {
    return {a.tok + b.tok, a.need + b.need, a.freed + b.freed};
}

struct PlanItem {
    int n;       // new tokens (0 for a released request)
    int len;     // tokens cached, clamped to the table's capacity
    int had;     // blocks they take
    int need;    // further blocks (0 if the request is released or too long)
    bool drop;   // released
    bool fits;   // the new length is within the block table
    bool bad;    // a length out of range
};

__device__ __forceinline__ PlanItem plan_item(const PlanArgs& p, int b) {
    PlanItem it;
    const int cap = p.max_blocks * p.block_size;  // < 2^31, checked on the host
    const int raw = p.new_len[b], len = p.cache_len[b];
    it.len = min(max(len, 0), cap);
    it.bad = len != it.len;
    it.drop = raw < 0;
    it.n = max(raw, 0);
    it.fits = static_cast<long long>(it.len) + it.n <= cap;
    it.had = (it.len + p.block_size - 1) / p.block_size;
    it.need = 0;
    if (!it.drop && it.fits) it.need = (it.len + it.n + p.block_size - 1) / p.block_size - it.had;
    return it;
}

__global__ void __launch_bounds__(1024) fa_cache_plan_kernel(const __grid_constant__ PlanArgs p) {
    extern __shared__ __align__(16) int psm[];
    int* tok_off = psm;                // [B + 1] first token of each request
    int* blk_off = tok_off + p.B + 1;  // [B] first ring entry of its new (or released) blocks
    int* lens = blk_off + p.B;         // [B] length; -1: refused; <= -2: released, length -2 - lens
    __shared__ PlanSum warp_sum[32];
    __shared__ int granted_s, invalid_s, short_s;
    const int tid = threadIdx.x, nth = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = nth >> 5;
    const uint32_t rank = cluster_rank(), ranks = cluster_size();
    const int cap = p.num_blocks;
    int head = p.free_state[0], count = p.free_state[1];
    const bool state_bad = head < 0 || head >= cap || count < 0 || count > cap;
    head = head < 0 || head >= cap ? 0 : head;
    count = min(max(count, 0), cap);
    if (tid == 0) {
        granted_s = 0;
        invalid_s = state_bad;
        short_s = 0;
        if (rank == 0) *p.status = 0;
    }
    // prefix sums over the requests, `per` consecutive ones for each thread
    const int per = (p.B + nth - 1) / nth;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    PlanSum mine{0, 0, 0};
    for (int b = b0; b < b1; ++b) {
        const PlanItem it = plan_item(p, b);
        mine = plan_add(mine, {it.n, it.need, it.drop ? it.had : 0});
    }
    PlanSum inc = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const PlanSum up{__shfl_up_sync(0xffffffffu, inc.tok, off), __shfl_up_sync(0xffffffffu, inc.need, off),
                         __shfl_up_sync(0xffffffffu, inc.freed, off)};
        if (lane >= off) inc = plan_add(inc, up);
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    PlanSum base{0, 0, 0}, all{0, 0, 0};
    for (int w = 0; w < nw; ++w) {
        if (w < warp) base = plan_add(base, warp_sum[w]);
        all = plan_add(all, warp_sum[w]);
    }
    PlanSum run{base.tok + inc.tok - mine.tok, base.need + inc.need - mine.need, base.freed + inc.freed - mine.freed};
    bool invalid = all.tok > p.total, refused = false;
    int granted = 0;
    for (int b = b0; b < b1; ++b) {
        const PlanItem it = plan_item(p, b);
        const bool room = it.need == 0 || run.need + it.need <= count;
        // tokens past the slot array (the lengths add up to more than total)
        const bool listed = run.tok + it.n <= p.total;
        tok_off[b] = static_cast<int>(min(run.tok, static_cast<long long>(p.total)));
        if (it.drop) {
            blk_off[b] = static_cast<int>(min(run.freed, static_cast<long long>(cap)));
            lens[b] = -2 - it.len;
        } else if (room && it.fits && listed) {
            blk_off[b] = static_cast<int>(run.need);
            lens[b] = it.len;
            if (it.need) granted = static_cast<int>(run.need + it.need);
        } else {
            blk_off[b] = 0;
            lens[b] = -1;
            refused |= !room;
        }
        invalid |= it.bad || !it.fits;
        run = plan_add(run, {it.n, it.need, it.drop ? it.had : 0});
    }
    if (tid == nth - 1) tok_off[p.B] = static_cast<int>(min(all.tok, static_cast<long long>(p.total)));
    if (granted) atomicMax(&granted_s, granted);
    if (invalid) invalid_s = 1;
    if (refused) short_s = 1;
    cluster_sync_all();  // every CTA has read the lengths and the state; the status word is zero
    granted = granted_s;
    const int ntok = tok_off[p.B];
    // tokens: four consecutive ones per thread share one search
    const int stride = static_cast<int>(ranks) * nth * 4;
    for (int t0 = (static_cast<int>(rank) * nth + tid) * 4; t0 < p.total; t0 += stride) {
        int lo = 0, hi = p.B;  // last request that starts at or before t0
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (tok_off[mid] <= t0) lo = mid; else hi = mid;
        }
        int b = lo;
        const int t1 = min(t0 + 4, p.total);
        for (int t = t0; t < t1; ++t) {
            int slot = -1;
            if (t < ntok) {
                while (t >= tok_off[b + 1]) ++b;
                const int len = lens[b];
                if (len >= 0) {
                    const int pos = len + t - tok_off[b], j = pos / p.block_size, r = pos - j * p.block_size;
                    const int had = (len + p.block_size - 1) / p.block_size;
                    int32_t* row = p.block_table + static_cast<size_t>(b) * p.max_blocks;
                    int blk;
                    if (j < had) {
                        blk = row[j];
                    } else {
                        long long at = static_cast<long long>(head) + blk_off[b] + (j - had);
                        at = at >= cap ? at - cap : at;
                        blk = p.free_blocks[at];
                        if (r == 0) row[j] = blk;
                    }
                    if (blk >= 0 && blk < cap) slot = blk * p.block_size + r;
                    else invalid = true;
                }
            }
            p.slots[t] = slot;
        }
    }
    // released blocks go to the back of the ring, a warp for each request;
    // pushes that the ring has no room for (a block returned twice) are dropped
    const int room = cap - count;
    if (all.freed > room) invalid = true;
    for (int b = static_cast<int>(rank) * nw + warp; b < p.B && all.freed; b += static_cast<int>(ranks) * nw) {
        if (lens[b] > -2) continue;
        const int len = -2 - lens[b], had = (len + p.block_size - 1) / p.block_size;
        const int32_t* row = p.block_table + static_cast<size_t>(b) * p.max_blocks;
        for (int j = lane; j < had; j += 32) {
            const int blk = row[j];
            const bool ok = blk >= 0 && blk < cap;
            if (!ok) invalid = true;
            const long long k = static_cast<long long>(blk_off[b]) + j;
            if (k < room) p.free_blocks[(static_cast<long long>(head) + count + k) % cap] = ok ? blk : -1;
        }
    }
    if (rank == 0) {
        for (int b = tid; b < p.B; b += nth) {
            p.cu_seqlens[b] = tok_off[b];
            const int len = lens[b], n = tok_off[b + 1] - tok_off[b];
            // a refused request keeps its length
            if (len != -1) p.cache_len_out[b] = len < 0 ? 0 : len + n;
            else if (p.cache_len_out != p.cache_len) p.cache_len_out[b] = p.cache_len[b];
        }
        if (tid == 0) {
            p.cu_seqlens[p.B] = ntok;
            const int back = static_cast<int>(min(all.freed, static_cast<long long>(room)));
            const long long h2 = static_cast<long long>(head) + granted;
            p.free_state_out[0] = static_cast<int>(h2 >= cap ? h2 - cap : h2);
            p.free_state_out[1] = count - granted + back;
            invalid |= invalid_s != 0;
            if (short_s) atomicCAS(p.status, 0, FA_DEV_NO_BLOCKS);
        }
    }
    // a length or id out of range counts more than a list that ran out
    if (invalid) atomicExch(p.status, FA_DEV_INVALID);
}

cudaError_t launch_cache_plan(const PlanArgs& a, cudaStream_t stream, int* nlaunch) {
    const size_t smem = (static_cast<size_t>(a.B) * 3 + 1) * sizeof(int);
    cudaError_t e = cudaFuncSetAttribute(fa_cache_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (3 * kPlanMaxB + 4) * sizeof(int));
    if (e != cudaSuccess) return e;
    const bool big = a.B > 1024 || a.total > 4096;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = big ? 8 : 1;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(big ? 8 : 1);
    cfg.blockDim = dim3(big ? 1024 : 256);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, fa_cache_plan_kernel, a);
    *nlaunch = 1;
    return e != cudaSuccess ? e : cudaGetLastError();
}

// --------------------------------------------------------------------------
// append
// --------------------------------------------------------------------------
// The new rows of one block and head share a scale 2^e with
// e = max(-126, ceil(log2(amax / 448))) over their finite values, or the
// block's scale so far (rounded up to a power of two) where that is larger;
// rows the block holds already are then moved to the new scale. With powers
// of two x / scale is exact before its one rounding to E4M3, and a move only
// rounds what falls below the smallest normal number.
template <int D>
__global__ void __launch_bounds__(256) fa_cache_append_kernel(const __grid_constant__ AppendArgs p) {
    constexpr int LPR = D / 8;      // lanes per row, eight values (16 bytes) each
    constexpr int RPW = 32 / LPR;   // rows of one warp-wide load
    const int lane = threadIdx.x & 31;
    const long long w = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int t = static_cast<int>(w / (2 * p.H));
    if (t >= p.total) return;
    const int rest = static_cast<int>(w - static_cast<long long>(t) * (2 * p.H));
    const int h = rest >> 1;
    const int bs = p.block_size, nslots = p.num_blocks * bs;
    const int slot = p.slots[t];
    if (slot < 0 || slot >= nslots) return;
    const int blk = slot / bs;
    if (t > 0) {
        const int before = p.slots[t - 1];
        if (before >= 0 && before < nslots && before / bs == blk) return;  // an earlier token's warp takes the block
    }
    // the run: the following tokens whose slots lie in the same block
    int end = t + 1;
    for (;;) {
        const int u = end + lane;
        const int s = u < p.total ? p.slots[u] : -1;
        const uint32_t in = __ballot_sync(0xffffffffu, s >= 0 && s / bs == blk);
        if (in != 0xffffffffu) {
            end += __ffs(~in) - 1;
            break;
        }
        end += 32;
    }
    const uint16_t* src = static_cast<const uint16_t*>(rest & 1 ? p.v : p.k);
    uint8_t* cache = (rest & 1 ? p.v_cache : p.k_cache) + (static_cast<size_t>(blk) * p.H + h) * bs * D;
    float* scale = (rest & 1 ? p.v_scale : p.k_scale) + static_cast<size_t>(blk) * p.H + h;
    const int sub = lane / LPR, col = (lane % LPR) * 8;
    // largest finite magnitude, as bf16 bits (ordered like the values)
    uint32_t top = 0;
    for (int u = t + sub; u < end; u += RPW) {
        const uint4 x = *reinterpret_cast<const uint4*>(src + (static_cast<size_t>(u) * p.H + h) * D + col);
        const uint32_t wds[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = wds[i] & 0x7FFFu, hi = (wds[i] >> 16) & 0x7FFFu;
            top = max(top, lo < 0x7F80u ? lo : 0u);
            top = max(top, hi < 0x7F80u ? hi : 0u);
        }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    // amax / 448 = (1.m / 1.75) 2^(E - 135)
    const int e = max(static_cast<int>(top >> 7) - 135 + ((top & 127u) > 96u ? 1 : 0), -126);
    float s_new = exp2i(e), s_old = 0.f;
    const int first = slot - blk * bs;
    if (first > 0) {
        s_old = *scale;
        s_old = s_old > 0.f && s_old < CUDART_INF_F ? s_old : 0.f;
        const float up = __uint_as_float((__float_as_uint(s_old) + 0x7FFFFFu) & 0x7F800000u);
        if (up < CUDART_INF_F) s_new = fmaxf(s_new, up);
    }
    __syncwarp();
    if (first > 0 && s_new != s_old) {
        const float f = s_old / s_new;
        for (int i = lane * 16; i < first * D; i += 512) {
            uint4* at = reinterpret_cast<uint4*>(cache + i);
            const uint4 x = *at;
            uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float a, b, c, d;
                f2_split(f2_from_e4m3x2(y[k] & 0xFFFFu), a, b);
                f2_split(f2_from_e4m3x2(y[k] >> 16), c, d);
                y[k] = pack_e4m3x2(a * f, b * f) | (pack_e4m3x2(c * f, d * f) << 16);
            }
            *at = make_uint4(y[0], y[1], y[2], y[3]);
        }
    }
    if (lane == 0) *scale = s_new;
    const float inv = 1.f / s_new;  // a power of two: exact
    for (int u = t + sub; u < end; u += RPW) {
        const uint4 x = *reinterpret_cast<const uint4*>(src + (static_cast<size_t>(u) * p.H + h) * D + col);
        const uint32_t wds[4] = {x.x, x.y, x.z, x.w};
        uint32_t y[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t a = wds[2 * i], b = wds[2 * i + 1];
            y[i] = pack_e4m3x2(__uint_as_float(a << 16) * inv, __uint_as_float(a & 0xFFFF0000u) * inv) |
                   (pack_e4m3x2(__uint_as_float(b << 16) * inv, __uint_as_float(b & 0xFFFF0000u) * inv) << 16);
        }
        *reinterpret_cast<uint2*>(cache + static_cast<size_t>(p.slots[u] - blk * bs) * D + col) =
            make_uint2(y[0], y[1]);
    }
}

cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t stream, int* nlaunch) {
    const long long warps = static_cast<long long>(a.total) * a.H * 2;
    const unsigned grid = static_cast<unsigned>((warps + 7) / 8);
    if (a.d == 64)
        fa_cache_append_kernel<64><<<grid, 256, 0, stream>>>(a);
    else
        fa_cache_append_kernel<128><<<grid, 256, 0, stream>>>(a);
    *nlaunch = 1;
    return cudaGetLastError();
}

}  // namespace fa
