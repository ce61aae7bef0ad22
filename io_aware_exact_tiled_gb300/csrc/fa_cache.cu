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
// Bound: latency. 16 requests of a token each take 4.6 us (a launch alone 2),
// 4,096 requests with 117K tokens, a tenth of them released, 17 us: the scan 4,
// the tokens 6, released blocks 3.
constexpr int kPlanKeep = 4;
constexpr int kPlanMaxSmem = (3 * kPlanMaxB + 4) * sizeof(int);

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
    int need;    // further blocks (0 if the request is released or does not fit)
    bool drop;   // released
    bool fits;   // both lengths are within the block table
};

__device__ __forceinline__ int plan_blocks(const PlanArgs& p, int len) {  // len < 2^31 - 256
    return (len + (1 << p.bs_log2) - 1) >> p.bs_log2;
}

__device__ __forceinline__ PlanItem plan_item(const PlanArgs& p, int raw, int len) {
    PlanItem it;
    const int cap = p.max_blocks << p.bs_log2;  // < 2^31, checked on the host
    it.len = min(max(len, 0), cap);
    it.n = max(raw, 0);
    it.fits = len == it.len && static_cast<long long>(it.len) + it.n <= cap;
    it.drop = raw < 0 && it.fits;  // of a length out of range nobody knows which blocks are the request's
    it.had = plan_blocks(p, it.len);
    it.need = 0;
    if (!it.drop && it.fits) it.need = plan_blocks(p, it.len + it.n) - it.had;
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
    // the first few of them stay in registers, their loads in flight together
    int raw[kPlanKeep], len0[kPlanKeep];
#pragma unroll
    for (int k = 0; k < kPlanKeep; ++k) {
        raw[k] = b0 + k < b1 ? p.new_len[b0 + k] : 0;
        len0[k] = b0 + k < b1 ? p.cache_len[b0 + k] : 0;
    }
    auto each = [&](auto&& f) {
#pragma unroll
        for (int k = 0; k < kPlanKeep; ++k)
            if (b0 + k < b1) f(b0 + k, plan_item(p, raw[k], len0[k]));
        for (int b = b0 + kPlanKeep; b < b1; ++b) f(b, plan_item(p, p.new_len[b], p.cache_len[b]));
    };
    PlanSum mine{0, 0, 0};
    each([&](int, const PlanItem& it) { mine = plan_add(mine, {it.n, it.need, it.drop ? it.had : 0}); });
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
    each([&](int b, const PlanItem& it) {
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
        invalid |= !it.fits;
        run = plan_add(run, {it.n, it.need, it.drop ? it.had : 0});
    });
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
        int b = lo, blk = -1, blk_b = -1, blk_j = 0;  // the block looked up last
        const int t1 = min(t0 + 4, p.total);
        for (int t = t0; t < t1; ++t) {
            int slot = -1;
            if (t < ntok) {
                while (t >= tok_off[b + 1]) ++b;
                const int len = lens[b];
                if (len >= 0) {
                    const int pos = len + t - tok_off[b], j = pos >> p.bs_log2, r = pos & ((1 << p.bs_log2) - 1);
                    if (b != blk_b || j != blk_j) {
                        const int had = plan_blocks(p, len);
                        int32_t* row = p.block_table + static_cast<size_t>(b) * p.max_blocks;
                        blk_b = b;
                        blk_j = j;
                        if (j < had) {
                            blk = row[j];
                        } else {
                            long long at = static_cast<long long>(head) + blk_off[b] + (j - had);
                            at = at >= cap ? at - cap : at;
                            blk = p.free_blocks[at];
                            if (r == 0) row[j] = blk;  // the thread that has the block's first token
                        }
                    }
                    if (blk >= 0 && blk < cap) slot = (blk << p.bs_log2) + r;
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
        const int len = -2 - lens[b], had = plan_blocks(p, len);
        const int32_t* row = p.block_table + static_cast<size_t>(b) * p.max_blocks;
        for (int j = lane; j < had; j += 32) {
            const int blk = row[j];
            const bool ok = blk >= 0 && blk < cap;
            if (!ok) invalid = true;
            const long long k = static_cast<long long>(blk_off[b]) + j;
            long long at = static_cast<long long>(head) + count + k;
            at = at >= cap ? at - cap : at;
            if (k < room) p.free_blocks[at] = ok ? blk : -1;
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

// The largest cluster that a plan asks for (a debug build sets it lower, so that
// a test runs a smaller one).
#ifndef FA_PLAN_MAX_CLUSTER
#define FA_PLAN_MAX_CLUSTER 16
#endif

static cudaLaunchConfig_t plan_config(cudaLaunchAttribute* at, int ctas, int threads, size_t smem) {
    at->id = cudaLaunchAttributeClusterDimension;
    at->val.clusterDim.x = ctas;
    at->val.clusterDim.y = at->val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cfg;
}

// CTAs of the largest cluster that fits the current device with the most shared
// memory a plan takes (a part of a GPU may have no sixteen SMs together; one CTA
// always fits). Asked once for each device.
static cudaError_t plan_cluster(int* ctas) {
    static std::atomic<int> known[64];  // 0: not asked yet
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int n = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        for (n = FA_PLAN_MAX_CLUSTER; n > 1; n /= 2) {
            cudaLaunchAttribute at;
            const cudaLaunchConfig_t cfg = plan_config(&at, n, 1024, kPlanMaxSmem);
            int fit = 0;
            if (cudaOccupancyMaxActiveClusters(&fit, fa_cache_plan_kernel, &cfg) == cudaSuccess && fit > 0) break;
            cudaGetLastError();  // a size that the device does not know is one that does not fit
        }
        if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    }
    *ctas = n;
    return cudaSuccess;
}

cudaError_t launch_cache_plan(const PlanArgs& a, cudaStream_t stream, int* nlaunch) {
    const size_t smem = (static_cast<size_t>(a.B) * 3 + 1) * sizeof(int);
    static std::atomic<uint64_t> done{0};
    cudaError_t e = once_per_device(done, [] {
        cudaError_t r =
            cudaFuncSetAttribute(fa_cache_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPlanMaxSmem);
        if (r == cudaSuccess)
            r = cudaFuncSetAttribute(fa_cache_plan_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        return r;
    });
    if (e != cudaSuccess) return e;
    // One CTA where latency is all there is (16 requests of a token each: 4.6 us),
    // a cluster of 16 where there are many requests or tokens (4096 requests,
    // 117K tokens: 22 us with eight CTAs, 17 with sixteen).
    const bool big = a.B > 1024 || a.total > 4096;
    int ctas = 1;
    if (big && (e = plan_cluster(&ctas)) != cudaSuccess) return e;
    cudaLaunchAttribute at;
    cudaLaunchConfig_t cfg = plan_config(&at, ctas, big ? 1024 : 256, smem);
    cfg.stream = stream;
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
//
// A CTA takes the runs (consecutive tokens whose slots lie in one block) that
// start among its `span` tokens, for one head and one of K and V. One or two
// runs, as in a prompt, are each the whole CTA's: a thread holds 16 bytes of L
// rows, so the data are read once and the scale found on the way. More runs, as
// in a decoding batch, go to a warp each, which reads its rows twice (they stay
// in the L1 cache).
struct AppendRun {
    const uint16_t* src;  // this head's first row: token t is src + t * H * D
    uint8_t* cache;       // the block's rows of this head
    float* scale;
    size_t stride;        // H * D
};

// Largest finite magnitude of N x eight bf16 values, as bf16 bits (ordered like
// the values): of both halves of the words at once, again without the infinities
// and NaN if there were any.
template <int N>
__device__ __forceinline__ uint32_t append_amax(const uint4 (&x)[N], uint32_t top) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
        m = __vmaxu2(m, __vmaxu2(__vmaxu2(x[i].x & 0x7FFF7FFFu, x[i].y & 0x7FFF7FFFu),
                                 __vmaxu2(x[i].z & 0x7FFF7FFFu, x[i].w & 0x7FFF7FFFu)));
    uint32_t t = max(m & 0xFFFFu, m >> 16);
    if (t >= 0x7F80u) {
        t = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t lo = w[k] & 0x7FFFu, hi = (w[k] >> 16) & 0x7FFFu;
                t = max(t, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
            }
        }
    }
    return max(top, t);
}
__device__ __forceinline__ uint2 append_quantise(uint4 x, float inv) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t y[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t a = w[2 * i], b = w[2 * i + 1];
        y[i] = pack_e4m3x2(__uint_as_float(a << 16) * inv, __uint_as_float(a & 0xFFFF0000u) * inv) |
               (pack_e4m3x2(__uint_as_float(b << 16) * inv, __uint_as_float(b & 0xFFFF0000u) * inv) << 16);
    }
    return make_uint2(y[0], y[1]);
}
// The scale of a run whose largest magnitude is `top`, given the block's scale
// so far (0: none).
__device__ __forceinline__ float append_scale(uint32_t top, float old) {
    // amax / 448 = (1.m / 1.75) 2^(E - 135)
    const int e = max(static_cast<int>(top >> 7) - 135 + ((top & 127u) > 96u ? 1 : 0), -126);
    const float s = exp2i(e), up = __uint_as_float((__float_as_uint(old) + 0x7FFFFFu) & 0x7F800000u);
    return up < CUDART_INF_F ? fmaxf(s, up) : s;
}
__device__ __forceinline__ float append_old_scale(const float* scale) {
    const float s = *scale;
    return s > 0.f && s < CUDART_INF_F ? s : 0.f;
}
// Rows in front of the run to a new scale: factor f, 16 bytes a step.
__device__ __forceinline__ void append_move(uint8_t* cache, int bytes, float f, int i, int step) {
    for (i *= 16; i < bytes; i += step * 16) {
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

// As many CTAs of an SM as their rows in registers allow with few spills (d =
// 128, prompts of 20,000 tokens, blocks of 64 / 128 / 256: 97 / 94 / 134 us with
// five, four and two, 83 / 89 / 116 with eight, five and three).
template <int D, int L>
__global__ void __launch_bounds__(256, L <= 4 ? 8 : L == 8 ? 5 : 3)
    fa_cache_append_kernel(const __grid_constant__ AppendArgs p, int span) {
    constexpr int LPR = D / 8;         // lanes per row, eight values (16 bytes) each
    constexpr int ROWS = 256 / LPR;    // rows of a CTA-wide load
    __shared__ int slot_of[512];       // slot of tokens t0 .. (-1: none)
    __shared__ int leads[256], nlead;
    __shared__ uint32_t warp_top[8];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // the heads of a span follow one another: they share its rows' DRAM pages
    const int part = static_cast<int>(blockIdx.x / (2u * p.H)), hv = static_cast<int>(blockIdx.x - part * (2u * p.H));
    const int h = hv >> 1, bs = p.block_size, nslots = p.num_blocks * bs, bs_log2 = 31 - __clz(bs);
    const bool is_v = hv & 1;
    const long long t0 = static_cast<long long>(part) * span;
    auto slot_at = [&](long long t) {
        if (t < 0 || t >= p.total) return -1;
        const int s = p.slots[t];
        return s >= 0 && s < nslots ? s : -1;
    };
    auto blk_of = [&](int i) { return slot_of[i] >> bs_log2; };
    // slots of the span's tokens and of those that its last run may reach
    for (int i = tid; i < span + bs; i += 256) slot_of[i] = slot_at(t0 + i);
    if (tid == 0) nlead = 0;
    __syncthreads();
    if (tid < span && slot_of[tid] >= 0 && blk_of(tid) != (tid ? blk_of(tid - 1) : slot_at(t0 - 1) >> bs_log2))
        leads[atomicAdd(&nlead, 1)] = tid;
    __syncthreads();
    const int n = nlead;
    if (n == 0) return;
    AppendRun r;
    r.src = static_cast<const uint16_t*>(is_v ? p.v : p.k) + static_cast<size_t>(h) * D;
    r.stride = static_cast<size_t>(p.H) * D;
    auto open = [&](int lead) {  // returns the run's first row in its block
        const size_t at = static_cast<size_t>(blk_of(lead)) * p.H + h;
        r.cache = (is_v ? p.v_cache : p.k_cache) + at * bs * D;
        r.scale = (is_v ? p.v_scale : p.k_scale) + at;
        return slot_of[lead] & (bs - 1);
    };
    auto run_end = [&](int lead) {  // first token behind the run, as far as slot_of reaches (block_size tokens)
        const int blk = blk_of(lead);
        for (int e = lead + 1;; e += 32) {
            const int i = e + lane;
            const uint32_t in = __ballot_sync(0xffffffffu, i < min(lead + bs, span + bs) && blk_of(i) == blk);
            if (in != 0xffffffffu) return e + __ffs(~in) - 1;
        }
    };
    if (n <= 2) {
        // ------------------------------------------------ the CTA takes the runs in turn
        const int row = tid / LPR, col = (tid % LPR) * 8;
        for (int k = 0; k < n; ++k) {
            const int lead = leads[k], end = run_end(lead), first = open(lead);
            uint4 x[L];
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const int t = lead + i * ROWS + row;
                x[i] = make_uint4(0u, 0u, 0u, 0u);
                if (t < end) x[i] = *reinterpret_cast<const uint4*>(r.src + (t0 + t) * r.stride + col);
            }
            const float old = first > 0 ? append_old_scale(r.scale) : 0.f;
            top = append_amax(x, top);
            top = __reduce_max_sync(0xffffffffu, top);
            if (lane == 0) warp_top[warp] = top;
            __syncthreads();  // every thread has read the scale so far, too
#pragma unroll
            for (int w = 0; w < 8; ++w) top = max(top, warp_top[w]);
            const float s = append_scale(top, old), inv = 1.f / s;  // a power of two: exact
            if (first > 0 && s != old) append_move(r.cache, first * D, old / s, tid, 256);
            if (tid == 0) *r.scale = s;
            // the run's own rows, after the moved ones of a slot that it writes again
            __syncthreads();
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const int t = lead + i * ROWS + row;
                if (t < end)
                    *reinterpret_cast<uint2*>(r.cache + (slot_of[t] & (bs - 1)) * D + col) = append_quantise(x[i], inv);
            }
        }
        return;
    }
    // ---------------------------------------------------- a warp for each run
    constexpr int RPW = 32 / LPR;
    const int sub = lane / LPR, col = (lane % LPR) * 8;
    for (int k = warp; k < n; k += 8) {
        const int lead = leads[k], end = run_end(lead), first = open(lead);
        const float old = first > 0 ? append_old_scale(r.scale) : 0.f;
        uint32_t top = 0;
        for (int t = lead + sub; t < end; t += RPW) {
            const uint4 x[1] = {*reinterpret_cast<const uint4*>(r.src + (t0 + t) * r.stride + col)};
            top = append_amax(x, top);
        }
        top = __reduce_max_sync(0xffffffffu, top);
        const float s = append_scale(top, old), inv = 1.f / s;
        if (first > 0 && s != old) append_move(r.cache, first * D, old / s, lane, 32);
        __syncwarp();
        if (lane == 0) *r.scale = s;
        for (int t = lead + sub; t < end; t += RPW) {
            const uint4 x = *reinterpret_cast<const uint4*>(r.src + (t0 + t) * r.stride + col);
            *reinterpret_cast<uint2*>(r.cache + (slot_of[t] & (bs - 1)) * D + col) = append_quantise(x, inv);
        }
    }
}

template <int D, int L>
static void launch_append(const AppendArgs& a, cudaStream_t stream) {
    // Tokens of a CTA: sixteen in a small batch, so that the many runs of a
    // decoding batch spread over the GPU (128 requests of a token 3.9 us; prompts
    // of 19,900 tokens 203 us with sixteen, 116 with 64, before other changes), 64
    // in a large one (64 in blocks of 16, 20,000 tokens of prompts, d = 128: 118
    // us, 184 with one block), 128 where blocks are so small that each warp should
    // have one (the same prompts: 104 us, d = 64 60 and 74; 2,048 requests of a
    // token, d = 128: 16 us, 11 with 64).
    const int span = a.total > 8192 && a.block_size * D <= 2048 ? 128 : a.total > 1024 ? 64 : 16;
    const unsigned grid = static_cast<unsigned>((a.total + span - 1) / span) * 2u * a.H;
    fa_cache_append_kernel<D, L><<<grid, 256, 0, stream>>>(a, span);
}

cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t stream, int* nlaunch) {
    const int rows = a.d == 64 ? 32 : 16, l = (a.block_size + rows - 1) / rows;
    if (a.d == 64) {
        if (l == 1) launch_append<64, 1>(a, stream);
        else if (l == 2) launch_append<64, 2>(a, stream);
        else if (l == 4) launch_append<64, 4>(a, stream);
        else launch_append<64, 8>(a, stream);
    } else {
        if (l == 1) launch_append<128, 1>(a, stream);
        else if (l == 2) launch_append<128, 2>(a, stream);
        else if (l == 4) launch_append<128, 4>(a, stream);
        else if (l == 8) launch_append<128, 8>(a, stream);
        else launch_append<128, 16>(a, stream);
    }
    *nlaunch = 1;
    return cudaGetLastError();
}

}  // namespace fa
