// Internal interface of the paged 8-bit key/value cache: the block plan and
// the quantising append (fa_cache.cu) and attention over the cache
// (fa_paged.cu).
#pragma once

#include <atomic>

#include <cuda_runtime.h>
#include <stdint.h>

namespace fa {

// Status code a kernel leaves when the free list ran out (FA_ERR_NO_BLOCKS).
enum : int { FA_DEV_NO_BLOCKS = 5 };

constexpr int kPlanMaxB = 16384;      // requests of one plan (offsets of all of them sit in shared memory)
constexpr int kPagedCtas = 152;       // one persistent CTA per SM
constexpr int kPagedMaxRows = 32;     // tallest row tile of the split-key kernel
constexpr int kPagedTileRows = 256;   // query rows of a unit of the row-tile kernel

struct PlanArgs {
    const int32_t *new_len, *cache_len;
    int32_t* cache_len_out;
    int32_t* block_table;  // [B][max_blocks]
    int32_t* free_blocks;  // ring [num_blocks]
    const int32_t* free_state;  // {head, count}
    int32_t* free_state_out;
    int32_t* cu_seqlens;  // [B + 1]
    int32_t* slots;       // [total]
    int B, max_blocks, num_blocks, bs_log2, total;
    int* status;
};

struct AppendArgs {
    const void *k, *v;  // [total][H][d] bf16
    uint8_t *k_cache, *v_cache;  // [num_blocks][H][block_size][d] E4M3
    float *k_scale, *v_scale;    // [num_blocks][H]
    const int32_t* slots;        // [total]
    int total, H, d, num_blocks, block_size;
};

struct PagedArgs {
    const void* q;  // [total][Hq][d] bf16
    const uint8_t *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    void* o;     // [total][Hq][d] bf16
    float* lse;  // [Hq][total]
    const int32_t *cu_seqlens, *cache_len, *block_table;
    int B, Hq, Hkv, total, max_new, max_blocks, num_blocks, block_size, d;
    float scale;
    int causal;
    // workspace; the counters are zero at the start
    int* status;
    int* counters;       // [B * Hkv] finished pieces of the split-key kernel's units
    float *pm, *pl;      // [2 * kPagedCtas][kPagedMaxRows]
    float* po;           // [2 * kPagedCtas][kPagedMaxRows][d]
    int* tile_counters;  // [2 * max_tile_units], of the row-tile kernel's row tiles
    int max_tile_units;
    float *tile_pm, *tile_pl;  // [2 * kPagedCtas][kPagedTileRows]
    float* tile_po;            // [2 * kPagedCtas][kPagedTileRows][d]
    cudaEvent_t ev_begin, ev_end;  // optional, recorded around the attention kernels
};

// Query rows (new tokens x heads of a group) up to which a request can be the
// split-key kernel's. Above 24 rows of d = 128 its registers do not hold O (64
// requests of 8,000 tokens, 32 rows: 479 us there, 332 to 342 in the
// row-tile kernel); at d = 64 they do (232 us and 290).
inline int paged_max_rows(int d) { return d == 64 ? 32 : 24; }
// Whether a request of max_new new tokens goes to the row-tile kernel.
inline bool paged_has_tiles(int max_new, int group, int d) {
    return static_cast<long long>(max_new) * group > paged_max_rows(d);
}
// Rows up to which a request of this call is the split-key kernel's, the height
// of its tile: what the longest request has, or, where that one is the row-tile
// kernel's, what one new token has, as the host knows no more. A batch with a
// prompt in it is mostly decoding otherwise, and a taller tile than their rows
// need slows those requests down (a prompt of 2,000 tokens beside 63 requests of
// 8,000 tokens, one new token each, 4 rows: 170 us in a tile of eight rows, 274
// in one of 32 at d = 64; 254 and 334 at d = 128). Requests of a few tokens
// beside a prompt pay for it (three each, 12 rows: 351 us in the row-tile kernel,
// 276 in a tile of 32; 437 and 341): they are better off in a call of their own.
inline int paged_split_rows(int max_new, int group, int d) {
    const int rows = paged_has_tiles(max_new, group, d) ? group : max_new * group;
    return ((rows < paged_max_rows(d) ? rows : paged_max_rows(d)) + 7) / 8 * 8;
}
// Units of the row-tile kernel that B requests of together `total` tokens can
// have (none if no request can be that long).
inline long long paged_max_tile_units(int B, int Hq, int Hkv, int total, int max_new, int d) {
    const long long group = Hq / Hkv;
    if (!paged_has_tiles(max_new, static_cast<int>(group), d)) return 0;
    return Hkv * (B + total * group / kPagedTileRows);
}

// Runs `set` (function attributes) once for each device; `done` remembers
// which, for up to 64 devices.
template <typename F>
inline cudaError_t once_per_device(std::atomic<uint64_t>& done, F&& set) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = set();
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

#ifdef __CUDACC__
// x / d for 0 <= x, 0 < d: in 32 bits where x has no more.
__device__ __forceinline__ long long div_short(long long x, long long d) {
    if (((x | d) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(d);
    return x / d;
}
// Two E4M3 numbers (low 16 bits) to an f16 pair, exactly.
__device__ __forceinline__ uint32_t f16x2_from_e4m3x2(uint32_t x) {
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
#endif

// Division of 0 <= x < 2^31 by a divisor that the host knows: with
// l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1 the quotient is
// (umulhi(m, x) + x) >> l (Granlund and Montgomery, PLDI 1994).
struct FastDiv {
    uint32_t d, m, l;
#ifdef __CUDACC__
    __device__ __forceinline__ int div(int x) const {
        return static_cast<int>((__umulhi(m, static_cast<uint32_t>(x)) + static_cast<uint32_t>(x)) >> l);
    }
#endif
};
inline FastDiv make_fast_div(int d) {
    uint32_t l = 0;
    while ((1ull << l) < static_cast<uint64_t>(d)) ++l;
    const uint64_t m = ((((1ull << l) - d) << 32) / d) + 1;
    return {static_cast<uint32_t>(d), static_cast<uint32_t>(m), l};
}

cudaError_t launch_cache_plan(const PlanArgs& a, cudaStream_t stream, int* nlaunch);
cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t stream, int* nlaunch);
cudaError_t launch_paged_tile(const PagedArgs& a, cudaStream_t stream);
cudaError_t launch_fwd_paged(const PagedArgs& a, cudaStream_t stream, int* nlaunch);

}  // namespace fa
