// Internal interface of the paged 8-bit key/value cache: the block plan and
// the quantising append (fa_cache.cu) and attention over the cache
// (fa_paged.cu).
#pragma once

#include <atomic>

#include <cuda_runtime.h>
#include <stdint.h>
#include <math.h>

namespace fa {

// Status code a kernel leaves when the free list ran out (FA_ERR_NO_BLOCKS).
enum : int { FA_DEV_NO_BLOCKS = 5 };

constexpr int kPlanMaxB = 16384;      // requests of one plan (offsets of all of them sit in shared memory)
constexpr int kPagedCtas = 152;       // one persistent CTA per SM
constexpr int kPagedMaxRows = 32;     // tallest row tile of the split-key kernel
constexpr float kPagedLag = 8.f;      // us that a row-tile CTA's start and end take longer than a split-key CTA's
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

// A unit of the row-tile kernel whose key tiles were cut between CTAs, for the
// kernel that merges its pieces: rows row0 .. (token row / G, head hk * G + row %
// G, of tokens tok0 ..) of at most `rows`, pieces in slots piece(cta), cta = first .. last.
struct PagedCut {
    int valid, tok0, row0, rows, hk, first, last, parts;  // parts of a row in each piece: 1, 2 (row tiles) or 4 (and lanes 64 ..)
    long long line0, quota;
    __host__ __device__ int piece(int cta) const { return 2 * cta + (line0 <= quota * cta ? 0 : 1); }
};

// What a call with shared prefixes adds to its two passes (all zero otherwise).
// A pass leaves rows in ml and o (maximum and minus the sum, whose sign bit says
// that the row is there; output, normalised) for the other pass, or for the
// kernel that merges.
struct PagedJoin {
    const int32_t* first;   // the prefixes' pass: its request b is requests first[b] .. first[b + 1] - 1
    const int32_t* groups;  // requests groups[0] .. groups[ngroups] - 1 have a prefix
    int ngroups, requests;
    int leaves;             // this pass leaves the rows that have a prefix
    float2* ml;             // [total][Hq]; of the other pass where this one does not leave its rows
    float* o;               // [total][Hq][d]
    PagedCut* cuts;         // [2 * kPagedCtas], prefixes' pass of the row-tile kernel; zero at the start
    // both passes at once: what the other one reads and how it works, for the
    // number of CTAs that it gets
    const int32_t *other_len, *other_cu;
    int other_n, other_cap;      // its requests, and the longest that one may be
    int other_rows, other_cost;  // split-key kernel: rows of the row-tile kernel's units, and what one costs
    float place_us, other_us;  // time of a place on this pass's line and on the other's
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
    int split_rows;  // requests of no more rows are the split-key kernel's
    PagedJoin join;
    // workspace; the counters are zero at the start
    int* status;
    int* counters;       // [B * Hkv] finished pieces of the split-key kernel's units
    float *pm, *pl;      // [2 * kPagedCtas][kPagedMaxRows]
    float* po;           // [2 * kPagedCtas][kPagedMaxRows][d]
    int* tile_counters;  // [2 * max_tile_units], of the row-tile kernel's row tiles
    int max_tile_units;
    // [2 * kPagedCtas][kPagedTileRows] and the same [d]; the prefixes' pass has kPagedCtas
    // more, where the two parts of a unit of one row tile lie that is whole in a CTA
    float *tile_pm, *tile_pl, *tile_po;
    cudaEvent_t ev_begin, ev_end;  // optional, recorded around the attention kernels
    int one_tile;  // units of one row tile (the prefixes' pass)
    int chained;  // launched while the kernel before it may still run (see paged_wait_before)
};

inline cudaLaunchConfig_t paged_config(int threads, size_t smem, cudaStream_t stream, bool chained,
                                       cudaLaunchAttribute* at) {
    at->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at->val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(kPagedCtas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = chained ? 1 : 0;
    return cfg;
}

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
inline long long paged_max_tile_units(int B, int Hq, int Hkv, int total, int max_new, int d,
                                      int rows = kPagedTileRows) {
    const long long group = Hq / Hkv;
    if (!paged_has_tiles(max_new, static_cast<int>(group), d)) return 0;
    return Hkv * (B + total * group / rows);
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
// Programmatic dependent launch: a kernel of a chain may start once every CTA of
// the one before has let it (paged_let_next), and waits (paged_wait_before) where
// it needs that one's results, at the latest before it ends, so that the end of
// the last kernel is the end of all.
__device__ __forceinline__ void paged_let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void paged_wait_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Asynchronous copy of four bytes to shared memory, in groups.
__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>  // all but the newest N groups of this thread have landed
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Two E4M3 numbers (low 16 bits) to an f16 pair, exactly.
__device__ __forceinline__ uint32_t f16x2_from_e4m3x2(uint32_t x) {
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(x));
    return r;
}
// Of a call with shared prefixes: the requests i0 .. i1 - 1 that request i0 of
// this pass stands for. False if the offsets are none.
__device__ __forceinline__ bool paged_members(const PagedJoin& j, int& i0, int& i1) {
    if (!j.first) return true;
    const int a = j.first[i0], b = j.first[i1];
    i0 = min(max(a, 0), j.requests);
    i1 = min(max(b, i0), j.requests);
    return i0 == a && i1 == b;
}
__device__ __forceinline__ bool paged_joins(const PagedJoin& j, int b) {
    return b >= j.groups[0] && b < j.groups[j.ngroups];
}
// Places of the row-tile kernel's line that a request of `rows` rows and `len` keys
// has for each key head, all keys seen by all rows.
__device__ __forceinline__ long long paged_tile_places(int len, int cap, int rows, int unit, int cost) {
    const long long tiles = max(1, (min(max(len, 0), cap) + 127) >> 7);
    return (tiles + cost) * ((rows + unit - 1) / unit);
}
// Whether this pass leaves request b's rows to another kernel.
__device__ __forceinline__ bool paged_leaves(const PagedJoin& j, int b) {
    return j.leaves && (j.first || paged_joins(j, b));
}
// CTAs of this pass where both run at once: n of the prefixes' and the rest of the
// other such that kPagedLag + a / n = b / (kPagedCtas - n), a and b being the
// prefixes' work and the other, in us of a CTA.
__device__ __forceinline__ int paged_share(const PagedJoin& j, long long mine, long long other) {
    if (!j.other_len || mine == 0) return kPagedCtas;
    const float x = j.place_us * static_cast<float>(mine), y = j.other_us * static_cast<float>(other);
    const float a = j.first ? x : y, b = j.first ? y : x, c = a + b - kPagedLag * kPagedCtas;
    const float n = (sqrtf(c * c + 4.f * kPagedLag * kPagedCtas * a) - c) / (2.f * kPagedLag);
    const int pre = min(max(static_cast<int>(n + 0.5f), 1), kPagedCtas - 1);
    return j.first ? pre : kPagedCtas - pre;
}
// What a pass leaves of a row: its maximum and minus its sum, a NaN's sign set too
// (by an instruction that is no arithmetic: that would drop a NaN's sign).
__device__ __forceinline__ float2 paged_leave(float m, float l) {
    uint32_t y;
    asm("or.b32 %0, %1, 0x80000000;" : "=r"(y) : "r"(__float_as_uint(l)));
    return make_float2(m, __uint_as_float(y));
}
// Maximum and sum that the other pass left of a row.
__device__ __forceinline__ float2 paged_left(const PagedJoin& j, size_t row) {
    const float2 b = __ldcg(&j.ml[row]);
    return make_float2(b.x, -b.y);
}
// Softmax over two sets of keys with maxima m (log2 units) and sums l (both
// times 2^6, as the kernels keep them): the weights of the own output (not
// normalised) and of the prefix's (normalised), and L.
struct PagedWeights {
    float own, prefix, lse;
};
__device__ __forceinline__ PagedWeights paged_weights(float m, float l, float2 b) {
    const float la = log2f(l), lb = log2f(b.y), ln2 = 0.69314718055994530942f;
    const float d = l == 0.f ? -INFINITY : b.y == 0.f ? INFINITY : (m - b.x) + (la - lb);
    const float e = exp2f(-fabsf(d)), big = 1.f / (1.f + e), small = e * big;
    PagedWeights w;
    w.own = l == 0.f ? 0.f : (d >= 0.f ? big : small) / l;
    w.prefix = b.y == 0.f ? 0.f : d >= 0.f ? small : big;
    w.lse = ((d >= 0.f ? (m - 6.f) + la : (b.x - 6.f) + lb) + log2f(1.f + e)) * ln2;
    if (l == 0.f && b.y == 0.f) w.lse = -INFINITY;
    return w;
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

// Key tiles' time that a unit of the row-tile kernel takes beside its tiles', and
// chunks' time of a split-key unit (see there).
constexpr int paged_tile_cost(int d) { return d == 64 ? 6 : 8; }
constexpr int paged_split_cost(int d) { return d == 64 ? 48 : 32; }

// Sets up both passes of a call with shared prefixes to run at once. Times of a
// place on either line of work, in us: a tile of 128 keys for one or for two row
// tiles; a chunk of 32 keys for 8, 16, .. rows (64 requests behind 32,768 tokens 121
// us, 143 with one pass after the other; a serving step of 32 behind 4,096: 52 and 62).
inline void paged_run_both(PagedArgs& prefix, PagedArgs& own, float2* own_ml, float* own_o) {
    const int nt = own.split_rows / 8;
    prefix.join.place_us = prefix.d == 64 ? (prefix.one_tile ? 1.15f : 1.65f) : (prefix.one_tile ? 1.3f : 2.3f);
    prefix.join.other_us = prefix.d == 64 ? 0.20f + 0.05f * (nt - 1) : 0.18f + 0.05f * (nt - 1);
    prefix.join.other_len = own.cache_len;
    prefix.join.other_cu = own.cu_seqlens;
    prefix.join.other_n = own.B;
    prefix.join.other_cap = own.max_blocks * own.block_size;
    prefix.join.other_cost = paged_split_cost(own.d);
    own.join.place_us = prefix.join.other_us;
    own.join.other_us = prefix.join.place_us;
    own.join.other_len = prefix.cache_len;
    own.join.other_n = prefix.B;
    own.join.other_cap = prefix.max_blocks * prefix.block_size;
    own.join.other_rows = prefix.one_tile ? 128 : kPagedTileRows;
    own.join.other_cost = paged_tile_cost(own.d);
    own.join.leaves = 1;
    own.join.ml = own_ml;
    own.join.o = own_o;
}

cudaError_t launch_cache_plan(const PlanArgs& a, cudaStream_t stream, int* nlaunch);
cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t stream, int* nlaunch);
cudaError_t launch_paged_tile(const PagedArgs& a, cudaStream_t stream);
cudaError_t launch_fwd_paged_prefix(const PagedArgs& prefix, const PagedArgs& own, cudaStream_t stream, int* nlaunch);
cudaError_t launch_fwd_paged(const PagedArgs& a, cudaStream_t stream, int* nlaunch);

}  // namespace fa
