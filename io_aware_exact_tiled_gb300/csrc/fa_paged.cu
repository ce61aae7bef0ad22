// Attention over the paged 8-bit cache: the query rows of each request's new
// tokens against everything that the request's block table names.
//
// What it computes, for request b with n new tokens and length len, key head
// hk, query head h = hk * G + g and new token i at position p = len - n + i:
//   s_j = scale * (q . k8_j) * ks(block of j, hk),     j <= p (causal) or j < len
//   O = sum_j softmax(s)_j vs(block of j, hk) v8_j,    L = logsumexp(s)
// with k8, v8 the E4M3 numbers of the cache and ks, vs their block scales.
//
// Bound: every cached byte is read once and serves the n * G query rows of
// its head, so with few rows the time is the cache's bytes over HBM's rate.
// What has to be kept off that path is the conversion of the bytes and the
// wait for the block table in front of each copy. Measured, d = 128, one token
// for each request, against a copy's 6,766 GB/s: 16 requests of 8,192 to 16,383
// tokens, 32 key heads, 252 us = 6,630 GB/s of cache; 64 requests of 1 to 16,384
// tokens, 8 key heads, 193 us = 5,950; one request of 262,001 tokens, 96 us =
// 5,590. At d = 64, or with more rows, the issue slots bound it: 64 requests of
// 8,000 tokens, 8 key heads, 8 / 16 / 24 / 32 rows: 115 / 148 / 191 / 231 us
// (bytes alone: 77), d = 128 170 / 215 / 266 us (155).
//
// Design:
//   * Work is counted in chunks of 32 keys. A unit is (request, key head), with
//     at most RT = 8, 16, 24 or (d = 64) 32 query rows (fa_paged_tile.cu takes
//     requests of more). The chunks of the long units form one line (with room in front of
//     each unit for what its start and end cost) that is cut into equal quotas,
//     one for each persistent CTA, so ragged lengths balance by themselves and
//     one long request spreads over the whole GPU. A unit that
//     was cut leaves partial (m, l, O) in the workspace and the CTA that
//     finishes last merges them, in the order of the CTAs (the same result
//     every time). Short units (up to a third of a warp's even share of all
//     chunks) are not worth a CTA's barriers: each is one warp's, from its Q
//     to its output.
//   * Each of a CTA's eight to sixteen warps streams its own chunks (of a long
//     unit every eighth to sixteenth) through its own ring of TMA boxes with its
//     own mbarriers: no barrier between warps before a long unit ends. Block ids are fetched
//     three chunks ahead of the copies that need them.
//   * S^T = K Q^T and O^T = V^T P^T as m16n8k16 products with f16 operands
//     and fp32 sums, keys respectively head columns along M, the query rows
//     along N: eight rows cost no more than one. E4M3 converts to f16 exactly,
//     and so does Q down to 2^-31 of its row's maximum (within 2^-39 of it
//     below) after a power of two is taken out of each row. The k index of either product may be permuted
//     freely: K rows are read sixteen bytes a lane as they lie, and V's bytes
//     of two keys are interleaved by a byte permute; the permutations are
//     chosen so that no read of the 128-byte-swizzled tiles meets a bank
//     conflict.
//   * P is rounded to f16 relative to 2^-6 of the running reference maximum,
//     which only moves when a row grows by more than 2^8: weights keep their
//     11 bits down to 2^-20 of the maximum and vanish below 2^-30.
//   * ks multiplies S, vs the product of each chunk: neither scale is folded
//     into an 8- or 16-bit number.
#include <limits.h>
#include <math_constants.h>

#include "fa_paged.h"
#include "sm103_ptx.cuh"
#include "tmap.h"

namespace fa {

constexpr float kPgLn2 = 0.69314718055994530942f;
constexpr float kPgRescale = 8.0f;  // log2 units
constexpr float kPgOffset = 6.0f;   // log2 of the factor on P before its rounding to f16
constexpr int kPgChunk = 32;        // keys of a chunk
constexpr int kPgAhead = 3;         // chunks between the fetch of a block id and its use

// FA_DEBUG_DROP_ARRIVE (debug builds only): the first chunk's V is not
// requested in the first warp of each CTA, so that this warp's bounded wait
// runs out; a test checks that every warp gives up cleanly.
#ifdef FA_DEBUG_DROP_ARRIVE
#define FA_DROP_THIS_COPY(first_chunk) ((first_chunk) && threadIdx.x < 32)
#else
#define FA_DROP_THIS_COPY(first_chunk) false
#endif

template <int D, int NT, bool B16>
struct PgCfg {
    static constexpr int RT = 8 * NT;                     // query rows of a unit
    // Warps: what hides a chunk's chain of loads, products, exponentials and
    // shuffles is other warps, as many as the registers allow with few spills,
    // and as many on each scheduler (64 requests of 8,000 tokens, d = 64: 8 rows
    // 137 us with 8 warps, 118 with 12, 115 with 16; 16 rows 165 with 8, 174 with
    // 10, 146 with 12, 212 with 16).
    static constexpr int W = D == 64 && NT <= 2 ? (NT == 1 ? 16 : 12) : 8;
    static constexpr int THREADS = 32 * W;
    static constexpr int STAGES = D == 64 ? (NT >= 3 ? 4 : NT == 2 ? 3 : 2) : (NT == 1 ? 3 : 2);
    // chunks' time that a long unit's rows, barriers and merge take (64 requests
    // of 1 to 16,384 tokens: d = 128 271 us with 1, 192 with 32, 196 with 48; d = 64
    // 212 with 1, 126 with 48, 129 with 72)
    static constexpr int COST = D == 64 ? 48 : 32;
    static constexpr int TILE = kPgChunk * D;             // bytes of a chunk's K (or V)
    static constexpr int SUBS = B16 ? 2 : 1;              // boxes of a tile
    static constexpr int BOX = TILE / SUBS;
    static constexpr int KK = D / 16;                     // k steps of S
    static constexpr int MI = D / 16;                     // m tiles of O^T
    static constexpr int RED_F = 4 * NT * 32;             // floats of one m tile of a warp's O^T
    static constexpr int RED_M = 4;                       // m tiles merged at a time
    static constexpr int RING_OFF = 0;
    static constexpr int RING = W * STAGES * 2 * TILE;
    static constexpr int RED_OFF = RING_OFF + RING;       // fp32 [W][RED_M][RED_F] or f16 Q of each warp's unit
    static constexpr int Q_BYTES = RT * D * 2;            // f16 fragments of Q
    static constexpr int Q_OFF = RED_OFF + W * RED_M * RED_F * 4;  // of a long unit
    static constexpr int ML_OFF = Q_OFF + Q_BYTES;        // fp32 [W + 1][RT][2]
    static constexpr int ROW_OFF = ML_OFF + (W + 1) * RT * 8;  // [W] {score factor, visible keys} of each row
    static constexpr int META_OFF = ROW_OFF + W * RT * 8;  // float4 [W][STAGES]: ks0, ks1, vs0, vs1
    static constexpr int NAN_OFF = META_OFF + W * STAGES * 16;  // int [W][D] first key with a NaN value
    static constexpr int ID_OFF = NAN_OFF + W * D * 4;  // int [W][4][2] block ids on their way
    static constexpr int BAR_OFF = ID_OFF + W * 32;
    static constexpr int USED = BAR_OFF + W * STAGES * 8;
    static constexpr int SMEM = USED + 1024;
    static_assert(W * RED_M * RED_F * 4 >= W * Q_BYTES, "Q of the warps' units");
    static_assert(SMEM <= 232448 - 6144, "shared memory, beside the static arrays");
};

struct PagedParams {
    const uint16_t* q;
    const float *k_scale, *v_scale;
    uint16_t* o;
    float* lse;
    const int32_t *cu_seqlens, *cache_len, *block_table;
    int B, Hq, Hkv, G, total, max_new, max_blocks, num_blocks, bs_log2;
    float scale_log2;
    int causal;
    int split_rows;  // requests of more rows are the row-tile kernel's
    FastDiv by_g;    // division by G
    int *status, *counters;
    float *pm, *pl, *po;
};

// m16n8k16, f16 operands, fp32 sums.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transpose of the warp's 8 x 8 matrix of 16-bit elements.
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t saddr) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(saddr));
    return v;
}
// Asynchronous copy of four bytes to shared memory, in groups.
__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>  // all but the newest N groups of this thread have landed
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Bytes of x that are E4M3 NaN (0x7F or 0xFF) as 0x80 bits.
__device__ __forceinline__ uint32_t e4m3_nan_bits(uint32_t x) { return ((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// Key of a 16-key group that row r (0..15) of the key-side MMA tile holds.
// d = 128: a shared-memory row per key; d = 64: two keys share a row. Either
// order makes the two rows of a quarter-warp's K read (r = 2q, 2q + 1) and the
// four rows of its V read (r = 2t, or 2t + 1) lie in different banks.
template <int D>
__device__ __forceinline__ int pg_key(int r) {
    constexpr uint32_t kMap = D == 128 ? 0x36147250u : 0x65217430u;
    return (r & 8) | ((kMap >> (4 * (r & 7))) & 7u);
}
// Byte offset of 16-byte piece c of key j (0..31) in a chunk's swizzled tile.
template <int D>
__device__ __forceinline__ uint32_t pg_off(int j, int c) {
    if constexpr (D == 128) return static_cast<uint32_t>(j * 128 + ((c ^ (j & 7)) << 4));
    else return static_cast<uint32_t>((j >> 1) * 128 + (((((j & 1) << 2) | c) ^ ((j >> 1) & 7)) << 4));
}

// One unit's piece of a CTA's quota.
struct PgSeg {
    int b, hk;          // request, key head
    int n, len, tok0;   // new tokens (0: none, or the row-tile kernel's), length, first token
    int nchunk;         // chunks of each of the request's units; 0 without rows
    int c0, c1;         // this piece's chunks
    bool alone;         // a short unit, one warp's
    long long rline;    // position of the request's first chunk on its line
    long long line0;    // position of a long unit's first chunk on its line
};

// Loads request b (sizes clamped to what the tables can hold).
__device__ __forceinline__ void pg_request(const PagedParams& p, int b, PgSeg& s) {
    const int t0 = min(max(p.cu_seqlens[b], 0), p.total), t1 = min(max(p.cu_seqlens[b + 1], t0), p.total);
    s.tok0 = t0;
    s.n = min(t1 - t0, p.max_new);
    if (static_cast<long long>(s.n) * p.G > p.split_rows) s.n = 0;
    s.len = min(max(p.cache_len[b], 0), p.max_blocks << p.bs_log2);
    s.nchunk = s.n > 0 ? max(1, (s.len + kPgChunk - 1) / kPgChunk) : 0;
}

template <int D, int NT, bool B16>
__global__ void __launch_bounds__(PgCfg<D, NT, B16>::THREADS, 1)
    fa_paged_split_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                          const __grid_constant__ PagedParams p) {
    using C = PgCfg<D, NT, B16>;
    constexpr int RT = C::RT;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ long long scan_w[3][C::W];
    __shared__ long long short_base[C::THREADS + 1];  // chunks of short units in front of each thread's requests
    __shared__ int start_b, last_s;
    __shared__ long long start_line;
    __shared__ int nan_seen, abort_s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;

    // ---- all chunks, then the lines of long and of short units
    const int per = (p.B + C::THREADS - 1) / C::THREADS;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    long long mw = 0;
    bool bad = false;
    for (int b = b0; b < b1; ++b) {
        PgSeg s;
        pg_request(p, b, s);
        mw += static_cast<long long>(p.Hkv) * s.nchunk;
        const int raw = p.cu_seqlens[b], nxt = p.cu_seqlens[b + 1], len = p.cache_len[b];
        bad |= raw < 0 || nxt < raw || nxt > p.total || nxt - raw > p.max_new || len != s.len;
    }
    if (bad && blockIdx.x == 0) atomicCAS(p.status, 0, FA_DEV_INVALID | (90 << 8));
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::BAR_OFF) + warp * C::STAGES;
    if (tid == 0) {
        abort_s = 0;
        nan_seen = 0;
    }
    if (lane < C::STAGES) mbar_init(&bars[lane], 1);
    fence_barrier_init();
    int* first_nan = reinterpret_cast<int*>(sm + C::NAN_OFF);
    for (int i = tid; i < C::W * D; i += C::THREADS) first_nan[i] = INT_MAX;
    long long sum = mw;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (lane == 0) scan_w[0][warp] = sum;
    __syncthreads();
    long long W = 0;
    for (int w = 0; w < C::W; ++w) W += scan_w[0][w];
    // A unit of up to a third of a warp's even share of all chunks is short, and
    // one of up to twelve chunks always: a long unit costs its CTA barriers and a
    // merge, a short one keeps a single warp busy, at the end while others have
    // nothing left. d = 128, one token, 8 heads of keys: 1,024 requests of 1 to
    // 600 tokens 197 us (up to a sixth: 251; none short: 302), 256 requests of 1 to
    // 2,000 tokens 143 us (up to a half: 160; to the whole share: 172).
    const long long share = W / (kPagedCtas * C::W);
    int T = static_cast<int>(min(max(share / 3, 12ll), 1ll << 30));
    auto line_long = [&](const PgSeg& s) {
        return s.nchunk > T ? static_cast<long long>(p.Hkv) * (s.nchunk + C::COST) : 0ll;
    };
    auto line_short = [&](const PgSeg& s) { return s.nchunk <= T ? static_cast<long long>(p.Hkv) * s.nchunk : 0ll; };
    long long ml_ = 0, ms = 0, ma = 0;  // long, short, all as long ones
    for (int b = b0; b < b1; ++b) {
        PgSeg s;
        pg_request(p, b, s);
        ml_ += line_long(s);
        ms += line_short(s);
        if (s.nchunk > 0) ma += static_cast<long long>(p.Hkv) * (s.nchunk + C::COST);
    }
    long long il = ml_, is_ = ms, ia = ma;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, il, off), c = __shfl_up_sync(0xffffffffu, is_, off);
        const long long d = __shfl_up_sync(0xffffffffu, ia, off);
        if (lane >= off) {
            il += a;
            is_ += c;
            ia += d;
        }
    }
    __syncthreads();
    if (lane == 31) {
        scan_w[0][warp] = il;
        scan_w[1][warp] = is_;
        scan_w[2][warp] = ia;
    }
    __syncthreads();
    long long Wl = 0, Ws = 0, Wa = 0, bw = il - ml_, bs = is_ - ms, ba = ia - ma;
#pragma unroll
    for (int w = 0; w < C::W; ++w) {
        if (w < warp) {
            bw += scan_w[0][w];
            bs += scan_w[1][w];
            ba += scan_w[2][w];
        }
        Wl += scan_w[0][w];
        Ws += scan_w[1][w];
        Wa += scan_w[2][w];
    }
    // A few short units among long ones would only come after everything else:
    // they are taken as long ones (64 requests of 1 to 16,384 tokens: 192 us, 232
    // with a warp each for the short ones).
    if (Ws * 8 < W) {
        T = 0;
        Wl = Wa;
        Ws = 0;
        bw = ba;
        ml_ = ma;
        bs = 0;
    }
    // equal quotas of the long line, at least one chunk for each warp
    const long long quota = max((Wl + kPagedCtas - 1) / kPagedCtas, static_cast<long long>(C::W));
    const long long x0 = quota * blockIdx.x, x1 = min(x0 + quota, Wl);
    // the short units that start in this warp's part of their line; parts that
    // follow one another lie in different CTAs
    const long long part = (Ws + kPagedCtas * C::W - 1) / (kPagedCtas * C::W);
    const long long y0 = part * (warp * kPagedCtas + static_cast<int>(blockIdx.x)), y1 = min(y0 + part, Ws);
    short_base[tid] = bs;
    if (tid == C::THREADS - 1) short_base[C::THREADS] = Ws;
    if (x0 < x1 && x0 >= bw && x0 < bw + ml_) {
        for (int b = b0; b < b1; ++b) {
            PgSeg s;
            pg_request(p, b, s);
            const long long w = line_long(s);
            if (x0 < bw + w) {
                start_b = b;
                start_line = bw;
                break;
            }
            bw += w;
        }
    }
    __syncthreads();

    // ---- the pieces of this warp: first its share of the CTA's pieces of long
    // units, then its short units
    auto place = [&](PgSeg& s, long long x) -> bool {  // long: the piece that starts at x, here or in a later request
        for (;;) {
            const long long w = line_long(s);
            if (x < s.rline + w) break;
            s.rline += w;
            ++s.b;
            pg_request(p, s.b, s);
        }
        const long long r = x - s.rline;
        s.hk = static_cast<int>(div_short(r, s.nchunk + C::COST));
        const int rest = static_cast<int>(r - static_cast<long long>(s.hk) * (s.nchunk + C::COST));
        s.line0 = x - rest + C::COST;
        s.c0 = max(rest - C::COST, 0);
        s.c1 = static_cast<int>(min(static_cast<long long>(s.nchunk), x1 - s.line0));
        return s.c1 > s.c0;  // not only the room in front of a unit
    };
    auto settle = [&](PgSeg& s) -> bool {  // short: hk names the wanted unit of request b, or one past its last
        while (s.hk >= p.Hkv || s.nchunk == 0 || s.nchunk > T) {
            s.rline += line_short(s);
            if (s.rline >= y1) return false;
            ++s.b;
            s.hk = 0;
            pg_request(p, s.b, s);
        }
        s.c0 = 0;
        s.c1 = s.nchunk;
        return s.rline + static_cast<long long>(s.hk) * s.nchunk < y1;
    };
    auto first_short = [&](PgSeg& s) -> bool {
        if (y0 >= y1) return false;
        s.alone = true;
        // the thread whose requests hold position y0
        int lo = 0;
        for (int i = 0; i < C::W; ++i) {
            const uint32_t in = __ballot_sync(0xffffffffu, short_base[i * 32 + lane] <= y0);
            if (in) lo = i * 32 + 31 - __clz(in);
        }
        s.b = lo * per;
        s.rline = short_base[lo];
        pg_request(p, s.b, s);
        for (;;) {
            const long long w = line_short(s);
            if (y0 < s.rline + w) break;
            s.rline += w;
            ++s.b;
            pg_request(p, s.b, s);
        }
        s.hk = static_cast<int>(div_short(y0 - s.rline + s.nchunk - 1, s.nchunk));
        return settle(s);
    };
    auto next = [&](PgSeg& s) -> bool {
        if (s.alone) {
            ++s.hk;
            return settle(s);
        }
        const long long x = s.line0 + s.c1;
        return (x < x1 && place(s, x)) || first_short(s);
    };
    PgSeg cs, is;  // pieces being consumed and being requested
    cs.alone = false;
    bool work = false;
    if (x0 < x1) {
        cs.b = start_b;
        cs.rline = start_line;
        pg_request(p, cs.b, cs);
        work = place(cs, x0);
    }
    work = work || first_short(cs);
    is = cs;
    bool iwork = work;

    const WaitCtx cx{reinterpret_cast<volatile int*>(&abort_s), p.status};
    uint8_t* ring = sm + C::RING_OFF + warp * C::STAGES * 2 * C::TILE;
    float4* meta = reinterpret_cast<float4*>(sm + C::META_OFF) + warp * C::STAGES;
    // ---- requests of this warp: chunk c0 + warp + W k of a long piece, c0 + k
    // of a short unit. A chunk's loads depend on one another (block id, then
    // the copies and the scales), so the ids come three chunks ahead of the
    // copies, and both they and the scales go to shared memory by asynchronous
    // copies. Step j commits one group: the ids of chunk j + 3 and the scales
    // of chunk j.
    auto chunk_of = [&](const PgSeg& s, int k) { return s.alone ? s.c0 + k : s.c0 + warp + C::W * k; };
    int* idq = reinterpret_cast<int*>(sm + C::ID_OFF) + warp * 8;  // [4][2] block ids
    int ik = 0, issued = 0, consumed = 0, fetched = 0;
    auto prefetch_q = [&](const PgSeg& s) {  // a unit's query rows, wanted soon
        if (lane >= s.n * p.G) return;
        const int tok = p.by_g.div(lane);
        const uint16_t* row = p.q + (static_cast<size_t>(s.tok0 + tok) * p.Hq + s.hk * p.G + (lane - tok * p.G)) * D;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(row));
        if (D == 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + 64));
    };
    if (work) prefetch_q(cs);
    int hk_in[kPgAhead] = {};  // (key head << bs_log2) + first row; -1: no chunk
    int in_len[kPgAhead] = {};  // boxes with keys in front of the last token's end
    auto fetch = [&](int at) {
        while (iwork && chunk_of(is, ik) >= is.c1) {
            iwork = next(is);
            ik = 0;
            if (iwork) prefetch_q(is);
        }
        hk_in[at] = -1;
        if (!iwork) return;
        const int key0 = chunk_of(is, ik) * kPgChunk, key = key0 + 16 * lane;
        hk_in[at] = (is.hk << p.bs_log2) + (B16 ? 0 : key0 & ((1 << p.bs_log2) - 1));
        in_len[at] = key0 >= is.len ? 0 : key0 + 16 < is.len ? 2 : 1;
        if (lane < C::SUBS && key < is.len)
            cp_async4(&idq[(fetched & 3) * 2 + lane],
                      &p.block_table[static_cast<size_t>(is.b) * p.max_blocks + (key >> p.bs_log2)]);
        ++fetched;
        ++ik;
    };
    auto issue = [&]() {
        cp_async_wait<2>();
        __syncwarp();
        const int hi = hk_in[0];
        if (hi >= 0) {
            const int st = issued % C::STAGES;
            if (lane == 0) mbar_arrive_expect_tx(&bars[st], 2 * C::TILE);
            __syncwarp();
            // lane 0 (and 1, for a second box) requests the copies, lanes 0..3 the scales
            const int sub = C::SUBS == 2 ? lane & 1 : 0, raw = idq[(issued & 3) * 2 + sub];
            const bool named = sub < in_len[0], good = named && raw >= 0 && raw < p.num_blocks;
            const int id = good ? raw : 0;
            if (lane < C::SUBS) {
                if (named && !good) atomicCAS(p.status, 0, FA_DEV_INVALID | (91 << 8));
                // rows of the [num_blocks * Hkv * block_size * d / 128, 128] matrix
                const long long key = ((static_cast<long long>(id) * p.Hkv) << p.bs_log2) + hi;
                const int row = static_cast<int>(D == 128 ? key : key >> 1);
                tma_load_2d(ring + (2 * st) * C::TILE + sub * C::BOX, &tmK, 0, row, &bars[st]);
                if (!FA_DROP_THIS_COPY(issued == 0))
                    tma_load_2d(ring + (2 * st + 1) * C::TILE + sub * C::BOX, &tmV, 0, row, &bars[st]);
            }
            if (lane < 4) {
                float* dst = reinterpret_cast<float*>(&meta[st]) + lane;
                if (good)
                    cp_async4(dst, (lane < 2 ? p.k_scale : p.v_scale) + static_cast<size_t>(id) * p.Hkv +
                                       (hi >> p.bs_log2));
                else
                    *dst = 0.f;
            }
            ++issued;
        }
#pragma unroll
        for (int i = 0; i + 1 < kPgAhead; ++i) {
            hk_in[i] = hk_in[i + 1];
            in_len[i] = in_len[i + 1];
        }
        fetch(kPgAhead - 1);
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kPgAhead; ++i) {
        fetch(i);
        cp_async_commit();
    }
#pragma unroll 1
    for (int i = 0; i < C::STAGES; ++i) issue();

    float2* ml = reinterpret_cast<float2*>(sm + C::ML_OFF);
    float* red = reinterpret_cast<float*>(sm + C::RED_OFF);
    bool ok = true;

#pragma unroll 1
    while (work) {
        // ---------------------------------------------------- the piece's rows
        const int nrow = cs.n * p.G;  // rows of the request: token * G + head of the group
        uint8_t* qs = cs.alone ? sm + C::RED_OFF + warp * C::Q_BYTES : sm + C::Q_OFF;
        float2* rowc = reinterpret_cast<float2*>(sm + C::ROW_OFF) + (cs.alone ? warp * RT : 0);
        int* nan_at = first_nan + (cs.alone ? warp * D : 0);
        // visible keys of the first and the last row
        auto visible = [&](int tok) { return p.causal ? min(max(cs.len - cs.n + tok + 1, 0), cs.len) : cs.len; };
        const int vis_min = visible(0), vis_max = visible(cs.n - 1);
        const int r0 = cs.alone ? 0 : warp, rstep = cs.alone ? 1 : C::W;
#pragma unroll 4
        for (int r = r0; r < RT; r += rstep) {
            // four values per lane; the row's power of two goes to its score factor
            uint2 x = make_uint2(0u, 0u);
            const int tok = p.by_g.div(r);
            if (r < nrow && lane < D / 4)
                x = *reinterpret_cast<const uint2*>(
                    p.q + (static_cast<size_t>(cs.tok0 + tok) * p.Hq + cs.hk * p.G + (r - tok * p.G)) * D + lane * 4);
            const uint32_t h4[4] = {x.x & 0xFFFFu, x.x >> 16, x.y & 0xFFFFu, x.y >> 16};
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) top = max(top, h4[i] & 0x7FFFu);
            top = __reduce_max_sync(0xffffffffu, top);
            const bool wild = top >= 0x7F80u;  // an infinity or a NaN: the row has no finite result
            const int e = top >> 7 && !wild ? min(max(static_cast<int>(top >> 7) - 141, -120), 120) : 0;
            const float f = exp2i(-e);
            if (lane < D / 4) {
                const int half = lane >> 4, tq = (lane >> 2) & 3, kk = half * 4 + (lane & 3);
                uint2 y;
                y.x = pack_f16x2(__uint_as_float(h4[0] << 16) * f, __uint_as_float(h4[1] << 16) * f);
                y.y = pack_f16x2(__uint_as_float(h4[2] << 16) * f, __uint_as_float(h4[3] << 16) * f);
                *reinterpret_cast<uint2*>(qs + (((r >> 3) * (C::KK / 2) + (kk >> 1)) * 32 + 4 * (r & 7) + tq) * 16 +
                                          (kk & 1) * 8) = y;
            }
            if (lane == 0)
                rowc[r] = make_float2(wild ? CUDART_NAN_F : p.scale_log2 * exp2i(e),
                                      __int_as_float(r < nrow ? visible(tok) : cs.len));
        }
        if (cs.alone) __syncwarp();
        else __syncthreads();
        float rc[NT][2], m[NT][2], l[NT][2];
        int lim[NT][2];
        float o[C::MI][NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float2 v = rowc[nt * 8 + 2 * t4 + e];
                rc[nt][e] = v.x;
                lim[nt][e] = __float_as_int(v.y);
                m[nt][e] = -CUDART_INF_F;
                l[nt][e] = 0.f;
            }
#pragma unroll
        for (int i = 0; i < C::MI; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][nt][e] = 0.f;

        // ---------------------------------------------------- its chunks
        uint32_t nan_bits = 0u;
#pragma unroll 1
        for (int c = chunk_of(cs, 0), cstep = chunk_of(cs, 1) - c; c < cs.c1; c += cstep) {
            const int st = consumed % C::STAGES;
            ok = mbar_wait_warp(&bars[st], (consumed / C::STAGES) & 1, cx, 92);
            if (!ok) break;
            cp_async_wait<C::STAGES - 1>();
            __syncwarp();
            const float4 mt4 = meta[st];
            const uint32_t kb = smem_u32(ring + 2 * st * C::TILE), vb = kb + C::TILE;
            const int key0 = c * kPgChunk;
            const bool edge = key0 + kPgChunk > vis_min;
            // ---- S^T = K Q^T
            float s[2][NT][4];
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[mt][nt][e] = 0.f;
#pragma unroll
            for (int cc = 0; cc < D / 64; ++cc) {
                uint4 kw[2][2];
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh)
                        kw[mt][hh] = lds128_u4(kb + pg_off<D>(mt * 16 + hh * 8 + pg_key<D>(g), t4 + 4 * cc));
#pragma unroll
                for (int k2 = 0; k2 < 2; ++k2) {
                    uint4 qf[NT];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        qf[nt] = lds128_u4(smem_u32(qs + ((nt * (C::KK / 2) + cc * 2 + k2) * 32 + lane) * 16));
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int mt = 0; mt < 2; ++mt) {
                            const uint32_t lo = (&kw[mt][0].x)[k2 * 2 + e], hi = (&kw[mt][1].x)[k2 * 2 + e];
                            const uint32_t a0 = f16x2_from_e4m3x2(lo), a2 = f16x2_from_e4m3x2(lo >> 16);
                            const uint32_t a1 = f16x2_from_e4m3x2(hi), a3 = f16x2_from_e4m3x2(hi >> 16);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma_f16(s[mt][nt], a0, a1, a2, a3, e ? qf[nt].z : qf[nt].x, e ? qf[nt].w : qf[nt].y);
                        }
                }
            }
            // ---- scale, mask, maximum
            bool grow = false;
            float mx[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float f0 = rc[nt][e] * mt4.x, f1 = rc[nt][e] * mt4.y;
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        s[0][nt][2 * hh + e] *= f0;
                        s[1][nt][2 * hh + e] *= f1;
                    }
                    if (edge) {
#pragma unroll
                        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                            for (int hh = 0; hh < 2; ++hh)
                                if (key0 + mt * 16 + hh * 8 + pg_key<D>(g) >= lim[nt][e])
                                    s[mt][nt][2 * hh + e] = -CUDART_INF_F;
                    }
                    mx[nt][e] = fmaxf(fmaxf(s[0][nt][e], s[0][nt][2 + e]), fmaxf(s[1][nt][e], s[1][nt][2 + e]));
                    grow |= mx[nt][e] > m[nt][e] + kPgRescale;
                }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = mx[nt][e];
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                        const float mn = fmaxf(m[nt][e], x);
                        const float al = m[nt][e] == -CUDART_INF_F ? 0.f : ex2_approx(m[nt][e] - mn);
                        m[nt][e] = mn;
                        l[nt][e] *= al;
#pragma unroll
                        for (int i = 0; i < C::MI; ++i) {
                            o[i][nt][e] *= al;
                            o[i][nt][2 + e] *= al;
                        }
                    }
            }
            // ---- P (f16) and its transposition into the B fragments
            uint32_t pb[2][NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float sh[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) sh[e] = m[nt][e] == -CUDART_INF_F ? 0.f : kPgOffset - m[nt][e];
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        const float p0 = ex2_approx(s[mt][nt][2 * hh] + sh[0]);
                        const float p1 = ex2_approx(s[mt][nt][2 * hh + 1] + sh[1]);
                        l[nt][0] += p0;
                        l[nt][1] += p1;
                        pb[mt][nt][hh] = movmatrix(pack_f16x2(p0, p1));
                    }
            }
            // ---- O^T += vs V^T P^T
            // (with many rows and d = 128, in two parts of the columns: the registers
            // hold no more)
            constexpr int VH = D == 128 && NT >= 3 ? 2 : 1, VW = D / 32 / VH;
#pragma unroll
            for (int vh = 0; vh < VH; ++vh) {
                uint32_t vw[2][4][VW];
#pragma unroll
                for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int j = ks * 16 + (r >> 1) * 8 + pg_key<D>(2 * t4 + (r & 1));
                        if constexpr (VW == 4) {
                            const uint4 x = lds128_u4(vb + pg_off<D>(j, g));
                            vw[ks][r][0] = x.x;
                            vw[ks][r][1] = x.y;
                            vw[ks][r][2] = x.z;
                            vw[ks][r][3] = x.w;
                        } else {
                            const uint2 x = D == 128 ? lds64(vb + pg_off<D>(j, g) + vh * 8)
                                                     : lds64(vb + pg_off<D>(j, g >> 1) + (g & 1) * 8);
                            vw[ks][r][0] = x.x;
                            vw[ks][r][1] = x.y;
                        }
                    }
                if (edge) {
                    // keys that no row sees count as zero whatever their bytes are;
                    // a NaN that only some rows see is taken out here and given
                    // back to those rows at the end (one test for all words: 2,048
                    // requests of 1 to 100 tokens 208 -> 154 us)
                    uint32_t any = 0u;
#pragma unroll
                    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int key = key0 + ks * 16 + (r >> 1) * 8 + pg_key<D>(2 * t4 + (r & 1));
#pragma unroll
                            for (int w = 0; w < VW; ++w) {
                                if (key >= vis_max) vw[ks][r][w] = 0u;
                                any |= e4m3_nan_bits(vw[ks][r][w]);
                            }
                        }
                    if (any) {
                        nan_bits = 1u;
#pragma unroll
                        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                const int key = key0 + ks * 16 + (r >> 1) * 8 + pg_key<D>(2 * t4 + (r & 1));
#pragma unroll
                                for (int w = 0; w < VW; ++w) {
                                    const uint32_t nb = e4m3_nan_bits(vw[ks][r][w]);
                                    if (!nb) continue;
#pragma unroll
                                    for (int y = 0; y < 4; ++y)
                                        if ((nb >> (8 * y)) & 0x80u) {
                                            atomicMin(&nan_at[g * (D / 8) + (vh * VW + w) * 4 + y], key);
                                            vw[ks][r][w] &= ~(0xFFu << (8 * y));
                                        }
                                }
                            }
                    }
                }
#pragma unroll
                for (int k = 0; k < 2 * VW; ++k) {
                    const int i = vh * 2 * VW + k;
                    float acc[NT][4];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[nt][e] = 0.f;
#pragma unroll
                    for (int ks = 0; ks < 2; ++ks) {
                        const uint32_t sel = k & 1 ? 0x7362u : 0x5140u;
                        const uint32_t x = __byte_perm(vw[ks][0][k >> 1], vw[ks][1][k >> 1], sel);
                        const uint32_t y = __byte_perm(vw[ks][2][k >> 1], vw[ks][3][k >> 1], sel);
                        const uint32_t a0 = f16x2_from_e4m3x2(x), a1 = f16x2_from_e4m3x2(x >> 16);
                        const uint32_t a2 = f16x2_from_e4m3x2(y), a3 = f16x2_from_e4m3x2(y >> 16);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_f16(acc[nt], a0, a1, a2, a3, pb[ks][nt][0], pb[ks][nt][1]);
                        if (B16 || ks == 1) {
                            const float vs = ks ? mt4.w : mt4.z;
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    o[i][nt][e] = fmaf(vs, acc[nt][e], o[i][nt][e]);
                                    if (B16) acc[nt][e] = 0.f;
                                }
                        }
                    }
                }
            }
            ++consumed;
            // The stage has been read: the copy that issue() requests into it
            // must find every lane's loads done, and a barrier alone does not
            // wait for loads whose values are still on their way. A vote on a
            // sum that took a word of each load of V does, with the branch on it
            // (to a fence, which changes nothing); the loads of K were done at
            // the vote on the maxima above.
            bool odd = __float_as_uint(o[0][0][0]) == 0x7F7F7F7Fu;
            if constexpr (VH == 2) odd |= __float_as_uint(o[2 * VW][0][0]) == 0x7F7F7F7Fu;
            if (__any_sync(0xffffffffu, odd)) __threadfence_block();
            __syncwarp();
            issue();
        }

        // row sums over the key lanes
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = l[nt][e];
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                x += __shfl_xor_sync(0xffffffffu, x, 8);
                x += __shfl_xor_sync(0xffffffffu, x, 16);
                l[nt][e] = x;
            }
        auto lse_of = [&](float mm, float ll) {
            return ll == 0.f ? -CUDART_INF_F : (mm - kPgOffset + log2f(ll)) * kPgLn2;
        };
        if (cs.alone) {
            // ------------------------------------------------ a short unit: its rows are this warp's
            if (!ok) break;
            const bool nans = __any_sync(0xffffffffu, nan_bits != 0u);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = nt * 8 + 2 * t4 + e, tok = p.by_g.div(r), hq = cs.hk * p.G + r - tok * p.G;
                    if (r >= nrow) continue;
                    const float inv = l[nt][e] == 0.f ? 0.f : 1.f / l[nt][e];
                    // columns g D/8 .. + D/8 of row r
                    uint32_t w[C::MI];
#pragma unroll
                    for (int i = 0; i < C::MI; ++i) {
                        float a = o[i][nt][e] * inv, b = o[i][nt][2 + e] * inv;
                        if (nans) {
                            a = nan_at[g * (D / 8) + 2 * i] < lim[nt][e] ? CUDART_NAN_F : a;
                            b = nan_at[g * (D / 8) + 2 * i + 1] < lim[nt][e] ? CUDART_NAN_F : b;
                        }
                        w[i] = pack_bf16x2(a, b);
                    }
                    uint4* dst = reinterpret_cast<uint4*>(
                        p.o + (static_cast<size_t>(cs.tok0 + tok) * p.Hq + hq) * D + g * (D / 8));
#pragma unroll
                    for (int i = 0; i < C::MI / 4; ++i)
                        dst[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                    if (g == 0)
                        p.lse[static_cast<size_t>(hq) * p.total + cs.tok0 + tok] = lse_of(m[nt][e], l[nt][e]);
                }
            __syncwarp();
            if (nans) {
                for (int i = lane; i < D; i += 32) nan_at[i] = INT_MAX;
                __syncwarp();
            }
            work = next(cs);
            continue;
        }
        // ---------------------------------------------------- merge of the warps
        if (nan_bits) nan_seen = 1;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (g == 0) ml[warp * RT + nt * 8 + 2 * t4 + e] = make_float2(m[nt][e], l[nt][e]);
        if (__syncthreads_or(!ok)) break;
        float fac[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float M = -CUDART_INF_F;
#pragma unroll
                for (int w = 0; w < C::W; ++w) M = fmaxf(M, ml[w * RT + nt * 8 + 2 * t4 + e].x);
                fac[nt][e] = m[nt][e] == -CUDART_INF_F ? 0.f : ex2_approx(m[nt][e] - M);
            }
        const bool whole = cs.c0 == 0 && cs.c1 == cs.nchunk;
        const int slot = 2 * static_cast<int>(blockIdx.x) + (cs.line0 <= x0 ? 0 : 1);
        if (tid < RT) {
            // the row's maximum and sum over the warps
            float M = -CUDART_INF_F, L = 0.f;
#pragma unroll
            for (int w = 0; w < C::W; ++w) M = fmaxf(M, ml[w * RT + tid].x);
#pragma unroll
            for (int w = 0; w < C::W; ++w) {
                const float2 v = ml[w * RT + tid];
                L += v.y * (v.x == -CUDART_INF_F ? 0.f : ex2_approx(v.x - M));
            }
            ml[C::W * RT + tid] = make_float2(M, L == 0.f ? 0.f : 1.f / L);
            if (!whole) {
                p.pm[slot * kPagedMaxRows + tid] = M;
                p.pl[slot * kPagedMaxRows + tid] = L;
            } else if (tid < nrow) {
                const int tok = p.by_g.div(tid), hq = cs.hk * p.G + tid - tok * p.G;
                p.lse[static_cast<size_t>(hq) * p.total + cs.tok0 + tok] = lse_of(M, L);
            }
        }
        // m tiles in turn: the warps' parts of RED_M tiles at a time
#pragma unroll
        for (int i0 = 0; i0 < C::MI; i0 += C::RED_M) {
#pragma unroll
            for (int i = i0; i < i0 + C::RED_M; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        // element (m tile, row, column pair): lanes of a store cover 32 banks
                        red[((warp * C::RED_M + i - i0) * 4 * NT + nt * 4 + e) * 32 + lane] =
                            o[i][nt][e] * fac[nt][e & 1];
            __syncthreads();
#pragma unroll
            for (int x = tid; x < C::RED_M * C::RED_F; x += C::THREADS) {
                float sum = 0.f;
#pragma unroll
                for (int w = 0; w < C::W; ++w) sum += red[w * C::RED_M * C::RED_F + x];
                const int ln = x & 31, q = x >> 5, e = q & 3, nt = (q >> 2) % NT, i = i0 + q / (4 * NT);
                const int r = nt * 8 + 2 * (ln & 3) + (e & 1);
                const int col = (ln >> 2) * (D / 8) + 2 * i + (e >> 1);
                if (nan_seen && nan_at[col] < __float_as_int(rowc[r].y)) sum = CUDART_NAN_F;
                if (!whole) {
                    p.po[(static_cast<size_t>(slot) * kPagedMaxRows + r) * D + col] = sum;
                } else if (r < nrow) {
                    const int tok = p.by_g.div(r), hq = cs.hk * p.G + r - tok * p.G;
                    p.o[(static_cast<size_t>(cs.tok0 + tok) * p.Hq + hq) * D + col] =
                        static_cast<uint16_t>(pack_bf16x2(sum * ml[C::W * RT + r].y, 0.f) & 0xFFFFu);
                }
            }
            __syncthreads();
        }
        if (tid < D) nan_at[tid] = INT_MAX;
        if (tid == 0) nan_seen = 0;
        if (!whole) {
            // the CTAs that hold pieces of this unit are consecutive; the last
            // one to get here merges them in order
            const int f = static_cast<int>(div_short(cs.line0, quota));
            const int e = static_cast<int>(div_short(cs.line0 + cs.nchunk - 1, quota));
            __threadfence();
            __syncthreads();
            if (tid == 0) last_s = atomicAdd(&p.counters[cs.b * p.Hkv + cs.hk], 1) == e - f;
            __syncthreads();
            if (last_s) {
                __threadfence();
                auto piece = [&](int cta) { return 2 * cta + (cs.line0 <= quota * cta ? 0 : 1); };
                // maxima and sums: a warp for each row, a lane for each piece
                for (int r = warp; r < nrow; r += C::W) {
                    float M = -CUDART_INF_F, L = 0.f;
                    for (int cta = f + lane; cta <= e; cta += 32)
                        M = fmaxf(M, __ldcg(&p.pm[piece(cta) * kPagedMaxRows + r]));
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
                    for (int cta = f + lane; cta <= e; cta += 32) {
                        const float mc = __ldcg(&p.pm[piece(cta) * kPagedMaxRows + r]);
                        L = fmaf(mc == -CUDART_INF_F ? 0.f : ex2_approx(mc - M),
                                 __ldcg(&p.pl[piece(cta) * kPagedMaxRows + r]), L);
                    }
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
                    if (lane == 0) {
                        ml[r] = make_float2(M, L == 0.f ? 0.f : 1.f / L);
                        const int tok = p.by_g.div(r), hq = cs.hk * p.G + r - tok * p.G;
                        p.lse[static_cast<size_t>(hq) * p.total + cs.tok0 + tok] = lse_of(M, L);
                    }
                }
                __syncthreads();
                // outputs: a thread for four columns of a row
                for (int x = tid; x < nrow * (D / 4); x += C::THREADS) {
                    const int r = x / (D / 4), c4 = x - r * (D / 4);
                    const float M = ml[r].x;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                    for (int cta = f; cta <= e; ++cta) {
                        const int sl = piece(cta);
                        const float mc = __ldcg(&p.pm[sl * kPagedMaxRows + r]);
                        const float4 v = __ldcg(reinterpret_cast<const float4*>(
                                                    p.po + (static_cast<size_t>(sl) * kPagedMaxRows + r) * D) + c4);
                        const float w = mc == -CUDART_INF_F ? 0.f : ex2_approx(mc - M);
                        acc.x = fmaf(w, v.x, acc.x);
                        acc.y = fmaf(w, v.y, acc.y);
                        acc.z = fmaf(w, v.z, acc.z);
                        acc.w = fmaf(w, v.w, acc.w);
                    }
                    const int tok = p.by_g.div(r), hq = cs.hk * p.G + r - tok * p.G;
                    const float iL = ml[r].y;
                    *reinterpret_cast<uint2*>(p.o + (static_cast<size_t>(cs.tok0 + tok) * p.Hq + hq) * D + c4 * 4) =
                        make_uint2(pack_bf16x2(acc.x * iL, acc.y * iL), pack_bf16x2(acc.z * iL, acc.w * iL));
                }
            }
        }
        work = next(cs);
        __syncthreads();
    }
    cp_async_wait<0>();
    // after a wait that gave up: let the copies still in flight land before
    // leaving (otherwise every copy requested has been consumed)
    for (int u = consumed; u < issued; ++u)
        mbar_wait_teardown(&bars[u % C::STAGES], (u / C::STAGES) & 1, 200000000ull);
}

template <int D, int NT, bool B16>
static cudaError_t launch_split(const PagedArgs& a, const PagedParams& p, cudaStream_t stream) {
    using C = PgCfg<D, NT, B16>;
    const uint64_t rows = static_cast<uint64_t>(a.num_blocks) * a.Hkv * a.block_size * D / 128;
    const uint32_t box = C::BOX / 128;
    CUtensorMap tk, tv;
    if (!make_tmap_2d_sw128(&tk, a.k_cache, rows, 128, 1, box, 128) ||
        !make_tmap_2d_sw128(&tv, a.v_cache, rows, 128, 1, box, 128))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = once_per_device(done, [] {
        return cudaFuncSetAttribute(fa_paged_split_kernel<D, NT, B16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    C::SMEM);
    });
    if (e != cudaSuccess) return e;
    fa_paged_split_kernel<D, NT, B16><<<kPagedCtas, C::THREADS, C::SMEM, stream>>>(tk, tv, p);
    return cudaGetLastError();
}

template <int D>
static cudaError_t launch_split_d(const PagedArgs& a, const PagedParams& p, cudaStream_t stream) {
    const bool b16 = a.block_size == 16;
    const int rows = p.split_rows;
    if (rows <= 8) return b16 ? launch_split<D, 1, true>(a, p, stream) : launch_split<D, 1, false>(a, p, stream);
    if (rows <= 16) return b16 ? launch_split<D, 2, true>(a, p, stream) : launch_split<D, 2, false>(a, p, stream);
    if constexpr (D == 64)
        if (rows > 24) return b16 ? launch_split<D, 4, true>(a, p, stream) : launch_split<D, 4, false>(a, p, stream);
    return b16 ? launch_split<D, 3, true>(a, p, stream) : launch_split<D, 3, false>(a, p, stream);
}

cudaError_t launch_fwd_paged(const PagedArgs& a, cudaStream_t stream, int* nlaunch) {
    PagedParams p;
    p.q = static_cast<const uint16_t*>(a.q);
    p.k_scale = a.k_scale;
    p.v_scale = a.v_scale;
    p.o = static_cast<uint16_t*>(a.o);
    p.lse = a.lse;
    p.cu_seqlens = a.cu_seqlens;
    p.cache_len = a.cache_len;
    p.block_table = a.block_table;
    p.B = a.B;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.G = a.Hq / a.Hkv;
    p.by_g = make_fast_div(p.G);
    p.split_rows = paged_split_rows(a.max_new, p.G, a.d);
    p.total = a.total;
    p.max_new = a.max_new;
    p.max_blocks = a.max_blocks;
    p.num_blocks = a.num_blocks;
    p.bs_log2 = 0;
    while ((1 << p.bs_log2) < a.block_size) ++p.bs_log2;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.causal = a.causal;
    p.status = a.status;
    p.counters = a.counters;
    p.pm = a.pm;
    p.pl = a.pl;
    p.po = a.po;
    if (a.ev_begin) cudaEventRecord(a.ev_begin, stream);
    cudaError_t e = a.d == 64 ? launch_split_d<64>(a, p, stream) : launch_split_d<128>(a, p, stream);
    *nlaunch = 1;
    if (e == cudaSuccess && paged_has_tiles(a.max_new, p.G, a.d)) {
        e = launch_paged_tile(a, stream);
        *nlaunch = 2;
    }
    if (a.ev_end) cudaEventRecord(a.ev_end, stream);
    return e;
}

}  // namespace fa
