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
// wait for the block table in front of each copy.
//
// Design:
//   * Work is counted in chunks of 32 keys. A unit is (request, key head), with
//     at most RT = 8, 16 or 32 query rows (fa_paged_tile.cu takes requests of
//     more); the units' chunks form one line that is cut into
//     equal quotas, one for each persistent CTA, so ragged lengths balance by
//     themselves and one long request spreads over the whole GPU. A unit that
//     was cut leaves partial (m, l, O) in the workspace and the CTA that
//     finishes last merges them, in the order of the CTAs (the same result
//     every time).
//   * Each of a CTA's eight warps streams its own chunks (every eighth one)
//     through its own ring of TMA boxes with its own mbarriers: no barrier
//     between warps before a unit ends. Block ids and scales are fetched for
//     32 chunks at once, a lane for each.
//   * S^T = K Q^T and O^T = V^T P^T as m16n8k16 products with f16 operands
//     and fp32 sums, keys respectively head columns along M, the query rows
//     along N: eight rows cost no more than one. E4M3 converts to f16 exactly,
//     and Q does up to 2^-25 of its row's maximum after a power of two is
//     taken out of each row. The k index of either product may be permuted
//     freely: K rows are read sixteen bytes a lane as they lie, and V's bytes
//     of two keys are interleaved by a byte permute; the permutations are
//     chosen so that no read of the 128-byte-swizzled tiles meets a bank
//     conflict.
//   * P is rounded to f16 relative to 2^-6 of the running reference maximum,
//     which only moves when a row grows by more than 2^8: weights keep their
//     11 bits down to 2^-20 of the maximum and vanish below 2^-30.
//   * ks multiplies S, vs the product of each chunk: neither scale is folded
//     into an 8- or 16-bit number.
#include <math_constants.h>

#include "fa_paged.h"
#include "sm103_ptx.cuh"
#include "tmap.h"

namespace fa {

constexpr float kPgLn2 = 0.69314718055994530942f;
constexpr float kPgRescale = 8.0f;  // log2 units
constexpr float kPgOffset = 6.0f;   // log2 of the factor on P before its rounding to f16
constexpr int kPgChunk = 32;        // keys of a chunk
constexpr int kPgWarps = 8;

template <int D, int NT, bool B16>
struct PgCfg {
    static constexpr int RT = 8 * NT;                     // query rows of a tile
    static constexpr int STAGES = NT == 4 ? 2 : (D == 64 ? 5 : 3);
    static constexpr int TILE = kPgChunk * D;             // bytes of a chunk's K (or V)
    static constexpr int SUBS = B16 ? 2 : 1;              // boxes of a tile
    static constexpr int BOX = TILE / SUBS;
    static constexpr int KK = D / 16;                     // k steps of S
    static constexpr int MI = D / 16;                     // m tiles of O^T
    static constexpr int RED_F = 4 * NT * 32;             // floats of one m tile of a warp's O^T
    static constexpr int RED_M = 4 / NT > 0 ? 4 / NT : 1; // m tiles merged at a time
    static constexpr int RING_OFF = 0;
    static constexpr int RING = kPgWarps * STAGES * 2 * TILE;
    static constexpr int RED_OFF = RING_OFF + RING;       // fp32 [8 warps][RED_M][RED_F]
    static constexpr int Q_OFF = RED_OFF + kPgWarps * RED_M * RED_F * 4;  // f16 fragments of Q
    static constexpr int ML_OFF = Q_OFF + RT * D * 2;     // fp32 [8 warps][RT][2]
    static constexpr int ROW_OFF = ML_OFF + kPgWarps * RT * 8;  // {score factor, visible keys} of each row
    static constexpr int META_OFF = ROW_OFF + RT * 8;     // float4 [8 warps][STAGES]: ks0, ks1, vs0, vs1
    static constexpr int NAN_OFF = META_OFF + kPgWarps * STAGES * 16;  // int [D] first key with a NaN value
    static constexpr int BAR_OFF = NAN_OFF + D * 4;
    static constexpr int USED = BAR_OFF + kPgWarps * STAGES * 8 + 64;
    static constexpr int SMEM = USED + 1024;
    static_assert(SMEM <= 232448 - 2048, "shared memory");
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
    long long line0;    // position of the unit's first chunk on the line of all chunks
};

// Loads request b (sizes clamped to what the tables can hold).
__device__ __forceinline__ void pg_request(const PagedParams& p, int b, PgSeg& s) {
    const int t0 = min(max(p.cu_seqlens[b], 0), p.total), t1 = min(max(p.cu_seqlens[b + 1], t0), p.total);
    s.tok0 = t0;
    s.n = min(t1 - t0, p.max_new);
    if (static_cast<long long>(s.n) * p.G > kPagedMaxRows) s.n = 0;
    s.len = min(max(p.cache_len[b], 0), p.max_blocks << p.bs_log2);
    s.nchunk = s.n > 0 ? max(1, (s.len + kPgChunk - 1) / kPgChunk) : 0;
}

template <int D, int NT, bool B16>
__global__ void __launch_bounds__(256, 1)
    fa_paged_split_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                          const __grid_constant__ PagedParams p) {
    using C = PgCfg<D, NT, B16>;
    constexpr int RT = C::RT;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ long long scan_w[kPgWarps];
    __shared__ int start_b, last_s;
    __shared__ long long start_line;
    __shared__ int nan_seen, abort_s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;

    // ---- the line of chunks: total length, and the request at this CTA's start
    const int per = (p.B + 255) / 256;
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
    long long iw = mw;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, iw, off);
        if (lane >= off) iw += a;
    }
    if (lane == 31) scan_w[warp] = iw;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::BAR_OFF) + warp * C::STAGES;
    if (tid == 0) {
        abort_s = 0;
        nan_seen = 0;
        for (int i = 0; i < kPgWarps * C::STAGES; ++i) mbar_init(reinterpret_cast<uint64_t*>(sm + C::BAR_OFF) + i, 1);
        fence_barrier_init();
    }
    int* first_nan = reinterpret_cast<int*>(sm + C::NAN_OFF);
    for (int i = tid; i < D; i += 256) first_nan[i] = INT_MAX;
    __syncthreads();
    long long W = 0, bw = 0;
    for (int w = 0; w < kPgWarps; ++w) {
        if (w < warp) bw += scan_w[w];
        W += scan_w[w];
    }
    // equal quotas, at least one chunk for each warp
    long long quota = (W + gridDim.x - 1) / gridDim.x;
    quota = quota < kPgWarps ? kPgWarps : quota;
    const long long x0 = quota * blockIdx.x, x1 = min(x0 + quota, W);
    if (x0 >= x1) return;  // uniform over the CTA
    bw += iw - mw;
    if (x0 >= bw && x0 < bw + mw) {
        for (int b = b0; b < b1; ++b) {
            PgSeg s;
            pg_request(p, b, s);
            const long long w = static_cast<long long>(p.Hkv) * s.nchunk;
            if (x0 < bw + w) {
                start_b = b;
                start_line = bw;
                break;
            }
            bw += w;
        }
    }
    __syncthreads();

    // the piece that starts at position x of the line, given a request at or
    // before it (which starts at rline)
    auto place = [&](PgSeg& s, long long& rline, long long x) {
        for (;;) {
            const long long w = static_cast<long long>(p.Hkv) * s.nchunk;
            if (x < rline + w) break;
            rline += w;
            ++s.b;
            pg_request(p, s.b, s);
        }
        const long long r = x - rline;
        s.hk = static_cast<int>(r / s.nchunk);
        s.c0 = static_cast<int>(r - static_cast<long long>(s.hk) * s.nchunk);
        s.line0 = x - s.c0;
        s.c1 = static_cast<int>(min(static_cast<long long>(s.nchunk), x1 - s.line0));
    };
    PgSeg cs, is;  // pieces being consumed and being requested
    long long crl = start_line, irl = start_line;
    cs.b = is.b = start_b;
    pg_request(p, cs.b, cs);
    pg_request(p, is.b, is);
    place(cs, crl, x0);
    place(is, irl, x0);

    const WaitCtx cx{reinterpret_cast<volatile int*>(&abort_s), p.status};
    uint8_t* ring = sm + C::RING_OFF + warp * C::STAGES * 2 * C::TILE;
    float4* meta = reinterpret_cast<float4*>(sm + C::META_OFF) + warp * C::STAGES;
    // ---- requests of this warp: chunk c0 + warp + 8 k of each piece
    int ik = 0, issued = 0, consumed = 0;
    bool idone = false;
    float bks[C::SUBS], bvs[C::SUBS];  // batch of 32 of them: block ids and scales, a lane each
    int bid[C::SUBS];
    auto fetch = [&]() {
        const int c = is.c0 + warp + kPgWarps * (ik + lane);
#pragma unroll
        for (int u = 0; u < C::SUBS; ++u) {
            bid[u] = 0;
            bks[u] = bvs[u] = 0.f;
            const int key = c * kPgChunk + u * 16;
            if (c < is.c1 && key < is.len) {
                const int id = p.block_table[static_cast<size_t>(is.b) * p.max_blocks + (key >> p.bs_log2)];
                if (id >= 0 && id < p.num_blocks) {
                    bid[u] = id;
                    bks[u] = p.k_scale[static_cast<size_t>(id) * p.Hkv + is.hk];
                    bvs[u] = p.v_scale[static_cast<size_t>(id) * p.Hkv + is.hk];
                } else {
                    atomicCAS(p.status, 0, FA_DEV_INVALID | (91 << 8));
                }
            }
        }
    };
    fetch();
    auto issue = [&]() {
        // the next chunk, if this warp has one
        while (!idone && is.c0 + warp + kPgWarps * ik >= is.c1) {
            const long long x = is.line0 + is.c1;
            if (x >= x1) {
                idone = true;
                break;
            }
            place(is, irl, x);
            ik = 0;
            fetch();
        }
        if (idone) return;
        const int c = is.c0 + warp + kPgWarps * ik, st = issued % C::STAGES;
        if (lane == (ik & 31)) {
            meta[st] = make_float4(bks[0], bks[C::SUBS - 1], bvs[0], bvs[C::SUBS - 1]);
            mbar_arrive_expect_tx(&bars[st], 2 * C::TILE);
#pragma unroll
            for (int u = 0; u < C::SUBS; ++u) {
                // rows of the [num_blocks * Hkv * block_size * d / 128, 128] matrix
                const int in = B16 ? 0 : (c * kPgChunk) & ((1 << p.bs_log2) - 1);
                const long long key = (static_cast<long long>(bid[u]) * p.Hkv + is.hk << p.bs_log2) + in;
                const int row = static_cast<int>(D == 128 ? key : key >> 1);
                tma_load_2d(ring + (2 * st) * C::TILE + u * C::BOX, &tmK, 0, row, &bars[st]);
                tma_load_2d(ring + (2 * st + 1) * C::TILE + u * C::BOX, &tmV, 0, row, &bars[st]);
            }
        }
        __syncwarp();
        ++issued;
        ++ik;
        if ((ik & 31) == 0) fetch();
    };
#pragma unroll 1
    for (int i = 0; i < C::STAGES; ++i) issue();

    uint8_t* qs = sm + C::Q_OFF;
    float2* rowc = reinterpret_cast<float2*>(sm + C::ROW_OFF);
    float2* ml = reinterpret_cast<float2*>(sm + C::ML_OFF);
    float* red = reinterpret_cast<float*>(sm + C::RED_OFF);
    bool ok = true;

#pragma unroll 1
    for (;;) {
        // ---------------------------------------------------- the piece's rows
        const int nrow = cs.n * p.G;  // rows of the request: token * G + head of the group
        // visible keys of the first and the last row
        auto visible = [&](int tok) { return p.causal ? min(max(cs.len - cs.n + tok + 1, 0), cs.len) : cs.len; };
        const int vis_min = visible(0), vis_max = visible(cs.n - 1);
        for (int r = warp; r < RT; r += kPgWarps) {
            // four values per lane; the row's power of two goes to its score factor
            uint2 x = make_uint2(0u, 0u);
            const int tok = r / p.G;
            if (r < nrow && lane < D / 4)
                x = *reinterpret_cast<const uint2*>(
                    p.q + (static_cast<size_t>(cs.tok0 + tok) * p.Hq + cs.hk * p.G + (r - tok * p.G)) * D + lane * 4);
            const uint32_t h4[4] = {x.x & 0xFFFFu, x.x >> 16, x.y & 0xFFFFu, x.y >> 16};
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t a = h4[i] & 0x7FFFu;
                top = max(top, a < 0x7F80u ? a : 0u);
            }
            top = __reduce_max_sync(0xffffffffu, top);
            const int e = top >> 7 ? min(max(static_cast<int>(top >> 7) - 127, -120), 120) : 0;
            const float f = exp2i(-e);
            if (lane < D / 4) {
                const int half = lane >> 4, tq = (lane >> 2) & 3, kk = half * 4 + (lane & 3);
                uint2 y;
                y.x = pack_f16x2(__uint_as_float(h4[0] << 16) * f, __uint_as_float(h4[1] << 16) * f);
                y.y = pack_f16x2(__uint_as_float(h4[2] << 16) * f, __uint_as_float(h4[3] << 16) * f);
                *reinterpret_cast<uint2*>(qs + (((r >> 3) * (C::KK / 2) + (kk >> 1)) * 32 + 4 * (r & 7) + tq) * 16 +
                                          (kk & 1) * 8) = y;
            }
            if (lane == 0) rowc[r] = make_float2(p.scale_log2 * exp2i(e), __int_as_float(r < nrow ? visible(tok) : cs.len));
        }
        __syncthreads();
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
#pragma unroll 1
        for (int c = cs.c0 + warp; c < cs.c1; c += kPgWarps) {
            const int st = consumed % C::STAGES;
            ok = mbar_wait_warp(&bars[st], (consumed / C::STAGES) & 1, cx, 92);
            if (!ok) break;
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
            uint32_t vw[2][4][D / 32];
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int j = ks * 16 + (r >> 1) * 8 + pg_key<D>(2 * t4 + (r & 1));
                    if constexpr (D == 128) {
                        const uint4 x = lds128_u4(vb + pg_off<D>(j, g));
                        vw[ks][r][0] = x.x;
                        vw[ks][r][1] = x.y;
                        vw[ks][r][2] = x.z;
                        vw[ks][r][3] = x.w;
                    } else {
                        const uint2 x = lds64(vb + pg_off<D>(j, g >> 1) + (g & 1) * 8);
                        vw[ks][r][0] = x.x;
                        vw[ks][r][1] = x.y;
                    }
                }
            if (edge) {
                // keys that no row sees count as zero whatever their bytes are;
                // a NaN that only some rows see is taken out here and given
                // back to those rows at the end
#pragma unroll
                for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int key = key0 + ks * 16 + (r >> 1) * 8 + pg_key<D>(2 * t4 + (r & 1));
#pragma unroll
                        for (int w = 0; w < D / 32; ++w) {
                            if (key >= vis_max) vw[ks][r][w] = 0u;
                            const uint32_t nb = e4m3_nan_bits(vw[ks][r][w]);
                            if (nb) {
                                nan_seen = 1;
#pragma unroll
                                for (int y = 0; y < 4; ++y)
                                    if ((nb >> (8 * y)) & 0x80u) {
                                        atomicMin(&first_nan[g * (D / 8) + w * 4 + y], key);
                                        vw[ks][r][w] &= ~(0xFFu << (8 * y));
                                    }
                            }
                        }
                    }
            }
#pragma unroll
            for (int i = 0; i < C::MI; ++i) {
                float acc[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[nt][e] = 0.f;
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    const uint32_t sel = i & 1 ? 0x7362u : 0x5140u;
                    const uint32_t x = __byte_perm(vw[ks][0][i >> 1], vw[ks][1][i >> 1], sel);
                    const uint32_t y = __byte_perm(vw[ks][2][i >> 1], vw[ks][3][i >> 1], sel);
                    const uint32_t a0 = f16x2_from_e4m3x2(x), a1 = f16x2_from_e4m3x2(x >> 16);
                    const uint32_t a2 = f16x2_from_e4m3x2(y), a3 = f16x2_from_e4m3x2(y >> 16);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_f16(acc[nt], a0, a1, a2, a3, pb[ks][nt][0], pb[ks][nt][1]);
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
            ++consumed;
            __syncwarp();  // the stage has been read
            issue();
        }

        // ---------------------------------------------------- merge of the warps
        // row sums over the key lanes
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = l[nt][e];
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                x += __shfl_xor_sync(0xffffffffu, x, 8);
                x += __shfl_xor_sync(0xffffffffu, x, 16);
                if (g == 0) ml[warp * RT + nt * 8 + 2 * t4 + e] = make_float2(m[nt][e], x);
            }
        if (__syncthreads_or(!ok)) break;
        float fac[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float M = -CUDART_INF_F;
                for (int w = 0; w < kPgWarps; ++w) M = fmaxf(M, ml[w * RT + nt * 8 + 2 * t4 + e].x);
                fac[nt][e] = m[nt][e] == -CUDART_INF_F ? 0.f : ex2_approx(m[nt][e] - M);
            }
        const bool whole = cs.c0 == 0 && cs.c1 == cs.nchunk;
        const int slot = 2 * static_cast<int>(blockIdx.x) + (cs.line0 <= x0 ? 0 : 1);
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
            for (int x = tid; x < C::RED_M * C::RED_F; x += 256) {
                float sum = 0.f;
#pragma unroll
                for (int w = 0; w < kPgWarps; ++w) sum += red[w * C::RED_M * C::RED_F + x];
                const int ln = x & 31, q = x >> 5, e = q & 3, nt = (q >> 2) % NT, i = i0 + q / (4 * NT);
                const int r = nt * 8 + 2 * (ln & 3) + (e & 1);
                const int col = (ln >> 2) * (D / 8) + 2 * i + (e >> 1);
                float M = -CUDART_INF_F, L = 0.f;
                for (int w = 0; w < kPgWarps; ++w) M = fmaxf(M, ml[w * RT + r].x);
                for (int w = 0; w < kPgWarps; ++w) {
                    const float2 v = ml[w * RT + r];
                    L += v.y * (v.x == -CUDART_INF_F ? 0.f : ex2_approx(v.x - M));
                }
                if (nan_seen && first_nan[col] < __float_as_int(rowc[r].y)) sum = CUDART_NAN_F;
                if (whole) {
                    if (r < nrow) {
                        const int tok = r / p.G, hq = cs.hk * p.G + r - tok * p.G;
                        const float out = L == 0.f ? 0.f : sum / L;
                        p.o[(static_cast<size_t>(cs.tok0 + tok) * p.Hq + hq) * D + col] =
                            static_cast<uint16_t>(pack_bf16x2(out, 0.f) & 0xFFFFu);
                        if (col == 0)
                            p.lse[static_cast<size_t>(hq) * p.total + cs.tok0 + tok] =
                                L == 0.f ? -CUDART_INF_F : (M - kPgOffset + log2f(L)) * kPgLn2;
                    }
                } else {
                    p.po[(static_cast<size_t>(slot) * kPagedMaxRows + r) * D + col] = sum;
                    if (col == 0) {
                        p.pm[slot * kPagedMaxRows + r] = M;
                        p.pl[slot * kPagedMaxRows + r] = L;
                    }
                }
            }
            __syncthreads();
        }
        if (tid < D) first_nan[tid] = INT_MAX;
        if (tid == 0) nan_seen = 0;
        if (!whole) {
            // the CTAs that hold pieces of this unit are consecutive; the last
            // one to get here merges them in order
            const int f = static_cast<int>(cs.line0 / quota), e = static_cast<int>((cs.line0 + cs.nchunk - 1) / quota);
            __threadfence();
            __syncthreads();
            if (tid == 0) last_s = atomicAdd(&p.counters[cs.b * p.Hkv + cs.hk], 1) == e - f;
            __syncthreads();
            if (last_s) {
                __threadfence();
                for (int x = tid; x < nrow * D; x += 256) {
                    const int r = x / D, col = x - r * D;
                    float M = -CUDART_INF_F, L = 0.f, acc = 0.f;
                    for (int cta = f; cta <= e; ++cta) {
                        const int sl = 2 * cta + (cs.line0 <= quota * cta ? 0 : 1);
                        M = fmaxf(M, __ldcg(&p.pm[sl * kPagedMaxRows + r]));
                    }
                    for (int cta = f; cta <= e; ++cta) {
                        const int sl = 2 * cta + (cs.line0 <= quota * cta ? 0 : 1);
                        const float mc = __ldcg(&p.pm[sl * kPagedMaxRows + r]);
                        const float w = mc == -CUDART_INF_F ? 0.f : ex2_approx(mc - M);
                        L = fmaf(w, __ldcg(&p.pl[sl * kPagedMaxRows + r]), L);
                        acc = fmaf(w, __ldcg(&p.po[(static_cast<size_t>(sl) * kPagedMaxRows + r) * D + col]), acc);
                    }
                    const int tok = r / p.G, hq = cs.hk * p.G + r - tok * p.G;
                    const float out = L == 0.f ? 0.f : acc / L;
                    p.o[(static_cast<size_t>(cs.tok0 + tok) * p.Hq + hq) * D + col] =
                        static_cast<uint16_t>(pack_bf16x2(out, 0.f) & 0xFFFFu);
                    if (col == 0)
                        p.lse[static_cast<size_t>(hq) * p.total + cs.tok0 + tok] =
                            L == 0.f ? -CUDART_INF_F : (M - kPgOffset + log2f(L)) * kPgLn2;
                }
            }
        }
        const long long x = cs.line0 + cs.c1;
        if (x >= x1) break;
        place(cs, crl, x);
        __syncthreads();
    }
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
    cudaError_t e =
        cudaFuncSetAttribute(fa_paged_split_kernel<D, NT, B16>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    fa_paged_split_kernel<D, NT, B16><<<kPagedCtas, 256, C::SMEM, stream>>>(tk, tv, p);
    return cudaGetLastError();
}

template <int D>
static cudaError_t launch_split_d(const PagedArgs& a, const PagedParams& p, cudaStream_t stream) {
    const bool b16 = a.block_size == 16;
    const long long rows = static_cast<long long>(a.max_new) * p.G;
    if (rows <= 8) return b16 ? launch_split<D, 1, true>(a, p, stream) : launch_split<D, 1, false>(a, p, stream);
    if (rows <= 16) return b16 ? launch_split<D, 2, true>(a, p, stream) : launch_split<D, 2, false>(a, p, stream);
    return b16 ? launch_split<D, 4, true>(a, p, stream) : launch_split<D, 4, false>(a, p, stream);
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
    if (e == cudaSuccess && paged_has_tiles(a.max_new, p.G)) {
        e = launch_paged_tile(a, stream);
        *nlaunch = 2;
    }
    if (a.ev_end) cudaEventRecord(a.ev_end, stream);
    return e;
}

}  // namespace fa
