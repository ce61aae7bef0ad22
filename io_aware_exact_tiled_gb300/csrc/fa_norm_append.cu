// The norm and rotation of fa_norm.cu for new tokens of a serving step: queries
// to an array, keys and values to the paged 8-bit cache as the append of
// fa_cache.cu stores them (the key's input to that is the rotated key in bf16).
//
// Bound: the tokens' bytes in large batches, latency in small ones.
//
// The first CTAs take the runs (consecutive tokens whose slots lie in one block)
// that start among `span` tokens, for a group of heads and one of K and V; the
// others take the queries (in large batches the kernel of fa_norm.cu does). One or
// two runs, as in a prompt, are each the whole CTA's: rows come by asynchronous
// copies, HPC heads ahead, and stay in registers from their norm to their
// rounding, which waits for the run's largest value. More runs, as in a decoding
// batch, go to a warp each, which reads its rows twice.
//
// Measured: 128 requests of a token, 32 + 8 heads, 10 us; four prompts of 17,400
// tokens, 32 heads each, d = 128, blocks of 64: 220 us (874 MB: 129 at the copy
// rate), 62 of them the queries' kernel and 158 this one, whose sixteen warps on
// an SM issue in 48 % of the cycles. One head a CTA with its rows loaded directly
// took 290 us in all, four heads 232, with copies ahead and angles kept 220.
#include <type_traits>

#include "fa_append.cuh"
#include "fa_norm.cuh"

namespace fa {

constexpr int kNaSeqs = 1024;  // offsets kept in shared memory

template <int D, bool INTER, int L, int HPC>
__global__ void __launch_bounds__(256, 2)
    fa_norm_append_kernel(const __grid_constant__ NormAppendArgs args, int span, int hpc, int kv_ctas, int q_parts) {
    using LN = NormLane<D, INTER>;
    constexpr int ROWS = 256 / LN::TPR;  // rows of a CTA-wide load
    extern __shared__ __align__(16) uint4 ring[];
    __shared__ uint64_t turns[D / 2];
    __shared__ __align__(16) float weights[2 * D];
    __shared__ int cu_s[kNaSeqs];
    __shared__ int slot_s[513], pos_s[512];  // slot of tokens t0 - 1 .. (-1: none), position of tokens t0 ..
    __shared__ int leads[256], nlead;
    __shared__ uint32_t warp_top[HPC][8];
    const NormArgs& p = args.n;
    const AppendArgs& a = args.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    norm_tables<uint16_t, D, INTER>(p, turns, weights, tid, 256);
    if (static_cast<int>(blockIdx.x) >= kv_ctas) {
        __syncthreads();
        norm_forward<uint16_t, D, INTER>(p, turns, weights, ring, (blockIdx.x - kv_ctas) * 8 + warp,
                                         (gridDim.x - kv_ctas) * 8, q_parts, warp, lane);
        return;
    }
    const int groups = (a.H + hpc - 1) / hpc;
    // the heads of a span follow one another: they share its rows' DRAM pages
    const int part = static_cast<int>(blockIdx.x / (2u * groups));
    const int gv = static_cast<int>(blockIdx.x - part * (2u * groups));
    const int h0 = (gv >> 1) * hpc, nh = min(hpc, a.H - h0);
    const int bs = a.block_size, nslots = a.num_blocks * bs, bs_log2 = 31 - __clz(bs);
    const bool is_v = gv & 1;
    const long long t0 = static_cast<long long>(part) * span;
    const bool near = p.B < kNaSeqs;
    if (near)
        for (int i = tid; i <= p.B; i += 256) cu_s[i] = p.cu_seqlens[i];
    if (tid == 0) nlead = 0;
    __syncthreads();
    const int* cu = near ? cu_s : p.cu_seqlens;
    int* slot_of = slot_s + 1;
    // slots and positions of the span's tokens, of the one in front of them and
    // of those that the last run may reach; a token of no sequence has none
    for (int i = tid - 1; i < span + bs; i += 256) {
        const long long t = t0 + i;
        int slot = -1;
        if (t >= 0 && t < a.total) {
            const int s = a.slots[t];
            int lo = 0, hi = p.B;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cu[mid] <= t) lo = mid;
                else hi = mid;
            }
            if (s >= 0 && s < nslots && cu[lo] <= t && t < cu[lo + 1]) {
                slot = s;
                if (i >= 0) pos_s[i] = packed_position(p, lo, static_cast<int>(t));
            }
        }
        slot_of[i] = slot;
    }
    __syncthreads();
    auto blk_of = [&](int i) { return slot_of[i] >> bs_log2; };
    if (tid < span && slot_of[tid] >= 0 && blk_of(tid) != blk_of(tid - 1)) leads[atomicAdd(&nlead, 1)] = tid;
    __syncthreads();
    const int n = nlead;
    if (n == 0) return;
    const LN ln(lane, p.rot);
    const float* w = p.k_weight ? weights + D : nullptr;
    const NormRows& in = is_v ? args.v : p.k;
    auto source = [&](int h, int t) {
        return static_cast<const uint16_t*>(in.data) + h * in.head + (t0 + t) * in.token;
    };
    auto block_at = [&](int lead, int h) { return static_cast<size_t>(blk_of(lead)) * a.H + h; };
    auto cache_at = [&](int lead, int h) { return (is_v ? a.v_cache : a.k_cache) + block_at(lead, h) * bs * D; };
    auto scale_at = [&](int lead, int h) { return (is_v ? a.v_scale : a.k_scale) + block_at(lead, h); };
    auto run_end = [&](int lead) {  // first token behind the run, as far as slot_of reaches (block_size tokens)
        const int blk = blk_of(lead);
        for (int e = lead + 1;; e += 32) {
            const int i = e + lane;
            const uint32_t same = __ballot_sync(0xffffffffu, i < min(lead + bs, span + bs) && blk_of(i) == blk);
            if (same != 0xffffffffu) return e + __ffs(~same) - 1;
        }
    };
    auto turn_of = [&](int t, NormTurn& turn) {  // this lane's angles of token t
        const uint64_t pos = static_cast<uint64_t>(static_cast<int64_t>(pos_s[t]));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float c[2], s[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int at = ln.freq(2 * i + y);
                turn_cos_sin(pos * (at < p.rot / 2 ? turns[at] : 0ull), c[y], s[y]);
            }
            turn.c[i] = f2_make(c[0], c[1]);
            turn.s[i] = f2_make(s[0], s[1]);
        }
    };
    auto finish = [&](NormRaw<uint16_t>& raw, const NormTurn& turn) {  // a row of K, in bf16
        NormVec x;
        raw.get<INTER>(x);
        norm_row<D, INTER>(x, w, ln, p.eps, turn);
        raw.set<INTER>(x);
    };
    auto store = [&](uint8_t* row, const NormRaw<uint16_t>& raw, float inv) {
        *reinterpret_cast<uint2*>(row + ln.a) = append_quantise(raw.w[0], inv);
        *reinterpret_cast<uint2*>(row + ln.b) = append_quantise(raw.w[1], inv);
    };
    if (n <= 2) {
        // ------------------------------------------------ the CTA takes the runs in turn,
        // HPC heads at a time; a lane's angles stay in shared memory for the next ones
        const int row = tid / LN::TPR;
        constexpr bool KEEP = L <= 2;
        // rows of the heads to come, on their way; each lane reads what it copied
        uint4* stage = ring + tid;  // [L][HPC][2][256]
        ulonglong2* kept = reinterpret_cast<ulonglong2*>(ring + L * HPC * 512) + tid;  // [L][4][256]
        for (int k = 0; k < n; ++k) {
            const int lead = leads[k], end = run_end(lead), first = slot_of[lead] & (bs - 1);
            auto request = [&](int i, int h1) {  // rows of set i, heads h1 ..
                const int t = lead + i * ROWS + row;
#pragma unroll
                for (int h = 0; h < HPC; ++h) {
                    if (t >= end || h1 + h >= h0 + nh) continue;
                    const uint16_t* src = source(h1 + h, t);
                    cp_async16(stage + ((i * HPC + h) * 2) * 256, src + ln.a);
                    cp_async16(stage + ((i * HPC + h) * 2 + 1) * 256, src + ln.b);
                }
            };
#pragma unroll
            for (int i = 0; i < L; ++i) request(i, h0);
            cp_async_commit();
            for (int h1 = h0; h1 < h0 + nh; h1 += HPC) {
                const int mh = min(HPC, h0 + nh - h1);
                NormRaw<uint16_t> raw[L][HPC];
                uint32_t top[HPC];
                float old[HPC];
#pragma unroll
                for (int h = 0; h < HPC; ++h) {
                    top[h] = 0;
                    old[h] = first > 0 && h < mh ? append_old_scale(scale_at(lead, h1 + h)) : 0.f;
                }
                cp_async_wait<0>();
#pragma unroll
                for (int i = 0; i < L; ++i) {
                    const int t = lead + i * ROWS + row;
#pragma unroll
                    for (int h = 0; h < HPC; ++h) {
                        raw[i][h].zero();
                        if (t < end && h < mh) {
                            raw[i][h].w[0] = stage[((i * HPC + h) * 2) * 256];
                            raw[i][h].w[1] = stage[((i * HPC + h) * 2 + 1) * 256];
                        }
                    }
                    if (!is_v) {
                        NormTurn turn;
                        if (!KEEP || h1 == h0) {
                            turn_of(min(t, end - 1), turn);
                            if (KEEP) {
#pragma unroll
                                for (int y = 0; y < 4; ++y)
                                    kept[(i * 4 + y) * 256] = make_ulonglong2(turn.c[y], turn.s[y]);
                            }
                        } else {
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const ulonglong2 v = kept[(i * 4 + y) * 256];
                                turn.c[y] = v.x;
                                turn.s[y] = v.y;
                            }
                        }
#pragma unroll
                        for (int h = 0; h < HPC; ++h) finish(raw[i][h], turn);
                    }
#pragma unroll
                    for (int h = 0; h < HPC; ++h) top[h] = append_amax(raw[i][h].w, top[h]);
                    request(i, h1 + HPC);  // into the place of the rows just taken
                }
                cp_async_commit();
#pragma unroll
                for (int h = 0; h < HPC; ++h) {
                    top[h] = __reduce_max_sync(0xffffffffu, top[h]);
                    if (lane == 0) warp_top[h][warp] = top[h];
                }
                __syncthreads();  // every thread has read the scales so far, too
                float inv[HPC];
#pragma unroll
                for (int h = 0; h < HPC; ++h) {
#pragma unroll
                    for (int x = 0; x < 8; ++x) top[h] = max(top[h], warp_top[h][x]);
                    const float s = append_scale(top[h], old[h]);
                    inv[h] = 1.f / s;  // a power of two: exact
                    if (h < mh) {
                        if (first > 0 && s != old[h])
                            append_move(cache_at(lead, h1 + h), first * D, old[h] / s, tid, 256);
                        if (tid == 0) *scale_at(lead, h1 + h) = s;
                    }
                }
                // the run's own rows, after the moved ones of a slot that it writes
                // again; and the maxima have been read
                __syncthreads();
#pragma unroll
                for (int i = 0; i < L; ++i) {
                    const int t = lead + i * ROWS + row;
#pragma unroll
                    for (int h = 0; h < HPC; ++h)
                        if (t < end && h < mh)
                            store(cache_at(lead, h1 + h) + (slot_of[t] & (bs - 1)) * D, raw[i][h], inv[h]);
                }
            }
        }
        cp_async_wait<0>();
        return;
    }
    // ---------------------------------------------------- a warp for each run and head
    for (int k = warp; k < n * nh; k += 8) {
        const int x = k / nh, h = h0 + k - x * nh;
        const int lead = leads[x], end = run_end(lead), first = slot_of[lead] & (bs - 1);
        const float old = first > 0 ? append_old_scale(scale_at(lead, h)) : 0.f;
        NormRaw<uint16_t> raw;
        auto take = [&](int t) {  // row t of the run
            raw.zero();
            if (t < end) raw.load(source(h, t), ln.a, ln.b);
            if (is_v) return;
            NormTurn turn;
            turn_of(min(t, end - 1), turn);
            finish(raw, turn);
        };
        uint32_t top = 0;
        const int last = lead + (end - 1 - lead) / LN::RPW * LN::RPW;  // first row of the last step
        for (int t = lead; t <= last; t += LN::RPW) {
            take(t + ln.g);
            top = append_amax(raw.w, top);
        }
        top = __reduce_max_sync(0xffffffffu, top);
        const float s = append_scale(top, old), inv = 1.f / s;
        uint8_t* cache = cache_at(lead, h);
        if (first > 0 && s != old) append_move(cache, first * D, old / s, lane, 32);
        __syncwarp();
        if (lane == 0) *scale_at(lead, h) = s;
        for (int t = lead; t <= last; t += LN::RPW) {
            if (lead != last) take(t + ln.g);  // a run of one step is still there
            if (t + ln.g < end) store(cache + (slot_of[t + ln.g] & (bs - 1)) * D, raw, inv);
        }
    }
}

template <int D, bool INTER, int L>
static cudaError_t launch(const NormAppendArgs& a, cudaStream_t stream, int* nlaunch) {
    constexpr int HPC = L >= 8 ? 1 : L == 4 ? 2 : 4;
    const int total = a.a.total, passes = (a.n.Hq * (D / 16) + 31) / 32;
    const int span = total > 8192 && a.a.block_size * D <= 2048 ? 128 : total > 1024 ? 64 : 16;
    const bool big = total > 1024;
    const int hpc = big ? 4 * HPC : 1;
    constexpr int kStage = L * HPC * 8192 + (L <= 2 ? L * 16384 : 0);
    constexpr int kSmem = kStage > kNormRing<uint16_t> ? kStage : kNormRing<uint16_t>;
    const unsigned kv = static_cast<unsigned>((total + span - 1) / span) * 2u * ((a.a.H + hpc - 1) / hpc);
    int parts = (152 * 16 + total - 1) / total;
    parts = parts > passes ? passes : parts;
    const long long want = (static_cast<long long>(total) * parts + 7) / 8;
    unsigned qc = static_cast<unsigned>(want < 152 * 8 ? want : 152 * 8);
    static std::atomic<uint64_t> done{0};
    cudaError_t e = once_per_device(done, [] {
        return cudaFuncSetAttribute(fa_norm_append_kernel<D, INTER, L, HPC>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    });
    if (e == cudaSuccess && big) {  // the queries in a kernel of their own, with more warps on an SM
        int n;
        e = launch_norm(a.n, stream, &n);
        qc = 0;
        *nlaunch = 2;
    }
    if (e != cudaSuccess) return e;
    fa_norm_append_kernel<D, INTER, L, HPC>
        <<<kv + qc, 256, kSmem, stream>>>(a, span, hpc, static_cast<int>(kv), parts);
    return cudaGetLastError();
}

cudaError_t launch_norm_append(const NormAppendArgs& a, cudaStream_t stream, int* nlaunch) {
    auto rows = [&](auto inter) -> cudaError_t {
        constexpr bool INTER = decltype(inter)::value;
        const int bs = a.a.block_size;
        if (a.n.d == 64) {
            if (bs <= 64) return launch<64, INTER, 1>(a, stream, nlaunch);
            if (bs == 128) return launch<64, INTER, 2>(a, stream, nlaunch);
            return launch<64, INTER, 4>(a, stream, nlaunch);
        } else {
            if (bs <= 32) return launch<128, INTER, 1>(a, stream, nlaunch);
            if (bs == 64) return launch<128, INTER, 2>(a, stream, nlaunch);
            if (bs == 128) return launch<128, INTER, 4>(a, stream, nlaunch);
            return launch<128, INTER, 8>(a, stream, nlaunch);
        }
    };
    *nlaunch = 1;
    return a.n.interleaved ? rows(std::true_type{}) : rows(std::false_type{});
}

}  // namespace fa
