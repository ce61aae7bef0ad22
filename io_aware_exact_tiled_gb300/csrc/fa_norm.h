// Internal interface of the per-head norm with rotation: forward and backward
// (fa_norm.cu) and the form that writes keys and values into the paged cache
// (fa_norm_append.cu). Arguments are already validated.
#pragma once

#include "fa_paged.h"

namespace fa {

// Rows of d elements: row (b, h, n) starts at data + b * batch + h * head + n * token.
struct NormRows {
    void* data;
    long long batch, head, token;  // in elements
};

constexpr int kNormThreads = 256;
constexpr int kNormBwdCtas = 2 * 152;  // partial sums of the weights' gradients

struct NormArgs {
    NormRows q, k;              // inputs
    NormRows q_out, k_out;      // forward: results; backward: upstream gradients
    NormRows dq, dk;            // backward: results
    const void *q_weight, *k_weight;  // [d] of the inputs' type, or null
    float *dq_weight, *dk_weight;     // [d], backward with weights
    const double* inv_freq;     // [rot / 2]
    const int32_t *cu_seqlens, *ends;  // packed batch: [B + 1]; null or [B]
    int B, N, tokens, Hq, Hkv, d, rot, interleaved, fp32;
    float eps;
    FastDiv by_n;  // division by N (dense batches)
    int* status;      // backward
    float* partial;   // backward: [kNormBwdCtas][2][d]
};

struct NormAppendArgs {
    NormArgs n;  // q, q_out and k; packed
    NormRows v;
    AppendArgs a;  // caches, scales and slots
};

cudaError_t launch_norm(const NormArgs& a, cudaStream_t stream, int* nlaunch);
cudaError_t launch_norm_bwd(const NormArgs& a, cudaStream_t stream, int* nlaunch);
cudaError_t launch_norm_append(const NormAppendArgs& a, cudaStream_t stream, int* nlaunch);

}  // namespace fa
