// Pieces of the appends to the paged 8-bit cache: a run's scale, its rounding,
// and the move of rows that a block holds already.
#pragma once

#include <math_constants.h>

#include "fa_paged.h"
#include "sm103_ptx.cuh"

namespace fa {

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

}  // namespace fa
