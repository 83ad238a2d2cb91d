// epilogue.hpp -- what a dense projection does to its float32 sums before it
// rounds them once: y = f(sum + bias) + residual.
#pragma once

#include "common.hpp"
#include "launch.hpp"

namespace wq {

// f in float32.  The sigmoid forms divide by 1 + exp(-2u), which passes to
// infinity where u does; a NaN stays one.  GELU is as good as erf is near -1, where
// float32's step is 2^-24: |z| 2^-24 of it, not of the value's own size (1.3e-4 at -4).
__device__ __forceinline__ float activate(float z, int f) {
    switch (f) {
        case ACT_RELU: return z < 0.0f ? 0.0f : z;
        case ACT_SILU: return silu_f32(z);
        case ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
        case ACT_GELU_TANH: {  // 0.5 z (1 + tanh u) = z / (1 + exp(-2 u)), u = sqrt(2 / pi) (z + 0.044715 z^3)
            const float u2 = 1.5957691216057308f * (z + 0.044715f * z * z * z);
            return z / (1.0f + __expf(-u2));
        }
        default: return z;
    }
}

// outputs n0 .. n0 + 3 of row m (n0 a multiple of 4) to y, whose rows are N long
template <bool BF16>
__device__ __forceinline__ void finish4(const Epilogue& ep, f32x4 o, int64_t m, int n0, int N, uint16_t* y) {
    if (ep.bias) {
        const u32x2 b = *reinterpret_cast<const u32x2*>(ep.bias + n0);
        const uint32_t lo = b[0], hi = b[1];
        o[0] += act_to_f32<BF16>((uint16_t)lo);
        o[1] += act_to_f32<BF16>((uint16_t)(lo >> 16));
        o[2] += act_to_f32<BF16>((uint16_t)hi);
        o[3] += act_to_f32<BF16>((uint16_t)(hi >> 16));
    }
    if (ep.act != ACT_NONE) {
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = activate(o[i], ep.act);
    }
    if (ep.residual || ep.in_place) {
        const u32x2 r = *reinterpret_cast<const u32x2*>(ep.in_place ? y + m * N + n0 : ep.residual + m * ep.r_stride + n0);
        const uint32_t lo = r[0], hi = r[1];
        o[0] += act_to_f32<BF16>((uint16_t)lo);
        o[1] += act_to_f32<BF16>((uint16_t)(lo >> 16));
        o[2] += act_to_f32<BF16>((uint16_t)hi);
        o[3] += act_to_f32<BF16>((uint16_t)(hi >> 16));
    }
    *reinterpret_cast<u32x2*>(y + m * N + n0) = u32x2{f32_to_act2<BF16>(o[0], o[1]), f32_to_act2<BF16>(o[2], o[3])};
}

}  // namespace wq
