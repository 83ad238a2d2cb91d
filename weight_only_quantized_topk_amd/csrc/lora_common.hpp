// lora_common.hpp -- pieces of the low-rank adapter kernels (lora.hip for small
// batches, lora_wide.hip for large ones).
#pragma once

#include "common.hpp"
#include "launch.hpp"

namespace wq {

// The wave's index as a scalar: what is decided by it is a branch of the whole
// wave (a matrix instruction does not look at the lanes' mask, so one under a
// lane-wise condition would run all the same)
__device__ __forceinline__ int wave_index() { return __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6); }

// The adapters of a tile of up to 64 tokens: lane i holds token i's (-1: none, an
// id out of range counts as none).  A pass takes the adapter of the first token
// that is left and all tokens that share it (`mine`).
template <int TOKENS>
__device__ __forceinline__ int tile_ids(const LoraArgs& g, int tile, int lane) {
    const int m = tile * TOKENS + lane;
    const int id = lane < TOKENS && m < g.M ? g.ids[m] : -1;
    return id < g.adapters ? max(id, -1) : -1;
}
__device__ __forceinline__ int next_adapter(int ids, uint64_t& left, uint64_t& mine) {
    const int a = __builtin_amdgcn_readlane(ids, __builtin_ctzll(left));
    mine = __ballot(ids == a);
    left &= ~mine;
    return a;
}

// One token's t by 8 threads (neighbouring lanes, gr = 0 .. 7, ranks 64 w + 8
// gr .. + 7): the K slices added up, scaled by a power of two to at most 1 and
// split in high and low 16-bit parts, put(w, hi, lo).  Returns what the
// products have to be multiplied by: the power back, times the adapter's scale.
template <bool BF16, int RG, class PUT>
__device__ __forceinline__ float split_token(const LoraArgs& g, int m, int gr, PUT put) {
    const int id = g.ids[m];
    const float scale = g.scales && id >= 0 && id < g.adapters ? g.scales[id] : 1.0f;
    const float* src = g.t + (size_t)m * g.R;
    float v[RG][8];
    float top = 0.0f;
#pragma unroll
    for (int w = 0; w < RG; ++w) {
        const int rank = 64 * w + 8 * gr;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[w][i] = 0.0f;
        if (rank < g.R) {
#pragma unroll 4
            for (int z = 0; z < g.ks; ++z) {
                const f32x4 p0 = *reinterpret_cast<const f32x4*>(src + (size_t)z * g.M * g.R + rank);
                const f32x4 p1 = *reinterpret_cast<const f32x4*>(src + (size_t)z * g.M * g.R + rank + 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[w][i] += p0[i];
                    v[w][4 + i] += p1[i];
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[w][i]));
        }
    }
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
    const uint32_t e = min(__float_as_uint(top) >> 23, 252u);
    const float f = __uint_as_float((253u - e) << 23);  // 2^(126 - e)
#pragma unroll
    for (int w = 0; w < RG; ++w) {
        u32x4 hi, lo;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t h[2], l[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float s = v[w][2 * i + k] * f;
                h[k] = f32_to_act<BF16>(s);
                // an infinity is all in its high part
                l[k] = fabsf(s) < __builtin_inff() ? f32_to_act<BF16>(s - act_to_f32<BF16>((uint16_t)h[k])) : 0;
            }
            hi[i] = h[0] | (h[1] << 16);
            lo[i] = l[0] | (l[1] << 16);
        }
        put(w, hi, lo);
    }
    return __uint_as_float((e + 1u) << 23) * scale;
}

constexpr int LORA_STEP = 64;       // channels of a step of the first product
constexpr int LORA_MAX_SLICES = 4;  // K slices of t

// large batches (lora_wide.hip)
bool lora_wide(int M, int K, int N, int R);
int lora_wide_k_slices(int M, int K, int R);
void launch_lora_wide(const LoraArgs& g, bool bf16, hipStream_t s);

}  // namespace wq
