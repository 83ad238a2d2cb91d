// kv_cache.hip -- rows of a paged key-value cache: written (and quantised) as
// tokens come, and read back.
//
// The cache is [pages, kv_heads, page_size, head_dim] for keys and for values:
// the rows of one head in a page lie next to each other, so attention reads a
// page of a head as one piece.  A row (one token, one head) is 16-bit, or E4M3
// codes with a scale of its own or one for all:
//   row scale:  c = max(max|v| / 448, 2^-100), code = E4M3(v * (1 / c))
//   static scale c given:                      code = E4M3(v / c)
//   back:       v = code * c in float32, rounded once
// (the codes and scales of rms_norm.hip).  Both kernels give a row LPR lanes of
// 8 values each, keys and values by the same thread; a workgroup takes
// consecutive tokens of one head, whose rows and scales are neighbours in the
// cache where a prompt fills its pages.
#include "common.hpp"
#include "kv_common.hpp"
#include "launch.hpp"

namespace wq {

namespace {

constexpr float E4M3_MAX = 448.0f;
constexpr float MIN_ROW_SCALE = 0x1p-100f;  // a row of zeros: a scale that still has a reciprocal

// clamped by comparisons, which a NaN passes unchanged (its code is NaN), then
// the hardware's nearest-even conversion
__device__ __forceinline__ float clamp_e4m3(float v) {
    v = v > E4M3_MAX ? E4M3_MAX : v;
    return v < -E4M3_MAX ? -E4M3_MAX : v;
}
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(clamp_e4m3(a), clamp_e4m3(b), 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(clamp_e4m3(c), clamp_e4m3(d), w, true);
}

template <bool BF16>
__device__ __forceinline__ void widen(u32x4 d, float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = act_to_f32<BF16>((uint16_t)(d[j >> 1] >> (16 * (j & 1))));
}

// one row's 8 values in this lane (zeros in lanes past the row) into the cache
template <bool BF16, int MODE, int LPR>
__device__ __forceinline__ void put(u32x4 d, bool active, int64_t row, int D, int at, uint8_t* cache, float* scales,
                                    float static_scale) {
    if constexpr (MODE == KV_16) {
        if (active) *reinterpret_cast<u32x4*>(cache + (row * D + at) * 2) = d;
    } else {
        float v[8];
        widen<BF16>(d, v);
        if constexpr (MODE == KV_E4M3_ROW) {
            float top = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(v[j]));
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
            const float c = fmaxf(top / E4M3_MAX, MIN_ROW_SCALE);
            const float inv = 1.0f / c;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= inv;
            if (active && at == 0) scales[row] = c;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = v[j] / static_scale;
        }
        if (active)
            *reinterpret_cast<u32x2*>(cache + row * D + at) =
                u32x2{codes4(v[0], v[1], v[2], v[3]), codes4(v[4], v[5], v[6], v[7])};
    }
}

template <bool BF16, int MODE, int LPR>
__global__ __launch_bounds__(256) void kv_write_kernel(KvRowsArgs g) {
    const int lane = threadIdx.x % LPR, at = 8 * lane;
    const int64_t t = (int64_t)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
    const int h = blockIdx.y;
    if (t >= g.T) return;  // (whole rows: the lanes of a row's maximum leave together)
    const int64_t slot = g.slots[t];
    if (slot < 0 || slot >= (int64_t)g.pages * g.page_size) return;
    const uint32_t page = (uint32_t)slot / (uint32_t)g.page_size, off = (uint32_t)slot - page * g.page_size;
    const int64_t row = ((int64_t)page * g.kv_heads + h) * g.page_size + off;
    const bool active = at < g.D;
    u32x4 k = {0, 0, 0, 0}, v = {0, 0, 0, 0};
    if (active) {
        k = ldg128(g.k16 + t * g.k_stride + (int64_t)h * g.D + at);
        v = ldg128(g.v16 + t * g.v_stride + (int64_t)h * g.D + at);
    }
    put<BF16, MODE, LPR>(k, active, row, g.D, at, g.k, g.ks, g.k_scale);
    put<BF16, MODE, LPR>(v, active, row, g.D, at, g.v, g.vs, g.v_scale);
}

template <bool BF16, int MODE>
__device__ __forceinline__ u32x4 get(const uint8_t* cache, const float* scales, float static_scale, int64_t row, int D,
                                     int at) {
    if constexpr (MODE == KV_16) {
        return ldg128(cache + (row * D + at) * 2);
    } else {
        const u32x2 d = *reinterpret_cast<const u32x2*>(cache + row * D + at);
        const float c = MODE == KV_E4M3_ROW ? scales[row] : static_scale;
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t w = d[i];
            const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
            o[2 * i] = f32_to_act2<BF16>(lo[0] * c, lo[1] * c);
            o[2 * i + 1] = f32_to_act2<BF16>(hi[0] * c, hi[1] * c);
        }
        return o;
    }
}

template <bool BF16, int MODE, int LPR>
__global__ __launch_bounds__(256) void kv_read_kernel(KvRowsArgs g) {
    const int lane = threadIdx.x % LPR, at = 8 * lane;
    const int64_t t = (int64_t)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
    const int h = blockIdx.y;
    if (t >= g.T || at >= g.D) return;
    const int64_t slot = g.slots[t];
    u32x4 k = {0, 0, 0, 0}, v = {0, 0, 0, 0};
    if (slot >= 0 && slot < (int64_t)g.pages * g.page_size) {
        const uint32_t page = (uint32_t)slot / (uint32_t)g.page_size, off = (uint32_t)slot - page * g.page_size;
        const int64_t row = ((int64_t)page * g.kv_heads + h) * g.page_size + off;
        k = get<BF16, MODE>(g.k, g.ks, g.k_scale, row, g.D, at);
        v = get<BF16, MODE>(g.v, g.vs, g.v_scale, row, g.D, at);
    }
    *reinterpret_cast<u32x4*>(g.k16 + t * g.k_stride + (int64_t)h * g.D + at) = k;
    *reinterpret_cast<u32x4*>(g.v16 + t * g.v_stride + (int64_t)h * g.D + at) = v;
}

template <bool BF16, int MODE, int LPR>
void launch_lpr(const KvRowsArgs& g, bool write, hipStream_t s) {
    const dim3 grid((unsigned)(((int64_t)g.T + 256 / LPR - 1) / (256 / LPR)), g.kv_heads);
    if (write) hipLaunchKernelGGL((kv_write_kernel<BF16, MODE, LPR>), grid, dim3(256), 0, s, g);
    else hipLaunchKernelGGL((kv_read_kernel<BF16, MODE, LPR>), grid, dim3(256), 0, s, g);
}

template <bool BF16, int MODE>
void launch_mode(const KvRowsArgs& g, bool write, hipStream_t s) {
    if (g.D <= 64) launch_lpr<BF16, MODE, 8>(g, write, s);
    else if (g.D <= 128) launch_lpr<BF16, MODE, 16>(g, write, s);
    else launch_lpr<BF16, MODE, 32>(g, write, s);
}

template <bool BF16>
void launch_rows(const KvRowsArgs& g, bool write, hipStream_t s) {
    if (g.mode == KV_16) launch_mode<BF16, KV_16>(g, write, s);
    else if (g.mode == KV_E4M3_ROW) launch_mode<BF16, KV_E4M3_ROW>(g, write, s);
    else launch_mode<BF16, KV_E4M3_STATIC>(g, write, s);
}

}  // namespace

void launch_kv_rows(const KvRowsArgs& g, bool write, bool bf16, hipStream_t s) {
    if (bf16) launch_rows<true>(g, write, s);
    else launch_rows<false>(g, write, s);
}

}  // namespace wq
