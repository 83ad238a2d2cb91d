// kv_cache.hip -- rows of a paged key-value cache: written (and quantised) as
// tokens come, and read back.
//
// The cache is [pages, kv_heads, page_size, head_dim] for keys and for values:
// the rows of one head in a page lie next to each other, so attention reads a
// page of a head as one piece.  A row (one token, one head) is 16-bit, or E4M3
// codes with a scale of its own or one for all:
//   row scale:  c = max(max|v| / 448, 2^-100), written;  code = E4M3(v / c)
//   static scale c given:                                code = E4M3(v / c)
//   back:       v = code * c in float32, rounded once
// v / c is the float32 quotient: one reciprocal a row, then a product and one
// residual step, which gives the correctly rounded quotient where nothing over- or
// underflows (10 instructions a value less than a division: 0.9 us at the size below); the residual is
// taken as q c - v, whose zero is +0, so that q - 0 keeps the sign of a zero q.  Both kernels give a row LPR lanes of 8
// values each, keys and values by the same thread; a workgroup takes consecutive
// tokens of one head, whose rows and scales are neighbours in the cache where a prompt
// fills its pages.
// HBM bound: 8192 tokens of 8 heads of 128, bf16 to codes and scales (51 MB) 11.1
// us with a launch's 3 in it, 32768 back (204 MB) 31.5 us.  More tokens a thread
// were slower (by 0.8 and 3 us for 2 and 4), as were non-temporal reads of the new rows (by 1.6).
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
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

template <bool BF16>
__device__ __forceinline__ void widen(u32x4 d, float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = act_to_f32<BF16>((uint16_t)(d[j >> 1] >> (16 * (j & 1))));
}

template <int CTRL>
__device__ __forceinline__ float dpp_max(float v) {
    return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(v), __float_as_int(v), CTRL, 0xF, 0xF,
                                                               false)));
}
// over the LPR lanes of a row, in each of them: within 16 lanes by DPP
template <int LPR>
__device__ __forceinline__ float row_max(float v) {
    v = dpp_max<0xB1>(v);   // quad_perm [1,0,3,2]
    v = dpp_max<0x4E>(v);   // quad_perm [2,3,0,1]
    v = dpp_max<0x141>(v);  // row_half_mirror
    if constexpr (LPR > 8) v = dpp_max<0x140>(v);  // row_mirror
    if constexpr (LPR > 16) v = fmaxf(v, __shfl_xor(v, 16, 64));
    return v;
}

// one row's 8 values in this lane (zeros in lanes past the row) into the cache
template <bool BF16, int MODE, int LPR>
__device__ __forceinline__ void put(u32x4 d, bool active, int64_t row, int D, int at, uint8_t* cache, float* scales,
                                    float static_scale) {
    if constexpr (MODE == KV_16) {
        if (active) *reinterpret_cast<u32x4*>(cache + (row * D + at) * 2) = d;
    } else {
        float v[8], c = static_scale;
        widen<BF16>(d, v);
        if constexpr (MODE == KV_E4M3_ROW) {
            float top = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(v[j]));
            top = row_max<LPR>(top);
            c = fmaxf(top / E4M3_MAX, MIN_ROW_SCALE);
            if (active && at == 0) scales[row] = c;
        }
        const float inv = 1.0f / c;
        u32x2 code;
        if constexpr (MODE == KV_E4M3_ROW) {
            // a bf16 row of the largest values, or an infinity: the product alone, whose residual may not be finite
            const float cr = c > 0x1p100f ? 0.0f : c, ir = c > 0x1p100f ? 0.0f : inv;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float q = v[j] * inv;
                v[j] = fmaf(-fmaf(q, cr, -v[j]), ir, q);
            }
            // (at most 448 and a step, which the conversion rounds to 448)
            code = u32x2{codes4(v[0], v[1], v[2], v[3]), codes4(v[4], v[5], v[6], v[7])};
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {  // past the codes' range (the residual may be infinite): the product
                const float q = v[j] * inv;
                v[j] = fabsf(q) > 480.0f ? q : fmaf(-fmaf(q, c, -v[j]), inv, q);
            }
            code = u32x2{codes4(clamp_e4m3(v[0]), clamp_e4m3(v[1]), clamp_e4m3(v[2]), clamp_e4m3(v[3])),
                         codes4(clamp_e4m3(v[4]), clamp_e4m3(v[5]), clamp_e4m3(v[6]), clamp_e4m3(v[7]))};
        }
        if (active) *reinterpret_cast<u32x2*>(cache + row * D + at) = code;
    }
}

template <bool BF16, int MODE, int LPR>
__global__ __launch_bounds__(256) void kv_write_kernel(KvRowsArgs g) {
    const int lane = threadIdx.x % LPR, at = 8 * lane;
    const int64_t t = (int64_t)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
    const int h = blockIdx.y;
    if (t >= g.T) return;  // (whole rows: the lanes of a row's maximum leave together)
    const bool active = at < g.D;
    const int64_t slot = g.slots[t];
    u32x4 k = {0, 0, 0, 0}, v = {0, 0, 0, 0};
    if (active) {
        k = ldg128(g.k16 + t * g.k_stride + (int64_t)h * g.D + at);
        v = ldg128(g.v16 + t * g.v_stride + (int64_t)h * g.D + at);
    }
    if (slot < 0 || slot >= (int64_t)g.pages * g.page_size) return;
    const uint32_t page = (uint32_t)slot / (uint32_t)g.page_size, off = (uint32_t)slot - page * g.page_size;
    const int64_t row = ((int64_t)page * g.kv_heads + h) * g.page_size + off;
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

// NT: non-temporal stores
template <bool BF16, int MODE, int LPR, bool NT>
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
    u32x4* ko = reinterpret_cast<u32x4*>(g.k16 + t * g.k_stride + (int64_t)h * g.D + at);
    u32x4* vo = reinterpret_cast<u32x4*>(g.v16 + t * g.v_stride + (int64_t)h * g.D + at);
    if constexpr (NT) {
        __builtin_nontemporal_store(k, ko);
        __builtin_nontemporal_store(v, vo);
    } else {
        *ko = k;
        *vo = v;
    }
}

// Rows read from codes and more than the L2s hold (8 x 4 MB) are stored past them: 134
// MB 43 -> 31.5 us, 34 MB 10.9 -> 10.0 us.  Not copies of 16-bit rows (2 x 134 MB into
// memory that the last-level cache holds: 48 -> 55 us)
template <bool BF16, int MODE, int LPR>
void launch_lpr(const KvRowsArgs& g, bool write, hipStream_t s) {
    const dim3 grid((unsigned)(((int64_t)g.T + 256 / LPR - 1) / (256 / LPR)), g.kv_heads);
    if (write)
        hipLaunchKernelGGL((kv_write_kernel<BF16, MODE, LPR>), grid, dim3(256), 0, s, g);
    else if (MODE != KV_16 && (int64_t)g.T * g.kv_heads * g.D * 4 >= (32 << 20))
        hipLaunchKernelGGL((kv_read_kernel<BF16, MODE, LPR, MODE != KV_16>), grid, dim3(256), 0, s, g);
    else
        hipLaunchKernelGGL((kv_read_kernel<BF16, MODE, LPR, false>), grid, dim3(256), 0, s, g);
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
