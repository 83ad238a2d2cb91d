// rms_norm.hip -- residual addition + root-mean-square norm of a row, with a
// 16-bit output, E4M3 codes, or both (the input of the FP8 layer).
//
//   s = x + r              (float32; r' = s rounded to 16 bits, the new residual)
//   y = s / sqrt(mean(s^2) + eps) * w
//   row scale:  c = max(max|y| / 448, 2^-100), code = E4M3(y * (1 / c))
//   static scale c given:                      code = E4M3(y / c)
//
// Everything between the loads and the stores is float32: s is not rounded
// before it is squared, y is not rounded before it is quantised.  A row is
// read once: its values stay in registers between the sum of squares, the
// maximum and the store, a wave or a workgroup per row, of as many threads
// as keep 8 or 16 values each (16 bytes an access).  HBM bound for many rows: 8192
// x 5120 bf16 with residual, 16-bit and coded outputs moves 378 MB in 73.5 us, 5.14
// TB/s, what a large copy reaches.  One row of 4096: 2.8 us, the latency of two loads
// and two reductions; 333 rows of 1001 (single 2-byte accesses) 4.9 us, 8192 of 5121 195.
// Above 16384 values a row is read again for each step, by 2-byte accesses: 4096 rows
// of 20480 520 us.
#include "common.hpp"
#include "launch.hpp"

#include <algorithm>

namespace wq {

namespace {

constexpr float E4M3_MAX = 448.0f;
constexpr float MIN_ROW_SCALE = 0x1p-100f;  // a row of zeros: a scale that still has a reciprocal

struct Add {
    static __device__ __forceinline__ float of(float a, float b) { return a + b; }
};
struct Max {  // fmaxf: a NaN does not win, so the scale of a row with one is that of its numbers
    static __device__ __forceinline__ float of(float a, float b) { return fmaxf(a, b); }
};

// a launch holds at most 2^32 threads along x: workgroups beyond GRID_X go on along y
constexpr int GRID_X = 1 << 20;
__device__ __forceinline__ int64_t block_index() { return (int64_t)blockIdx.y * GRID_X + blockIdx.x; }
dim3 row_grid(int64_t blocks) {
    return dim3((unsigned)std::min<int64_t>(blocks, GRID_X), (unsigned)((blocks + GRID_X - 1) / GRID_X));
}

template <class OP, int CTRL>
__device__ __forceinline__ float dpp_step(float v) {
    const int o = __builtin_amdgcn_update_dpp(__float_as_int(v), __float_as_int(v), CTRL, 0xF, 0xF, false);
    return OP::of(v, __int_as_float(o));
}

// over the 64 lanes of a wave, in every lane: within rows of 16 lanes by DPP,
// then across the rows by two shuffles
template <class OP>
__device__ __forceinline__ float wave_all(float v) {
    v = dpp_step<OP, 0xB1>(v);   // quad_perm [1,0,3,2]
    v = dpp_step<OP, 0x4E>(v);   // quad_perm [2,3,0,1]
    v = dpp_step<OP, 0x141>(v);  // row_half_mirror
    v = dpp_step<OP, 0x140>(v);  // row_mirror
    v = OP::of(v, __shfl_xor(v, 16, 64));
    v = OP::of(v, __shfl_xor(v, 32, 64));
    return v;
}

// over the TPR threads of a row (whole waves); buf is used by one call only
template <class OP, int TPR>
__device__ __forceinline__ float row_all(float v, float* buf) {
    v = wave_all<OP>(v);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
        __syncthreads();
        v = buf[0];
#pragma unroll
        for (int i = 1; i < TPR / 64; ++i) v = OP::of(v, buf[i]);
    }
    return v;
}

// E4M3 code pairs: clamped to +-448 by comparisons, which a NaN passes
// unchanged (its code is NaN), then the hardware's nearest-even conversion
__device__ __forceinline__ float clamp_e4m3(float v) {
    v = v > E4M3_MAX ? E4M3_MAX : v;
    return v < -E4M3_MAX ? -E4M3_MAX : v;
}
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(clamp_e4m3(a), clamp_e4m3(b), 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(clamp_e4m3(c), clamp_e4m3(d), w, true);
}

// VEC consecutive 16-bit values as floats: one 16-byte access (VEC 8) or one value (VEC 1)
template <bool BF16, int VEC>
__device__ __forceinline__ void load_vec(const uint16_t* p, float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        const u32x4 d = ldg128(p);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = act_to_f32<BF16>((uint16_t)(d[j >> 1] >> (16 * (j & 1))));
    } else {
        v[0] = act_to_f32<BF16>(*p);
    }
}
template <bool BF16, int VEC>
__device__ __forceinline__ void store_vec(uint16_t* p, const float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        u32x4 d;
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] = f32_to_act2<BF16>(v[2 * j], v[2 * j + 1]);
        *reinterpret_cast<u32x4*>(p) = d;
    } else {
        *p = f32_to_act<BF16>(v[0]);
    }
}
template <int VEC>
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        *reinterpret_cast<u32x2*>(p) = u32x2{codes4(v[0], v[1], v[2], v[3]), codes4(v[4], v[5], v[6], v[7])};
    } else {
        *p = (uint8_t)codes4(v[0], 0.0f, 0.0f, 0.0f);
    }
}

// the sum of squares above which (or as a NaN) a row is looked at again, and
// the power of two that its values are then taken down by: bf16 rows beyond
// about 1e17, whose squares pass float32's range
constexpr float SUM_MAX = 3.0e38f;
constexpr float DOWN = 0x1p-96f;

// The row's sum of squares, in an order that the launch shape does not change
// (the shape goes by the number of rows, a row's bits must not): each vector of 8
// by itself, the 64 consecutive vectors of a wave, then these sums in ascending
// order, whether one wave holds several of them or several waves one each.
// Single values: one chain a thread, in shapes that go by the width only.
template <int VEC, int TPR, int VPT>
__device__ __forceinline__ float row_squares(const float (&v)[VPT][VEC], float* buf) {
    constexpr int SUMS = VEC == 1 ? 1 : VPT;
    float p[SUMS];
#pragma unroll
    for (int k = 0; k < SUMS; ++k) p[k] = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) p[i % SUMS] = fmaf(v[i][j], v[i][j], p[i % SUMS]);
#pragma unroll
    for (int k = 0; k < SUMS; ++k) p[k] = wave_all<Add>(p[k]);
    float total;
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int k = 0; k < SUMS; ++k) buf[k * (TPR / 64) + (threadIdx.x >> 6)] = p[k];
        }
        __syncthreads();
        total = buf[0];
#pragma unroll
        for (int k = 1; k < SUMS * (TPR / 64); ++k) total += buf[k];
    } else {
        total = p[0];
#pragma unroll
        for (int k = 1; k < SUMS; ++k) total += p[k];
    }
    return total;
}

// A row in registers: TPR threads, VPT vectors of VEC values each.
template <bool BF16, int VEC, int TPR, int VPT>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void rms_norm_kernel(RmsNormArgs g) {
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
    static_assert(RPB == 1 || TPR == 64, "rows that share a workgroup are one wave each: no barrier");
    __shared__ float buf[4][VPT * (TPR / 64)];
    const int tid = threadIdx.x % TPR;
    const int64_t row = block_index() * RPB + threadIdx.x / TPR;
    if (row >= g.rows) return;
    const uint16_t* x = g.x + row * g.x_stride;
    const uint16_t* r = g.r ? g.r + row * g.r_stride : nullptr;

    float v[VPT][VEC];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (i * TPR + tid) * VEC;
        if (c < g.n) load_vec<BF16, VEC>(x + c, v[i]);
        else
#pragma unroll
            for (int j = 0; j < VEC; ++j) v[i][j] = 0.0f;
    }
    if (r) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * TPR + tid) * VEC;
            if (c < g.n) {
                float t[VEC];
                load_vec<BF16, VEC>(r + c, t);
#pragma unroll
                for (int j = 0; j < VEC; ++j) v[i][j] += t[j];
            }
        }
    }
    if (g.r_out) {  // each value is read by the thread that writes it: r_out may be r, or x
        uint16_t* ro = g.r_out + row * g.ro_stride;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * TPR + tid) * VEC;
            if (c < g.n) store_vec<BF16, VEC>(ro + c, v[i]);
        }
    }
    if (!g.out && !g.codes) return;

    float ss = row_squares<VEC, TPR, VPT>(v, buf[0]);
    float eps = g.eps;
    if (!(ss <= SUM_MAX)) {  // the same for the whole row
        float am = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) am = fmaxf(am, fabsf(v[i][j]));
        am = row_all<Max, TPR>(am, buf[1]);
        if (am < __builtin_inff()) {  // finite (or a NaN beside finite values, which keeps the sum a NaN)
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j) v[i][j] *= DOWN;
            ss = row_squares<VEC, TPR, VPT>(v, buf[2]);
            eps = 0.0f;  // nothing beside such a sum
        }
    }
    const float inv = rsqrtf(ss / (float)g.n + eps);

    float am = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (i * TPR + tid) * VEC;
        if (c < g.n) {
            float w[VEC];
            if (g.w) load_vec<BF16, VEC>(g.w + c, w);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                v[i][j] *= inv;
                if (g.w) v[i][j] *= w[j];
                am = fmaxf(am, fabsf(v[i][j]));
            }
            if (g.out) store_vec<BF16, VEC>(g.out + row * g.out_stride + c, v[i]);
        }
    }
    if (!g.codes) return;
    uint8_t* q = g.codes + row * g.n;
    if (g.scales) {
        const float scale = fmaxf(row_all<Max, TPR>(am, buf[3]) / E4M3_MAX, MIN_ROW_SCALE);
        if (tid == 0) g.scales[row] = scale;
        const float up = 1.0f / scale;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) v[i][j] *= up;
    } else {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) v[i][j] = __fdiv_rn(v[i][j], g.static_scale);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (i * TPR + tid) * VEC;
        if (c < g.n) store_codes<VEC>(q + c, v[i]);
    }
}

// Rows of any width, read again for each step (from the caches where they
// fit): widths beyond the registers of a workgroup.  r_out and out are written
// in the last step only, each value by the thread that reads it.
template <bool BF16>
__global__ __launch_bounds__(1024) void rms_norm_long_kernel(RmsNormArgs g) {
    __shared__ float buf[4][16];
    const int64_t row = block_index();
    if (row >= g.rows) return;
    const uint16_t* x = g.x + row * g.x_stride;
    const uint16_t* r = g.r ? g.r + row * g.r_stride : nullptr;
    auto value = [&](int c) {
        const float s = act_to_f32<BF16>(x[c]);
        return r ? s + act_to_f32<BF16>(r[c]) : s;
    };
    float ss = 0.0f;
    for (int c = threadIdx.x; c < g.n; c += 1024) {
        const float s = value(c);
        ss = fmaf(s, s, ss);
    }
    ss = row_all<Add, 1024>(ss, buf[0]);
    float f = 1.0f;
    if (!(ss <= SUM_MAX)) {
        float am = 0.0f;
        for (int c = threadIdx.x; c < g.n; c += 1024) am = fmaxf(am, fabsf(value(c)));
        am = row_all<Max, 1024>(am, buf[1]);
        if (am < __builtin_inff()) {
            f = DOWN;
            ss = 0.0f;
            for (int c = threadIdx.x; c < g.n; c += 1024) {
                const float s = value(c) * f;
                ss = fmaf(s, s, ss);
            }
            ss = row_all<Add, 1024>(ss, buf[2]);
        }
    }
    const float inv = rsqrtf(ss / (float)g.n + (f == 1.0f ? g.eps : 0.0f));
    auto normed = [&](float s, int c) {
        const float y = s * f * inv;
        return g.w ? y * act_to_f32<BF16>(g.w[c]) : y;
    };
    float up = 1.0f;
    if (g.codes && g.scales) {
        float am = 0.0f;
        for (int c = threadIdx.x; c < g.n; c += 1024) am = fmaxf(am, fabsf(normed(value(c), c)));
        const float scale = fmaxf(row_all<Max, 1024>(am, buf[3]) / E4M3_MAX, MIN_ROW_SCALE);
        if (threadIdx.x == 0) g.scales[row] = scale;
        up = 1.0f / scale;
    }
    for (int c = threadIdx.x; c < g.n; c += 1024) {
        const float s = value(c);
        const float y = normed(s, c);
        if (g.r_out) g.r_out[row * g.ro_stride + c] = f32_to_act<BF16>(s);
        if (g.out) g.out[row * g.out_stride + c] = f32_to_act<BF16>(y);
        if (g.codes) {
            const float q[1] = {g.scales ? y * up : __fdiv_rn(y, g.static_scale)};
            store_codes<1>(g.codes + row * g.n + c, q);
        }
    }
}

template <bool BF16, int VEC, int TPR, int VPT>
void launch_cfg(const RmsNormArgs& g, hipStream_t s) {
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
    hipLaunchKernelGGL((rms_norm_kernel<BF16, VEC, TPR, VPT>), row_grid(((int64_t)g.rows + RPB - 1) / RPB),
                       dim3(TPR < 256 ? 256 : TPR), 0, s, g);
}

template <bool BF16>
void launch_t(const RmsNormArgs& g, hipStream_t s) {
    const bool vec = g.n % 8 == 0 && g.x_stride % 8 == 0 && (!g.r || g.r_stride % 8 == 0) &&
                     (!g.r_out || g.ro_stride % 8 == 0) && (!g.out || g.out_stride % 8 == 0);
    // Threads per row: one 16-byte access each is the shortest chain; up to a row
    // per CU that decides, beyond it fewer threads per row keep more rows under way.
    // us at 64 rows / 8192 rows (residual, 16-bit and coded outputs): n = 1024 by 256
    // threads 3.4 / 16.9, by 64 of two accesses 4.0 / 14.0; n = 4096 by 512 3.7 / 56.7,
    // by 256 of two 4.3 / 56.4; n = 5120 by 1024 4.0 / 82.7, by 512 of two 4.3 / 75.8, by
    // 256 of four 5.2 / 77.9; n = 16384 by 1024 of two 5.8 / 114 (4096 rows), by 512 of
    // four 6.8 / 121.
    const bool few = g.rows <= 256;
    if (vec) {
        if (g.n <= 512) return launch_cfg<BF16, 8, 64, 1>(g, s);
        if (g.n <= 1024 && !few) return launch_cfg<BF16, 8, 64, 2>(g, s);
        if (g.n <= 2048) return launch_cfg<BF16, 8, 256, 1>(g, s);
        if (g.n <= 4096) return launch_cfg<BF16, 8, 512, 1>(g, s);
        if (g.n <= 8192 && !few) return launch_cfg<BF16, 8, 512, 2>(g, s);
        if (g.n <= 8192) return launch_cfg<BF16, 8, 1024, 1>(g, s);
        if (g.n <= 16384) return launch_cfg<BF16, 8, 1024, 2>(g, s);
    } else {
        if (g.n <= 512) return launch_cfg<BF16, 1, 64, 8>(g, s);
        if (g.n <= 2048) return launch_cfg<BF16, 1, 256, 8>(g, s);
        if (g.n <= 8192) return launch_cfg<BF16, 1, 1024, 8>(g, s);
    }
    hipLaunchKernelGGL(rms_norm_long_kernel<BF16>, row_grid(g.rows), dim3(1024), 0, s, g);
}

}  // namespace

void launch_rms_norm(const RmsNormArgs& g, bool bf16, hipStream_t s) {
    if (bf16) launch_t<true>(g, s);
    else launch_t<false>(g, s);
}

}  // namespace wq
