// dense_split.hip -- the dense linear layer with an epilogue at few rows or few
// outputs, where one round of workgroups covers the output.
//
//   y[m, n] = f(sum_k x[m, k] W[n, k] + bias[n]) + residual[m, n]
//
// A workgroup owns RT 16-row weight tiles and 16 R token rows and its NW waves
// share K: wave w takes the packed chunks w, w + NW, ... (1 KiB a tile, the A operand
// of v_mfma_f32_16x16x32 as it lies), DEPTH of them in flight with their token
// rows, which come straight from memory as the B operand (64 bytes of each of
// 16 rows an access): no barrier and no LDS before the waves' sums are joined.
// Numerics as dense_decode.hip: int4 codes exact, the group's scale on the float32 sum of
// its 128 channels, int8 exact, the column's scale at the end; partial sums in wave order.
//
// The bound is latency: at K = 4096 a wave has 4 chunks (int4) or 8 (int8) of which
// up to 3 are in flight, so one or two waits for memory are not hidden, and a launch and the
// join of 8 waves stand beside them.  (A workgroup's own reading, K (RT tiles + 16 R rows of x), is far less:
// 0.19 MB at M = 29, N = 4096, 1.3 of the 8.7 us at 64 bytes a clock.)  Measured, a 1024 channels
// cost what STEP_US says, growing with the tile, so the tile is the smallest with which the
// grid is one round (256 workgroups); beyond that the streaming kernel, which shares
// its rows through LDS, is ahead.  Against it (N = 4096, K = 4096, int4 / int8, us): M = 4 14.5
// / 19.9 -> 5.5 / 6.2; M = 29 17.7 / 23.0 -> 8.7 / 8.3; M = 128 25.6 / 29.9 -> 16.0 / 15.4; K =
// 14336: M = 29 54 / 73 -> 21.6 / 25.1.  The reading of weights and x alone would take 1.8 / 3.4 us at M = 29,
// K = 4096 and 6.1 / 11.6 at K = 14336.
#include "common.hpp"
#include "epilogue.hpp"
#include "launch.hpp"

namespace wq {

namespace {

template <int WBITS, bool BF16, int RT, int R, int NW, int DEPTH>
__global__ __launch_bounds__(NW * 64) void dense_split_kernel(const uint16_t* __restrict__ x, int M, int K, int N,
                                                              const uint8_t* __restrict__ w,
                                                              const uint16_t* __restrict__ s, int groups,
                                                              uint16_t* __restrict__ y, Epilogue ep) {
    constexpr int KCHUNK = WFmt<WBITS>::KCHUNK;
    constexpr int KSTEPS = KCHUNK / 32;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds_split[];
    f32x4* red = reinterpret_cast<f32x4*>(lds_split);  // [NW][RT * R][64]
    const int lane = threadIdx.x & 63, r16 = lane & 15, q4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tiles = N / TILE_ROWS, t0 = blockIdx.x * RT, m0 = blockIdx.y * (16 * R);
    const int C = K / KCHUNK;
    // chunks wave + NW i, i < nw; past the last the last again, unused
    const int nw = wave < C ? (C - 1 - wave) / NW + 1 : 0;
    const int clast = wave < C ? wave + (nw - 1) * NW : C - 1;
    const uint8_t* wt[RT];
    const uint16_t* st[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {  // past the last tile the last again, not stored
        const int tt = min(t0 + t, tiles - 1);
        wt[t] = w + (size_t)tt * C * CHUNK_BYTES + lane * 16;
        st[t] = s + tt * TILE_ROWS + 4 * q4;
    }
    const uint16_t* xr[R];
#pragma unroll
    for (int r = 0; r < R; ++r) xr[r] = x + (size_t)min(m0 + 16 * r + r16, M - 1) * K + 8 * q4;
    u32x4 wv[DEPTH][RT], xv[DEPTH][R][KSTEPS];
    u32x2 sv[DEPTH][RT];
    auto load = [&](int i, int slot) {
        const int c = min(wave + NW * i, clast);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int k = 0; k < KSTEPS; ++k) xv[slot][r][k] = ldg128(xr[r] + (size_t)c * KCHUNK + 32 * k);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            wv[slot][t] = ldg128_stream(wt[t] + (size_t)c * CHUNK_BYTES);
            if constexpr (WBITS == 4)
                sv[slot][t] = *reinterpret_cast<const u32x2*>(st[t] + (size_t)(groups > 1 ? c : 0) * N);
        }
    };
    f32x4 acc[RT][R];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int r = 0; r < R; ++r) acc[t][r] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto body = [&](int i, auto U) {
        constexpr int u = decltype(U)::value;
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            if constexpr (WBITS == 4) {
                u32x4 a[KSTEPS];
#pragma unroll
                for (int k = 0; k < KSTEPS; ++k) a[k] = dequant_w4_f16(wv[u][t][k]);
                const uint32_t lo = sv[u][t][0], hi = sv[u][t][1];
                const float s0 = f16_to_f32((uint16_t)(lo & 0xffffu)), s1 = f16_to_f32((uint16_t)(lo >> 16));
                const float s2 = f16_to_f32((uint16_t)(hi & 0xffffu)), s3 = f16_to_f32((uint16_t)(hi >> 16));
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    f32x4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int k = 0; k < KSTEPS; ++k) part = mfma16x16x32<false>(a[k], xv[u][r][k], part);
                    acc[t][r][0] += part[0] * s0;
                    acc[t][r][1] += part[1] * s1;
                    acc[t][r][2] += part[2] * s2;
                    acc[t][r][3] += part[3] * s3;
                }
            } else {
#pragma unroll
                for (int k = 0; k < KSTEPS; ++k) {
                    const u32x4 a = dequant_w8x8<BF16>(wv[u][t][2 * k], wv[u][t][2 * k + 1]);
#pragma unroll
                    for (int r = 0; r < R; ++r) acc[t][r] = mfma16x16x32<BF16>(a, xv[u][r][k], acc[t][r]);
                }
            }
        }
        load(i + DEPTH, u);
    };
#pragma unroll
    for (int p = 0; p < DEPTH; ++p) load(p, p);
    int i0 = 0;
    for (; i0 + DEPTH <= nw; i0 += DEPTH) static_for<0, DEPTH>([&](auto U) { body(i0 + decltype(U)::value, U); });
    static_for<0, DEPTH - 1>([&](auto U) {
        if (i0 + decltype(U)::value < nw) body(i0 + decltype(U)::value, U);
    });
    constexpr int PARTS = RT * R;
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int r = 0; r < R; ++r) red[(wave * PARTS + t * R + r) * 64 + lane] = acc[t][r];
    __syncthreads();
    for (int p = wave; p < PARTS; p += NW) {
        f32x4 o = red[p * 64 + lane];
#pragma unroll
        for (int q = 1; q < NW; ++q) o += red[(q * PARTS + p) * 64 + lane];
        const int t = t0 + p / R, m = m0 + 16 * (p % R) + r16, n0 = t * TILE_ROWS + 4 * q4;
        if (m < M && t < tiles) {
            if constexpr (WBITS == 8) {
#pragma unroll
                for (int k = 0; k < 4; ++k) o[k] *= act_to_f32<BF16>(s[n0 + k]);
            }
            finish4<BF16>(ep, o, m, n0, N, y);
        }
    }
}

template <int WBITS, bool BF16, int RT, int R, int NW, int DEPTH>
void launch_cfg(const uint16_t* x, int M, int K, int N, const uint8_t* w, const uint16_t* s, int groups, uint16_t* y,
                const Epilogue& ep, hipStream_t st) {
    constexpr int LDS = NW * RT * R * 64 * 16;
    auto kern = dense_split_kernel<WBITS, BF16, RT, R, NW, DEPTH>;
    if (LDS > 65536)
        (void)hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, LDS);
    const dim3 grid((N / TILE_ROWS + RT - 1) / RT, (M + 16 * R - 1) / (16 * R));
    hipLaunchKernelGGL(kern, grid, dim3(NW * 64), LDS, st, x, M, K, N, w, s, groups, y, ep);
}
// the plans: RT, R, waves, chunks ahead (int4 holds more of x a chunk: no room for 8 x 2 tiles)
enum SplitPlan { SPLIT_1X1, SPLIT_2X1, SPLIT_4X1, SPLIT_4X2, SPLIT_4X4, SPLIT_8X2, SPLIT_NONE };

constexpr int ROUND = 256;  // workgroups of one round: one a CU

int64_t groups_of(int M, int N, int RT, int R) {
    return (int64_t)((N / TILE_ROWS + RT - 1) / RT) * ((M + 16 * R - 1) / (16 * R));
}

// The smallest tile whose workgroups are one round (the order of the reading each
// one does).  More than a round, against the streaming kernel at N = 20480, K = 7168: up
// to 8 rows 2 tiles (int4 / int8 at 4 rows 23 / 28.5 against 27.7 / 43.4 us), int8 up to 16
// rows 4 tiles (36.4 against 44.4; int4 29.4 against 28.0), int8 up to 32 rows 8 x 2 (43.9
// against 47.3).  1 or 2 rows: dense_decode_kernel there (N = 6144, K = 4096: 6.8 / 7.8
// against 7.0 / 8.0 us; N = 20480 18.4 / 27 against 22 / 28).  Above 128 rows the tile of one
// round against the large-batch kernel by the times both expect: 5 us and STEP_US a 1024
// channels here (M = 256, N = K = 4096 23 / 20.5 us, that kernel 24 / 23; N = 1024 11.8 / 10.9,
// that 18; but M = 160, K = 14336, N = 4096 70 / 60 us, that 46 / 42)
constexpr float STEP_US[] = {1.0f, 1.25f, 1.75f, 2.6f, 4.1f, 3.9f};

SplitPlan split_plan(int wbits, int M, int N) {
    if (groups_of(M, N, 1, 1) <= ROUND) return SPLIT_1X1;
    if (M <= 2) return SPLIT_NONE;
    if (groups_of(M, N, 2, 1) <= ROUND) return SPLIT_2X1;
    if (groups_of(M, N, 4, 1) <= ROUND) return SPLIT_4X1;
    if (groups_of(M, N, 4, 2) <= ROUND) return SPLIT_4X2;
    if (wbits == 4 && groups_of(M, N, 4, 4) <= ROUND) return SPLIT_4X4;
    if (wbits == 8 && groups_of(M, N, 8, 2) <= ROUND) return SPLIT_8X2;
    if (M > 128) return SPLIT_NONE;
    if (M <= 8) return SPLIT_2X1;
    if (wbits == 8 && M <= 16) return SPLIT_4X1;
    if (wbits == 8 && M <= 32) return SPLIT_8X2;
    return SPLIT_NONE;
}

template <int WBITS, bool BF16>
void launch_split(const uint16_t* x, int M, int K, int N, const uint8_t* w, const uint16_t* s, int groups, uint16_t* y,
                  const Epilogue& ep, hipStream_t st) {
    switch (split_plan(WBITS, M, N)) {
        case SPLIT_1X1: launch_cfg<WBITS, BF16, 1, 1, 8, 3>(x, M, K, N, w, s, groups, y, ep, st); break;
        case SPLIT_2X1: launch_cfg<WBITS, BF16, 2, 1, 8, 3>(x, M, K, N, w, s, groups, y, ep, st); break;
        case SPLIT_4X1: launch_cfg<WBITS, BF16, 4, 1, 8, 2>(x, M, K, N, w, s, groups, y, ep, st); break;
        case SPLIT_4X2: launch_cfg<WBITS, BF16, 4, 2, 8, 2>(x, M, K, N, w, s, groups, y, ep, st); break;
        default:
            if constexpr (WBITS == 4) launch_cfg<WBITS, BF16, 4, 4, 8, 1>(x, M, K, N, w, s, groups, y, ep, st);
            else launch_cfg<WBITS, BF16, 8, 2, 8, 2>(x, M, K, N, w, s, groups, y, ep, st);
    }
}

}  // namespace

bool dense_split_supported(int wbits, int M, int K, int N) {
    const SplitPlan p = split_plan(wbits, M, N);
    return p != SPLIT_NONE && (M <= 128 || 5.0f + (float)K / 1024.0f * STEP_US[p] <= dense_large_us(M, K, N));
}

void launch_dense_split(int wbits, bool bf16, const uint16_t* x, int M, int K, int N, const uint8_t* w,
                        const uint16_t* s, int groups, uint16_t* y, const Epilogue& ep, hipStream_t st) {
    if (wbits == 4) launch_split<4, false>(x, M, K, N, w, s, groups, y, ep, st);
    else if (bf16) launch_split<8, true>(x, M, K, N, w, s, groups, y, ep, st);
    else launch_split<8, false>(x, M, K, N, w, s, groups, y, ep, st);
}

}  // namespace wq
