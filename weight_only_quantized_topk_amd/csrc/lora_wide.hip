// lora_wide.hip -- the adapters of a large batch (prompts): the same two
// products as lora.hip, for tiles of 32 and 64 tokens.
//
// A matrix operand read straight from row-major memory has neighbouring lanes
// in different rows, 16 bytes in each of 64 cache lines an instruction; at this
// size the cache's lookups bounded both products.  Here everything passes
// through LDS from loads whose neighbouring lanes are neighbours in a row, the B
// rows once per workgroup, and y is accessed in 256-byte pieces of a row.
//
// 4096 rows of 11 prompts, rank 64, 7168 x 20480 bf16: 33 us (59 MB of x) and 85 us
// (336 MB of y read and written; 114 us from lora.hip's kernel), 118 us for what a
// copy of 423 MB does in 82.  The tiles in which a prompt ends take a second pass
// after the first: with one adapter for all rows the first product takes 19.5 us.
#include "lora_common.hpp"

#include <algorithm>

namespace wq {

namespace {

constexpr int DOWN_WAVES = 8;
constexpr int UP_WAVES = 4;
// a wave's lanes exchange values through LDS that no other wave touches: the
// accesses of one wave take effect in order, so only the compiler has to keep it
__device__ __forceinline__ void wave_lds_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

constexpr int TS = 2;  // 16-token tiles of the first product's workgroups

// t = x A^T: 32 tokens, one slice of K, 16 RT ranks a workgroup; its waves take
// the 64-channel steps of the slice in turn.  A wave's step: its 32 x rows and
// 16 RT rank rows of 128 bytes go through registers (two steps ahead) into the
// wave's own part of LDS, piece c of row r in slot c ^ (r % 8), so that the 8
// lanes of an access phase fall on different banks both ways; no barrier.
template <bool BF16, int RT>
__global__ __launch_bounds__(64 * DOWN_WAVES) void lora_wide_down_kernel(LoraArgs g) {
    constexpr int ROWS = 16 * (TS + RT);
    constexpr int LOADS = ROWS / 8;
    extern __shared__ u32x4 lds[];  // [DOWN_WAVES][ROWS][8], then the waves' sums [DOWN_WAVES][TS][RT][64]
    const int lane = threadIdx.x & 63;
    const int wave = wave_index();
    const int col = lane & 15, q = lane >> 4;
    const int groups = (g.R + 16 * RT - 1) / (16 * RT);
    const int slice = blockIdx.x % g.ks, r0 = blockIdx.x / g.ks % groups * (16 * RT);
    const int tile = blockIdx.x / (g.ks * groups);
    u32x4* own = lds + wave * ROWS * 8;

    const int steps = (g.K + LORA_STEP - 1) / LORA_STEP;
    const int s0 = (int)((int64_t)slice * steps / g.ks) + wave, s1 = (int)((int64_t)(slice + 1) * steps / g.ks);
    const int lrow = lane >> 3, piece = lane & 7;

    const int ids = tile_ids<16 * TS>(g, tile, lane);
    uint64_t left = __ballot(ids >= 0), mine;
    for (int j = 0; left; ++j) {
        const int a = next_adapter(ids, left, mine);
        if (j % (int)gridDim.y != (int)blockIdx.y) continue;
        const uint16_t* row[LOADS];  // rows past M or R: the last one (their results are dropped)
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int r = 8 * i + lrow;
            row[i] = i < 2 * TS ? g.x + (int64_t)min(tile * 16 * TS + r, g.M - 1) * g.x_stride
                                : g.a + ((size_t)a * g.R + min(r0 + r - 16 * TS, g.R - 1)) * g.K;
        }
        f32x4 acc[TS][RT];
#pragma unroll
        for (int t = 0; t < TS; ++t)
#pragma unroll
            for (int r = 0; r < RT; ++r) acc[t][r] = f32x4{0.f, 0.f, 0.f, 0.f};
        u32x4 va[LOADS], vb[LOADS];
        auto load = [&](int s, u32x4 (&v)[LOADS]) {
            const int c = min(LORA_STEP * s + 8 * piece, g.K - 8);
#pragma unroll
            for (int i = 0; i < LOADS; ++i) v[i] = ldg128(row[i] + c);
        };
        auto step = [&](int s, u32x4 (&v)[LOADS]) {
            if (LORA_STEP * (s + 1) > g.K) {  // channels past K: zeros on both sides
#pragma unroll
                for (int i = 0; i < LOADS; ++i)
                    v[i] = LORA_STEP * s + 8 * piece < g.K ? v[i] : u32x4{0u, 0u, 0u, 0u};
            }
#pragma unroll
            for (int i = 0; i < LOADS; ++i) own[(8 * i + lrow) * 8 + (piece ^ lrow)] = v[i];
            wave_lds_order();
            if (s + 2 * DOWN_WAVES < s1) load(s + 2 * DOWN_WAVES, v);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int slot = (q + 4 * h) ^ (col & 7);
                u32x4 xv[TS];
#pragma unroll
                for (int t = 0; t < TS; ++t) xv[t] = own[(16 * t + col) * 8 + slot];
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const u32x4 av = own[(16 * (TS + r) + col) * 8 + slot];
#pragma unroll
                    for (int t = 0; t < TS; ++t) acc[t][r] = mfma16x16x32<BF16>(av, xv[t], acc[t][r]);
                }
            }
            wave_lds_order();
        };
        if (s0 < s1) load(s0, va);
        if (s0 + DOWN_WAVES < s1) load(s0 + DOWN_WAVES, vb);
        for (int s = s0; s < s1; s += 2 * DOWN_WAVES) {
            step(s, va);
            if (s + DOWN_WAVES < s1) step(s + DOWN_WAVES, vb);
        }
        __syncthreads();
        f32x4* red = reinterpret_cast<f32x4*>(lds);
#pragma unroll
        for (int t = 0; t < TS; ++t)
#pragma unroll
            for (int r = 0; r < RT; ++r) red[((wave * TS + t) * RT + r) * 64 + lane] = acc[t][r];
        __syncthreads();
        for (int i = wave; i < TS * RT; i += DOWN_WAVES) {
            f32x4 sum = red[i * 64 + lane];
#pragma unroll
            for (int w = 1; w < DOWN_WAVES; ++w) sum += red[(w * TS * RT + i) * 64 + lane];
            const int rank = r0 + 16 * (i % RT) + 4 * q;
            const int tok = 16 * (i / RT) + col;
            if (((mine >> tok) & 1ull) && rank < g.R)
                *reinterpret_cast<f32x4*>(g.t + ((size_t)slice * g.M + tile * 16 * TS + tok) * g.R + rank) = sum;
        }
        __syncthreads();
    }
}

// y += scale * t B^T: 64 tokens (16 a wave), 128 outputs at a time.  The tokens'
// t is split once (lora_common.hpp) and kept in registers as matrix operands;
// the 128 B rows of a step, contiguous in memory, go through registers into
// one of two LDS buffers a step ahead, and the next step's y into registers.
// D's rows are tokens, its columns outputs: column c of weight tile k is output
// 8 c + k, so a lane's results of the 8 tiles are 8 outputs in a row of a token,
// and 16 lanes cover 256 bytes of it.  Piece p (8 ranks) of B row n is kept in
// slot p ^ (n / 8) of its row (of CP slots): 8 lanes of a read, rows 8 apart,
// fall on different banks.  RC: chunks of 32 ranks.
template <bool BF16, int RC>
__global__ __launch_bounds__(64 * UP_WAVES, RC <= 2 ? 3 : 1) void lora_wide_up_kernel(LoraArgs g, int per, int ranges) {
    constexpr int CP = 4 * RC;                    // slots of a B row
    constexpr int STAGE = 128 * CP / (64 * UP_WAVES);  // pieces a thread moves per step
    constexpr int BUF = 128 * CP;
    constexpr int SWZ = CP < 8 ? CP - 1 : 7;
    __shared__ u32x4 buf[2 * BUF];
    __shared__ __attribute__((aligned(16))) float back[64];
    const int lane = threadIdx.x & 63;
    const int wave = wave_index();
    const int col = lane & 15, q = lane >> 4;
    const int tile = blockIdx.x / ranges;
    const int first = blockIdx.x % ranges * per;
    const int count = min(per, (g.N + 127) / 128 - first);
    const int pieces = g.R / 8;

    // t: 8 threads a token, operands by way of the second buffer
    for (int tok = threadIdx.x >> 3; tok < 64; tok += 8 * UP_WAVES) {
        const int gr = threadIdx.x & 7;
        const float f = split_token<BF16, (RC + 1) / 2>(
            g, min(tile * 64 + tok, g.M - 1), gr, [&](int w, u32x4 hi, u32x4 lo) {
                const int c = 2 * w + (gr >> 2);
                if (c >= RC) return;
                u32x4* to = buf + BUF + ((tok >> 4) * RC + c) * 128 + 16 * (gr & 3) + (tok & 15);
                to[0] = hi;
                to[64] = lo;
            });
        if (gr == 0) back[tok] = f;
    }
    const int ids = tile_ids<64>(g, tile, lane);
    __syncthreads();
    u32x4 thi[RC], tlo[RC];
#pragma unroll
    for (int c = 0; c < RC; ++c) {
        thi[c] = buf[BUF + (wave * RC + c) * 128 + lane];
        tlo[c] = buf[BUF + (wave * RC + c) * 128 + 64 + lane];
    }
    const f32x4 fb = *reinterpret_cast<const f32x4*>(back + 16 * wave + 4 * q);
    __syncthreads();
    if (pieces < CP)  // ranks past R: zeros, which no step overwrites
        for (int i = threadIdx.x; i < 2 * BUF; i += 64 * UP_WAVES) {
            const int n = i / CP % 128;
            if (((i % CP) ^ ((n >> 3) & SWZ)) >= pieces) buf[i] = u32x4{0u, 0u, 0u, 0u};
        }

    // this thread's pieces of a step: B rows n0 .. n0 + 127 are one run of memory
    int slot[STAGE];
#pragma unroll
    for (int i = 0; i < STAGE; ++i) {
        const int p = (int)threadIdx.x + 64 * UP_WAVES * i;
        const int n = p / pieces;
        slot[i] = n < 128 ? n * CP + ((p - n * pieces) ^ ((n >> 3) & SWZ)) : -1;
    }

    uint64_t left = __ballot(ids >= 0), mine;
    for (int j = 0; left; ++j) {
        const int a = next_adapter(ids, left, mine);
        if (j % (int)gridDim.y != (int)blockIdx.y) continue;
        const uint32_t mw = (uint32_t)(mine >> (16 * wave)) & 0xFFFFu;  // of this wave's tokens
        const uint16_t* bw = g.b + (size_t)a * g.N * g.R;

        u32x4 sv[STAGE], yv[4];
        auto load_b = [&](int i) {
            const int n0 = 128 * (first + i);
            const int last = min(128, g.N - n0) * pieces - 1;
            const uint16_t* base = bw + (size_t)n0 * g.R;
#pragma unroll
            for (int k = 0; k < STAGE; ++k)
                if (64 * UP_WAVES * k < 128 * pieces)
                    sv[k] = ldg128(base + 8 * min((int)threadIdx.x + 64 * UP_WAVES * k, last));
        };
        auto store_b = [&](int i) {
#pragma unroll
            for (int k = 0; k < STAGE; ++k)
                if (slot[k] >= 0) buf[(i & 1) * BUF + slot[k]] = sv[k];
        };
        uint16_t* yt = g.y + (int64_t)(tile * 64 + 16 * wave) * g.y_stride;
        auto y_at = [&](int r, int n) { return yt + (uint32_t)((4 * q + r) * (int)g.y_stride + n); };
        auto load_y = [&](int i) {
            const int n = 128 * (first + i) + 8 * col;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (((mw >> (4 * q + r)) & 1u) && n < g.N) yv[r] = ldg128(y_at(r, n));
        };
        load_b(0);
        if (mw) load_y(0);
        store_b(0);
        __syncthreads();
        for (int i = 0; i < count; ++i) {
            if (i + 1 < count) load_b(i + 1);
            if (mw) {
                f32x4 acc[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) acc[k] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < RC; ++c) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const u32x4 b = buf[(i & 1) * BUF + (8 * col + k) * CP + ((4 * c + q) ^ (col & SWZ))];
                        acc[k] = mfma16x16x32<BF16>(thi[c], b, acc[k]);
                        acc[k] = mfma16x16x32<BF16>(tlo[c], b, acc[k]);
                    }
                }
                const int n = 128 * (first + i) + 8 * col;
                u32x4 out[4];
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t d = yv[r][w];
                        out[r][w] = f32_to_act2<BF16>(act_to_f32<BF16>((uint16_t)d) + acc[2 * w][r] * fb[r],
                                                      act_to_f32<BF16>((uint16_t)(d >> 16)) + acc[2 * w + 1][r] * fb[r]);
                    }
                if (i + 1 < count) load_y(i + 1);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (((mw >> (4 * q + r)) & 1u) && n < g.N) *reinterpret_cast<u32x4*>(y_at(r, n)) = out[r];
            }
            if (i + 1 < count) store_b(i + 1);
            __syncthreads();
        }
    }
}

int rank_tiles(int R) { return R <= 16 ? 1 : (R <= 32 ? 2 : 4); }

template <bool BF16, int RT>
void launch_down(const LoraArgs& g, hipStream_t s) {
    const int tiles = (g.M + 16 * TS - 1) / (16 * TS);
    const int groups = (g.R + 16 * RT - 1) / (16 * RT);
    const int wgs = tiles * g.ks * groups;
    const int side = std::max(1, std::min(std::min(16 * TS, g.adapters), 256 / wgs));
    const size_t lds = sizeof(u32x4) * 8 * 16 * (TS + RT) * DOWN_WAVES;
    static_assert(16 * (TS + RT) * 8 >= TS * RT * 64, "the waves' sums fit where the operands were");
    if (lds > 65536)
        (void)hipFuncSetAttribute(reinterpret_cast<const void*>(&lora_wide_down_kernel<BF16, RT>),
                                  hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    hipLaunchKernelGGL((lora_wide_down_kernel<BF16, RT>), dim3(wgs, side), dim3(64 * DOWN_WAVES), lds, s, g);
}

template <bool BF16, int RC>
void launch_up(const LoraArgs& g, hipStream_t s) {
    const int tiles = (g.M + 63) / 64;
    const int blocks = (g.N + 127) / 128;
    // steps of 128 outputs a workgroup takes, while 1024 workgroups are left: at most 8
    // (4096 rows, rank 64, 7168 x 20480, both products: 16 146 us, 8 128, 4 128, 2 143)
    const int per = (int)std::max<int64_t>(1, std::min<int64_t>(8, (int64_t)blocks * tiles / 1024));
    const int ranges = (blocks + per - 1) / per;
    const int side = (int)std::max<int64_t>(1, std::min<int64_t>(std::min(64, g.adapters), 1024 / ((int64_t)tiles * ranges)));
    hipLaunchKernelGGL((lora_wide_up_kernel<BF16, RC>), dim3((unsigned)(tiles * ranges), side), dim3(64 * UP_WAVES), 0,
                       s, g, per, ranges);
}

template <bool BF16>
void launch_t(const LoraArgs& g, hipStream_t s) {
    switch (rank_tiles(g.R)) {
        case 1: launch_down<BF16, 1>(g, s); break;
        case 2: launch_down<BF16, 2>(g, s); break;
        default: launch_down<BF16, 4>(g, s); break;
    }
    switch ((g.R + 31) / 32) {
        case 1: return launch_up<BF16, 1>(g, s);
        case 2: return launch_up<BF16, 2>(g, s);
        default: return launch_up<BF16, 4>(g, s);
    }
}

}  // namespace

// Large batches by the elements of x and y that pass: through LDS the loads are
// whole cache lines, at the price of a longer chain.  us here / in lora.hip, 8
// adapters in 11 prompts | in random order:
//   rank 8    4096 x 4096   2048 rows 22.9 / 21.0 | 45 / 53,  2730 rows 28.3 / 27.9 | 62 / 71,  4096 rows 29.7 / 34.0
//   rank 16   4096 x 4096   2048 rows 23.1 / 22.7 | 47 / 58,  2730 rows 28.9 / 30.7 | 63 / 79
//             7168 x 20480   348 rows 20.6 / 24.1 | 31 / 40,   697 rows 28.0 / 32.6 | 53 / 68
//   rank 24   4096 x 4096    341 rows 15.0 / 15.1 | 20 / 23,  1365 rows 21.0 / 21.2 | 44 / 56
//             7168 x 20480   261 rows 20.2 / 24.1 | 31 / 38,   5120 x 1536   512 rows 14.2 / 17.2 | 19 / 25
//   rank 32   4096 x 4096    341 rows 15.0 / 16.0 | 20 / 25,   5120 x 1536  2048 rows 21.6 / 26.7 | 45 / 83
//   rank 40   4096 x 4096    341 rows 20.5 / 18.2 | 28 / 29,   5120 x 1536   384 rows 16.0 / 20.6 | 23 / 30
//   rank 64   4096 x 4096    341 rows 20.7 / 21.0 | 28 / 39,   5120 x 1536   384 rows 16.4 / 22.8 | 23 / 37
//   rank 128  4096 x 4096    341 rows 28.4 / 31.0 | 44 / 67,   5120 x 1536   384 rows 26.3 / 32.9 | 43 / 74
// rank 64, 7168 x 20480, 100 rows: 30.1 / 24.2.  32 adapters in random order: rank 24
// 103 / 89 (4096 x 4096, 1365 rows) to 106 / 135 (5120 x 1536, 2048 rows), rank 128 101 / 154.
bool lora_wide(int M, int K, int N, int R) {
    return M >= 256 && R <= 128 && (int64_t)M * (K + 2 * (int64_t)N) > (R > 16 ? 3 << 20 : 32 << 20);
}

// K slices of the first product: a workgroup per CU (two measured the same, with
// twice the slices to add up), a step at least for each wave
int lora_wide_k_slices(int M, int K, int R) {
    const int ranks = 16 * rank_tiles(R);
    const int wgs = (M + 16 * TS - 1) / (16 * TS) * ((R + ranks - 1) / ranks);
    return std::max(1, std::min(std::min(LORA_MAX_SLICES, 256 / std::max(1, wgs)), K / LORA_STEP / DOWN_WAVES));
}

void launch_lora_wide(const LoraArgs& g, bool bf16, hipStream_t s) {
    if (bf16) launch_t<true>(g, s);
    else launch_t<false>(g, s);
}

}  // namespace wq
