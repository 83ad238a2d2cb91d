// lora.hip -- low-rank adapters of many requests added to a dense projection's
// output:  y[m] += scale_a * (x[m] A_a^T) B_a^T,  a = ids[m].
//
// Two launches: lora_down_kernel writes t = x A^T (fp32 [K slices, M, R]),
// lora_up_kernel adds scale * t B^T to y.  Both work on tiles of 16 TS tokens
// in the order they come in: a tile enumerates the different adapters among its
// tokens and takes one pass for each, of which every token keeps its own
// result (a select, not a product with zero: another request's infinities
// stay its own).  A prompt's tokens share one adapter, so its tiles take one
// pass; a decode batch's tile takes one per request, side by side in different
// workgroups, each adapter's weights read once.  Nothing has to be sorted or
// planned before.
//
// The intermediate t is scaled by a power of two to at most 1 per token (fp16 has
// the range then) and split in two 16-bit parts, hi + lo, which are both multiplied
// by the B rows (one register load of 32 ranks serves two matrix instructions).
// That holds t to 2^-16 of each value in bf16 (two parts of 8 bits), and to 2^-22 of
// it and 2^-24 of the token's largest in fp16 (two of 11, the least step of a value
// below 1 being 2^-24): far below y's own half step, 2^-8 and 2^-11, at two
// instructions a product, where 32-bit products have 1 / 16 of the rate.
//
// Bound by the chain of dependent loads (ids, weights, t, y), not by bytes: 8
// rows of 8 adapters, rank 16, 4096 x 4096 bf16, 4.5 + 4.9 us for 2.3 MB; 203 rows,
// rank 24, 5120 x 1544 fp16, 8.8 + 4.3 us.  Large batches: lora_wide.hip.
#include "lora_common.hpp"

#include <algorithm>

namespace wq {

namespace {

constexpr int UP_WAVES = 4;
constexpr int DOWN_WAVES = 8;

// t = x A^T of the tile's tokens over one slice of K and one group of 16 RT
// ranks.  The waves take the 64-channel steps of the slice in turn (a row's 128
// bytes, one cache line, by one wave), DEPTH of a wave's steps in flight; D's
// columns are tokens, its rows ranks; the waves' sums are added in LDS in wave
// order.  Loads are unconditional: rows past M or R read the last one (their
// results are dropped), steps past the slice its last step; the channels past
// the last whole step go through a step of their own with zeros on both sides.
template <bool BF16, int TS, int RT, int WAVES, int DEPTH>
__global__ __launch_bounds__(64 * WAVES) void lora_down_kernel(LoraArgs g) {
    __shared__ f32x4 red[WAVES][TS][RT][64];
    const int lane = threadIdx.x & 63;
    const int wave = wave_index();
    const int col = lane & 15, q = lane >> 4;
    const int tile = blockIdx.x;
    const int slice = blockIdx.z % g.ks, r0 = blockIdx.z / g.ks * (16 * RT);

    const int steps = g.K / LORA_STEP;
    const int s0 = (int)((int64_t)slice * steps / g.ks), s1 = (int)((int64_t)(slice + 1) * steps / g.ks);
    const int mine_steps = s0 + wave < s1 ? (s1 - s0 - wave + WAVES - 1) / WAVES : 0;

    const uint16_t* xr[TS];
#pragma unroll
    for (int t = 0; t < TS; ++t)
        xr[t] = g.x + (int64_t)min(tile * 16 * TS + 16 * t + col, g.M - 1) * g.x_stride + 8 * q;
    u32x4 xv[DEPTH][2][TS], av[DEPTH][2][RT];
    auto channel = [&](int i) { return LORA_STEP * (s0 + wave + WAVES * min(i, mine_steps - 1)); };
    auto load_x = [&](int i, int b) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int t = 0; t < TS; ++t) xv[b][h][t] = ldg128(xr[t] + channel(i) + 32 * h);
    };
    if (mine_steps > 0) {  // on its way while the tile's adapters are found
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) load_x(d, d);
    }
    const int ids = tile_ids<16 * TS>(g, tile, lane);

    bool first = true;
    uint64_t left = __ballot(ids >= 0), mine;
    for (int j = 0; left; ++j) {
        const int a = next_adapter(ids, left, mine);
        if (j % (int)gridDim.y != (int)blockIdx.y) continue;
        const uint16_t* ar[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r)
            ar[r] = g.a + ((size_t)a * g.R + min(r0 + 16 * r + col, g.R - 1)) * g.K + 8 * q;

        f32x4 acc[TS][RT];
#pragma unroll
        for (int t = 0; t < TS; ++t)
#pragma unroll
            for (int r = 0; r < RT; ++r) acc[t][r] = f32x4{0.f, 0.f, 0.f, 0.f};
        auto multiply = [&](const u32x4 (&av)[RT], const u32x4 (&xv)[TS]) {
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int t = 0; t < TS; ++t) acc[t][r] = mfma16x16x32<BF16>(av[r], xv[t], acc[t][r]);
        };
        if (mine_steps > 0) {
            auto load_a = [&](int i, int b) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < RT; ++r) av[b][h][r] = ldg128(ar[r] + channel(i) + 32 * h);
            };
#pragma unroll
            for (int d = 0; d < DEPTH; ++d) {
                if (!first) load_x(d, d);
                load_a(d, d);
            }
            first = false;
            for (int i = 0; i < mine_steps; i += DEPTH) {
#pragma unroll
                for (int d = 0; d < DEPTH; ++d) {
                    if (i + d < mine_steps) {
                        multiply(av[d][0], xv[d][0]);
                        multiply(av[d][1], xv[d][1]);
                    }
                    if (i + DEPTH < mine_steps) {
                        load_x(i + DEPTH + d, d);
                        load_a(i + DEPTH + d, d);
                    }
                }
            }
        }
        if (g.K % LORA_STEP && slice == g.ks - 1 && wave == WAVES - 1) {
            const u32x4 none = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = LORA_STEP * steps + 32 * h;
                const bool in = c + 8 * q < g.K;
                u32x4 xl[TS], al[RT];
#pragma unroll
                for (int t = 0; t < TS; ++t) xl[t] = in ? ldg128(xr[t] + c) : none;
#pragma unroll
                for (int r = 0; r < RT; ++r) al[r] = in ? ldg128(ar[r] + c) : none;
                multiply(al, xl);
            }
        }
#pragma unroll
        for (int t = 0; t < TS; ++t)
#pragma unroll
            for (int r = 0; r < RT; ++r) red[wave][t][r][lane] = acc[t][r];
        __syncthreads();
#pragma unroll
        for (int i = wave; i < TS * RT; i += WAVES) {
            const int t = i / RT, r = i % RT;
            f32x4 v = red[0][t][r][lane];
#pragma unroll
            for (int w = 1; w < WAVES; ++w) v += red[w][t][r][lane];
            const int rank = r0 + 16 * r + 4 * q;
            const int tok = 16 * t + col;
            if (((mine >> tok) & 1ull) && rank < g.R)
                *reinterpret_cast<f32x4*>(g.t + ((size_t)slice * g.M + tile * 16 * TS + tok) * g.R + rank) = v;
        }
        __syncthreads();
    }
}

// y += scale * t B^T for the tile's tokens and a range of outputs.  The
// workgroup adds up the K slices of its tokens' t (8 threads a token, 8 ranks
// each at a time), splits the sums and leaves them in LDS as matrix operands
// of 32 ranks, high and low parts; in a pass each wave takes 64 outputs at a time.
// Weight tile k holds outputs 32 (k / 2) + 8 (row / 4) + 4 (k % 2) + row % 4 of
// the 64, so that a lane's results of two tiles are 8 outputs in a row of one
// token (a 16-byte access) and the four lane groups' are 32: whole 64-byte
// pieces of y.  (With a lane's 16 results in a row, two accesses each touched
// half of every piece, and prompts took 1.5 times as long.)  The B rows and y of the next 64 outputs are in
// flight while these are added.  RC: chunks of 32 ranks held at a time; RG:
// groups of 64 ranks a token's t takes.
template <bool BF16, int TS, int RC, int RG>
__global__ __launch_bounds__(64 * UP_WAVES, RG == 1 ? 3 : 2) void lora_up_kernel(LoraArgs g, int per_wave) {
    constexpr int TOKENS = 16 * TS;
    extern __shared__ u32x4 frag[];  // [TS][R / 32 rounded up][hi, lo][64]
    __shared__ float back[TOKENS];   // what a token's products are multiplied by
    const int lane = threadIdx.x & 63;
    const int wave = wave_index();
    const int col = lane & 15, q = lane >> 4;
    const int tile = blockIdx.x;
    const int chunks = (g.R + 31) / 32;
    const int n_first = blockIdx.y * (64 * UP_WAVES * per_wave) + 64 * wave;  // the waves side by side
    const int n_count = max(0, min(per_wave, (g.N - n_first + 64 * UP_WAVES - 1) / (64 * UP_WAVES)));

    const int tok = threadIdx.x >> 3;
    if (tok < TOKENS) {
        const int gr = threadIdx.x & 7;
        const float f = split_token<BF16, RG>(g, min(tile * TOKENS + tok, g.M - 1), gr, [&](int w, u32x4 hi, u32x4 lo) {
            const int c = 2 * w + (gr >> 2);
            if (c >= chunks) return;  // (ranks past R in the last chunk are written, as zeros)
            u32x4* to = frag + ((tok >> 4) * chunks + c) * 128 + 16 * (gr & 3) + (tok & 15);
            to[0] = hi;
            to[64] = lo;
        });
        if (gr == 0) back[tok] = f;
    }

    const int ids = tile_ids<TOKENS>(g, tile, lane);
    __syncthreads();

    uint64_t left = __ballot(ids >= 0), mine;
    for (int j = 0; left; ++j) {
        const int a = next_adapter(ids, left, mine);
        if (j % (int)gridDim.z != (int)blockIdx.z) continue;
        const uint16_t* bw = g.b + (size_t)a * g.N * g.R;

        u32x4 bv[RC][4];
        u32x4 yv[TS][2];
        // (ranks past R: the last ones, replaced by zeros before use)
        auto load_b = [&](int n0, int c0) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int n = min(n0 + 32 * (k >> 1) + 8 * (col >> 2) + 4 * (k & 1) + (col & 3), g.N - 1);
#pragma unroll
                for (int r = 0; r < RC; ++r)
                    bv[r][k] = ldg128(bw + (uint32_t)(n * g.R + min(32 * (c0 + r) + 8 * q, g.R - 8)));
            }
        };
        // a token's outputs start (16 t + col) rows below the tile's first
        uint16_t* yt = g.y + (int64_t)tile * TOKENS * g.y_stride;
        auto y_at = [&](int t, int n) { return yt + (uint32_t)((16 * t + col) * (int)g.y_stride + n); };
        auto load_y = [&](int n0) {
#pragma unroll
            for (int t = 0; t < TS; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int n = n0 + 32 * h + 8 * q;
                    if (((mine >> (16 * t + col)) & 1ull) && n < g.N) yv[t][h] = ldg128(y_at(t, n));
                }
        };
        if (n_count > 0) {
            load_b(n_first, 0);
            load_y(n_first);
        }


        for (int i = 0; i < n_count; ++i) {
            const int n0 = n_first + 64 * UP_WAVES * i;
            f32x4 acc[TS][4];
#pragma unroll
            for (int t = 0; t < TS; ++t)
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[t][k] = f32x4{0.f, 0.f, 0.f, 0.f};
            for (int c0 = 0; c0 < chunks; c0 += RC) {
                if (c0 > 0) load_b(n0, c0);
#pragma unroll
                for (int r = 0; r < RC; ++r) {
                    if (c0 + r >= chunks) break;
                    if (32 * (c0 + r + 1) > g.R) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            bv[r][k] = 32 * (c0 + r) + 8 * q < g.R ? bv[r][k] : u32x4{0u, 0u, 0u, 0u};
                    }
#pragma unroll
                    for (int t = 0; t < TS; ++t) {
                        const u32x4* tv = frag + (t * chunks + c0 + r) * 128 + lane;
                        const u32x4 hi = tv[0], lo = tv[64];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            acc[t][k] = mfma16x16x32<BF16>(bv[r][k], hi, acc[t][k]);
                            acc[t][k] = mfma16x16x32<BF16>(bv[r][k], lo, acc[t][k]);
                        }
                    }
                }
            }
            if (i + 1 < n_count) load_b(n0 + 64 * UP_WAVES, 0);
            u32x4 out[TS][2];
#pragma unroll
            for (int t = 0; t < TS; ++t) {
                const float f = back[16 * t + col];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const int k = 8 * h + 2 * w;
                        const uint32_t d = yv[t][h][w];
                        const float v0 = act_to_f32<BF16>((uint16_t)d) + acc[t][k >> 2][k & 3] * f;
                        const float v1 = act_to_f32<BF16>((uint16_t)(d >> 16)) + acc[t][k >> 2][(k & 3) + 1] * f;
                        out[t][h][w] = f32_to_act2<BF16>(v0, v1);
                    }
            }
            if (i + 1 < n_count) load_y(n0 + 64 * UP_WAVES);
#pragma unroll
            for (int t = 0; t < TS; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int n = n0 + 32 * h + 8 * q;
                    if (((mine >> (16 * t + col)) & 1ull) && n < g.N)
                        *reinterpret_cast<u32x4*>(y_at(t, n)) = out[t][h];
                }
        }
    }
}

constexpr int TS = 1;  // 16-token tiles: workgroups to fill the chip

// ranks a workgroup takes at a time, in tiles of 16
int rank_tiles(int R) { return R <= 16 ? 1 : (R <= 32 ? 2 : 4); }

template <bool BF16, int RT>
void launch_cfg(const LoraArgs& g, hipStream_t s) {
    const int tiles = (g.M + 16 * TS - 1) / (16 * TS);
    const int groups = (g.R + 16 * RT - 1) / (16 * RT);
    // passes side by side: a workgroup for each adapter of a tile while there are few tiles
    const int most = std::min(std::min(16 * TS, g.adapters), g.M);
    const int side = std::max(1, std::min(most, 1024 / std::max(1, tiles * g.ks * groups)));
    hipLaunchKernelGGL((lora_down_kernel<BF16, TS, RT, DOWN_WAVES, 2>), dim3(tiles, side, g.ks * groups),
                       dim3(64 * DOWN_WAVES), 0, s, g);
    const int blocks = (g.N + 64 * UP_WAVES - 1) / (64 * UP_WAVES);
    const int per_wave = (int)std::max<int64_t>(1, std::min<int64_t>(4, (int64_t)blocks * tiles / 1024));
    const int ranges = (blocks + per_wave - 1) / per_wave;
    const int side2 = (int)std::max<int64_t>(1, std::min<int64_t>(most, 1024 / ((int64_t)tiles * ranges)));
    const dim3 grid(tiles, ranges, side2);
    const size_t lds = sizeof(u32x4) * 128 * TS * ((g.R + 31) / 32);
    if (g.R <= 64)
        hipLaunchKernelGGL((lora_up_kernel<BF16, TS, (RT + 1) / 2, 1>), grid, dim3(64 * UP_WAVES), lds, s, g, per_wave);
    else
        hipLaunchKernelGGL((lora_up_kernel<BF16, TS, 2, 4>), grid, dim3(64 * UP_WAVES), lds, s, g, per_wave);
}

template <bool BF16>
void launch_t(const LoraArgs& g, hipStream_t s) {
    switch (rank_tiles(g.R)) {
        case 1: return launch_cfg<BF16, 1>(g, s);
        case 2: return launch_cfg<BF16, 2>(g, s);
        default: return launch_cfg<BF16, 4>(g, s);
    }
}

}  // namespace

// K slices of the first product: workgroups to fill the chip, at most 4 (the
// second product adds them up), a step of 64 channels at least for each wave
int lora_k_slices(int M, int K, int N, int R) {
    if (lora_wide(M, K, N, R)) return lora_wide_k_slices(M, K, R);
    const int rows = 16 * TS, ranks = 16 * rank_tiles(R);
    const int wgs = (M + rows - 1) / rows * ((R + ranks - 1) / ranks);
    return std::max(1, std::min(std::min(LORA_MAX_SLICES, 512 / std::max(1, wgs)), K / LORA_STEP / DOWN_WAVES));
}

void launch_lora(const LoraArgs& g, bool bf16, hipStream_t s) {
    if (lora_wide(g.M, g.K, g.N, g.R)) return launch_lora_wide(g, bf16, s);
    if (bf16) launch_t<true>(g, s);
    else launch_t<false>(g, s);
}

}  // namespace wq
