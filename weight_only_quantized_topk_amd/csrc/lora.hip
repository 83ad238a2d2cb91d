// lora.hip -- low-rank adapters of many requests added to a dense projection's
// output:  y[m] += scale_a * (x[m] A_a^T) B_a^T,  a = ids[m].
//
// Two launches: lora_down_kernel writes t = x A^T (fp32 [K slices, M, R]),
// lora_up_kernel adds scale * t B^T to y.  Both work on tiles of 16 TS tokens
// in the order they come in: a tile enumerates the different adapters among its
// tokens and takes one pass for each, of which every token keeps its own
// result (a select, not a product with zero: another request's infinities
// stay its own).  A prompt's tokens share one adapter, so its tiles take one
// pass; a decode batch's tile takes one per request, each adapter's weights
// read once.  Nothing has to be sorted or planned before.
//
// The intermediate t stays in fp32's precision: it is scaled by a power of two
// to at most 1 per token (fp16 has the range then) and split in two 16-bit
// parts, hi + lo, whose products with the same B rows are both taken, as the
// two halves of one 32-deep matrix instruction's reduction (16 ranks each).
#include "common.hpp"
#include "launch.hpp"

#include <algorithm>

namespace wq {

namespace {

constexpr int RANK_GROUP = 64;  // ranks of one pass: 4 tiles of 16
constexpr int DOWN_WAVES = 4;
constexpr int UP_WAVES = 4;

// The adapters of a tile of up to 64 tokens: lane i holds token i's (-1: none,
// an id out of range counts as none), first marks each one's first token
struct TileIds {
    int id;
    uint64_t first;
};
__device__ __forceinline__ TileIds tile_ids(const LoraArgs& g, int tile, int tokens, int lane) {
    TileIds t;
    const int m = tile * tokens + lane;
    t.id = (lane < tokens && m < g.M) ? g.ids[m] : -1;
    if (t.id < 0 || t.id >= g.adapters) t.id = -1;
    bool seen = t.id < 0;
    for (int i = 0; i < tokens; ++i) seen = seen || (i < lane && __builtin_amdgcn_readlane(t.id, i) == t.id);
    t.first = __ballot(!seen);
    return t;
}

// t = x A^T of the tile's tokens over one slice of K and one group of 64 ranks.
// Four waves take the 32-channel steps of the slice in turn; D's columns are
// tokens, its rows ranks; the waves' sums are added in LDS in wave order.
template <bool BF16, int TS>
__global__ __launch_bounds__(64 * DOWN_WAVES) void lora_down_kernel(LoraArgs g) {
    constexpr int RT = RANK_GROUP / 16;
    __shared__ f32x4 red[DOWN_WAVES][TS][RT][64];
    const int lane = threadIdx.x & 63;
    const int wave = threadIdx.x >> 6;
    const int col = lane & 15, q = lane >> 4;
    const int tile = blockIdx.x;
    const int slice = blockIdx.z % g.ks, r0 = blockIdx.z / g.ks * RANK_GROUP;
    const int rts = min(RT, (g.R - r0 + 15) / 16);

    const TileIds ids = tile_ids(g, tile, 16 * TS, lane);
    const int passes = __popcll(ids.first);
    const int steps = (g.K + 31) / 32;
    const int s0 = (int)((int64_t)slice * steps / g.ks), s1 = (int)((int64_t)(slice + 1) * steps / g.ks);

    const uint16_t* xr[TS];
#pragma unroll
    for (int t = 0; t < TS; ++t)
        xr[t] = g.x + (int64_t)min(tile * 16 * TS + 16 * t + col, g.M - 1) * g.x_stride + 8 * q;

    uint64_t left = ids.first;
    for (int j = 0; j < passes; ++j, left &= left - 1) {
        if (j % (int)gridDim.y != (int)blockIdx.y) continue;
        const int a = __builtin_amdgcn_readlane(ids.id, __builtin_ctzll(left));
        const uint64_t mine = __ballot(ids.id == a);
        const uint16_t* ar = g.a + (size_t)a * g.R * g.K + 8 * q;
        const uint16_t* arow[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) arow[r] = ar + (size_t)min(r0 + 16 * r + col, g.R - 1) * g.K;

        f32x4 acc[TS][RT];
#pragma unroll
        for (int t = 0; t < TS; ++t)
#pragma unroll
            for (int r = 0; r < RT; ++r) acc[t][r] = f32x4{0.f, 0.f, 0.f, 0.f};
        u32x4 xv[2][TS], av[2][RT];
        auto load = [&](int s, int b) {
            const bool in = s < s1 && 32 * s + 8 * q < g.K;  // channels past K: zeros on both sides
#pragma unroll
            for (int t = 0; t < TS; ++t)
                xv[b][t] = in && ((mine >> (16 * t)) & 0xFFFFull) ? ldg128(xr[t] + 32 * s) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
            for (int r = 0; r < RT; ++r)
                av[b][r] = in && r < rts ? ldg128(arow[r] + 32 * s) : u32x4{0u, 0u, 0u, 0u};
        };
        auto compute = [&](int b) {
#pragma unroll
            for (int r = 0; r < RT; ++r)
                if (r < rts)
#pragma unroll
                    for (int t = 0; t < TS; ++t) acc[t][r] = mfma16x16x32<BF16>(av[b][r], xv[b][t], acc[t][r]);
        };
        load(s0 + wave, 0);
        for (int s = s0 + wave; s < s1; s += 2 * DOWN_WAVES) {
            load(s + DOWN_WAVES, 1);
            compute(0);
            load(s + 2 * DOWN_WAVES, 0);
            compute(1);
        }
#pragma unroll
        for (int t = 0; t < TS; ++t)
#pragma unroll
            for (int r = 0; r < RT; ++r) red[wave][t][r][lane] = acc[t][r];
        __syncthreads();
        for (int i = wave; i < TS * RT; i += DOWN_WAVES) {
            const int t = i / RT, r = i % RT;
            f32x4 v = red[0][t][r][lane];
#pragma unroll
            for (int w = 1; w < DOWN_WAVES; ++w) v += red[w][t][r][lane];
            const int rank = r0 + 16 * r + 4 * q;
            const int tok = 16 * t + col;
            if (((mine >> tok) & 1ull) && rank < g.R)
                *reinterpret_cast<f32x4*>(g.t + ((size_t)slice * g.M + tile * 16 * TS + tok) * g.R + rank) = v;
        }
        __syncthreads();
    }
}

// The two 16-bit parts of a token's t for one tile of 16 ranks, as the matrix
// instruction's B operand: lane group q holds ranks 8 (q % 2) .. + 7 of the
// tile, the high parts in groups 0 and 1, the low parts in 2 and 3
template <bool BF16>
__device__ __forceinline__ u32x4 split_part(const float (&v)[8], float f, bool low) {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t w = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float s = v[2 * i + h] * f;
            const uint16_t hi = f32_to_act<BF16>(s);
            const float rest = s - act_to_f32<BF16>(hi);
            const uint16_t lo = fabsf(s) < __builtin_inff() ? f32_to_act<BF16>(rest) : (uint16_t)0;
            w |= (uint32_t)(low ? lo : hi) << (16 * h);
        }
        o[i] = w;
    }
    return o;
}

// y += scale * t B^T for the tile's tokens and a range of outputs: a wave takes
// 64 outputs at a time.  Weight tile k holds outputs 16 (row / 4) + 4 k + row % 4
// of the 64, so that a lane's four results of the four tiles are 16 outputs in
// a row of one token: two 16-byte accesses of y.
template <bool BF16, int TS>
__global__ __launch_bounds__(64 * UP_WAVES) void lora_up_kernel(LoraArgs g, int per_wave) {
    constexpr int RT = RANK_GROUP / 16;
    const int lane = threadIdx.x & 63;
    const int wave = threadIdx.x >> 6;
    const int col = lane & 15, q = lane >> 4;
    const int tile = blockIdx.x;
    const TileIds ids = tile_ids(g, tile, 16 * TS, lane);
    const int groups = (g.R + RANK_GROUP - 1) / RANK_GROUP;
    const int n_first = (blockIdx.y * UP_WAVES + wave) * 64 * per_wave;

    for (uint64_t left = ids.first; left; left &= left - 1) {
        const int a = __builtin_amdgcn_readlane(ids.id, __builtin_ctzll(left));
        const uint64_t mine = __ballot(ids.id == a);
        const float scale = g.scales ? g.scales[a] : 1.0f;
        const uint16_t* bw = g.b + (size_t)a * g.N * g.R;

        u32x4 tv[TS][RT];
        float back[TS];
        auto load_t = [&](int grp) {
            const int r0 = grp * RANK_GROUP + 8 * (q & 1);
#pragma unroll
            for (int t = 0; t < TS; ++t) {
                back[t] = 0.0f;
                if (!((mine >> (16 * t)) & 0xFFFFull)) continue;
                const float* src = g.t + (size_t)min(tile * 16 * TS + 16 * t + col, g.M - 1) * g.R + r0;
                float v[RT][8];
                float top = 0.0f;
#pragma unroll
                for (int r = 0; r < RT; ++r) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[r][i] = 0.0f;
                    if (r0 + 16 * r < g.R)
                        for (int z = 0; z < g.ks; ++z) {
                            const f32x4 lo = *reinterpret_cast<const f32x4*>(src + (size_t)z * g.M * g.R + 16 * r);
                            const f32x4 hi = *reinterpret_cast<const f32x4*>(src + (size_t)z * g.M * g.R + 16 * r + 4);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                v[r][i] += lo[i];
                                v[r][4 + i] += hi[i];
                            }
                        }
#pragma unroll
                    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[r][i]));
                }
                top = fmaxf(top, __shfl_xor(top, 16, 64));  // the token's other 8 ranks of each tile
                const uint32_t e = min(__float_as_uint(top) >> 23, 252u);
                const float f = __uint_as_float((253u - e) << 23);  // 2^(126 - e)
                back[t] = __uint_as_float((e + 1u) << 23) * scale;
#pragma unroll
                for (int r = 0; r < RT; ++r) tv[t][r] = split_part<BF16>(v[r], f, q >= 2);
            }
        };
        if (groups == 1) load_t(0);

        for (int i = 0; i < per_wave; ++i) {
            const int n0 = n_first + 64 * i;
            if (n0 >= g.N) break;
            float out[TS][16];
#pragma unroll
            for (int t = 0; t < TS; ++t)
#pragma unroll
                for (int k = 0; k < 16; ++k) out[t][k] = 0.0f;
            for (int grp = 0; grp < groups; ++grp) {
                if (groups > 1) load_t(grp);
                f32x4 acc[TS][4];
#pragma unroll
                for (int t = 0; t < TS; ++t)
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[t][k] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const int rank = grp * RANK_GROUP + 16 * r + 8 * (q & 1);
                    if (grp * RANK_GROUP + 16 * r >= g.R) continue;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int n = min(n0 + 16 * (col >> 2) + 4 * k + (col & 3), g.N - 1);
                        const u32x4 w = rank < g.R ? ldg128(bw + (size_t)n * g.R + rank) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
                        for (int t = 0; t < TS; ++t)
                            if ((mine >> (16 * t)) & 0xFFFFull) acc[t][k] = mfma16x16x32<BF16>(w, tv[t][r], acc[t][k]);
                    }
                }
#pragma unroll
                for (int t = 0; t < TS; ++t)
#pragma unroll
                    for (int k = 0; k < 16; ++k) out[t][k] = fmaf(acc[t][k >> 2][k & 3], back[t], out[t][k]);
            }
#pragma unroll
            for (int t = 0; t < TS; ++t) {
                if (!((mine >> (16 * t + col)) & 1ull)) continue;
                uint16_t* y = g.y + (int64_t)(tile * 16 * TS + 16 * t + col) * g.y_stride + n0 + 16 * q;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (n0 + 16 * q + 8 * h >= g.N) continue;
                    u32x4 d = ldg128(y + 8 * h);
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const float v0 = act_to_f32<BF16>((uint16_t)d[w]) + out[t][8 * h + 2 * w];
                        const float v1 = act_to_f32<BF16>((uint16_t)(d[w] >> 16)) + out[t][8 * h + 2 * w + 1];
                        d[w] = (uint32_t)f32_to_act<BF16>(v0) | ((uint32_t)f32_to_act<BF16>(v1) << 16);
                    }
                    *reinterpret_cast<u32x4*>(y + 8 * h) = d;
                }
            }
        }
    }
}

// 16-token tiles up to 512 tokens (workgroups to fill the chip), 64 above (the
// adapters' weights are read once per tile)
int token_tiles(int M) { return M <= 512 ? 1 : 4; }

template <bool BF16, int TS>
void launch_ts(LoraArgs g, hipStream_t s) {
    const int tiles = (g.M + 16 * TS - 1) / (16 * TS);
    const int groups = (g.R + RANK_GROUP - 1) / RANK_GROUP;
    // passes side by side: a workgroup for each adapter of a tile while there are few tiles
    const int most = std::min(std::min(16 * TS, g.adapters), g.M);
    const int side = std::max(1, std::min(most, 1024 / std::max(1, tiles * g.ks * groups)));
    hipLaunchKernelGGL((lora_down_kernel<BF16, TS>), dim3(tiles, side, g.ks * groups), dim3(64 * DOWN_WAVES), 0, s, g);
    const int blocks = (g.N + 64 * UP_WAVES - 1) / (64 * UP_WAVES);
    const int per_wave = std::max(1, std::min(4, (int)((int64_t)blocks * tiles / 1024)));
    hipLaunchKernelGGL((lora_up_kernel<BF16, TS>), dim3(tiles, (blocks + per_wave - 1) / per_wave),
                       dim3(64 * UP_WAVES), 0, s, g, per_wave);
}

}  // namespace

// K slices of the first product: workgroups to fill the chip, at least 2 steps
// of 32 channels for each of their four waves
int lora_k_slices(int M, int K, int R) {
    const int ts = token_tiles(M);
    const int wgs = (M + 16 * ts - 1) / (16 * ts) * ((R + RANK_GROUP - 1) / RANK_GROUP);
    const int steps = (K + 31) / 32;
    return std::max(1, std::min(std::min(16, 512 / std::max(1, wgs)), steps / (2 * DOWN_WAVES)));
}

void launch_lora(const LoraArgs& g, bool bf16, hipStream_t s) {
    const bool wide = token_tiles(g.M) > 1;
    if (bf16) wide ? launch_ts<true, 4>(g, s) : launch_ts<true, 1>(g, s);
    else wide ? launch_ts<false, 4>(g, s) : launch_ts<false, 1>(g, s);
}

}  // namespace wq
