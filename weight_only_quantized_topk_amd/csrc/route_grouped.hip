// route_grouped.hip -- moe_route_grouped: 16 or 64 lanes per token
// (route_grouped.hpp), 256 lanes a workgroup; with the sort for small batches in
// one workgroup, as route_align_kernel: the pairs' experts stay in LDS, up to 64
// pairs are sorted by one wave, more by the whole workgroup.
// Bound by instructions: the exponentials in double (one per expert where a bias,
// the groups' two best or the softmax's sum need them) and the rounds of the
// choice.  Kernel time: one token of 160 experts with its sort 6.0 us, 61 tokens
// of 96 experts 4.7 us (and 4.4 us the sort), 8192 tokens of 256 experts, sigmoid
// with a bias and 8 groups, 14.1 us (a read of its logits: 1.6 us).
#include "route_grouped.hpp"

#include <algorithm>

#include "route_sort.hpp"

namespace wq {

template <int W, int PL>
__global__ __launch_bounds__(256) void route_grouped_kernel(RouteGroupedArgs g, GroupedLayout y) {
    const int m = blockIdx.x * (256 / W) + threadIdx.x / W;
    const int r = threadIdx.x % W;
    if (W == 64 && m >= g.M) return;  // a whole wave
    route_token_grouped<W, PL>(g, y, min(m, g.M - 1), m < g.M, r, (threadIdx.x & 63) - r, nullptr);
}

template <int PL>
__global__ __launch_bounds__(ALIGN_THREADS) void route_grouped_align_kernel(RouteGroupedArgs g, GroupedLayout y, int BS,
                                                                            int nbits, int32_t* __restrict__ sorted,
                                                                            int32_t* __restrict__ expert_ids,
                                                                            int32_t* __restrict__ ntpp, int cap) {
    extern __shared__ int smem[];
    const int lane = threadIdx.x & 63;
    const int wave = threadIdx.x >> 6;
    const int T = g.M * g.topk;
    int* sids = smem;
    if (wave < g.M) route_token_grouped<64, PL>(g, y, wave, true, lane, 0, sids + wave * g.topk);
    __syncthreads();
    if (T <= ROUTE_ALIGN_WAVE_MAX) {
        if (wave == 0) align_pairs(sids, T, BS, cap, lane, sorted, expert_ids, ntpp);
        return;
    }
    align_body(sids, T, g.E, BS, nbits, sorted, expert_ids, ntpp, cap, smem + T);
}

// f(PL) for the experts a lane holds
template <class F>
static void with_per_lane(int per, F f) {
    if (per <= 1) f(std::integral_constant<int, 1>{});
    else if (per <= 2) f(std::integral_constant<int, 2>{});
    else if (per <= 4) f(std::integral_constant<int, 4>{});
    else if (per <= 8) f(std::integral_constant<int, 8>{});
    else if (per <= 12) f(std::integral_constant<int, 12>{});
    else if (per <= 16) f(std::integral_constant<int, 16>{});
    else f(std::integral_constant<int, 32>{});
}

// Lanes per token: 16 lanes and four tokens a wave take fewer instructions per
// token, 64 lanes the shorter chain (a lane's exponentials in double and its
// compares follow one another): 16 lanes pay from 400 tokens per expert of a lane where
// every expert has its exponential, from 200 where the slots alone have one.  us with
// 16 / 64 lanes, sigmoid with a bias and groups' two best | renormalised softmax:
//   96 experts (8 per lane)   3000 tokens  5.7 /  4.7,  3600  5.7 /  5.3 | 1200  3.5 / 3.6,  1800  3.5 / 3.7
//   128 experts (8 per lane)  2720 tokens  7.3 /  6.5,  3200  7.3 /  7.4 | 1600  5.0 / 5.1,  3200  5.1 / 6.7
//   160 experts (12 per lane) 4096 tokens  8.3 /  8.3,  5000  9.4 /  9.7 | 2000  5.2 / 4.8,  3000  5.2 / 5.6
//   256 experts (16 per lane) 5440 tokens 12.8 / 12.0,  8000 13.0 / 14.8 | 3200  6.5 / 7.1,  5440  7.3 / 9.2
//   8 experts (1 per lane)     200 tokens  2.7 /  2.9                    |  200  2.5 / 2.8
static bool route_by_16(const RouteGroupedArgs& g, const GroupedLayout& few) {
    const bool slots_only = !g.bias && !(g.top2 && g.groups > 1) && (g.sigmoid || g.renormalize);
    return few.lpg > 0 && few.per <= 16 && g.M >= (slots_only ? 200 : 400) * few.per;
}

void launch_route_grouped(const RouteGroupedArgs& g, hipStream_t s) {
    const GroupedLayout few = grouped_layout(g.E, g.groups, 16);
    if (route_by_16(g, few)) {
        with_per_lane(few.per, [&](auto P) {
            if constexpr (decltype(P)::value <= 16)
                hipLaunchKernelGGL((route_grouped_kernel<16, decltype(P)::value>), dim3((g.M + 15) / 16), dim3(256), 0, s,
                                   g, few);
        });
        return;
    }
    const GroupedLayout y = grouped_layout(g.E, g.groups, 64);
    with_per_lane(y.per, [&](auto P) {
        hipLaunchKernelGGL((route_grouped_kernel<64, decltype(P)::value>), dim3((g.M + 3) / 4), dim3(256), 0, s, g, y);
    });
}

// with the sort in one workgroup, a wave per token: up to 16 tokens.  (Up to 64
// tokens by 16 lanes each, in the one workgroup: 61 tokens, 96 experts 12.4 us;
// two launches 8.6 us.)
bool route_grouped_fused(const RouteGroupedArgs& g) { return route_align_fused(g.M, g.topk); }

void launch_route_grouped_align(const RouteGroupedArgs& g, int BS, int32_t* sorted, int32_t* expert_ids,
                                int32_t* ntpp, int cap, hipStream_t s) {
    const GroupedLayout y = grouped_layout(g.E, g.groups, 64);
    const int T = g.M * g.topk;
    const bool one_wave = T <= ROUTE_ALIGN_WAVE_MAX;
    const int threads = one_wave ? 64 * g.M : ALIGN_THREADS;
    int nbits = 0;  // of an expert id
    while ((1 << nbits) < g.E) ++nbits;
    const size_t lds = sizeof(int) * ((size_t)T + (one_wave ? 0 : (size_t)g.E * ALIGN_WAVES));
    with_per_lane(y.per, [&](auto P) {
        constexpr int PL = decltype(P)::value;
        if (lds > 65536)
            (void)hipFuncSetAttribute(reinterpret_cast<const void*>(&route_grouped_align_kernel<PL>),
                                      hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        hipLaunchKernelGGL(route_grouped_align_kernel<PL>, dim3(1), dim3(threads), lds, s, g, y, BS, nbits, sorted,
                           expert_ids, ntpp, cap);
    });
}

}  // namespace wq
