// route_grouped.hpp -- one token's routing with scores, a balancing bias and
// expert groups, by one 64-lane wave, and the padded sort of up to 64 pairs
// over any number of experts by one wave.
//
//   s_e = softmax over all experts, or sigmoid, of the logits     (double)
//   c_e = float(s_e + b_e) with a bias; without one the order is that of the
//         logits themselves, and c_e = float(s_e)
//   group value = its best expert's order value, or c_1 + c_2 of its two
//         largest c (one float addition); the topk_group best groups are open
//   slots = the topk best experts of the open groups
//   w_j = scale * s_j, over the slots' sum of s when renormalised; a sum of
//         zero gives weights of zero
// Equal values: the lower group, the lower expert.  A NaN ranks below every
// number, so the slots always name topk different experts.
//
// Layout: the groups, padded to a power of two, share the wave's lanes evenly
// (LPG lanes each) and a lane holds PL consecutive experts of its group, so
// experts ascend with (lane, slot): the lowest expert of the largest value is
// found by a ballot's first lane.  The largest 32-bit key of a wave is taken
// by DPP within rows of 16 lanes and four scalar reads across them: no LDS.  A
// round of the choice is that, a ballot and PL compares per lane.
#pragma once

#include "common.hpp"
#include "launch.hpp"
#include "route_common.hpp"

namespace wq {

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xF, 0xF, false);
}

// the largest value of each aligned run of `width` lanes (a power of two), in
// every lane of the run
__device__ __forceinline__ uint32_t run_max(uint32_t v, int width) {
    if (width >= 2) v = max(v, dpp_u32<0xB1>(v));    // quad_perm [1,0,3,2]
    if (width >= 4) v = max(v, dpp_u32<0x4E>(v));    // quad_perm [2,3,0,1]
    if (width >= 8) v = max(v, dpp_u32<0x141>(v));   // row_half_mirror
    if (width >= 16) v = max(v, dpp_u32<0x140>(v));  // row_mirror
    if (width >= 32) v = max(v, (uint32_t)__shfl_xor((int)v, 16, 64));
    if (width >= 64) v = max(v, (uint32_t)__shfl_xor((int)v, 32, 64));
    return v;
}

// the two largest of each run, likewise (hi >= lo)
__device__ __forceinline__ void pair_merge(uint32_t& hi, uint32_t& lo, uint32_t ohi, uint32_t olo) {
    lo = max(min(hi, ohi), max(lo, olo));
    hi = max(hi, ohi);
}
__device__ __forceinline__ void run_max2(uint32_t& hi, uint32_t& lo, int width) {
    if (width >= 2) pair_merge(hi, lo, dpp_u32<0xB1>(hi), dpp_u32<0xB1>(lo));
    if (width >= 4) pair_merge(hi, lo, dpp_u32<0x4E>(hi), dpp_u32<0x4E>(lo));
    if (width >= 8) pair_merge(hi, lo, dpp_u32<0x141>(hi), dpp_u32<0x141>(lo));
    if (width >= 16) pair_merge(hi, lo, dpp_u32<0x140>(hi), dpp_u32<0x140>(lo));
    for (int off = 16; off < width; off <<= 1)
        pair_merge(hi, lo, (uint32_t)__shfl_xor((int)hi, off, 64), (uint32_t)__shfl_xor((int)lo, off, 64));
}

// the largest value of the wave, as a scalar
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
    v = max(v, dpp_u32<0xB1>(v));
    v = max(v, dpp_u32<0x4E>(v));
    v = max(v, dpp_u32<0x141>(v));
    v = max(v, dpp_u32<0x140>(v));  // every lane holds its row's
    const uint32_t a = (uint32_t)__builtin_amdgcn_readlane((int)v, 0), b = (uint32_t)__builtin_amdgcn_readlane((int)v, 16);
    const uint32_t c = (uint32_t)__builtin_amdgcn_readlane((int)v, 32), d = (uint32_t)__builtin_amdgcn_readlane((int)v, 48);
    return max(max(a, b), max(c, d));
}

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}

__device__ __forceinline__ float load_logit(const void* p, int dtype, size_t i) {
    if (dtype == 2) return static_cast<const float*>(p)[i];
    const uint16_t h = static_cast<const uint16_t*>(p)[i];
    return dtype == 1 ? bf16_to_f32(h) : f16_to_f32(h);
}

// lanes per group and experts per lane (host and device)
__host__ __device__ __forceinline__ int grouped_lanes(int groups) {
    int p = 1;
    while (p < groups) p <<= 1;
    return 64 / p;
}
__host__ __device__ __forceinline__ int grouped_per_lane(int E, int groups) {
    const int lpg = grouped_lanes(groups);
    return (E / groups + lpg - 1) / lpg;
}

// routes token m; lane j < topk writes slot j (and the expert to lds_ids[j] if given)
template <int PL>
__device__ __forceinline__ void route_token_grouped(const RouteGroupedArgs& g, int m, int lane, int lpg, int per,
                                                    int* lds_ids) {
    const int gs = g.E / g.groups;
    const int grp = lane / lpg;
    const int first = (lane - grp * lpg) * per;  // of the group's experts
    const int count = grp < g.groups ? min(per, gs - first) : 0;  // may be negative
    const int e0 = grp * gs + first;

    float l[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) l[i] = i < count ? load_logit(g.logits, g.dtype, (size_t)m * g.E + e0 + i) : 0.0f;

    // softmax: the row's largest logit, and the sum of the exponentials where it is needed
    const bool two = g.top2 && g.groups > 1;
    const bool all = g.bias || two;  // the choice needs every expert's score
    double mx = 0.0, total = 1.0;
    double ex[PL];
    if (!g.sigmoid && (all || !g.renormalize)) {
        uint32_t k = 0;
#pragma unroll
        for (int i = 0; i < PL; ++i) k = max(k, i < count ? order_key(l[i]) : 0u);
        mx = (double)key_value(wave_max_u32(k));
        double part = 0.0;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            // a row of -inf only has scores of zero
            ex[i] = i < count && mx != -__builtin_inf() ? exp((double)l[i] - mx) : 0.0;
            part += ex[i];
        }
        total = wave_sum_f64(part);
        if (total == 0.0) total = 1.0;
    } else if (g.sigmoid && all) {
#pragma unroll
        for (int i = 0; i < PL; ++i) ex[i] = 1.0 / (1.0 + exp(-(double)l[i]));
    }

    uint32_t key[PL];
    uint32_t avail = 0;  // bit i: slot i holds an expert that may still be chosen
    uint32_t hi = 0, lo = 0;  // of this lane's c
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        key[i] = order_key(l[i]);
        if (all) {
            const double sc = ex[i] / total;
            const float c = g.bias ? (float)(sc + (double)(i < count ? g.bias[e0 + i] : 0.0f)) : (float)sc;
            const uint32_t ck = order_key(c);
            if (g.bias) key[i] = ck;
            if (i < count) {
                lo = max(lo, min(hi, ck));
                hi = max(hi, ck);
            }
        }
        if (i < count) avail |= 1u << i;
    }

    if (g.groups > 1 && g.topk_group < g.groups) {
        uint32_t gk = 0;
        if (two) {
            run_max2(hi, lo, lpg);
            gk = order_key(key_value(hi) + key_value(lo));
        } else {
#pragma unroll
            for (int i = 0; i < PL; ++i) gk = max(gk, (avail >> i) & 1u ? key[i] : 0u);
            gk = run_max(gk, lpg);
        }
        int ahead = 0;
        for (int o = 0; o < g.groups; ++o) {
            const uint32_t ok = (uint32_t)__builtin_amdgcn_readlane((int)gk, o * lpg);
            ahead += (ok > gk || (ok == gk && o < grp)) ? 1 : 0;
        }
        if (ahead >= g.topk_group) avail = 0;
    }

    float sel_l = 0.0f;  // lane j < topk: slot j's logit and expert
    int sel_e = 0;
    for (int j = 0; j < g.topk; ++j) {
        uint32_t bk = 0;
        int bi = -1;
        float bl = 0.0f;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            const bool better = ((avail >> i) & 1u) && (bi < 0 || key[i] > bk);
            bk = better ? key[i] : bk;
            bl = better ? l[i] : bl;
            bi = better ? i : bi;
        }
        const uint32_t top = wave_max_u32(bk);
        const uint64_t at = __ballot(bi >= 0 && bk == top);
        const int wl = __builtin_ctzll(at);  // the open groups hold topk experts (checked on the host): at != 0
        const int e = __builtin_amdgcn_readlane(e0 + bi, wl);
        const float le = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(bl), wl));
        if (lane == wl) avail &= ~(1u << bi);
        if (lane == j) {
            sel_l = le;
            sel_e = e;
        }
    }

    // the weights, from the slots' logits: renormalised softmax weights do not
    // pass through scores that may have underflowed
    double s = 0.0;
    const bool slot = lane < g.topk;
    if (g.sigmoid) {
        s = slot ? 1.0 / (1.0 + exp(-(double)sel_l)) : 0.0;
    } else if (g.renormalize) {
        uint32_t k = slot ? order_key(sel_l) : 0u;
        const double top = (double)key_value(wave_max_u32(k));
        s = slot && top != -__builtin_inf() ? exp((double)sel_l - top) : 0.0;
    } else {
        s = slot && mx != -__builtin_inf() ? exp((double)sel_l - mx) : 0.0;
    }
    double denom = total;
    if (g.sigmoid) denom = 1.0;
    if (g.renormalize) {
        denom = 0.0;
        for (int j = 0; j < g.topk; ++j) denom += __shfl(s, j, 64);  // ascending slot order
        if (denom == 0.0) denom = 1.0;
    }
    if (slot) {
        const size_t o = (size_t)m * g.topk + lane;
        g.w_out[o] = (float)(s / denom * (double)g.scale);
        g.ids_out[o] = sel_e;
        if (lds_ids) lds_ids[lane] = sel_e;
    }
}

// The padded sort of at most 64 pairs over any number of experts by one wave
// (lane i holds pair i's expert, in [0, E)): the outputs of moe_align.  An
// expert's first pair speaks for it: it carries the padded size of its run,
// and a pair's offset is the sum over the speakers of smaller experts.
__device__ __forceinline__ void align_pairs(const int* ids, int T, int BS, int cap, int lane, int32_t* sorted,
                                            int32_t* expert_ids, int32_t* ntpp) {
    const int e = lane < T ? ids[lane] : -1;
    int rank = 0, cnt = 0;
    for (int i = 0; i < T; ++i) {
        const bool same = __builtin_amdgcn_readlane(e, i) == e;
        rank += (same && i < lane) ? 1 : 0;
        cnt += same ? 1 : 0;
    }
    const bool speaks = lane < T && rank == 0;
    const int size = speaks ? (cnt + BS - 1) / BS * BS : 0;
    int at = 0, total = 0;
    for (int i = 0; i < T; ++i) {
        const int z = __builtin_amdgcn_readlane(size, i);
        at += __builtin_amdgcn_readlane(e, i) < e ? z : 0;
        total += z;
    }
    if (lane < T) sorted[at + rank] = lane;
    if (speaks) {
        for (int p = at + cnt; p < at + size; ++p) sorted[p] = T;
        for (int b = at / BS; b < (at + size) / BS; ++b) expert_ids[b] = e;
    }
    for (int p = total + lane; p < cap; p += 64) sorted[p] = T;
    for (int b = total / BS + lane; b < cap / BS; b += 64) expert_ids[b] = -1;
    if (lane == 0) *ntpp = total;
}

}  // namespace wq
