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
// Equal values: the lower group, the lower expert.  A NaN (c_e of a NaN logit,
// all of a row's under softmax) ranks below every number, so the slots always
// name topk different experts.
//
// Layout: W lanes take a token (64, or 16 and four tokens a wave).  The groups,
// padded to a power of two, share them evenly (LPG lanes each) and a lane holds
// PL consecutive experts of its group, so experts ascend with (lane, slot).  The
// largest 32-bit key of the token is taken by DPP (and scalar reads across the
// wave's rows of 16 lanes), then the lowest expert that holds it likewise: no
// LDS.  With 16 lanes a round of the choice costs 4.5 PL instructions and 10 for
// four tokens at once; a wave per token has the shorter chain.
#pragma once

#include "common.hpp"
#include "launch.hpp"
#include "route_common.hpp"

namespace wq {

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xF, 0xF, false);
}

struct MaxU32 {
    static __device__ __forceinline__ uint32_t of(uint32_t a, uint32_t b) { return max(a, b); }
};
struct MinU32 {
    static __device__ __forceinline__ uint32_t of(uint32_t a, uint32_t b) { return min(a, b); }
};

// over each aligned run of `width` lanes (a power of two), in every lane of it
template <class OP>
__device__ __forceinline__ uint32_t run_all(uint32_t v, int width) {
    if (width >= 2) v = OP::of(v, dpp_u32<0xB1>(v));    // quad_perm [1,0,3,2]
    if (width >= 4) v = OP::of(v, dpp_u32<0x4E>(v));    // quad_perm [2,3,0,1]
    if (width >= 8) v = OP::of(v, dpp_u32<0x141>(v));   // row_half_mirror
    if (width >= 16) v = OP::of(v, dpp_u32<0x140>(v));  // row_mirror
    if (width >= 32) v = OP::of(v, (uint32_t)__shfl_xor((int)v, 16, 64));
    if (width >= 64) v = OP::of(v, (uint32_t)__shfl_xor((int)v, 32, 64));
    return v;
}

// over the W lanes of a token: every lane's (W 16), or a scalar (W 64)
template <class OP, int W>
__device__ __forceinline__ uint32_t token_all(uint32_t v) {
    v = run_all<OP>(v, 16);
    if constexpr (W == 64) {
        const uint32_t a = (uint32_t)__builtin_amdgcn_readlane((int)v, 0), b = (uint32_t)__builtin_amdgcn_readlane((int)v, 16);
        const uint32_t c = (uint32_t)__builtin_amdgcn_readlane((int)v, 32), d = (uint32_t)__builtin_amdgcn_readlane((int)v, 48);
        return OP::of(OP::of(a, b), OP::of(c, d));
    }
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

template <int W>
__device__ __forceinline__ double token_sum(double v) {
#pragma unroll
    for (int off = W / 2; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}

// 1 / d for d >= 1 by the hardware's estimate and two Newton steps (the last
// bit may differ from the rounded quotient, far below the float that is
// compared); 0 for an infinite d (the steps would give a NaN), a NaN for a NaN
__device__ __forceinline__ double inverse(double d) {
    double r = __builtin_amdgcn_rcp(d);
    r = fma(r, fma(-d, r, 1.0), r);
    r = fma(r, fma(-d, r, 1.0), r);
    return d == __builtin_inf() ? 0.0 : r;
}

// the score of a logit but for the softmax's sum: exp(l - ref), or 1 / (1 +
// exp(-l)); one exponential in the code for both.  dead: a score of 0
__device__ __forceinline__ double raw_score(float l, double ref, bool sigmoid, bool dead) {
    const double ex = exp(sigmoid ? -(double)l : (double)l - ref);
    const double s = sigmoid ? inverse(1.0 + ex) : ex;
    return dead ? 0.0 : s;
}

__device__ __forceinline__ float load_logit(const void* p, int dtype, size_t i) {
    if (dtype == 2) return static_cast<const float*>(p)[i];
    const uint16_t h = static_cast<const uint16_t*>(p)[i];
    return dtype == 1 ? bf16_to_f32(h) : f16_to_f32(h);
}

// four logits from an index that is a multiple of four
__device__ __forceinline__ f32x4 load_logits4(const void* p, int dtype, size_t i) {
    if (dtype == 2) return *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
    const u32x2 d = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(p) + i);
    const uint16_t h[4] = {(uint16_t)d[0], (uint16_t)(d[0] >> 16), (uint16_t)d[1], (uint16_t)(d[1] >> 16)};
    f32x4 v;
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = dtype == 1 ? bf16_to_f32(h[k]) : f16_to_f32(h[k]);
    return v;
}

// how W lanes share a token's experts (made on the host)
struct GroupedLayout {
    int lpg;   // lanes per group
    int per;   // experts per lane
    int vec4;  // a lane's experts begin and end at multiples of four, in every row
};
inline GroupedLayout grouped_layout(int E, int groups, int W) {
    int p = 1;
    while (p < groups) p <<= 1;
    GroupedLayout y;
    y.lpg = W / p;  // 0: more groups than lanes
    if (y.lpg == 0) return y;
    const int gs = E / groups;
    y.per = (gs + y.lpg - 1) / y.lpg;
    y.vec4 = y.per > 2 && gs % 4 == 0 && E % 4 == 0;
    if (y.vec4) y.per = (y.per + 3) / 4 * 4;
    return y;
}

// routes the token of this lane's W lanes (live: there is one; others go along
// and write nothing); r: the lane's place among them, base: their first lane.
// Lane r < topk writes slot r (and the expert to lds_ids[r] if given)
template <int W, int PL>
__device__ __forceinline__ void route_token_grouped(const RouteGroupedArgs& g, const GroupedLayout& y, int m, bool live,
                                                    int r, int base, int* lds_ids) {
    const int gs = g.E / g.groups;
    const int grp = r / y.lpg;
    const int first = (r - grp * y.lpg) * y.per;  // of the group's experts
    const int count = grp < g.groups ? min(y.per, gs - first) : 0;  // may be negative
    const int e0 = grp * gs + first;
    const size_t at = (size_t)m * g.E;

    float l[PL];  // (past the lane's experts: others')
    if (y.vec4 && PL % 4 == 0) {
#pragma unroll
        for (int i = 0; i < PL / 4; ++i) {
            const f32x4 v = load_logits4(g.logits, g.dtype, at + min(e0 + 4 * i, g.E - 4));
#pragma unroll
            for (int k = 0; k < 4; ++k) l[4 * i + k] = v[k];
        }
    } else {
#pragma unroll
        for (int i = 0; i < PL; ++i) l[i] = load_logit(g.logits, g.dtype, at + min(e0 + i, g.E - 1));
    }

    // the scores, where they are needed: every expert's for the choice, or the softmax's sum
    const bool two = g.top2 && g.groups > 1;
    const bool all = g.bias || two;  // the choice needs every expert's score
    double mx = 0.0, total = 1.0;
    double sc[PL];
    if (all || !(g.sigmoid || g.renormalize)) {
        if (!g.sigmoid) {
            uint32_t k = 0;
#pragma unroll
            for (int i = 0; i < PL; ++i) k = max(k, i < count ? order_key(l[i]) : 0u);
            mx = (double)key_value(token_all<MaxU32, W>(k));
        }
        double part = 0.0;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            // a row of -inf only has scores of zero
            sc[i] = raw_score(l[i], mx, g.sigmoid, i >= count || mx == -__builtin_inf());
            part += sc[i];
        }
        if (!g.sigmoid) {
            total = token_sum<W>(part);
            if (total == 0.0) total = 1.0;
            const double up = 1.0 / total;
#pragma unroll
            for (int i = 0; i < PL; ++i) sc[i] *= up;
        }
    }

    // keys of the choice: 0 for none (left), at least 1 for an expert (a NaN: 1)
    uint32_t key[PL];
    uint32_t hi = 0, lo = 0;  // of this lane's c
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        uint32_t k = order_key(l[i]);
        if (all) {
            const float c = g.bias ? (float)(sc[i] + (double)g.bias[min(e0 + i, g.E - 1)]) : (float)sc[i];
            const uint32_t ck = order_key(c);
            if (g.bias) k = ck;
            if (i < count) {
                lo = max(lo, min(hi, ck));
                hi = max(hi, ck);
            }
        }
        key[i] = i < count ? max(k, 1u) : 0u;
    }

    if (g.groups > 1 && g.topk_group < g.groups) {
        uint32_t gk = 0;
        if (two) {
            run_max2(hi, lo, y.lpg);
            gk = order_key(key_value(hi) + key_value(lo));
        } else {
#pragma unroll
            for (int i = 0; i < PL; ++i) gk = max(gk, key[i]);
            gk = run_all<MaxU32>(gk, y.lpg);
        }
        int ahead = 0;
        for (int o = 0; o < g.groups; ++o) {
            uint32_t ok;
            if constexpr (W == 64) ok = (uint32_t)__builtin_amdgcn_readlane((int)gk, o * y.lpg);
            else ok = (uint32_t)__shfl((int)gk, base + o * y.lpg, 64);
            ahead += (ok > gk || (ok == gk && o < grp)) ? 1 : 0;
        }
        if (ahead >= g.topk_group) {
#pragma unroll
            for (int i = 0; i < PL; ++i) key[i] = 0u;
        }
    }

    int sel_e = 0;  // lane r < topk: slot r's expert
    for (int j = 0; j < g.topk; ++j) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < PL; ++i) best = max(best, key[i]);
        // the open groups hold topk experts (checked on the host): top >= 1
        const uint32_t top = token_all<MaxU32, W>(best);
        uint32_t e = 0xffffffffu;
#pragma unroll
        for (int i = PL - 1; i >= 0; --i) e = key[i] == top ? (uint32_t)(e0 + i) : e;
        e = token_all<MinU32, W>(e);
#pragma unroll
        for (int i = 0; i < PL; ++i) key[i] = (uint32_t)(e0 + i) == e ? 0u : key[i];
        if (r == j) sel_e = (int)e;
    }

    // the weights, from the slots' logits (read again): renormalised softmax
    // weights do not pass through scores that may have underflowed
    const bool slot = r < g.topk;
    const float sl = slot ? load_logit(g.logits, g.dtype, at + sel_e) : 0.0f;
    double ref = mx;
    if (!g.sigmoid && g.renormalize) ref = (double)key_value(token_all<MaxU32, W>(slot ? order_key(sl) : 0u));
    const double s = raw_score(sl, ref, g.sigmoid, !slot || (!g.sigmoid && ref == -__builtin_inf()));
    double denom = g.sigmoid ? 1.0 : total;
    if (g.renormalize) {
        denom = 0.0;
        for (int j = 0; j < g.topk; ++j) denom += __shfl(s, base + j, 64);  // ascending slot order
        if (denom == 0.0) denom = 1.0;
    }
    if (slot && live) {
        const size_t o = (size_t)m * g.topk + r;
        g.w_out[o] = (float)(s / denom * (double)g.scale);
        g.ids_out[o] = sel_e;
        if (lds_ids) lds_ids[r] = sel_e;
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
