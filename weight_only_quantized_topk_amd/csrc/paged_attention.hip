// paged_attention.hip -- attention of one new token a sequence over a paged
// key-value cache.
//
//   s_t = scale * q . k_t,  p_t = exp(s_t - max s),  out = sum p_t v_t / sum p_t,
//   lse = max s + log sum p_t
//
// over the sequence's tokens (the last `window` of them), for each query head
// with the keys and values of its group's head; k_t, v_t 16-bit rows or E4M3
// codes times their row's scale.  A row of the cache takes part in 2 products
// of 2 operations a value for each of the group's G heads, so at most 2 G
// operations a byte (4 G for codes): HBM bound.
//
// The cache is read once for every 16 heads of a group begun, straight to registers.  A wave takes tiles of 32
// tokens; the group's heads (up to 16 at a time) are the 16 columns of
// v_mfma_f32_16x16x32:
//   S^T [token, head] = K Q^T: lane l holds 8 channels of token l % 16 as they lie
//       in memory, the A operand;
//   O^T [channel, head] += V^T P^T: S^T comes out with head l % 16 and tokens
//       4 (l / 16) + i of each half in lane l, and as the order of the tokens in
//       a product is free, that is the B operand as it stands.  Lane l loads
//       VEC channels from VEC (l % 16) of the same 8 tokens, and the A operand of
//       channel e of each is 4 byte permutations of its own registers.
// No value crosses lanes but the running maximum, and nothing goes through LDS
// until the waves' results are joined (but Q where registers are short).  P is 16-bit in two parts (value, and
// what that rounding left out), each multiplied by the same V operand: right to 2^-16
// (bf16) or 2^-22 (fp16, or 2^-37 of the largest if that is more) of itself; with one part its rounding alone would be as
// large as the output's.  Under E4M3 values P carries the row's scale, in bf16 for its range.
// Scores, statistics and sums are float32.  The maximum is raised only
// when a score passes it by 2^8 (fp16: 2^2), so p is up to that and the accumulators are
// seldom rescaled.
//
// Split over the length: every workgroup reads the batch's lengths and finds
// from them alone the same cut: the sequences' steps (a tile for each of 4 waves, 128
// tokens; a sequence of none has one step) one after another in as many equal shares as the
// chip holds workgroups (256 CUs x 4, 3 or 2 by the registers that head_dim takes),
// so one long sequence among short ones is shared out and no workgroup waits for another.
// A workgroup goes through its share without a pause between sequences: the rows of the next step are
// asked for as the registers of this one come free, and the pages of 32 steps
// by one vector load a block ahead.  (Pages read singly by scalar loads cost 3 to
// 5 % more; a whole tile more in flight does not fit in the registers.)  A sequence that lies in one share is written at
// once; the pieces of the others, at most two a share, go as (O, max, sum) in
// float32 to the workspace and are joined in ascending order by a second
// kernel.  No atomics: the same inputs and grid give the same bits.  Caches
// of few tokens a sequence, and batches that fill the chip with short sequences, have a workgroup a
// sequence and no second kernel (the rule is at paged_attn_splits).
//
// Measured (device time in a graph; a large copy reaches 5.2 TB/s here): one
// sequence of 131072 tokens, 64 heads over 8 of 128 in bf16 (537 MB) 99.6 us;
// 61 sequences of up to 8192 tokens, E4M3 rows (536 MB) 105 us; 256 of up to 1024,
// 16 heads of 64 (538 MB) 106 us: 5.1 to 5.4 TB/s, the rate of reading.  Far from it: widths that run
// padded (16 sequences of up to 4096, 8 heads of 32 in E4M3 rows 23 us, 3.6 by their bytes), groups of more than 16 heads (2 groups
// of 17 of 128, the same lengths: 24.8 us, of 16 21.0, by their bytes 6.5).  Short
// ones are bound by two launches, the walk over lengths and tables and the join:
// 9 us for one sequence of 1024 tokens (4 MB), of these 3 to 4 the second kernel.
#include "common.hpp"
#include "kv_common.hpp"
#include "launch.hpp"

#include <algorithm>

namespace wq {

namespace {

constexpr int NW = 4;              // waves of a workgroup
constexpr int TILE = 32;           // tokens of a wave's step
// head_dim rounded up, and the waves a SIMD (workgroups a CU) that its registers leave room for
constexpr int dim_of(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }
constexpr int waves_of(int DM) { return DM == 256 ? 2 : DM == 128 ? 3 : 4; }
template <int MODE, int DM>
constexpr bool q_in_lds = MODE == KV_16 && DM == 256;
template <int MODE, int DM>
constexpr int join_channels = q_in_lds<MODE, DM> ? 128 : DM;  // (leaves Q room for two workgroups a CU)
constexpr float M_NONE = -3.4028234e38f;  // the running maximum before any score
// scores may pass the running maximum by SLACK, and weights are held times 2^BIAS (exponents of 2).  fp16 weights
// need the bias: their least step is 2^-24, so without one (p up to 2^8) the second part of a weight below 2^-3 was
// short and one below 2^-25 was nothing, which the sum still had: behind one token 2^25 above all others a long
// context's output lost up to a quarter (500 tokens in a workgroup).  With 2^13, and a slack of 2 so that p 2^13 stays below
// 2^15, the two parts are right to 2^-37 of the largest weight; times are the same (256 sequences of up to 1024, 16 heads of 64:
// 106 us).  bf16 has float32's exponents
template <bool PBF>
constexpr float SLACK = PBF ? 8.0f : 2.0f;
template <bool PBF>
constexpr float BIAS = PBF ? 0.0f : 13.0f;
template <bool PBF>
constexpr float UNBIAS = PBF ? 1.0f : 0x1p-13f;
constexpr float LN2 = 0.693147180559945309f;

// a sequence's tokens [lo, len), its first tile beginning at lo rounded down to
// half a tile, and its steps of a workgroup (NW tiles, the last one partly idle);
// at least one, so that every sequence is in some workgroup's share
__device__ __forceinline__ int len_of(const PagedAttnArgs& g, int len) { return min(max(len, 0), g.width * g.page_size); }
__device__ __forceinline__ int lo_of(const PagedAttnArgs& g, int len) { return g.window > 0 ? max(0, len - g.window) : 0; }
__device__ __forceinline__ int begin_of(const PagedAttnArgs& g, int len) { return lo_of(g, len) & ~(KV_TOKENS - 1); }
__device__ __forceinline__ int steps_of(const PagedAttnArgs& g, int len) {
    return max(1, (len - begin_of(g, len) + NW * TILE - 1) / (NW * TILE));
}

// a wave-uniform index into an array that the kernel does not write: a scalar
// load, which the counter of the vector loads in flight does not wait for
__device__ __forceinline__ int uniform_at(const int32_t* p, int64_t i) {
    return *(const __attribute__((address_space(4))) int32_t*)(p + i);
}

template <int CTRL, int ROW_MASK>
__device__ __forceinline__ int dpp_add(int v) {
    return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROW_MASK, 0xF, false);
}
// inclusive sums over the lanes of a wave: within rows of 16 lanes, then the
// rows' last lanes onto the rows behind
__device__ __forceinline__ int wave_scan(int v) {
    v = dpp_add<0x111, 0xF>(v);  // row_shr 1, 2, 4, 8
    v = dpp_add<0x112, 0xF>(v);
    v = dpp_add<0x114, 0xF>(v);
    v = dpp_add<0x118, 0xF>(v);
    v = dpp_add<0x142, 0xA>(v);  // row_bcast 15
    v = dpp_add<0x143, 0xC>(v);  // row_bcast 31
    return v;
}

// workgroup x's share of the batch's steps, one sequence's after another's: `steps`
// from step `off` of sequence b on (0: none); every share but the last has `cut`
struct Share {
    int b, off, steps, cut;
};
__device__ __forceinline__ Share share_of(const PagedAttnArgs& g, int x) {
    if (g.splits == 0) return Share{x, 0, steps_of(g, len_of(g, g.lengths[x])), 0};
    const int lane = threadIdx.x & 63;
    const int each = (g.B + 63) / 64;  // consecutive sequences of a lane
    const int b0 = lane * each, b1 = min(b0 + each, g.B);
    int sum = 0;
    for (int b = b0; b < b1; ++b) sum += steps_of(g, len_of(g, g.lengths[b]));
    const int upto = wave_scan(sum);
    const int total = __builtin_amdgcn_readlane(upto, 63);
    const int cut = (total + g.splits - 1) / g.splits;
    const int64_t lo64 = (int64_t)x * cut;
    if (lo64 >= total) return Share{0, 0, 0, cut};
    const int lo = (int)lo64, hi = min(lo + cut, total);
    const int owner = __ffsll((unsigned long long)__ballot(upto > lo)) - 1;
    int off = lo - (__builtin_amdgcn_readlane(upto, owner) - __builtin_amdgcn_readlane(sum, owner));
    int b = owner * each;
    for (; b < g.B - 1; ++b) {
        const int n = steps_of(g, len_of(g, g.lengths[b]));
        if (off < n) break;
        off -= n;
    }
    return Share{b, off, hi - lo, cut};
}

template <bool BF16>
__device__ __forceinline__ uint32_t codes2(uint32_t w, bool hi) {
    // (the half has to be a constant)
    if constexpr (BF16) {
        const bf16x2 r = hi ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true)
                            : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false);
        return __builtin_bit_cast(uint32_t, r);
    } else {
        const f16x2 r = hi ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true)
                           : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false);
        return __builtin_bit_cast(uint32_t, r);
    }
}

// a buffer resource over the rows from base on (raw addressing: byte offsets)
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_at(const uint8_t* base) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), (short)0, -1, 0x00020000);
}

template <int N>
struct Dwords {
    uint32_t d[N];
};
template <int BYTES, int AUX>
__device__ __forceinline__ Dwords<BYTES / 4> load_bytes(__amdgpu_buffer_rsrc_t rows, int voff, int soff) {
    Dwords<BYTES / 4> r;
    if constexpr (BYTES == 4) {
        r.d[0] = __builtin_amdgcn_raw_buffer_load_b32(rows, voff, soff, AUX);
    } else if constexpr (BYTES == 8) {
        const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(rows, voff, soff, AUX);
        r.d[0] = v[0];
        r.d[1] = v[1];
    } else {
#pragma unroll
        for (int i = 0; i < BYTES / 16; ++i) {
            const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(rows, voff + 16 * i, soff, AUX);
#pragma unroll
            for (int j = 0; j < 4; ++j) r.d[4 * i + j] = v[j];
        }
    }
    return r;
}

// a pair of weights as 16-bit values and what their rounding left out
template <bool BF16>
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
    hi = f32_to_act2<BF16>(a, b);
    lo = f32_to_act2<BF16>(a - act_to_f32<BF16>((uint16_t)hi), b - act_to_f32<BF16>((uint16_t)(hi >> 16)));
}
// The same beside values that may be infinite: both parts above 0 where the weight is, so that an infinity times
// either is itself (0 or less than 0 made the channel NaN).  The first part is rounded towards 0; the second is
// raised by 2^-23 of the weight (bf16), or to fp16's least step.  As many instructions as above or fewer
template <bool BF16>
__device__ __forceinline__ void split2_above(float a, float b, uint32_t& hi, uint32_t& lo) {
    if constexpr (BF16) {
        const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
        hi = __builtin_amdgcn_perm(ub, ua, 0x07060302u);
        lo = f32_to_act2<true>(fmaf(a, 1.0f + 0x1p-23f, -__uint_as_float(ua & 0xffff0000u)),
                               fmaf(b, 1.0f + 0x1p-23f, -__uint_as_float(ub & 0xffff0000u)));
    } else {
        hi = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(a, b));
        const float ha = f16_to_f32((uint16_t)hi), hb = f16_to_f32((uint16_t)(hi >> 16));
        lo = f32_to_act2<false>(__builtin_amdgcn_fmed3f(a - ha, ha, 0x1p-24f), __builtin_amdgcn_fmed3f(b - hb, hb, 0x1p-24f));
    }
}

// DM: head_dim rounded up to 64, 128 or 256 (FULL: it is DM)
// NT: the cache's rows are read with non-temporal loads.
// (3 or 4 waves a SIMD: without the bound the compiler keeps the accumulators in
// the other register file and moves them there and back in every step)
template <bool BF16, int MODE, int DM, bool FULL, bool NT>
__global__ __launch_bounds__(NW * 64, waves_of(DM)) void paged_attention_kernel(PagedAttnArgs g) {
    constexpr int AUX = NT ? 2 : 0;
    constexpr bool F8 = MODE != KV_16;
    constexpr bool ROW = MODE == KV_E4M3_ROW;
    constexpr bool PBF = BF16 || F8;              // P's type: E4M3 values and scales go as bf16
    constexpr int ELT = F8 ? 1 : 2;
    constexpr int KD = F8 ? 64 : 32;              // channels of one 16-byte K load of the 4 lane groups
    constexpr int KL = DM / KD;                   // such loads a token row
    constexpr int VEC = DM / 16;                  // V channels of a lane
    constexpr int VD = VEC * ELT / 4;             // their dwords
    constexpr int JC = join_channels<MODE, DM>;   // channels that the waves join at a time
    constexpr int LD = JC + 4;
    extern __shared__ __attribute__((aligned(16))) float lds[];

    const int D = FULL ? DM : g.D;
    const int lane = threadIdx.x & 63, r = lane & 15, q4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int group = g.heads / g.kv_heads;
    const int htiles = (group + 15) / 16;
    const int kvh = blockIdx.y / htiles, h0 = (blockIdx.y - kvh * htiles) * 16;
    const int nh = min(16, group - h0);           // heads of this workgroup
    const int head0 = kvh * group + h0;
    const uint32_t page16 = (uint32_t)g.page_size / KV_TOKENS;
    // u / page16 by one multiplication: the host checks the range
    const uint32_t magic = (uint32_t)(0xffffffffu / page16 + 1);
    auto column_of = [&](uint32_t u) { return page16 == 1 ? u : __umulhi(u, magic); };

    // half a tile: 16 tokens, in one page; those past the sequence read its last
    struct Half {
        int64_t rows;  // (page, head)'s first row in the cache + the position in the page
        bool good;
    };
    u32x4 kv[2][KL];
    Dwords<VD> vv[8];
    f32x4 ksv[2], vsv[2];
    // the wave-uniform part of an address is the resource's base, the lane's a
    // 32-bit offset
    const int koff = r * (D * ELT) + 16 * q4, voff = 4 * q4 * (D * ELT) + r * (VEC * ELT);
    auto kload = [&](const Half (&h)[2]) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const __amdgpu_buffer_rsrc_t rows = rows_at(g.k + h[s].rows * (D * ELT));
#pragma unroll
            for (int c = 0; c < KL; ++c) {
                if (!FULL) kv[s][c] = u32x4{0, 0, 0, 0};
                if (FULL || KD * c + (16 / ELT) * q4 < D)
                    kv[s][c] = __builtin_amdgcn_raw_buffer_load_b128(rows, koff + KD * c * ELT, 0, AUX);
            }
            if constexpr (ROW) ksv[s] = *reinterpret_cast<const f32x4*>(g.ks + h[s].rows + 4 * q4);
        }
    };
    auto vload = [&](const Half (&h)[2]) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const __amdgpu_buffer_rsrc_t rows = rows_at(g.v + h[s].rows * (D * ELT));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (!FULL)
#pragma unroll
                    for (int i = 0; i < VD; ++i) vv[4 * s + j].d[i] = 0;
                if (FULL) vv[4 * s + j] = load_bytes<VEC * ELT, AUX>(rows, voff + j * (DM * ELT), 0);
                else if (r * VEC < D) vv[4 * s + j] = load_bytes<VEC * ELT, AUX>(rows, voff, j * (D * ELT));
            }
            if constexpr (ROW) vsv[s] = *reinterpret_cast<const f32x4*>(g.vs + h[s].rows + 4 * q4);
        }
    };

    const Share share = share_of(g, blockIdx.x);
    int left = __builtin_amdgcn_readfirstlane(share.steps);
    const int cut = __builtin_amdgcn_readfirstlane(share.cut);
    int goes_on = 0, begins = 0;  // pieces of the sequence that begins here and ends in another share; it
    if (left > 0) {
        // a sequence's steps in the share (up to s1), and blocks of AHEAD of them, whose pages one vector load
        // fetches a block ahead: lane 2 k + s has that of half s of this wave's tile in the block's k-th step
        constexpr int AHEAD = 32;
        struct Part {
            int b, len, s1;
        };
        auto part_of = [&](int b, int off) {
            const int len = len_of(g, uniform_at(g.lengths, b));
            return Part{b, len, min(steps_of(g, len), off + left)};
        };
        // the block after the one from `base` on: of the same sequence, or of the next
        auto follow = [&](const Part& p, int base, Part& q, int& qbase) {
            if (base + AHEAD < p.s1) {
                q = p;
                qbase = base + AHEAD;
                return true;
            }
            if (left <= 0 || p.b + 1 >= g.B) return false;
            q = part_of(p.b + 1, 0);
            left -= q.s1;
            qbase = 0;
            return true;
        };
        // half s of the wave's tile in step i, the sequence's last 16 tokens past the end
        auto half16 = [&](const Part& p, int i, int s) {
            return (uint32_t)min(begin_of(g, p.len) + TILE * (NW * i + wave) + KV_TOKENS * s, max(p.len - 1, 0)) / KV_TOKENS;
        };
        auto pages_of = [&](const Part& p, int base) {
            return g.table[(int64_t)p.b * g.width + column_of(half16(p, min(base + (lane >> 1), p.s1 - 1), lane & 1))];
        };
        auto half_at = [&](const Part& p, int i, int s, int page) {
            const uint32_t u = half16(p, i, s), col = column_of(u);
            Half h;
            h.good = page >= 0 && page < g.pages;  // a bad page holds no tokens
            h.rows = ((int64_t)(h.good ? page : 0) * g.kv_heads + kvh) * g.page_size + (u - col * page16) * KV_TOKENS;
            return h;
        };
        // Q, the B operand of every K step: head r, the channels in K's order; in registers, or where there are
        // too few of them (16-bit rows at DM 256, 104 bytes a lane spilled) in LDS, each lane its own: 64 sequences
        // of up to 8192 tokens, 8 heads of 256: 408 against 516 us.  E4M3 rows leave room: 38 against 42 us
        // (16 x up to 4096)
        constexpr bool QLDS = q_in_lds<MODE, DM>;
        u32x4 qv[QLDS ? 1 : DM / 32];
        u32x4* qs = reinterpret_cast<u32x4*>(lds + 2 * NW * 16 + NW * nh * LD) + wave * (DM / 32) * 64 + lane;
        auto qload = [&](int b) {
#pragma unroll
            for (int c = 0; c < DM / 32; ++c) {
                const int ch = F8 ? 64 * (c / 2) + 16 * q4 + 8 * (c % 2) : 32 * c + 8 * q4;
                u32x4 v = {0, 0, 0, 0};
                if (r < nh && ch < D) v = ldg128(g.q + (int64_t)b * g.q_stride + (int64_t)(head0 + r) * D + ch);
                if constexpr (QLDS) qs[64 * c] = v;
                else qv[c] = v;
            }
        };
        auto q_at = [&](int c) {
            if constexpr (QLDS) return qs[64 * c];
            else return qv[c];
        };

        int s0 = __builtin_amdgcn_readfirstlane(share.off);  // the sequence's first step in the share
        Part pt = part_of(__builtin_amdgcn_readfirstlane(share.b), s0), np = pt;
        left -= pt.s1 - s0;
        int base = s0, nbase = 0;
        int pages = pages_of(pt, base), npages = 0;
        bool more = follow(pt, base, np, nbase);
        if (more) npages = pages_of(np, nbase);
        f32x4 acc[VEC];
        float m, l;  // head r's running maximum (the same in its 4 lanes); the lane's own sum
        auto clear = [&]() {
            m = M_NONE;
            l = 0.0f;
#pragma unroll
            for (int e = 0; e < VEC; ++e) acc[e] = f32x4{0.f, 0.f, 0.f, 0.f};
        };
        clear();
        Half cur[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) cur[s] = half_at(pt, s0, s, __builtin_amdgcn_readlane(pages, s));
        qload(pt.b);
        kload(cur);
        vload(cur);
        for (int i = s0;;) {
            // the next step, of this block or the next one, is loaded while this one is multiplied (this one again
            // after the last)
            const bool last = i + 1 >= pt.s1, cross = last || i + 1 >= base + AHEAD, on = cross && more;
            const Part qt = on ? np : pt;
            const int ni = on ? nbase : cross ? i : i + 1;
            Half nxt[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int here = __builtin_amdgcn_readlane(pages, 2 * ((cross ? i : i + 1) - base) + s);
                nxt[s] = half_at(qt, ni, s, on ? __builtin_amdgcn_readlane(npages, s) : here);
            }
            if (on) {
                pages = npages;
                base = nbase;
                more = follow(qt, base, np, nbase);
                if (more) npages = pages_of(np, nbase);
            }

            f32x4 sc[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                sc[s] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < KL; ++c) {
                    if constexpr (F8) {
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const uint32_t w0 = kv[s][c][2 * half], w1 = kv[s][c][2 * half + 1];
                            const u32x4 a = {codes2<BF16>(w0, false), codes2<BF16>(w0, true), codes2<BF16>(w1, false),
                                             codes2<BF16>(w1, true)};
                            sc[s] = mfma16x16x32<BF16>(a, q_at(2 * c + half), sc[s]);
                        }
                    } else {
                        sc[s] = mfma16x16x32<BF16>(kv[s][c], q_at(c), sc[s]);
                    }
                }
                if constexpr (ROW) sc[s] *= ksv[s];
            }
            kload(nxt);
            if (last && on) qload(qt.b);

            // scores in exponents of 2; tokens outside the span or in a bad page have none
            const int tok = begin_of(g, pt.len) + TILE * (NW * i + wave), lo = lo_of(g, pt.len);
            const bool edge = tok < lo || tok + TILE > pt.len || !cur[0].good || !cur[1].good;
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = sc[j / 4][j % 4] * g.qk_scale;
            if (edge) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int k = tok + 16 * (j / 4) + 4 * q4 + j % 4;
                    const bool live = k >= lo && k < pt.len && cur[j / 4].good;
                    x[j] = live ? x[j] : -INFINITY;
                    // what lies there may be anything, and 0 * NaN is one
#pragma unroll
                    for (int w = 0; w < VD; ++w) vv[j].d[w] = live ? vv[j].d[w] : 0;
                    if constexpr (ROW) vsv[j / 4][j % 4] = live ? vsv[j / 4][j % 4] : 0.0f;
                }
            }
            float top = x[0];
#pragma unroll
            for (int j = 1; j < 8; ++j) top = fmaxf(top, x[j]);
            if (__any(top - m > SLACK<PBF>)) {  // (m + SLACK may round up past a score from 2^25 on)
                top = fmaxf(top, m);
                top = fmaxf(top, __shfl_xor(top, 16, 64));
                top = fmaxf(top, __shfl_xor(top, 32, 64));
                const float f = __builtin_amdgcn_exp2f(m - top);
                m = top;
                l *= f;
#pragma unroll
                for (int e = 0; e < VEC; ++e) acc[e] *= f;
            }
            u32x4 phi, plo;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] = __builtin_amdgcn_exp2f(x[j] - m + BIAS<PBF>);
                l += x[j];
                if constexpr (ROW) x[j] *= vsv[j / 4][j % 4];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t hi, lo;
                if constexpr (F8) split2<PBF>(x[2 * j], x[2 * j + 1], hi, lo);
                else split2_above<BF16>(x[2 * j], x[2 * j + 1], hi, lo);
                phi[j] = hi;
                plo[j] = lo;
            }
            // channel e of each lane's VEC: tokens 2 j and 2 j + 1 side by side
            if constexpr (F8) {
#pragma unroll
                for (int w = 0; w < VEC / 2; ++w) {  // channels 2 w and 2 w + 1: bytes of dword w / 2
                    u32x4 a0, a1;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t lo = vv[2 * j].d[w / 2], hi = vv[2 * j + 1].d[w / 2];
                        const uint32_t pair = __builtin_amdgcn_perm(hi, lo, w % 2 ? 0x07030602u : 0x05010400u);
                        a0[j] = codes2<PBF>(pair, false);
                        a1[j] = codes2<PBF>(pair, true);
                    }
                    acc[2 * w] = mfma16x16x32<PBF>(a0, phi, acc[2 * w]);
                    acc[2 * w + 1] = mfma16x16x32<PBF>(a1, phi, acc[2 * w + 1]);
                    acc[2 * w] = mfma16x16x32<PBF>(a0, plo, acc[2 * w]);
                    acc[2 * w + 1] = mfma16x16x32<PBF>(a1, plo, acc[2 * w + 1]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    u32x4 a;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t lo = vv[2 * j].d[e / 2], hi = vv[2 * j + 1].d[e / 2];
                        a[j] = __builtin_amdgcn_perm(hi, lo, e % 2 ? 0x07060302u : 0x05040100u);
                    }
                    acc[e] = mfma16x16x32<PBF>(a, phi, acc[e]);
                    acc[e] = mfma16x16x32<PBF>(a, plo, acc[e]);
                }
            }
            vload(nxt);
#pragma unroll
            for (int s = 0; s < 2; ++s) cur[s] = nxt[s];
            if (!last) {
                i = ni;
                continue;
            }

            // join the waves: lane l holds channels [4 VEC q4, +4 VEC) of head r
            float* lm = lds;                  // [NW][16]
            float* ll = lds + NW * 16;        // [NW][16]
            float* lacc = lds + 2 * NW * 16;  // [NW][nh][LD]
            l += __shfl_xor(l, 16, 64);
            l += __shfl_xor(l, 32, 64);
            const int steps = steps_of(g, pt.len);
            const bool whole = s0 == 0 && pt.s1 == steps;
#pragma unroll
            for (int jc = 0; jc < DM; jc += JC) {
                __syncthreads();  // what was there is read
                if (jc == 0 && q4 == 0) {
                    lm[wave * 16 + r] = m;
                    ll[wave * 16 + r] = l;
                }
                if (r < nh && (JC == DM || 4 * VEC * q4 / JC == jc / JC)) {
                    float* o = lacc + (wave * nh + r) * LD + 4 * VEC * q4 - jc;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int e = 0; e < VEC; e += 4)
                            *reinterpret_cast<f32x4*>(o + VEC * k + e) =
                                f32x4{acc[e][k], acc[e + 1][k], acc[e + 2][k], acc[e + 3][k]};
                }
                __syncthreads();
                const int quads = min(D - jc, JC) / 4;
                for (int id = threadIdx.x; id < nh * quads; id += NW * 64) {
                    const int hd = id / quads, c = 4 * (id - hd * quads);
                    float mx = lm[hd], sum = 0.0f;
#pragma unroll
                    for (int w = 1; w < NW; ++w) mx = fmaxf(mx, lm[w * 16 + hd]);
                    f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int w = 0; w < NW; ++w) {
                        const float f = __builtin_amdgcn_exp2f(lm[w * 16 + hd] - mx) * UNBIAS<PBF>;
                        sum += f * ll[w * 16 + hd];
                        o += f * *reinterpret_cast<const f32x4*>(lacc + (w * nh + hd) * LD + c);
                    }
                    const int64_t head = head0 + hd;
                    const bool first = jc == 0 && c == 0;
                    if (whole) {
                        // no token with a weight: zeros, and -inf
                        const float inv = sum == 0.0f ? 0.0f : g.v_scale / sum;
                        *reinterpret_cast<u32x2*>(g.out + (int64_t)pt.b * g.out_stride + head * D + jc + c) =
                            u32x2{f32_to_act2<BF16>(o[0] * inv, o[1] * inv), f32_to_act2<BF16>(o[2] * inv, o[3] * inv)};
                        if (g.lse && first)
                            g.lse[(int64_t)pt.b * g.heads + head] = sum == 0.0f ? -INFINITY : (mx + log2f(sum)) * LN2;
                    } else {
                        const int64_t slot = (int64_t)(2 * blockIdx.x + (s0 == 0)) * g.heads + head;
                        *reinterpret_cast<f32x4*>(g.part_o + slot * D + jc + c) = o;
                        if (first) {
                            g.part_ml[2 * slot] = mx;
                            g.part_ml[2 * slot + 1] = sum;
                        }
                    }
                }
            }
            if (!on) {
                if (s0 == 0 && !whole) {
                    goes_on = 1 + (steps - pt.s1 + cut - 1) / cut;
                    begins = pt.b;
                }
                break;
            }
            pt = qt;
            i = s0 = 0;
            clear();
        }
    }
    if (g.splits > 0 && blockIdx.y == 0 && threadIdx.x == 0) {
        g.part_at[2 * blockIdx.x] = begins;
        g.part_at[2 * blockIdx.x + 1] = goes_on;
    }
}

// The pieces of sequences in more than one share: 256 threads as rows of D / 4
// vectors of 4 channels.  The rows are shared out over `hb` heads; a head's rows take
// every so many-th piece, JOIN_AHEAD of them loaded together with their statistics, and
// are joined through LDS where there are several.  A workgroup looks at `shares`
// of them one after another, in each of which at most one such sequence begins.
constexpr int JOIN_AHEAD = 8;

template <bool BF16>
__global__ __launch_bounds__(256) void paged_join_kernel(PagedAttnArgs g, int shares, int hb) {
    __shared__ f32x4 so[256];
    __shared__ float sm[256], sl[256];
    const int tid = threadIdx.x;
    const int quads = g.D / 4, per = 256 / quads / hb;  // rows of a head
    const int row = tid / quads, c = 4 * (tid - row * quads);
    const int head = blockIdx.x * hb + row / per, first = row - row / per * per;
    const bool mine_too = row < per * hb && head < g.heads;
    // lane k of every wave: the k-th share's sequence and its pieces (0: none begins there to be joined)
    const int mine = blockIdx.y * shares + (tid & 63);
    const bool there = (tid & 63) < shares && mine < g.splits;
    const int bs = there ? g.part_at[2 * mine] : 0, ns = there ? g.part_at[2 * mine + 1] : 0;
    for (uint64_t todo = __ballot(ns > 0); todo != 0; todo &= todo - 1) {
        const int k0 = __ffsll((unsigned long long)todo) - 1;
        const int x = blockIdx.y * shares + k0;
        const int n = __builtin_amdgcn_readlane(ns, k0), b = __builtin_amdgcn_readlane(bs, k0);
        float m = M_NONE, l = 0.0f;
        f32x4 o = {0.f, 0.f, 0.f, 0.f};
        for (int p0 = first; p0 < n && mine_too; p0 += per * JOIN_AHEAD) {
            float pm[JOIN_AHEAD], pl[JOIN_AHEAD];
            f32x4 po[JOIN_AHEAD];
#pragma unroll
            for (int k = 0; k < JOIN_AHEAD; ++k) {
                // piece 0 is share x's second, piece p share x + p's first; past the last: it again, without weight
                const int p = min(p0 + k * per, n - 1);
                const int64_t slot = (int64_t)(2 * (x + p) + (p == 0)) * g.heads + head;
                pm[k] = p0 + k * per < n ? g.part_ml[2 * slot] : M_NONE;
                pl[k] = p0 + k * per < n ? g.part_ml[2 * slot + 1] : 0.0f;
                po[k] = *reinterpret_cast<const f32x4*>(g.part_o + slot * g.D + c);
            }
            float top = m;
#pragma unroll
            for (int k = 0; k < JOIN_AHEAD; ++k) top = fmaxf(top, pm[k]);
            const float f0 = __builtin_amdgcn_exp2f(m - top);
            m = top;
            l *= f0;
            o *= f0;
#pragma unroll
            for (int k = 0; k < JOIN_AHEAD; ++k) {
                const float f = p0 + k * per < n ? __builtin_amdgcn_exp2f(pm[k] - top) : 0.0f;
                l += f * pl[k];
                if (p0 + k * per < n) o += f * po[k];  // (a repeated piece may hold infinities)
            }
        }
        if (per > 1) {
            so[tid] = o;
            sm[tid] = m;
            sl[tid] = l;
            __syncthreads();
            if (first == 0 && mine_too) {
                float top = m;
                for (int i = 1; i < per; ++i) top = fmaxf(top, sm[tid + i * quads]);
                const float f0 = __builtin_amdgcn_exp2f(m - top);
                o *= f0;
                l *= f0;
                for (int i = 1; i < per; ++i) {
                    const float f = __builtin_amdgcn_exp2f(sm[tid + i * quads] - top);
                    l += f * sl[tid + i * quads];
                    o += f * so[tid + i * quads];
                }
                m = top;
            }
            __syncthreads();
        }
        if (first == 0 && mine_too) {
            const float inv = l == 0.0f ? 0.0f : g.v_scale / l;
            *reinterpret_cast<u32x2*>(g.out + (int64_t)b * g.out_stride + (int64_t)head * g.D + c) =
                u32x2{f32_to_act2<BF16>(o[0] * inv, o[1] * inv), f32_to_act2<BF16>(o[2] * inv, o[3] * inv)};
            if (g.lse && c == 0) g.lse[(int64_t)b * g.heads + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * LN2;
        }
    }
}

template <bool BF16, int MODE, int DM, bool FULL, bool NT>
void launch_kernel(const PagedAttnArgs& g, hipStream_t s) {
    const int group = g.heads / g.kv_heads;
    const int nh = std::min(group, 16);
    const size_t lds = (2 * NW * 16 + (size_t)NW * nh * (join_channels<MODE, DM> + 4)) * sizeof(float) +
                       (q_in_lds<MODE, DM> ? NW * (DM / 32) * 64 * 16 : 0);  // what is joined, and Q
    auto kern = paged_attention_kernel<BF16, MODE, DM, FULL, NT>;
    if (lds > 65536)
        (void)hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize,
                                  (int)lds);
    const dim3 grid(g.splits > 0 ? g.splits : g.B, g.kv_heads * ((group + 15) / 16));
    hipLaunchKernelGGL(kern, grid, dim3(NW * 64), lds, s, g);
}

// Non-temporal loads where the keys and values are more than the last-level
// cache (256 MB) holds from one step to the next: one sequence of 131072 tokens, 8
// heads of 128 in bf16 (537 MB), 99.5 against 105 us; 61 sequences of up to 8192 in
// E4M3 (536 MB) 105 against 111.  A cache that fits is read from there (56 MB: 20.8
// against 24.1), and sequences of a workgroup each are slower with them (119
// against 107 us, 256 x up to 1024 tokens, 16 heads of 64).  The host knows the whole cache's size only, not
// what a batch reads of it: a small batch in a large pool, called again and again over the same pages, gets them too (7 sequences
// under a window of 4096, 56 MB of a pool of 2 GB: 25.6 us)
template <bool BF16, int MODE, int DM, bool FULL>
void launch_full(const PagedAttnArgs& g, hipStream_t s) {
    const int64_t bytes = (int64_t)g.pages * g.page_size * g.kv_heads * g.D * (MODE == KV_16 ? 4 : 2);
    if (FULL && g.splits > 0 && bytes > (256 << 20)) launch_kernel<BF16, MODE, DM, FULL, FULL>(g, s);
    else launch_kernel<BF16, MODE, DM, FULL, false>(g, s);
}

template <bool BF16, int MODE>
void launch_dim(const PagedAttnArgs& g, hipStream_t s) {
    if (g.D == 64) launch_full<BF16, MODE, 64, true>(g, s);
    else if (g.D == 128) launch_full<BF16, MODE, 128, true>(g, s);
    else if (g.D == 256) launch_full<BF16, MODE, 256, true>(g, s);
    else if (g.D < 64) launch_full<BF16, MODE, 64, false>(g, s);
    else if (g.D < 128) launch_full<BF16, MODE, 128, false>(g, s);
    else launch_full<BF16, MODE, 256, false>(g, s);
}

template <bool BF16>
void launch_type(const PagedAttnArgs& g, hipStream_t s) {
    if (g.mode == KV_16) launch_dim<BF16, KV_16>(g, s);
    else if (g.mode == KV_E4M3_ROW) launch_dim<BF16, KV_E4M3_ROW>(g, s);
    else launch_dim<BF16, KV_E4M3_STATIC>(g, s);
    if (g.splits > 0) {
        // a workgroup has few shares that begin a sequence to join: at a quarter of the shares a sequence seldom two, one
        // after another (4 sequences of up to 8192, 8 heads of 64: 19.6 -> 15.0 us against all of them; single shares
        // 16.3, by workgroups without work).  A row a
        // head where a sequence has few pieces (48 heads, 228 sequences in 256 shares: 17 us a head a workgroup)
        const int shares = std::max(1, std::min(64, g.splits / g.B / 4)), rows = 256 / (g.D / 4);
        const int hb = g.splits <= JOIN_AHEAD * g.B ? std::min(rows, g.heads) : 1;
        hipLaunchKernelGGL(paged_join_kernel<BF16>, dim3((g.heads + hb - 1) / hb, (g.splits + shares - 1) / shares),
                           dim3(256), 0, s, g, shares, hb);
    }
}

}  // namespace

// Shares: as many as are resident at once on 256 CUs, rounded down (one more each
// makes a second round of a whole share: 131072 tokens of 3 heads of 64 / 256 in bf16 29.5 / 112 us against 26.6 /
// 103), none smaller than a tile a wave.  A workgroup a sequence and no second kernel where none is long (a step
// takes it 0.6, 1.1 or 2.7 us at DM 64, 128, 256, the join and its launch 4 to 8): device time, split against
// not, 8 heads of 64 / 128 / 256 in bf16,
//   up to 500 tokens, 1 sequence        8.0 /  6.5    8.9 /  8.6   14.4 / 17.4 us
//                    32 sequences      14.8 /  7.3   17.3 / 10.9   30.7 / 22.4
//   up to 1009 tokens, 1 sequence       8.1 /  9.0    9.0 / 12.9   15.9 / 25.9
//                      8 sequences     11.8 /  9.4   15.1 / 13.5   24.5 / 27.4
//                     16 sequences     16.0 /  9.3   17.2 / 13.9   32.9 / 28.0
//                     64 sequences     21.8 / 17.3   36.3 / 35.5   76.5 / 77.0
//   up to 2000 tokens, 1 sequence       9.6 / 14.2   11.7 / 21.5   17.0 / 45.2
//                     64 sequences     36.8 / 36.0   59.8 / 64.4    135 / 136
// (8 waves a workgroup there: 64 or 128 KB a step keep a CU busy as it is, 17.2 -> 18.9 us at 32 sequences of 1009)
// max_tokens is what the block table has room for: under a table wider than the lengths short
// sequences are split as long ones are (32 of up to 500 tokens, 8 heads of 128: 11.1 us with a table of 500 tokens, 16.8 with one
// of 131072)
int paged_attn_splits(int B, int heads, int kv_heads, int D, int64_t max_tokens) {
    const int DM = dim_of(D), RESIDENT = 256 * waves_of(DM);
    const int units = kv_heads * ((heads / kv_heads + 15) / 16);
    // (a window may begin anywhere in 16 tokens)
    const int64_t whole = ((int64_t)B * units >= (DM == 256 ? 128 : 64) ? 1024 : DM == 256 ? 256 : 512) + KV_TOKENS;
    if (max_tokens <= whole) return 0;
    const int64_t steps = (max_tokens + NW * TILE - 1) / (NW * TILE);
    return (int)std::min<int64_t>(std::max(1, RESIDENT / units), B * steps);
}

void launch_paged_attention(const PagedAttnArgs& g, bool bf16, hipStream_t s) {
    if (bf16) launch_type<true>(g, s);
    else launch_type<false>(g, s);
}

}  // namespace wq
