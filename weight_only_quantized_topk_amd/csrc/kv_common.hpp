// kv_common.hpp -- the paged key-value cache as its kernels take it
// (kv_cache.hip, paged_attention.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace wq {

// what a cache row holds
constexpr int KV_16 = 0;           // 16-bit values of the activation type
constexpr int KV_E4M3_ROW = 1;     // E4M3 codes, a float32 scale a row
constexpr int KV_E4M3_STATIC = 2;  // E4M3 codes, one scale for the keys and one for the values

constexpr int KV_TOKENS = 16;      // page sizes are multiples of it
constexpr int KV_MAX_DIM = 256;    // head_dim: a multiple of 16 up to it

// rows of a cache against rows of 16-bit tensors [T, kv_heads, D]; strides in elements
struct KvRowsArgs {
    uint8_t* k;               // cache [pages, kv_heads, page_size, D]
    uint8_t* v;
    float* ks;                // [pages, kv_heads, page_size], KV_E4M3_ROW
    float* vs;
    float k_scale, v_scale;   // KV_E4M3_STATIC
    uint16_t* k16;            // token rows, kv_heads * D values each
    uint16_t* v16;
    const int64_t* slots;     // [T] page * page_size + position; outside the cache: no row
    int64_t k_stride, v_stride;
    int T, pages, kv_heads, page_size, D, mode;
};
void launch_kv_rows(const KvRowsArgs& g, bool write, bool bf16, hipStream_t s);

// attention of one token a sequence (paged_attention.hip); strides in elements
struct PagedAttnArgs {
    const uint8_t* k;
    const uint8_t* v;
    const float* ks;
    const float* vs;
    const uint16_t* q;        // [B, heads, D]
    const int32_t* table;     // [B, width] page of each page_size tokens
    const int32_t* lengths;   // [B]
    uint16_t* out;            // [B, heads, D]
    float* lse;               // [B, heads] or null
    float* part_o;            // workspace of a split: [splits, 2, heads, D]
    float* part_ml;           // [splits, 2, heads, 2]
    int32_t* part_at;         // [splits, 2]: the sequence that begins in a share and goes on in the next, its pieces
    int64_t q_stride, out_stride;
    float qk_scale;           // on the products, for exponents of 2 (the keys' static scale within)
    float v_scale;            // on the output (the values' static scale, or 1)
    int B, heads, kv_heads, D, pages, page_size, width, window, mode;
    int splits;               // shares that the batch's tokens are cut into; 0: a sequence each
};
// shares of a call, for which its grid and workspace have room; max_tokens: the
// most that a sequence reads
int paged_attn_splits(int B, int heads, int kv_heads, int D, int64_t max_tokens);
void launch_paged_attention(const PagedAttnArgs& g, bool bf16, hipStream_t s);

}  // namespace wq
