// abi.cpp -- the C ABI of libwqmoe.so (declared in include/wqmoe.h): argument
// validation, device checks, kernel dispatch, and the offline packers.
//
// Every entry point validates all sizes, pointers and formats on the host
// before the first HIP call, so a rejected call launches nothing and the
// validation itself runs (and is tested) on machines without a GPU.  Device
// pointers must live on the current device: a multi-device process that hands
// a kernel another device's buffer gets WQ_ERR_DEVICE instead of an illegal
// access (the failure reported for moe_align_block_size_kernel on a second
// device in "Marlin moe integration", nm-vllm PR 266, review thread).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <string>
#include <thread>
#include <vector>

#include "../../include/wqmoe.h"
#include "kv_common.hpp"
#include "launch.hpp"

namespace {

thread_local std::string g_last_error;

wq_status fail(wq_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    g_last_error = buf;
    return st;
}

wq_status ok() {
    g_last_error.clear();
    return WQ_OK;
}

#define WQ_REQUIRE(cond, st, ...)              \
    do {                                       \
        if (!(cond)) return fail(st, __VA_ARGS__); \
    } while (0)

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// host-side pointer sanity (no HIP call): non-null and 16-byte aligned
wq_status check_ptr(const void* p, const char* name) {
    WQ_REQUIRE(p != nullptr, WQ_ERR_INVALID, "%s is NULL", name);
    WQ_REQUIRE(aligned16(p), WQ_ERR_INVALID, "%s is not 16-byte aligned", name);
    return WQ_OK;
}

// device check: the pointer is device (or managed) memory of the current device
wq_status current_device(int* cur) {
    if (hipGetDevice(cur) != hipSuccess) return fail(WQ_ERR_HIP, "hipGetDevice failed");
    return WQ_OK;
}

wq_status check_dev(const void* p, const char* name, int cur) {
    hipPointerAttribute_t attr;
    if (hipPointerGetAttributes(&attr, p) != hipSuccess) {
        (void)hipGetLastError();
        return fail(WQ_ERR_DEVICE, "%s is not a HIP allocation", name);
    }
    if (attr.type != hipMemoryTypeDevice && attr.type != hipMemoryTypeManaged)
        return fail(WQ_ERR_DEVICE, "%s is not device memory", name);
    if (attr.type == hipMemoryTypeDevice && attr.device != cur)
        return fail(WQ_ERR_DEVICE, "%s lives on device %d, current device is %d", name, attr.device, cur);
    return WQ_OK;
}

wq_status check_dev(const void* p, const char* name) {
    int cur = -1;
    const wq_status st = current_device(&cur);
    return st != WQ_OK ? st : check_dev(p, name, cur);
}

#define WQ_TRY(expr)                      \
    do {                                  \
        wq_status _st = (expr);           \
        if (_st != WQ_OK) return _st;     \
    } while (0)

wq_status after_launch(const char* what) {
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(WQ_ERR_HIP, "%s: launch failed: %s", what, hipGetErrorString(e));
    return ok();
}

// ---------------------------------------------------------------------------
// The no-allocation entry point's workspace: one file-scope device array per
// GPU, held from the library's load until the process ends.  Host code never
// uses the array's name as an address (on the host it names a stand-in):
// the device address comes from hipGetSymbolAddress, once per device with that
// device current, and is kept per device.
// ---------------------------------------------------------------------------
static __device__ __align__(256) uint8_t scratch[WQ_NOALLOC_SCRATCH_BYTES];

constexpr int MAX_DEVICES = 64;
std::atomic<void*> g_scratch_addr[MAX_DEVICES];
std::mutex g_scratch_mu;

// device address of the current device's scratch array
wq_status scratch_for_current_device(void** out) {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess) return fail(WQ_ERR_HIP, "hipGetDevice failed");
    if (dev < 0 || dev >= MAX_DEVICES) return fail(WQ_ERR_UNSUPPORTED, "device %d >= %d", dev, MAX_DEVICES);
    void* p = g_scratch_addr[dev].load(std::memory_order_acquire);
    if (p == nullptr) {
        std::lock_guard<std::mutex> lock(g_scratch_mu);
        p = g_scratch_addr[dev].load(std::memory_order_relaxed);
        if (p == nullptr) {
            const hipError_t e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
            if (e != hipSuccess || p == nullptr) {
                (void)hipGetLastError();
                return fail(WQ_ERR_HIP, "hipGetSymbolAddress(scratch) on device %d: %s", dev, hipGetErrorString(e));
            }
            g_scratch_addr[dev].store(p, std::memory_order_release);
        }
    }
    *out = p;
    return WQ_OK;
}

bool valid_block_size(int bs) { return bs == 16 || bs == 32 || bs == 64 || bs == 128 || bs == 256; }

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

constexpr int64_t MAX_PAIRS = 1 << 24;

template <class F>
void parallel_for(int n, F f) {
    unsigned hw = std::max(1u, std::min(32u, std::thread::hardware_concurrency()));
    int nt = std::min<int>(n, (int)hw);
    if (nt <= 1) {
        for (int i = 0; i < n; ++i) f(i);
        return;
    }
    std::vector<std::thread> th;
    for (int t = 0; t < nt; ++t)
        th.emplace_back([=]() {
            for (int i = t; i < n; i += nt) f(i);
        });
    for (auto& x : th) x.join();
}

}  // namespace

extern "C" {

int wq_version(void) { return 1; }

const char* wq_status_string(wq_status s) {
    switch (s) {
        case WQ_OK: return "ok";
        case WQ_ERR_INVALID: return "invalid argument";
        case WQ_ERR_UNSUPPORTED: return "unsupported";
        case WQ_ERR_DEVICE: return "wrong device";
        case WQ_ERR_HIP: return "HIP runtime error";
        default: return "unknown status";
    }
}

const char* wq_last_error(void) { return g_last_error.c_str(); }

// ---------------------------------------------------------------------------
size_t moe_align_capacity(int M, int topk, int E, int block_size) {
    if (M < 0 || topk <= 0 || E <= 0 || block_size <= 0) return 0;
    const int64_t T = (int64_t)M * topk;
    const int64_t nz = std::min<int64_t>(T, E);
    const int64_t cap = T + nz * (block_size - 1);
    return (size_t)((cap + block_size - 1) / block_size * block_size);
}

wq_status moe_route(const float* d_logits, int M, int E, int topk, int renormalize, float* d_topk_weights,
                    int32_t* d_topk_ids, void* stream) {
    try {
        WQ_REQUIRE(M >= 0, WQ_ERR_INVALID, "M = %d < 0", M);
        WQ_REQUIRE(E >= 1 && topk >= 1 && topk <= E, WQ_ERR_INVALID, "need 1 <= topk <= E (topk %d, E %d)", topk, E);
        WQ_REQUIRE(E <= 1024, WQ_ERR_UNSUPPORTED, "E = %d > 1024", E);
        WQ_REQUIRE(topk <= 16, WQ_ERR_UNSUPPORTED, "topk = %d > 16", topk);
        WQ_REQUIRE((int64_t)M * topk <= MAX_PAIRS, WQ_ERR_UNSUPPORTED, "M*topk > 2^24");
        if (M == 0) return ok();
        WQ_TRY(check_ptr(d_logits, "logits"));
        WQ_TRY(check_ptr(d_topk_weights, "topk_weights"));
        WQ_TRY(check_ptr(d_topk_ids, "topk_ids"));
        WQ_TRY(check_dev(d_logits, "logits"));
        WQ_TRY(check_dev(d_topk_weights, "topk_weights"));
        WQ_TRY(check_dev(d_topk_ids, "topk_ids"));
        wq::launch_route(d_logits, M, E, topk, renormalize ? 1 : 0, d_topk_weights, d_topk_ids,
                         (hipStream_t)stream);
        return after_launch("moe_route");
    } catch (...) {
        return fail(WQ_ERR_HIP, "moe_route: unexpected exception");
    }
}

wq_status moe_align(const int32_t* d_topk_ids, int M, int topk, int E, int block_size, int32_t* d_sorted_token_ids,
                    int32_t* d_expert_ids, int32_t* d_num_tokens_post_padded, size_t capacity, void* stream) {
    try {
        WQ_REQUIRE(M >= 0 && topk >= 1 && E >= 1, WQ_ERR_INVALID, "bad sizes M %d topk %d E %d", M, topk, E);
        WQ_REQUIRE(E <= 1024, WQ_ERR_UNSUPPORTED, "E = %d > 1024", E);
        WQ_REQUIRE(valid_block_size(block_size), WQ_ERR_UNSUPPORTED, "block_size %d not in {16,32,64,128,256}",
                   block_size);
        WQ_REQUIRE((int64_t)M * topk <= MAX_PAIRS, WQ_ERR_UNSUPPORTED, "M*topk > 2^24");
        const size_t need = moe_align_capacity(M, topk, E, block_size);
        WQ_REQUIRE(capacity >= need, WQ_ERR_INVALID, "capacity %zu < required %zu", capacity, need);
        WQ_REQUIRE(capacity % (size_t)block_size == 0, WQ_ERR_INVALID, "capacity not a multiple of block_size");
        WQ_REQUIRE(capacity <= (size_t)0x7fffffff, WQ_ERR_UNSUPPORTED, "capacity too large");
        if (M > 0) WQ_TRY(check_ptr(d_topk_ids, "topk_ids"));
        WQ_TRY(check_ptr(d_sorted_token_ids, "sorted_token_ids"));
        WQ_TRY(check_ptr(d_expert_ids, "expert_ids"));
        WQ_TRY(check_ptr(d_num_tokens_post_padded, "num_tokens_post_padded"));
        if (M > 0) WQ_TRY(check_dev(d_topk_ids, "topk_ids"));
        WQ_TRY(check_dev(d_sorted_token_ids, "sorted_token_ids"));
        WQ_TRY(check_dev(d_expert_ids, "expert_ids"));
        WQ_TRY(check_dev(d_num_tokens_post_padded, "num_tokens_post_padded"));
        wq::launch_align(d_topk_ids, M * topk, E, block_size, d_sorted_token_ids, d_expert_ids,
                         d_num_tokens_post_padded, (int)capacity, (hipStream_t)stream);
        return after_launch("moe_align");
    } catch (...) {
        return fail(WQ_ERR_HIP, "moe_align: unexpected exception");
    }
}

// the launches of moe_route_align (arguments already validated)
static wq_status launch_routing(const float* d_logits, int M, int E, int topk, int renormalize, int block_size,
                               float* d_topk_weights, int32_t* d_topk_ids, int32_t* d_sorted_token_ids,
                               int32_t* d_expert_ids, int32_t* d_num_tokens_post_padded, size_t capacity,
                               hipStream_t s, const char* who) {
    const int rn = renormalize ? 1 : 0;
    if (M > 0 && wq::route_align_fused(M, topk)) {
        wq::launch_route_align(d_logits, M, E, topk, rn, d_topk_weights, d_topk_ids, block_size, d_sorted_token_ids,
                               d_expert_ids, d_num_tokens_post_padded, (int)capacity, s);
    } else {
        if (M > 0) {
            wq::launch_route(d_logits, M, E, topk, rn, d_topk_weights, d_topk_ids, s);
            WQ_TRY(after_launch(who));
        }
        wq::launch_align(d_topk_ids, M * topk, E, block_size, d_sorted_token_ids, d_expert_ids,
                         d_num_tokens_post_padded, (int)capacity, s);
    }
    return after_launch(who);
}

wq_status moe_route_align(const float* d_logits, int M, int E, int topk, int renormalize, int block_size,
                          float* d_topk_weights, int32_t* d_topk_ids, int32_t* d_sorted_token_ids,
                          int32_t* d_expert_ids, int32_t* d_num_tokens_post_padded, size_t capacity, void* stream) {
    try {
        WQ_REQUIRE(M >= 0, WQ_ERR_INVALID, "M = %d < 0", M);
        WQ_REQUIRE(E >= 1 && topk >= 1 && topk <= E, WQ_ERR_INVALID, "need 1 <= topk <= E (topk %d, E %d)", topk, E);
        WQ_REQUIRE(E <= 1024, WQ_ERR_UNSUPPORTED, "E = %d > 1024", E);
        WQ_REQUIRE(topk <= 16, WQ_ERR_UNSUPPORTED, "topk = %d > 16", topk);
        WQ_REQUIRE(valid_block_size(block_size), WQ_ERR_UNSUPPORTED, "block_size %d not in {16,32,64,128,256}",
                   block_size);
        WQ_REQUIRE((int64_t)M * topk <= MAX_PAIRS, WQ_ERR_UNSUPPORTED, "M*topk > 2^24");
        const size_t need = moe_align_capacity(M, topk, E, block_size);
        WQ_REQUIRE(capacity >= need, WQ_ERR_INVALID, "capacity %zu < required %zu", capacity, need);
        WQ_REQUIRE(capacity % (size_t)block_size == 0, WQ_ERR_INVALID, "capacity not a multiple of block_size");
        WQ_REQUIRE(capacity <= (size_t)0x7fffffff, WQ_ERR_UNSUPPORTED, "capacity too large");
        if (M > 0) {
            WQ_TRY(check_ptr(d_logits, "logits"));
            WQ_TRY(check_ptr(d_topk_weights, "topk_weights"));
            WQ_TRY(check_ptr(d_topk_ids, "topk_ids"));
        }
        WQ_TRY(check_ptr(d_sorted_token_ids, "sorted_token_ids"));
        WQ_TRY(check_ptr(d_expert_ids, "expert_ids"));
        WQ_TRY(check_ptr(d_num_tokens_post_padded, "num_tokens_post_padded"));
        if (M > 0) {
            WQ_TRY(check_dev(d_logits, "logits"));
            WQ_TRY(check_dev(d_topk_weights, "topk_weights"));
            WQ_TRY(check_dev(d_topk_ids, "topk_ids"));
        }
        WQ_TRY(check_dev(d_sorted_token_ids, "sorted_token_ids"));
        WQ_TRY(check_dev(d_expert_ids, "expert_ids"));
        WQ_TRY(check_dev(d_num_tokens_post_padded, "num_tokens_post_padded"));
        return launch_routing(d_logits, M, E, topk, renormalize, block_size, d_topk_weights, d_topk_ids,
                              d_sorted_token_ids, d_expert_ids, d_num_tokens_post_padded, capacity,
                              (hipStream_t)stream, "moe_route_align");
    } catch (...) {
        return fail(WQ_ERR_HIP, "moe_route_align: unexpected exception");
    }
}

// ---------------------------------------------------------------------------
// moe_route_grouped: the arguments both calls share
static wq_status route_grouped_args(wq::RouteGroupedArgs& g, const void* d_logits, int dtype, int M, int E, int topk,
                                    int scoring, const float* d_bias, int n_group, int topk_group, int group_score,
                                    int renormalize, float routed_scale, float* d_topk_weights, int32_t* d_topk_ids) {
    WQ_REQUIRE(dtype == WQ_F32 || dtype == WQ_F16 || dtype == WQ_BF16, WQ_ERR_INVALID, "bad logits dtype %d", dtype);
    WQ_REQUIRE(M >= 0, WQ_ERR_INVALID, "M = %d < 0", M);
    WQ_REQUIRE(E >= 1 && topk >= 1 && topk <= E, WQ_ERR_INVALID, "need 1 <= topk <= E (topk %d, E %d)", topk, E);
    WQ_REQUIRE(E <= 1024, WQ_ERR_UNSUPPORTED, "E = %d > 1024", E);
    WQ_REQUIRE(topk <= 16, WQ_ERR_UNSUPPORTED, "topk = %d > 16", topk);
    WQ_REQUIRE((int64_t)M * topk <= MAX_PAIRS, WQ_ERR_UNSUPPORTED, "M*topk > 2^24");
    WQ_REQUIRE(scoring == WQ_SCORE_SOFTMAX || scoring == WQ_SCORE_SIGMOID, WQ_ERR_INVALID, "bad scoring %d", scoring);
    WQ_REQUIRE(group_score == WQ_GROUP_MAX || group_score == WQ_GROUP_TOP2, WQ_ERR_INVALID, "bad group_score %d",
               group_score);
    WQ_REQUIRE(n_group >= 1 && E % n_group == 0, WQ_ERR_INVALID, "n_group %d does not divide E %d", n_group, E);
    WQ_REQUIRE(n_group <= 64, WQ_ERR_UNSUPPORTED, "n_group = %d > 64", n_group);
    WQ_REQUIRE(topk_group >= 1 && topk_group <= n_group, WQ_ERR_INVALID, "need 1 <= topk_group <= n_group (%d, %d)",
               topk_group, n_group);
    WQ_REQUIRE((int64_t)topk <= (int64_t)topk_group * (E / n_group), WQ_ERR_INVALID,
               "topk %d > the %d open groups' %d experts", topk, topk_group, topk_group * (E / n_group));
    WQ_REQUIRE(group_score != WQ_GROUP_TOP2 || n_group == 1 || E / n_group >= 2, WQ_ERR_INVALID,
               "groups of one expert have no two best");
    WQ_REQUIRE(std::isfinite(routed_scale), WQ_ERR_INVALID, "routed_scale is not finite");
    if (M > 0) {
        WQ_TRY(check_ptr(d_logits, "logits"));
        if (d_bias) WQ_TRY(check_ptr(d_bias, "bias"));
        WQ_TRY(check_ptr(d_topk_weights, "topk_weights"));
        WQ_TRY(check_ptr(d_topk_ids, "topk_ids"));
    }
    g = wq::RouteGroupedArgs{d_logits, d_bias, d_topk_weights, d_topk_ids, dtype, M, E, topk, n_group, topk_group,
                             scoring == WQ_SCORE_SIGMOID ? 1 : 0, group_score == WQ_GROUP_TOP2 ? 1 : 0,
                             renormalize ? 1 : 0, routed_scale};
    return WQ_OK;
}

static wq_status route_grouped_devs(const wq::RouteGroupedArgs& g, int cur) {
    WQ_TRY(check_dev(g.logits, "logits", cur));
    if (g.bias) WQ_TRY(check_dev(g.bias, "bias", cur));
    WQ_TRY(check_dev(g.w_out, "topk_weights", cur));
    WQ_TRY(check_dev(g.ids_out, "topk_ids", cur));
    return WQ_OK;
}

wq_status moe_route_grouped(const void* d_logits, int logits_dtype, int M, int E, int topk, int scoring,
                            const float* d_bias, int n_group, int topk_group, int group_score, int renormalize,
                            float routed_scale, float* d_topk_weights, int32_t* d_topk_ids, void* stream) {
    try {
        wq::RouteGroupedArgs g{};
        WQ_TRY(route_grouped_args(g, d_logits, logits_dtype, M, E, topk, scoring, d_bias, n_group, topk_group,
                                  group_score, renormalize, routed_scale, d_topk_weights, d_topk_ids));
        if (M == 0) return ok();
        int cur = -1;
        WQ_TRY(current_device(&cur));
        WQ_TRY(route_grouped_devs(g, cur));
        wq::launch_route_grouped(g, (hipStream_t)stream);
        return after_launch("moe_route_grouped");
    } catch (...) {
        return fail(WQ_ERR_HIP, "moe_route_grouped: unexpected exception");
    }
}

wq_status moe_route_grouped_align(const void* d_logits, int logits_dtype, int M, int E, int topk, int scoring,
                                  const float* d_bias, int n_group, int topk_group, int group_score, int renormalize,
                                  float routed_scale, int block_size, float* d_topk_weights, int32_t* d_topk_ids,
                                  int32_t* d_sorted_token_ids, int32_t* d_expert_ids,
                                  int32_t* d_num_tokens_post_padded, size_t capacity, void* stream) {
    try {
        wq::RouteGroupedArgs g{};
        WQ_TRY(route_grouped_args(g, d_logits, logits_dtype, M, E, topk, scoring, d_bias, n_group, topk_group,
                                  group_score, renormalize, routed_scale, d_topk_weights, d_topk_ids));
        WQ_REQUIRE(valid_block_size(block_size), WQ_ERR_UNSUPPORTED, "block_size %d not in {16,32,64,128,256}",
                   block_size);
        const size_t need = moe_align_capacity(M, topk, E, block_size);
        WQ_REQUIRE(capacity >= need, WQ_ERR_INVALID, "capacity %zu < required %zu", capacity, need);
        WQ_REQUIRE(capacity % (size_t)block_size == 0, WQ_ERR_INVALID, "capacity not a multiple of block_size");
        WQ_REQUIRE(capacity <= (size_t)0x7fffffff, WQ_ERR_UNSUPPORTED, "capacity too large");
        WQ_TRY(check_ptr(d_sorted_token_ids, "sorted_token_ids"));
        WQ_TRY(check_ptr(d_expert_ids, "expert_ids"));
        WQ_TRY(check_ptr(d_num_tokens_post_padded, "num_tokens_post_padded"));
        int cur = -1;
        WQ_TRY(current_device(&cur));
        if (M > 0) WQ_TRY(route_grouped_devs(g, cur));
        WQ_TRY(check_dev(d_sorted_token_ids, "sorted_token_ids", cur));
        WQ_TRY(check_dev(d_expert_ids, "expert_ids", cur));
        WQ_TRY(check_dev(d_num_tokens_post_padded, "num_tokens_post_padded", cur));
        hipStream_t s = (hipStream_t)stream;
        if (M > 0 && wq::route_grouped_fused(g)) {
            wq::launch_route_grouped_align(g, block_size, d_sorted_token_ids, d_expert_ids, d_num_tokens_post_padded,
                                           (int)capacity, s);
            return after_launch("moe_route_grouped_align");
        }
        if (M > 0) {
            wq::launch_route_grouped(g, s);
            WQ_TRY(after_launch("moe_route_grouped_align"));
        }
        wq::launch_align(d_topk_ids, M * topk, E, block_size, d_sorted_token_ids, d_expert_ids,
                         d_num_tokens_post_padded, (int)capacity, s);
        return after_launch("moe_route_grouped_align");
    } catch (...) {
        return fail(WQ_ERR_HIP, "moe_route_grouped_align: unexpected exception");
    }
}

// ---------------------------------------------------------------------------
// two arrays of `rows` rows (row starts `stride` bytes apart, `width` bytes
// used of each) that share a byte
static bool rows_overlap(const void* pa, int64_t sa, int64_t wa, const void* pb, int64_t sb, int64_t wb, int64_t rows) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(pa), b = reinterpret_cast<uintptr_t>(pb);
    const uintptr_t ea = a + (uintptr_t)((rows - 1) * sa + wa), eb = b + (uintptr_t)((rows - 1) * sb + wb);
    if (ea <= b || eb <= a) return false;
    if (rows == 1 || sa != sb) return true;  // other strides over one range: taken to overlap
    const uintptr_t d = b >= a ? (b - a) % (uintptr_t)sa : (uintptr_t)sa - 1 - (a - b - 1) % (uintptr_t)sa;
    return !(d >= (uintptr_t)wa && d + (uintptr_t)wb <= (uintptr_t)sa);  // b's rows in the gaps of a's
}

wq_status wq_rms_norm(const void* d_x, int64_t x_stride, const void* d_residual, int64_t residual_stride,
                      const void* d_weight, int rows, int n, float eps, int act_dtype, void* d_residual_out,
                      int64_t residual_out_stride, void* d_out, int64_t out_stride, uint8_t* d_codes, float* d_scales,
                      float static_scale, void* stream) {
    try {
        const char* who = "wq_rms_norm";
        WQ_REQUIRE(act_dtype == WQ_F16 || act_dtype == WQ_BF16, WQ_ERR_INVALID, "%s: bad act dtype", who);
        WQ_REQUIRE(rows >= 0 && n >= 1, WQ_ERR_INVALID, "%s: bad sizes rows %d n %d", who, rows, n);
        WQ_REQUIRE(n <= (1 << 30), WQ_ERR_UNSUPPORTED, "%s: n = %d > 2^30", who, n);
        WQ_REQUIRE(std::isfinite(eps) && eps >= 1e-30f, WQ_ERR_INVALID, "%s: eps must be finite and >= 1e-30", who);
        if (rows == 0) return ok();  // (empty arrays may have no address)
        WQ_REQUIRE(d_residual_out || d_out || d_codes, WQ_ERR_INVALID, "%s: no output", who);
        WQ_REQUIRE(d_codes || !d_scales, WQ_ERR_INVALID, "%s: row scales without codes", who);
        WQ_REQUIRE(!d_codes || d_scales || (std::isfinite(static_scale) && static_scale > 0.0f), WQ_ERR_INVALID,
                   "%s: static_scale must be finite and > 0", who);
        struct Rows {
            const void* p;
            int64_t stride, width;  // bytes
            const char* name;
        };
        const int64_t most = INT64_MAX / 4 / rows;
        const Rows in[3] = {{d_x, x_stride * 2, (int64_t)n * 2, "x"},
                            {d_residual, residual_stride * 2, (int64_t)n * 2, "residual"},
                            {d_weight, 0, (int64_t)n * 2, "weight"}};
        const Rows out[4] = {{d_residual_out, residual_out_stride * 2, (int64_t)n * 2, "residual_out"},
                             {d_out, out_stride * 2, (int64_t)n * 2, "out"},
                             {d_codes, n, n, "codes"},
                             {d_scales, 4, 4, "scales"}};
        const int64_t strides[4] = {x_stride, residual_stride, residual_out_stride, out_stride};
        const void* strided[4] = {d_x, d_residual, d_residual_out, d_out};
        for (int i = 0; i < 4; ++i)
            WQ_REQUIRE(!strided[i] || (strides[i] >= n && strides[i] <= most), WQ_ERR_INVALID,
                       "%s: row stride %lld (n %d)", who, (long long)strides[i], n);
        WQ_TRY(check_ptr(d_x, "x"));
        for (const Rows* a : {&in[1], &in[2], &out[0], &out[1], &out[2], &out[3]})
            if (a->p) WQ_TRY(check_ptr(a->p, a->name));
        for (int o = 0; o < 4; ++o) {
            if (!out[o].p) continue;
            for (int i = 0; i < 3; ++i) {
                if (!in[i].p) continue;
                const bool same = o < 2 && i < 2 && in[i].p == out[o].p && in[i].stride == out[o].stride;
                // the weight is one row: every row of the output against it
                const bool clash = i == 2 ? rows_overlap(out[o].p, 0, (rows - 1) * out[o].stride + out[o].width,
                                                         in[i].p, 0, in[i].width, 1)
                                          : rows_overlap(out[o].p, out[o].stride, out[o].width, in[i].p, in[i].stride,
                                                         in[i].width, rows);
                WQ_REQUIRE(same || !clash, WQ_ERR_INVALID, "%s: %s overlaps %s", who, out[o].name, in[i].name);
            }
            for (int p = 0; p < o; ++p)
                WQ_REQUIRE(!out[p].p || !rows_overlap(out[o].p, out[o].stride, out[o].width, out[p].p, out[p].stride,
                                                      out[p].width, rows),
                           WQ_ERR_INVALID, "%s: %s overlaps %s", who, out[o].name, out[p].name);
        }
        int cur = -1;
        WQ_TRY(current_device(&cur));
        WQ_TRY(check_dev(d_x, "x", cur));
        for (const Rows* a : {&in[1], &in[2], &out[0], &out[1], &out[2], &out[3]})
            if (a->p) WQ_TRY(check_dev(a->p, a->name, cur));
        wq::RmsNormArgs g{};
        g.x = static_cast<const uint16_t*>(d_x);
        g.r = static_cast<const uint16_t*>(d_residual);
        g.w = static_cast<const uint16_t*>(d_weight);
        g.r_out = static_cast<uint16_t*>(d_residual_out);
        g.out = static_cast<uint16_t*>(d_out);
        g.codes = d_codes;
        g.scales = d_scales;
        g.x_stride = x_stride;
        g.r_stride = residual_stride;
        g.ro_stride = residual_out_stride;
        g.out_stride = out_stride;
        g.rows = rows;
        g.n = n;
        g.eps = eps;
        g.static_scale = static_scale;
        wq::launch_rms_norm(g, act_dtype == WQ_BF16, (hipStream_t)stream);
        return after_launch(who);
    } catch (...) {
        return fail(WQ_ERR_HIP, "wq_rms_norm: unexpected exception");
    }
}

// ---------------------------------------------------------------------------
// fp32 slabs of M*topk x n_out the DOWN stage may write (one per K slice)
static int down_slabs(int M, int topk, int E, int n_out, int k_in) {
    return std::max(wq::prefill_down_split_max(M * topk, E, n_out, k_in), wq::tiny_down_slabs(M, k_in));
}

size_t moe_gemm_workspace_bytes(int stage, int M, int topk, int E, int n_out, int k_in, size_t capacity,
                                int act_order) {
    if (M < 0 || topk <= 0 || E <= 0 || n_out <= 0 || k_in <= 0) return 0;
    size_t b = 0;
    if ((stage == WQ_STAGE_GATE_UP || stage == WQ_STAGE_RAW) && act_order) b += round256(capacity * k_in * 2);
    if (stage == WQ_STAGE_DOWN) b += round256((size_t)down_slabs(M, topk, E, n_out, k_in) * M * topk * n_out * sizeof(float));
    return b;
}

// A GATE_UP call that also routes the batch (moe_route_gate_up): the logits
// and the routing outputs; the desc's sorted_token_ids / expert_ids /
// num_tokens_post_padded are then written, not read.
struct RouteRequest {
    const float* logits;
    int renormalize;
    float* topk_weights;
    int32_t* topk_ids;
};

// noalloc: the workspace is the library's scratch array (d_workspace must be
// NULL and workspace_bytes 0; a need above its size is refused)
static wq_status moe_gemm(const wq_moe_gemm_desc* d, int wbits, void* stream, const char* who, bool noalloc = false,
                          const RouteRequest* route = nullptr) {
    WQ_REQUIRE(d != nullptr, WQ_ERR_INVALID, "%s: desc is NULL", who);
    WQ_REQUIRE(d->struct_size >= sizeof(wq_moe_gemm_desc), WQ_ERR_INVALID, "%s: struct_size %zu < %zu", who,
               d->struct_size, sizeof(wq_moe_gemm_desc));
    const int stage = d->stage;
    WQ_REQUIRE(stage == WQ_STAGE_GATE_UP || stage == WQ_STAGE_DOWN || stage == WQ_STAGE_RAW, WQ_ERR_INVALID,
               "%s: bad stage %d", who, stage);
    WQ_REQUIRE(d->act_dtype == WQ_F16 || d->act_dtype == WQ_BF16, WQ_ERR_INVALID, "%s: bad act dtype", who);
    if (wbits == 4) WQ_REQUIRE(d->act_dtype == WQ_F16, WQ_ERR_UNSUPPORTED, "%s: int4 path takes fp16 activations", who);
    WQ_REQUIRE(d->M >= 0 && d->topk >= 1 && d->E >= 1 && d->topk <= d->E, WQ_ERR_INVALID,
               "%s: bad M/topk/E (%d/%d/%d)", who, d->M, d->topk, d->E);
    WQ_REQUIRE(d->E <= 1024, WQ_ERR_UNSUPPORTED, "%s: E > 1024", who);
    WQ_REQUIRE((int64_t)d->M * d->topk <= MAX_PAIRS, WQ_ERR_UNSUPPORTED, "%s: M*topk > 2^24", who);
    WQ_REQUIRE(d->n_out > 0 && d->k_in > 0, WQ_ERR_INVALID, "%s: bad n_out/k_in", who);
    const int kchunk = wbits == 4 ? wq::WFmt<4>::KCHUNK : wq::WFmt<8>::KCHUNK;
    WQ_REQUIRE(d->k_in % kchunk == 0, WQ_ERR_UNSUPPORTED, "%s: k_in %d not a multiple of %d", who, d->k_in, kchunk);
    WQ_REQUIRE(d->n_out % (stage == WQ_STAGE_GATE_UP ? 32 : 16) == 0, WQ_ERR_UNSUPPORTED,
               "%s: n_out %d not a multiple of %d", who, d->n_out, stage == WQ_STAGE_GATE_UP ? 32 : 16);
    if (wbits == 4)
        WQ_REQUIRE(d->group_size == 128 || d->group_size == -1, WQ_ERR_UNSUPPORTED, "%s: group_size %d", who,
                   d->group_size);
    else
        WQ_REQUIRE(d->group_size == -1, WQ_ERR_UNSUPPORTED, "%s: int8 weights take per-column scales (-1)", who);
    WQ_REQUIRE(valid_block_size(d->block_size), WQ_ERR_UNSUPPORTED, "%s: block_size %d", who, d->block_size);
    const size_t need_cap = moe_align_capacity(d->M, d->topk, d->E, d->block_size);
    WQ_REQUIRE(d->capacity >= need_cap && d->capacity % (size_t)d->block_size == 0 &&
                   d->capacity <= (size_t)0x7fffffff,
               WQ_ERR_INVALID, "%s: capacity %zu (need >= %zu, multiple of block_size)", who, d->capacity, need_cap);
    const bool act_order = d->d_k_perm != nullptr;
    WQ_REQUIRE(!act_order || (wbits == 4 && stage != WQ_STAGE_DOWN), WQ_ERR_INVALID,
               "%s: k_perm only applies to int4 GATE_UP/RAW", who);
    if (route) {
        WQ_REQUIRE(stage == WQ_STAGE_GATE_UP, WQ_ERR_INVALID, "%s: routing goes with the GATE_UP stage", who);
        WQ_REQUIRE(d->topk <= 16, WQ_ERR_UNSUPPORTED, "%s: topk = %d > 16", who, d->topk);
    }
    const size_t ws = moe_gemm_workspace_bytes(stage, d->M, d->topk, d->E, d->n_out, d->k_in, d->capacity, act_order);
    if (noalloc) {
        WQ_REQUIRE(d->d_workspace == nullptr && d->workspace_bytes == 0, WQ_ERR_INVALID,
                   "%s: takes no workspace (d_workspace must be NULL, workspace_bytes 0)", who);
        WQ_REQUIRE(ws <= (size_t)WQ_NOALLOC_SCRATCH_BYTES, WQ_ERR_UNSUPPORTED,
                   "%s: needs %zu bytes of workspace, more than the %zu-byte scratch", who, ws,
                   (size_t)WQ_NOALLOC_SCRATCH_BYTES);
    } else {
        WQ_REQUIRE(d->workspace_bytes >= ws, WQ_ERR_INVALID, "%s: workspace %zu < required %zu", who,
                   d->workspace_bytes, ws);
    }
    if (d->M == 0) {
        if (!route) return ok();
        // no tokens: the routing arrays are still written (an empty sort)
        WQ_TRY(check_ptr(d->d_sorted_token_ids, "sorted_token_ids"));
        WQ_TRY(check_ptr(d->d_expert_ids, "expert_ids"));
        WQ_TRY(check_ptr(d->d_num_tokens_post_padded, "num_tokens_post_padded"));
        WQ_TRY(check_dev(d->d_sorted_token_ids, "sorted_token_ids"));
        WQ_TRY(check_dev(d->d_expert_ids, "expert_ids"));
        WQ_TRY(check_dev(d->d_num_tokens_post_padded, "num_tokens_post_padded"));
        return launch_routing(nullptr, 0, d->E, d->topk, route->renormalize, d->block_size, nullptr, nullptr,
                              const_cast<int32_t*>(d->d_sorted_token_ids), const_cast<int32_t*>(d->d_expert_ids),
                              const_cast<int32_t*>(d->d_num_tokens_post_padded), d->capacity, (hipStream_t)stream,
                              who);
    }
    WQ_TRY(check_ptr(d->d_a, "a"));
    WQ_TRY(check_ptr(d->d_w_packed, "w_packed"));
    WQ_TRY(check_ptr(d->d_scales, "scales"));
    WQ_TRY(check_ptr(d->d_sorted_token_ids, "sorted_token_ids"));
    WQ_TRY(check_ptr(d->d_expert_ids, "expert_ids"));
    WQ_TRY(check_ptr(d->d_num_tokens_post_padded, "num_tokens_post_padded"));
    WQ_TRY(check_ptr(d->d_out, "out"));
    if (act_order) WQ_TRY(check_ptr(d->d_k_perm, "k_perm"));
    if (stage == WQ_STAGE_DOWN) WQ_TRY(check_ptr(d->d_topk_weights, "topk_weights"));
    if (ws && !noalloc) WQ_TRY(check_ptr(d->d_workspace, "workspace"));
    if (route) {
        WQ_TRY(check_ptr(route->logits, "logits"));
        WQ_TRY(check_ptr(route->topk_weights, "topk_weights"));
        WQ_TRY(check_ptr(route->topk_ids, "topk_ids"));
        WQ_TRY(check_dev(route->logits, "logits"));
        WQ_TRY(check_dev(route->topk_weights, "topk_weights"));
        WQ_TRY(check_dev(route->topk_ids, "topk_ids"));
    }

    WQ_TRY(check_dev(d->d_a, "a"));
    WQ_TRY(check_dev(d->d_w_packed, "w_packed"));
    WQ_TRY(check_dev(d->d_scales, "scales"));
    WQ_TRY(check_dev(d->d_sorted_token_ids, "sorted_token_ids"));
    WQ_TRY(check_dev(d->d_expert_ids, "expert_ids"));
    WQ_TRY(check_dev(d->d_num_tokens_post_padded, "num_tokens_post_padded"));
    WQ_TRY(check_dev(d->d_out, "out"));
    if (act_order) WQ_TRY(check_dev(d->d_k_perm, "k_perm"));
    if (stage == WQ_STAGE_DOWN) WQ_TRY(check_dev(d->d_topk_weights, "topk_weights"));
    if (ws && !noalloc) WQ_TRY(check_dev(d->d_workspace, "workspace"));
    void* workspace = d->d_workspace;
    if (ws && noalloc) WQ_TRY(scratch_for_current_device(&workspace));

    hipStream_t s = (hipStream_t)stream;
    const bool bf16 = d->act_dtype == WQ_BF16;
    wq::GemmArgs g{};
    g.a = static_cast<const uint16_t*>(d->d_a);
    g.w = static_cast<const uint8_t*>(d->d_w_packed);
    g.s = static_cast<const uint16_t*>(d->d_scales);
    g.sorted = d->d_sorted_token_ids;
    g.expert_ids = d->d_expert_ids;
    g.ntpp = d->d_num_tokens_post_padded;
    g.topk_w = d->d_topk_weights;
    g.out = d->d_out;
    g.M = d->M;
    g.topk = d->topk;
    g.E = d->E;
    g.n_out = d->n_out;
    g.k_in = d->k_in;
    g.block_size = d->block_size;
    g.groups = (wbits == 4 && d->group_size == 128) ? d->k_in / 128 : 1;
    g.a_direct = (stage == WQ_STAGE_DOWN) ? 1 : 0;
    g.cap = (int)d->capacity;

    if (stage == WQ_STAGE_DOWN && wq::tiny_down_combine_supported(wbits, d->M, d->topk, d->n_out, d->k_in)) {
        // one token: the top-k sum is folded into the DOWN kernel
        wq::launch_tiny_down_combine(wbits, bf16, g, static_cast<uint16_t*>(d->d_out), s);
        return after_launch(who);
    }
    const int slabs = stage == WQ_STAGE_DOWN ? down_slabs(d->M, d->topk, d->E, d->n_out, d->k_in) : 1;
    const bool tiny = wq::tiny_supported(wbits, stage, d->M, d->k_in, g.groups, slabs);
    const bool large = !tiny && wq::prefill_supported(d->n_out, d->k_in, d->block_size);
    WQ_REQUIRE(!large || wq::prefill_fits(d->capacity, d->k_in), WQ_ERR_UNSUPPORTED,
               "%s: activations of %zu rows x %d channels exceed 4 GiB (large-batch kernel)", who, d->capacity,
               d->k_in);
    bool gathered = false;  // the act-order rows already gathered by the routing launch
    if (route) {
        // one launch: the small-batch kernel routes and sorts the batch itself,
        // and for one token of an act-order layer each workgroup also gathers
        // the token's row in its expert's channel order
        const bool fold = !tiny && !large &&
                          wq::decode_route_supported(stage, d->M, d->topk, d->E, (int)d->capacity, d->block_size) &&
                          (!act_order || wq::decode_route_ao_supported(d->M, d->topk, d->n_out, d->k_in));
        if (fold) {
            wq::RouteArgs ra;
            ra.logits = route->logits;
            ra.renormalize = route->renormalize ? 1 : 0;
            ra.w_out = route->topk_weights;
            ra.ids_out = route->topk_ids;
            // the desc's routing arrays are outputs of this call
            ra.sorted_out = const_cast<int32_t*>(d->d_sorted_token_ids);
            ra.expert_ids_out = const_cast<int32_t*>(d->d_expert_ids);
            ra.ntpp_out = const_cast<int32_t*>(d->d_num_tokens_post_padded);
            ra.perm = act_order ? d->d_k_perm : nullptr;
            wq::launch_gemm_decode_route(wbits, bf16, g, ra, s);
            return after_launch(who);
        }
        if (act_order && !tiny &&
            wq::route_gather_supported(d->M, d->topk, d->E, (int)d->capacity, d->block_size)) {
            // one launch routes, sorts and gathers the act-order rows
            uint16_t* a1 = static_cast<uint16_t*>(workspace);
            wq::launch_route_align_gather(route->logits, d->M, d->E, d->topk, route->renormalize ? 1 : 0,
                                          route->topk_weights, route->topk_ids,
                                          d->block_size, const_cast<int32_t*>(d->d_sorted_token_ids),
                                          const_cast<int32_t*>(d->d_expert_ids),
                                          const_cast<int32_t*>(d->d_num_tokens_post_padded), (int)d->capacity, g.a,
                                          d->d_k_perm, d->k_in, a1, s);
            WQ_TRY(after_launch(who));
            g.a = a1;
            g.a_direct = 1;
            gathered = true;
        } else {
            WQ_TRY(launch_routing(route->logits, d->M, d->E, d->topk, route->renormalize, d->block_size,
                                  route->topk_weights, route->topk_ids, const_cast<int32_t*>(d->d_sorted_token_ids),
                                  const_cast<int32_t*>(d->d_expert_ids),
                                  const_cast<int32_t*>(d->d_num_tokens_post_padded), d->capacity, s, who));
        }
    }
    if (act_order && !tiny && !gathered) {
        uint16_t* a1 = static_cast<uint16_t*>(workspace);
        wq::launch_gather_perm(g.a, d->d_k_perm, g.sorted, g.expert_ids, g.ntpp, d->M, d->topk, d->k_in,
                               d->block_size, g.cap, a1, s);
        WQ_TRY(after_launch(who));
        g.a = a1;
        g.a_direct = 1;
    }
    float* y = nullptr;
    if (stage == WQ_STAGE_DOWN) {
        y = static_cast<float*>(workspace);
        g.out = y;
        // a large-batch DOWN that does not split K writes each pair's routed
        // row rounded once to the activation type (half the bytes of the
        // per-pair rows each way); split slices keep fp32 partial sums
        g.y_act = (large && wq::prefill_down_split(d->M * d->topk, d->E, d->n_out, d->k_in, d->block_size) == 1)
                      ? 1 : 0;
    }
    int ksplit = 1;
    if (tiny) ksplit = wq::launch_gemm_tiny(wbits, bf16, stage, g, act_order ? d->d_k_perm : nullptr, slabs, s);
    else if (large) ksplit = wq::launch_gemm_prefill(wbits, bf16, stage, g, s);
    else wq::launch_gemm_decode(wbits, bf16, stage, g, s);
    WQ_TRY(after_launch(who));
    if (stage == WQ_STAGE_DOWN) {
        if (g.y_act) {
            WQ_REQUIRE(ksplit == 1, WQ_ERR_HIP, "%s: DOWN split K after all", who);
            wq::launch_combine_act(reinterpret_cast<const uint16_t*>(y), d->M, d->topk, d->n_out, bf16,
                                   static_cast<uint16_t*>(d->d_out), s);
        } else {
            wq::launch_combine(y, d->M, d->topk, d->n_out, ksplit, bf16, static_cast<uint16_t*>(d->d_out), s);
        }
        WQ_TRY(after_launch(who));
    }
    return ok();
}

wq_status moe_w4a16_gemm(const wq_moe_gemm_desc* d, void* stream) {
    try {
        return moe_gemm(d, 4, stream, "moe_w4a16_gemm");
    } catch (...) {
        return fail(WQ_ERR_HIP, "moe_w4a16_gemm: unexpected exception");
    }
}

wq_status moe_w8a16_gemm(const wq_moe_gemm_desc* d, void* stream) {
    try {
        return moe_gemm(d, 8, stream, "moe_w8a16_gemm");
    } catch (...) {
        return fail(WQ_ERR_HIP, "moe_w8a16_gemm: unexpected exception");
    }
}

wq_status moe_route_gate_up(const float* d_logits, int renormalize, float* d_topk_weights, int32_t* d_topk_ids,
                            const wq_moe_gemm_desc* d, int wbits, void* stream) {
    try {
        WQ_REQUIRE(wbits == 4 || wbits == 8, WQ_ERR_INVALID, "moe_route_gate_up: wbits %d not 4 or 8", wbits);
        const RouteRequest rr{d_logits, renormalize, d_topk_weights, d_topk_ids};
        return moe_gemm(d, wbits, stream, "moe_route_gate_up", false, &rr);
    } catch (...) {
        return fail(WQ_ERR_HIP, "moe_route_gate_up: unexpected exception");
    }
}

wq_status moe_w8a16_gemm_noalloc(const wq_moe_gemm_desc* d, void* stream) {
    try {
        return moe_gemm(d, 8, stream, "moe_w8a16_gemm_noalloc", true);
    } catch (...) {
        return fail(WQ_ERR_HIP, "moe_w8a16_gemm_noalloc: unexpected exception");
    }
}

// ---------------------------------------------------------------------------
// FP8 (E4M3) W8A8 grouped GEMM
// ---------------------------------------------------------------------------
static int fp8_down_slabs(int M, int topk, int E, int n_out, int k_in) {
    const int T = M * topk;
    return std::max(wq::fp8_down_split(T, E, n_out, k_in, 64), wq::fp8_down_split(T, E, n_out, k_in, 128));
}

size_t moe_fp8_gemm_workspace_bytes(int stage, int M, int topk, int E, int n_out, int k_in) {
    if (M < 0 || topk <= 0 || E <= 0 || n_out <= 0 || k_in <= 0) return 0;
    if (stage == WQ_STAGE_GATE_UP || stage == WQ_STAGE_RAW) return round256((size_t)M * k_in);  // x codes
    if (stage == WQ_STAGE_DOWN)
        return round256((size_t)fp8_down_slabs(M, topk, E, n_out, k_in) * M * topk * n_out * sizeof(float));
    return 0;
}

// codes: d_a holds E4M3 codes of x, with a scale per row (row_scales) or
// in_scale for all; nothing is quantised and no workspace is needed
static wq_status fp8_gemm(const wq_moe_gemm_desc* d, float in_scale, float out_scale, void* stream, const char* who,
                          bool codes = false, const float* row_scales = nullptr) {
    WQ_REQUIRE(d != nullptr, WQ_ERR_INVALID, "%s: desc is NULL", who);
    WQ_REQUIRE(d->struct_size >= sizeof(wq_moe_gemm_desc), WQ_ERR_INVALID, "%s: struct_size %zu < %zu", who,
               d->struct_size, sizeof(wq_moe_gemm_desc));
    const int stage = d->stage;
    WQ_REQUIRE(stage == WQ_STAGE_GATE_UP || stage == WQ_STAGE_DOWN || stage == WQ_STAGE_RAW, WQ_ERR_INVALID,
               "%s: bad stage %d", who, stage);
    WQ_REQUIRE(!codes || stage != WQ_STAGE_DOWN, WQ_ERR_INVALID, "%s: the DOWN stage takes moe_fp8_w8a8_gemm", who);
    WQ_REQUIRE(d->act_dtype == WQ_F16 || d->act_dtype == WQ_BF16, WQ_ERR_INVALID, "%s: bad act dtype", who);
    WQ_REQUIRE(d->M >= 0 && d->topk >= 1 && d->E >= 1 && d->topk <= d->E, WQ_ERR_INVALID,
               "%s: bad M/topk/E (%d/%d/%d)", who, d->M, d->topk, d->E);
    WQ_REQUIRE(d->E <= 1024, WQ_ERR_UNSUPPORTED, "%s: E > 1024", who);
    WQ_REQUIRE((int64_t)d->M * d->topk <= MAX_PAIRS, WQ_ERR_UNSUPPORTED, "%s: M*topk > 2^24", who);
    WQ_REQUIRE(d->n_out > 0 && d->k_in > 0, WQ_ERR_INVALID, "%s: bad n_out/k_in", who);
    WQ_REQUIRE(d->k_in % wq::FP8_KCHUNK == 0, WQ_ERR_UNSUPPORTED, "%s: k_in %d not a multiple of %d", who, d->k_in,
               wq::FP8_KCHUNK);
    WQ_REQUIRE(d->n_out % (stage == WQ_STAGE_GATE_UP ? 32 : 16) == 0, WQ_ERR_UNSUPPORTED,
               "%s: n_out %d not a multiple of %d", who, d->n_out, stage == WQ_STAGE_GATE_UP ? 32 : 16);
    WQ_REQUIRE(d->group_size == -1, WQ_ERR_UNSUPPORTED, "%s: FP8 weights take per-column scales (-1)", who);
    WQ_REQUIRE(d->d_k_perm == nullptr, WQ_ERR_INVALID, "%s: no act-order for FP8 weights", who);
    WQ_REQUIRE(row_scales || (std::isfinite(in_scale) && in_scale > 0.0f), WQ_ERR_INVALID, "%s: in_scale must be finite and > 0",
               who);
    WQ_REQUIRE(stage != WQ_STAGE_GATE_UP || (std::isfinite(out_scale) && out_scale > 0.0f), WQ_ERR_INVALID,
               "%s: out_scale must be finite and > 0", who);
    WQ_REQUIRE(valid_block_size(d->block_size), WQ_ERR_UNSUPPORTED, "%s: block_size %d", who, d->block_size);
    const size_t need_cap = moe_align_capacity(d->M, d->topk, d->E, d->block_size);
    WQ_REQUIRE(d->capacity >= need_cap && d->capacity % (size_t)d->block_size == 0 &&
                   d->capacity <= (size_t)0x7fffffff,
               WQ_ERR_INVALID, "%s: capacity %zu (need >= %zu, multiple of block_size)", who, d->capacity, need_cap);
    const size_t ws = codes ? 0 : moe_fp8_gemm_workspace_bytes(stage, d->M, d->topk, d->E, d->n_out, d->k_in);
    WQ_REQUIRE(d->workspace_bytes >= ws, WQ_ERR_INVALID, "%s: workspace %zu < required %zu", who, d->workspace_bytes,
               ws);
    const bool large = wq::fp8_prefill_supported(d->n_out, d->k_in, d->block_size);
    // the large-batch kernel addresses its activation codes with 32-bit byte offsets
    const size_t a_rows = stage == WQ_STAGE_DOWN ? d->capacity : (size_t)d->M;
    WQ_REQUIRE(!large || a_rows * (size_t)d->k_in <= (size_t)0xffffffffu, WQ_ERR_UNSUPPORTED,
               "%s: activations of %zu rows x %d codes exceed 4 GiB (large-batch kernel)", who, a_rows, d->k_in);
    // its token tiles lie along grid y
    WQ_REQUIRE(!codes || !large || d->capacity / (d->block_size == 64 ? 64 : 128) <= 65535, WQ_ERR_UNSUPPORTED,
               "%s: capacity %zu exceeds 65535 token tiles", who, d->capacity);
    if (d->M == 0) return ok();
    WQ_TRY(check_ptr(d->d_a, "a"));
    WQ_TRY(check_ptr(d->d_w_packed, "w_packed"));
    WQ_TRY(check_ptr(d->d_scales, "scales"));
    WQ_TRY(check_ptr(d->d_sorted_token_ids, "sorted_token_ids"));
    WQ_TRY(check_ptr(d->d_expert_ids, "expert_ids"));
    WQ_TRY(check_ptr(d->d_num_tokens_post_padded, "num_tokens_post_padded"));
    WQ_TRY(check_ptr(d->d_out, "out"));
    if (stage == WQ_STAGE_DOWN) WQ_TRY(check_ptr(d->d_topk_weights, "topk_weights"));
    if (!codes) WQ_TRY(check_ptr(d->d_workspace, "workspace"));
    if (row_scales) WQ_TRY(check_ptr(row_scales, "row_scales"));
    WQ_TRY(check_dev(d->d_a, "a"));
    WQ_TRY(check_dev(d->d_w_packed, "w_packed"));
    WQ_TRY(check_dev(d->d_scales, "scales"));
    WQ_TRY(check_dev(d->d_sorted_token_ids, "sorted_token_ids"));
    WQ_TRY(check_dev(d->d_expert_ids, "expert_ids"));
    WQ_TRY(check_dev(d->d_num_tokens_post_padded, "num_tokens_post_padded"));
    WQ_TRY(check_dev(d->d_out, "out"));
    if (stage == WQ_STAGE_DOWN) WQ_TRY(check_dev(d->d_topk_weights, "topk_weights"));
    if (!codes) WQ_TRY(check_dev(d->d_workspace, "workspace"));
    if (row_scales) WQ_TRY(check_dev(row_scales, "row_scales"));

    hipStream_t s = (hipStream_t)stream;
    const bool bf16 = d->act_dtype == WQ_BF16;
    wq::Fp8GemmArgs g{};
    g.w = static_cast<const uint8_t*>(d->d_w_packed);
    g.s = static_cast<const float*>(d->d_scales);
    g.sorted = d->d_sorted_token_ids;
    g.expert_ids = d->d_expert_ids;
    g.ntpp = d->d_num_tokens_post_padded;
    g.topk_w = d->d_topk_weights;
    g.out = d->d_out;
    g.M = d->M;
    g.topk = d->topk;
    g.E = d->E;
    g.n_out = d->n_out;
    g.k_in = d->k_in;
    g.block_size = d->block_size;
    g.cap = (int)d->capacity;
    g.in_scale = in_scale;
    g.out_scale = out_scale;
    if (codes) {
        g.a = static_cast<const uint8_t*>(d->d_a);
        g.a_direct = 0;
        g.x_codes = 1;
        g.row_scales = row_scales;
    } else if (stage == WQ_STAGE_DOWN) {
        g.a = static_cast<const uint8_t*>(d->d_a);  // H codes in sorted order
        g.a_direct = 1;
        if (wq::fp8_down_combine_supported(d->M, d->topk, d->n_out, d->k_in)) {
            wq::launch_fp8_down_combine(bf16, g, s);  // g.out: the output row
            return after_launch(who);
        }
        g.out = d->d_workspace;                     // fp32 Y slabs
    } else if (wq::fp8_fold_quant_supported(stage, d->M, d->n_out, d->k_in, d->block_size)) {
        g.x16 = static_cast<const uint16_t*>(d->d_a);  // quantised inside the GEMM
        g.x_bf16 = bf16 ? 1 : 0;
        g.a_direct = 0;
    } else {
        uint8_t* xq = static_cast<uint8_t*>(d->d_workspace);
        wq::launch_fp8_quant(static_cast<const uint16_t*>(d->d_a), d->M, d->k_in, bf16, in_scale, xq, s);
        WQ_TRY(after_launch(who));
        g.a = xq;
        g.a_direct = 0;
    }
    const int ks = wq::launch_gemm_fp8(stage, g, s);
    WQ_TRY(after_launch(who));
    if (stage == WQ_STAGE_DOWN) {
        wq::launch_combine(static_cast<const float*>(d->d_workspace), d->M, d->topk, d->n_out, ks, bf16,
                           static_cast<uint16_t*>(d->d_out), s);
        WQ_TRY(after_launch(who));
    }
    return ok();
}

wq_status moe_fp8_w8a8_gemm(const wq_moe_gemm_desc* d, float in_scale, float out_scale, void* stream) {
    try {
        return fp8_gemm(d, in_scale, out_scale, stream, "moe_fp8_w8a8_gemm");
    } catch (...) {
        return fail(WQ_ERR_HIP, "moe_fp8_w8a8_gemm: unexpected exception");
    }
}

wq_status moe_fp8_codes_gemm(const wq_moe_gemm_desc* d, const float* d_row_scales, float in_scale, float out_scale,
                             void* stream) {
    try {
        return fp8_gemm(d, in_scale, out_scale, stream, "moe_fp8_codes_gemm", true, d_row_scales);
    } catch (...) {
        return fail(WQ_ERR_HIP, "moe_fp8_codes_gemm: unexpected exception");
    }
}

static wq_status sparse24_gemm(int bits, const void* d_x, int M, int K, int N, const void* d_vals, const void* d_meta,
                               const void* d_scales, int group_size, void* d_y, int act_dtype, void* stream,
                               const char* who) {
    WQ_REQUIRE(M >= 0 && K > 0 && N > 0, WQ_ERR_INVALID, "%s: bad sizes M %d K %d N %d", who, M, K, N);
    WQ_REQUIRE(act_dtype == WQ_F16, WQ_ERR_UNSUPPORTED, "%s: fp16 activations only", who);
    WQ_REQUIRE(group_size == 128 || group_size == -1, WQ_ERR_UNSUPPORTED, "%s: group_size %d (128 or -1)", who,
               group_size);
    WQ_REQUIRE(K % 256 == 0, WQ_ERR_UNSUPPORTED, "%s: K %d not a multiple of 256", who, K);
    WQ_REQUIRE(N % 16 == 0, WQ_ERR_UNSUPPORTED, "%s: N %d not a multiple of 16", who, N);
    WQ_REQUIRE((M + 15) / 16 <= 65535, WQ_ERR_UNSUPPORTED, "%s: M too large", who);
    if (M == 0) return ok();
    WQ_TRY(check_ptr(d_x, "x"));
    WQ_TRY(check_ptr(d_vals, "vals"));
    WQ_TRY(check_ptr(d_meta, "meta"));
    WQ_TRY(check_ptr(d_scales, "scales"));
    WQ_TRY(check_ptr(d_y, "y"));
    WQ_TRY(check_dev(d_x, "x"));
    WQ_TRY(check_dev(d_vals, "vals"));
    WQ_TRY(check_dev(d_meta, "meta"));
    WQ_TRY(check_dev(d_scales, "scales"));
    WQ_TRY(check_dev(d_y, "y"));
    wq::launch_sparse24(bits, static_cast<const uint16_t*>(d_x), M, K, N, static_cast<const uint8_t*>(d_vals),
                        static_cast<const uint8_t*>(d_meta), static_cast<const uint16_t*>(d_scales), group_size,
                        static_cast<uint16_t*>(d_y), (hipStream_t)stream);
    return after_launch(who);
}

wq_status sparse24_w4a16_gemm(const void* d_x, int M, int K, int N, const void* d_vals, const void* d_meta,
                              const void* d_scales, int group_size, void* d_y, int act_dtype, void* stream) {
    try {
        return sparse24_gemm(4, d_x, M, K, N, d_vals, d_meta, d_scales, group_size, d_y, act_dtype, stream,
                             "sparse24_w4a16_gemm");
    } catch (...) {
        return fail(WQ_ERR_HIP, "sparse24_w4a16_gemm: unexpected exception");
    }
}

wq_status sparse24_w8a16_gemm(const void* d_x, int M, int K, int N, const void* d_vals, const void* d_meta,
                              const void* d_scales, int group_size, void* d_y, int act_dtype, void* stream) {
    try {
        return sparse24_gemm(8, d_x, M, K, N, d_vals, d_meta, d_scales, group_size, d_y, act_dtype, stream,
                             "sparse24_w8a16_gemm");
    } catch (...) {
        return fail(WQ_ERR_HIP, "sparse24_w8a16_gemm: unexpected exception");
    }
}

// ---------------------------------------------------------------------------
// Dense single-expert linear.  1..4 rows (without act-order): one small-batch
// kernel with the rows staged in LDS, no workspace.  Otherwise the grouped
// kernels with E = 1 and top-1 on identity routing written into the workspace,
// the DOWN stage with unit routed weights (rows gathered by token, not by
// sorted position: x has M rows), the combine rounding the fp32 result to the
// activation type.
// ---------------------------------------------------------------------------
namespace {
struct DenseLayout {
    int bs, ks;
    size_t cap, off_sorted, off_eids, off_ntpp, off_w, off_a1, off_y, total;
};

// batch-size dispatch of the grouped path (above 128 rows, or with act-order;
// up to 128 rows without act-order one dense kernel runs, no workspace): the
// small-batch kernel (blocks of 16 rows) up to 24 rows, the large-batch kernel
// with 64-row tiles up to 192 (one expert gives few token tiles: 128-row tiles
// left the GPU part idle, Yi-34B shape int4 M = 128 0.114 -> 0.091 ms, M = 192
// 0.114 -> 0.106 ms; at 256 rows and above they are faster), 128-row tiles above
int dense_block_size(int M, int N, int K) {
    const int bs = M <= 24 ? 16 : (M <= 192 ? 64 : 128);
    return (bs == 16 || wq::prefill_supported(N, K, bs)) ? bs : 16;
}

DenseLayout dense_layout(int M, int K, int N, bool act_order) {
    DenseLayout L{};
    L.bs = dense_block_size(M, N, K);
    L.cap = moe_align_capacity(M, 1, 1, L.bs);
    L.ks = (L.bs == 16) ? 1 : wq::prefill_down_split(M, 1, N, K, L.bs);
    size_t o = 0;
    L.off_sorted = o;
    o += round256(L.cap * 4);
    L.off_eids = o;
    o += round256(L.cap / L.bs * 4);
    L.off_ntpp = o;
    o += 256;
    L.off_w = o;
    o += round256((size_t)M * 4);
    L.off_a1 = o;
    if (act_order) o += round256(L.cap * (size_t)K * 2);
    L.off_y = o;
    o += round256((size_t)L.ks * M * N * sizeof(float));
    L.total = o;
    return L;
}

wq_status dense_gemm(int wbits, const void* d_x, int M, int K, int N, const void* d_w, const void* d_scales,
                     int group_size, const int32_t* d_k_perm, void* d_y, int act_dtype, void* d_ws, size_t ws_bytes,
                     void* stream, const char* who) {
    WQ_REQUIRE(M >= 0 && K > 0 && N > 0, WQ_ERR_INVALID, "%s: bad sizes M %d K %d N %d", who, M, K, N);
    WQ_REQUIRE(M <= MAX_PAIRS, WQ_ERR_UNSUPPORTED, "%s: M > 2^24", who);
    WQ_REQUIRE(act_dtype == WQ_F16 || act_dtype == WQ_BF16, WQ_ERR_INVALID, "%s: bad act dtype", who);
    if (wbits == 4) WQ_REQUIRE(act_dtype == WQ_F16, WQ_ERR_UNSUPPORTED, "%s: int4 path takes fp16 activations", who);
    const int kchunk = wbits == 4 ? wq::WFmt<4>::KCHUNK : wq::WFmt<8>::KCHUNK;
    WQ_REQUIRE(K % kchunk == 0, WQ_ERR_UNSUPPORTED, "%s: K %d not a multiple of %d", who, K, kchunk);
    WQ_REQUIRE(N % 16 == 0, WQ_ERR_UNSUPPORTED, "%s: N %d not a multiple of 16", who, N);
    if (wbits == 4)
        WQ_REQUIRE(group_size == 128 || group_size == -1, WQ_ERR_UNSUPPORTED, "%s: group_size %d", who, group_size);
    const bool act_order = d_k_perm != nullptr;
    const size_t need = dense_gemm_workspace_bytes(M, K, N, act_order);
    WQ_REQUIRE(ws_bytes >= need, WQ_ERR_INVALID, "%s: workspace %zu < required %zu", who, ws_bytes, need);
    if (M == 0) return ok();
    WQ_TRY(check_ptr(d_x, "x"));
    WQ_TRY(check_ptr(d_w, "w_packed"));
    WQ_TRY(check_ptr(d_scales, "scales"));
    WQ_TRY(check_ptr(d_y, "y"));
    if (act_order) WQ_TRY(check_ptr(d_k_perm, "k_perm"));  // read with 128-bit loads by the gather
    WQ_TRY(check_dev(d_x, "x"));
    WQ_TRY(check_dev(d_w, "w_packed"));
    WQ_TRY(check_dev(d_scales, "scales"));
    WQ_TRY(check_dev(d_y, "y"));
    if (act_order) WQ_TRY(check_dev(d_k_perm, "k_perm"));
    hipStream_t s = (hipStream_t)stream;
    const bool bf16 = act_dtype == WQ_BF16;
    const int groups = (wbits == 4 && group_size == 128) ? K / 128 : 1;
    if (need == 0) {  // 1..4 rows: one kernel, no workspace
        wq::launch_dense_decode(wbits, bf16, static_cast<const uint16_t*>(d_x), M, K, N,
                                static_cast<const uint8_t*>(d_w), static_cast<const uint16_t*>(d_scales), groups,
                                static_cast<uint16_t*>(d_y), s);
        return after_launch(who);
    }
    WQ_TRY(check_ptr(d_ws, "workspace"));
    WQ_TRY(check_dev(d_ws, "workspace"));
    WQ_REQUIRE(reinterpret_cast<uintptr_t>(d_ws) % 256 == 0, WQ_ERR_INVALID, "%s: workspace not 256-byte aligned",
               who);

    const DenseLayout L = dense_layout(M, K, N, act_order);
    WQ_REQUIRE(L.bs == 16 || wq::prefill_fits(L.cap, K), WQ_ERR_UNSUPPORTED,
               "%s: activations of %d rows x %d channels exceed 4 GiB (large-batch kernel)", who, M, K);
    uint8_t* ws = static_cast<uint8_t*>(d_ws);
    int32_t* sorted = reinterpret_cast<int32_t*>(ws + L.off_sorted);
    int32_t* eids = reinterpret_cast<int32_t*>(ws + L.off_eids);
    int32_t* ntpp = reinterpret_cast<int32_t*>(ws + L.off_ntpp);
    float* tw = reinterpret_cast<float*>(ws + L.off_w);
    float* y = reinterpret_cast<float*>(ws + L.off_y);
    wq::launch_identity_route(M, (int)L.cap, L.bs, sorted, eids, ntpp, tw, s);
    WQ_TRY(after_launch(who));

    wq::GemmArgs g{};
    g.a = static_cast<const uint16_t*>(d_x);
    g.w = static_cast<const uint8_t*>(d_w);
    g.s = static_cast<const uint16_t*>(d_scales);
    g.sorted = sorted;
    g.expert_ids = eids;
    g.ntpp = ntpp;
    g.topk_w = tw;
    g.out = y;
    g.M = M;
    g.topk = 1;
    g.E = 1;
    g.n_out = N;
    g.k_in = K;
    g.block_size = L.bs;
    g.groups = groups;
    g.a_direct = 0;  // x row = token of the pair (x has M rows, no pad rows)
    g.cap = (int)L.cap;
    if (act_order) {
        uint16_t* a1 = reinterpret_cast<uint16_t*>(ws + L.off_a1);
        wq::launch_gather_perm(g.a, d_k_perm, sorted, eids, ntpp, M, 1, K, L.bs, g.cap, a1, s);
        WQ_TRY(after_launch(who));
        g.a = a1;
        g.a_direct = 1;
    }
    int ks = 1;
    if (L.bs != 16) ks = wq::launch_gemm_prefill(wbits, bf16, wq::STAGE_DOWN, g, s);
    else wq::launch_gemm_decode(wbits, bf16, wq::STAGE_DOWN, g, s);
    WQ_TRY(after_launch(who));
    wq::launch_combine(y, M, 1, N, ks, bf16, static_cast<uint16_t*>(d_y), s);
    return after_launch(who);
}
}  // namespace

size_t dense_gemm_workspace_bytes(int M, int K, int N, int act_order) {
    if (M < 0 || K <= 0 || N <= 0 || M > MAX_PAIRS) return 0;
    if (M == 0) return 0;
    if (!act_order && wq::dense_decode_supported(M, K)) return 0;  // the single-kernel small-batch path
    return dense_layout(M, K, N, act_order != 0).total;
}

wq_status dense_w4a16_gemm(const void* d_x, int M, int K, int N, const void* d_w_packed, const void* d_scales,
                           int group_size, const int32_t* d_k_perm, void* d_y, int act_dtype, void* d_workspace,
                           size_t workspace_bytes, void* stream) {
    try {
        return dense_gemm(4, d_x, M, K, N, d_w_packed, d_scales, group_size, d_k_perm, d_y, act_dtype, d_workspace,
                          workspace_bytes, stream, "dense_w4a16_gemm");
    } catch (...) {
        return fail(WQ_ERR_HIP, "dense_w4a16_gemm: unexpected exception");
    }
}

wq_status dense_w8a16_gemm(const void* d_x, int M, int K, int N, const void* d_w_packed, const void* d_scales,
                           void* d_y, int act_dtype, void* d_workspace, size_t workspace_bytes, void* stream) {
    try {
        return dense_gemm(8, d_x, M, K, N, d_w_packed, d_scales, -1, nullptr, d_y, act_dtype, d_workspace,
                          workspace_bytes, stream, "dense_w8a16_gemm");
    } catch (...) {
        return fail(WQ_ERR_HIP, "dense_w8a16_gemm: unexpected exception");
    }
}

// ---------------------------------------------------------------------------
static const char* lora_sizes(int M, int K, int N, int R, int adapters) {
    if (M < 0 || K <= 0 || N <= 0 || R <= 0 || adapters <= 0) return "sizes must be positive (M >= 0)";
    if (M > MAX_PAIRS || K > (1 << 24) || N > (1 << 24) || R > 256) return "M, K or N > 2^24, or rank > 256";
    if (K % 8 || N % 8 || R % 8) return "K, N and the rank must be multiples of 8";
    if ((int64_t)N * R > INT32_MAX) return "N * rank >= 2^31";
    return nullptr;
}

size_t dense_lora_workspace_bytes(int M, int K, int N, int R, int adapters) {
    if (M == 0 || lora_sizes(M, K, N, R, adapters)) return 0;
    return round256((size_t)wq::lora_k_slices(M, K, N, R) * M * R * sizeof(float));
}

wq_status dense_lora_gemm(const void* d_x, int64_t x_stride, int M, int K, int N, int R, int adapters,
                          const int32_t* d_adapter_ids, const void* d_a, const void* d_b, const float* d_scales,
                          void* d_y, int64_t y_stride, int act_dtype, void* d_workspace, size_t workspace_bytes,
                          void* stream) {
    try {
        const char* who = "dense_lora_gemm";
        WQ_REQUIRE(act_dtype == WQ_F16 || act_dtype == WQ_BF16, WQ_ERR_INVALID, "%s: bad act dtype", who);
        WQ_REQUIRE(M >= 0 && K > 0 && N > 0 && R > 0 && adapters > 0, WQ_ERR_INVALID,
                   "%s: bad sizes M %d K %d N %d rank %d adapters %d", who, M, K, N, R, adapters);
        const char* bad = lora_sizes(M, K, N, R, adapters);
        WQ_REQUIRE(!bad, WQ_ERR_UNSUPPORTED, "%s: %s", who, bad);
        if (M == 0) return ok();
        const int64_t most = INT64_MAX / 4 / M;
        WQ_REQUIRE(x_stride >= K && x_stride <= most, WQ_ERR_INVALID, "%s: x row stride %lld (K %d)", who,
                   (long long)x_stride, K);
        WQ_REQUIRE(y_stride >= N && y_stride <= most, WQ_ERR_INVALID, "%s: y row stride %lld (N %d)", who,
                   (long long)y_stride, N);
        WQ_REQUIRE(y_stride <= (1 << 25), WQ_ERR_UNSUPPORTED, "%s: y row stride %lld > 2^25", who,
                   (long long)y_stride);
        WQ_REQUIRE(x_stride % 8 == 0 && y_stride % 8 == 0, WQ_ERR_UNSUPPORTED,
                   "%s: row strides must be multiples of 8 (%lld, %lld)", who, (long long)x_stride,
                   (long long)y_stride);
        const size_t need = dense_lora_workspace_bytes(M, K, N, R, adapters);
        WQ_REQUIRE(workspace_bytes >= need, WQ_ERR_INVALID, "%s: workspace %zu < required %zu", who, workspace_bytes,
                   need);
        struct Flat {
            const void* p;
            size_t bytes;
            const char* name;
        };
        const Flat flat[5] = {{d_adapter_ids, (size_t)M * 4, "adapter_ids"},
                              {d_a, (size_t)adapters * R * K * 2, "a"},
                              {d_b, (size_t)adapters * N * R * 2, "b"},
                              {d_scales, (size_t)adapters * 4, "scales"},
                              {d_workspace, need, "workspace"}};
        WQ_TRY(check_ptr(d_x, "x"));
        WQ_TRY(check_ptr(d_y, "y"));
        for (const Flat& f : flat)
            if (f.p || &f != &flat[3]) WQ_TRY(check_ptr(f.p, f.name));
        WQ_REQUIRE(!rows_overlap(d_x, x_stride * 2, (int64_t)K * 2, d_y, y_stride * 2, (int64_t)N * 2, M),
                   WQ_ERR_INVALID, "%s: y overlaps x", who);
        const int64_t x_span = ((M - 1) * x_stride + K) * 2, y_span = ((M - 1) * y_stride + N) * 2;
        for (const Flat& f : flat)
            WQ_REQUIRE(!f.p || !rows_overlap(d_y, 0, y_span, f.p, 0, (int64_t)f.bytes, 1), WQ_ERR_INVALID,
                       "%s: y overlaps %s", who, f.name);
        for (int i = 0; i < 4; ++i)
            WQ_REQUIRE(!flat[i].p || !rows_overlap(d_workspace, 0, (int64_t)need, flat[i].p, 0,
                                                   (int64_t)flat[i].bytes, 1),
                       WQ_ERR_INVALID, "%s: the workspace overlaps %s", who, flat[i].name);
        WQ_REQUIRE(!rows_overlap(d_workspace, 0, (int64_t)need, d_x, 0, x_span, 1), WQ_ERR_INVALID,
                   "%s: the workspace overlaps x", who);
        int cur = -1;
        WQ_TRY(current_device(&cur));
        WQ_TRY(check_dev(d_x, "x", cur));
        WQ_TRY(check_dev(d_y, "y", cur));
        for (const Flat& f : flat)
            if (f.p) WQ_TRY(check_dev(f.p, f.name, cur));
        wq::LoraArgs g{};
        g.x = static_cast<const uint16_t*>(d_x);
        g.ids = d_adapter_ids;
        g.a = static_cast<const uint16_t*>(d_a);
        g.b = static_cast<const uint16_t*>(d_b);
        g.scales = d_scales;
        g.y = static_cast<uint16_t*>(d_y);
        g.t = static_cast<float*>(d_workspace);
        g.x_stride = x_stride;
        g.y_stride = y_stride;
        g.M = M;
        g.K = K;
        g.N = N;
        g.R = R;
        g.adapters = adapters;
        g.ks = wq::lora_k_slices(M, K, N, R);
        wq::launch_lora(g, act_dtype == WQ_BF16, (hipStream_t)stream);
        return after_launch(who);
    } catch (...) {
        return fail(WQ_ERR_HIP, "dense_lora_gemm: unexpected exception");
    }
}

// ---------------------------------------------------------------------------
// paged key-value cache
// ---------------------------------------------------------------------------
namespace {
struct Span8 {  // a contiguous array
    const void* p;
    int64_t bytes;
    const char* name;
};

struct KvCacheView {
    int mode;
    Span8 arrays[4];  // k, v, k_scales, v_scales (the last two NULL without row scales)
};

// the descriptor's checks that need no device
wq_status kv_cache_args(const wq_kv_cache* c, int act_dtype, KvCacheView* out, const char* who) {
    WQ_REQUIRE(c != nullptr, WQ_ERR_INVALID, "%s: cache is NULL", who);
    WQ_REQUIRE(c->struct_size == sizeof(wq_kv_cache), WQ_ERR_INVALID, "%s: cache struct_size %zu, expected %zu", who,
               c->struct_size, sizeof(wq_kv_cache));
    WQ_REQUIRE(act_dtype == WQ_F16 || act_dtype == WQ_BF16, WQ_ERR_INVALID, "%s: bad act dtype", who);
    WQ_REQUIRE(c->dtype == WQ_E4M3 || c->dtype == act_dtype, WQ_ERR_INVALID,
               "%s: cache dtype %d: the act dtype or WQ_E4M3", who, c->dtype);
    WQ_REQUIRE(c->pages >= 1 && c->kv_heads >= 1 && c->page_size >= 1 && c->head_dim >= 1, WQ_ERR_INVALID,
               "%s: bad cache sizes: pages %d kv_heads %d page_size %d head_dim %d", who, c->pages, c->kv_heads,
               c->page_size, c->head_dim);
    WQ_REQUIRE(c->page_size % wq::KV_TOKENS == 0 && c->page_size <= 4096, WQ_ERR_UNSUPPORTED,
               "%s: page_size %d: a multiple of 16, at most 4096", who, c->page_size);
    WQ_REQUIRE(c->head_dim % 16 == 0 && c->head_dim <= wq::KV_MAX_DIM, WQ_ERR_UNSUPPORTED,
               "%s: head_dim %d: a multiple of 16, at most 256", who, c->head_dim);
    WQ_REQUIRE((int64_t)c->pages * c->page_size <= INT32_MAX && c->kv_heads <= 65535, WQ_ERR_UNSUPPORTED,
               "%s: pages * page_size >= 2^31, or more than 65535 kv_heads", who);
    const bool e4m3 = c->dtype == WQ_E4M3, rows = e4m3 && (c->d_k_scales || c->d_v_scales);
    WQ_REQUIRE(e4m3 || (!c->d_k_scales && !c->d_v_scales), WQ_ERR_INVALID, "%s: scales of a 16-bit cache", who);
    WQ_REQUIRE(!rows || (c->d_k_scales && c->d_v_scales), WQ_ERR_INVALID,
               "%s: row scales for the keys and the values, or for neither", who);
    auto usable = [](float s) { return s >= 0x1p-100f && s <= 0x1p100f; };
    WQ_REQUIRE(!e4m3 || rows || (usable(c->k_scale) && usable(c->v_scale)), WQ_ERR_INVALID,
               "%s: k_scale and v_scale must be within 2^-100 and 2^100", who);
    const int64_t n = (int64_t)c->pages * c->page_size * c->kv_heads;  // rows: < 2^47
    const int64_t bytes = n * c->head_dim * (e4m3 ? 1 : 2);
    out->mode = !e4m3 ? wq::KV_16 : rows ? wq::KV_E4M3_ROW : wq::KV_E4M3_STATIC;
    out->arrays[0] = {c->d_k, bytes, "cache k"};
    out->arrays[1] = {c->d_v, bytes, "cache v"};
    out->arrays[2] = {rows ? c->d_k_scales : nullptr, n * 4, "cache k_scales"};
    out->arrays[3] = {rows ? c->d_v_scales : nullptr, n * 4, "cache v_scales"};
    for (int i = 0; i < (rows ? 4 : 2); ++i) WQ_TRY(check_ptr(out->arrays[i].p, out->arrays[i].name));
    return WQ_OK;
}

bool spans_overlap(const Span8& a, const Span8& b) {
    return a.p && b.p && rows_overlap(a.p, 0, a.bytes, b.p, 0, b.bytes, 1);
}

// no array of a shares memory with one of b
wq_status apart(const Span8* a, int na, const Span8* b, int nb, const char* who) {
    for (int i = 0; i < na; ++i)
        for (int j = 0; j < nb; ++j)
            WQ_REQUIRE(!spans_overlap(a[i], b[j]), WQ_ERR_INVALID, "%s: %s overlaps %s", who, a[i].name, b[j].name);
    return WQ_OK;
}

wq_status kv_rows(const wq_kv_cache* c, void* d_k, int64_t k_stride, void* d_v, int64_t v_stride,
                  const int64_t* d_slots, int T, int act_dtype, bool write, void* stream, const char* who) {
    KvCacheView view;
    WQ_REQUIRE(T >= 0, WQ_ERR_INVALID, "%s: T = %d", who, T);
    WQ_REQUIRE(T <= MAX_PAIRS, WQ_ERR_UNSUPPORTED, "%s: T = %d > 2^24", who, T);
    WQ_TRY(kv_cache_args(c, act_dtype, &view, who));
    if (T == 0) return ok();  // (empty arrays may have no address)
    const int64_t n = (int64_t)c->kv_heads * c->head_dim, most = INT64_MAX / 4 / T;
    WQ_REQUIRE(k_stride >= n && k_stride <= most && v_stride >= n && v_stride <= most, WQ_ERR_INVALID,
               "%s: row strides %lld, %lld (rows of %lld)", who, (long long)k_stride, (long long)v_stride,
               (long long)n);
    WQ_REQUIRE(k_stride % 8 == 0 && v_stride % 8 == 0, WQ_ERR_UNSUPPORTED, "%s: row strides must be multiples of 8", who);
    WQ_TRY(check_ptr(d_k, "k"));
    WQ_TRY(check_ptr(d_v, "v"));
    WQ_TRY(check_ptr(d_slots, "slots"));
    const Span8 rows[3] = {{d_k, ((int64_t)(T - 1) * k_stride + n) * 2, "k"},
                           {d_v, ((int64_t)(T - 1) * v_stride + n) * 2, "v"},
                           {d_slots, (int64_t)T * 8, "slots"}};
    WQ_TRY(apart(view.arrays, 4, rows, 3, who));
    if (write) {
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < i; ++j)
                WQ_REQUIRE(!spans_overlap(view.arrays[i], view.arrays[j]), WQ_ERR_INVALID, "%s: %s overlaps %s", who,
                           view.arrays[i].name, view.arrays[j].name);
    } else {  // (the rows of k and v may lie in each other's gaps)
        WQ_REQUIRE(!rows_overlap(d_k, k_stride * 2, n * 2, d_v, v_stride * 2, n * 2, T), WQ_ERR_INVALID,
                   "%s: k overlaps v", who);
        WQ_REQUIRE(!spans_overlap(rows[0], rows[2]) && !spans_overlap(rows[1], rows[2]), WQ_ERR_INVALID,
                   "%s: k or v overlaps slots", who);
    }
    int cur = -1;
    WQ_TRY(current_device(&cur));
    for (const Span8& a : view.arrays)
        if (a.p) WQ_TRY(check_dev(a.p, a.name, cur));
    for (const Span8& a : rows) WQ_TRY(check_dev(a.p, a.name, cur));
    wq::KvRowsArgs g{};
    g.k = static_cast<uint8_t*>(c->d_k);
    g.v = static_cast<uint8_t*>(c->d_v);
    g.ks = c->d_k_scales;
    g.vs = c->d_v_scales;
    g.k_scale = c->k_scale;
    g.v_scale = c->v_scale;
    g.k16 = static_cast<uint16_t*>(d_k);
    g.v16 = static_cast<uint16_t*>(d_v);
    g.slots = d_slots;
    g.k_stride = k_stride;
    g.v_stride = v_stride;
    g.T = T;
    g.pages = c->pages;
    g.kv_heads = c->kv_heads;
    g.page_size = c->page_size;
    g.D = c->head_dim;
    g.mode = view.mode;
    wq::launch_kv_rows(g, write, act_dtype == WQ_BF16, (hipStream_t)stream);
    return after_launch(who);
}
}  // namespace

wq_status wq_kv_cache_write(const wq_kv_cache* c, const void* d_k, int64_t k_stride, const void* d_v,
                            int64_t v_stride, const int64_t* d_slots, int T, int act_dtype, void* stream) {
    try {
        return kv_rows(c, const_cast<void*>(d_k), k_stride, const_cast<void*>(d_v), v_stride, d_slots, T, act_dtype,
                       true, stream, "wq_kv_cache_write");
    } catch (...) {
        return fail(WQ_ERR_HIP, "wq_kv_cache_write: unexpected exception");
    }
}

wq_status wq_kv_cache_read(const wq_kv_cache* c, const int64_t* d_slots, int T, void* d_k, int64_t k_stride,
                           void* d_v, int64_t v_stride, int act_dtype, void* stream) {
    try {
        return kv_rows(c, d_k, k_stride, d_v, v_stride, d_slots, T, act_dtype, false, stream, "wq_kv_cache_read");
    } catch (...) {
        return fail(WQ_ERR_HIP, "wq_kv_cache_read: unexpected exception");
    }
}

// ---------------------------------------------------------------------------
static const char* attn_sizes(int B, int heads, int kv_heads, int head_dim, int page_size, int table_width, int window) {
    if (B < 0 || heads <= 0 || kv_heads <= 0 || head_dim <= 0 || page_size <= 0 || table_width <= 0 || window < 0)
        return "sizes must be positive (B, window >= 0)";
    if (heads % kv_heads) return "heads must be a multiple of kv_heads";
    return nullptr;
}
static const char* attn_limits(int B, int heads, int kv_heads, int page_size, int table_width) {
    const int64_t tokens = (int64_t)table_width * page_size, tiles = tokens / 32 + 2, p16 = page_size / 16;
    if (B > 65535) return "more than 65535 sequences";
    if (heads > 65535) return "more than 65535 heads";
    if (tokens > (1 << 30)) return "table_width * page_size > 2^30";
    // a token's page from its index by one multiplication, exact below this
    if ((int64_t)table_width * p16 * p16 >= ((int64_t)1 << 32)) return "table_width * (page_size / 16)^2 >= 2^32";
    if (tiles * B > INT32_MAX / 2) return "sequences * table_width * page_size >= 2^35";
    return nullptr;
}
struct AttnLayout {
    int splits;
    size_t off_ml, off_at, total;
};
static AttnLayout attn_layout(int B, int heads, int kv_heads, int head_dim, int page_size, int table_width, int window) {
    int64_t most = (int64_t)table_width * page_size;
    if (window > 0) most = std::min<int64_t>(most, (int64_t)window + wq::KV_TOKENS - 1);  // it begins anywhere in 16
    AttnLayout L{};
    L.splits = wq::paged_attn_splits(B, heads, kv_heads, head_dim, most);
    if (L.splits == 0) return L;
    const size_t n = (size_t)2 * L.splits * heads;  // two pieces a share
    L.off_ml = round256(n * head_dim * sizeof(float));
    L.off_at = L.off_ml + round256(n * 2 * sizeof(float));
    L.total = L.off_at + round256((size_t)L.splits * 2 * sizeof(int32_t));
    return L;
}

size_t wq_paged_attention_workspace_bytes(int B, int heads, int kv_heads, int head_dim, int page_size, int table_width,
                                          int window) {
    if (B == 0 || attn_sizes(B, heads, kv_heads, head_dim, page_size, table_width, window) ||
        attn_limits(B, heads, kv_heads, page_size, table_width))
        return 0;
    return attn_layout(B, heads, kv_heads, head_dim, page_size, table_width, window).total;
}

wq_status wq_paged_attention(const wq_kv_cache* c, const void* d_q, int64_t q_stride, int B, int heads,
                             const int32_t* d_block_table, int table_width, const int32_t* d_lengths, float scale,
                             int window, void* d_out, int64_t out_stride, float* d_lse, int act_dtype,
                             void* d_workspace, size_t workspace_bytes, void* stream) {
    try {
        const char* who = "wq_paged_attention";
        KvCacheView view;
        WQ_TRY(kv_cache_args(c, act_dtype, &view, who));
        const char* bad = attn_sizes(B, heads, c->kv_heads, c->head_dim, c->page_size, table_width, window);
        WQ_REQUIRE(!bad, WQ_ERR_INVALID, "%s: %s", who, bad);
        bad = attn_limits(B, heads, c->kv_heads, c->page_size, table_width);
        WQ_REQUIRE(!bad, WQ_ERR_UNSUPPORTED, "%s: %s", who, bad);
        const bool fixed = view.mode == wq::KV_E4M3_STATIC;
        const float qk_scale = (float)((double)scale * (fixed ? (double)c->k_scale : 1.0) * 1.4426950408889634);
        WQ_REQUIRE(std::isfinite(qk_scale), WQ_ERR_INVALID, "%s: scale (times k_scale) must be finite", who);
        const AttnLayout L =
            attn_layout(B, heads, c->kv_heads, c->head_dim, c->page_size, table_width, window);
        if (B == 0) return ok();  // (empty arrays may have no address)
        WQ_REQUIRE(workspace_bytes >= L.total, WQ_ERR_INVALID, "%s: workspace %zu < required %zu", who,
                   workspace_bytes, L.total);
        const int64_t n = (int64_t)heads * c->head_dim, most = INT64_MAX / 4 / B;
        WQ_REQUIRE(q_stride >= n && q_stride <= most && out_stride >= n && out_stride <= most, WQ_ERR_INVALID,
                   "%s: row strides %lld, %lld (rows of %lld)", who, (long long)q_stride, (long long)out_stride,
                   (long long)n);
        WQ_REQUIRE(q_stride % 8 == 0 && out_stride % 8 == 0, WQ_ERR_UNSUPPORTED,
                   "%s: row strides must be multiples of 8", who);
        const Span8 in[3] = {{d_q, ((int64_t)(B - 1) * q_stride + n) * 2, "q"},
                             {d_block_table, (int64_t)B * table_width * 4, "block_table"},
                             {d_lengths, (int64_t)B * 4, "lengths"}};
        const Span8 out[3] = {{d_out, ((int64_t)(B - 1) * out_stride + n) * 2, "out"},
                              {d_lse, (int64_t)B * heads * 4, "lse"},
                              {L.total ? d_workspace : nullptr, (int64_t)L.total, "workspace"}};
        for (const Span8& a : in) WQ_TRY(check_ptr(a.p, a.name));
        WQ_TRY(check_ptr(d_out, "out"));
        if (d_lse) WQ_TRY(check_ptr(d_lse, "lse"));
        if (L.total) WQ_TRY(check_ptr(d_workspace, "workspace"));
        // rows of out may lie between q's (two column ranges of one array)
        WQ_REQUIRE(!rows_overlap(d_q, q_stride * 2, n * 2, d_out, out_stride * 2, n * 2, B), WQ_ERR_INVALID,
                   "%s: out overlaps q", who);
        for (int o = 0; o < 3; ++o) {
            for (int i = o == 0 ? 1 : 0; i < 3; ++i)
                WQ_REQUIRE(!spans_overlap(out[o], in[i]), WQ_ERR_INVALID, "%s: %s overlaps %s", who, out[o].name,
                           in[i].name);
            for (int i = 0; i < o; ++i)
                WQ_REQUIRE(!spans_overlap(out[o], out[i]), WQ_ERR_INVALID, "%s: %s overlaps %s", who, out[o].name,
                           out[i].name);
        }
        WQ_TRY(apart(out, 3, view.arrays, 4, who));
        int cur = -1;
        WQ_TRY(current_device(&cur));
        for (const Span8& a : view.arrays)
            if (a.p) WQ_TRY(check_dev(a.p, a.name, cur));
        for (const Span8& a : in) WQ_TRY(check_dev(a.p, a.name, cur));
        for (const Span8& a : out)
            if (a.p) WQ_TRY(check_dev(a.p, a.name, cur));
        uint8_t* ws = static_cast<uint8_t*>(d_workspace);
        wq::PagedAttnArgs g{};
        g.k = static_cast<const uint8_t*>(c->d_k);
        g.v = static_cast<const uint8_t*>(c->d_v);
        g.ks = c->d_k_scales;
        g.vs = c->d_v_scales;
        g.q = static_cast<const uint16_t*>(d_q);
        g.table = d_block_table;
        g.lengths = d_lengths;
        g.out = static_cast<uint16_t*>(d_out);
        g.lse = d_lse;
        if (L.splits) {
            g.part_o = reinterpret_cast<float*>(ws);
            g.part_ml = reinterpret_cast<float*>(ws + L.off_ml);
            g.part_at = reinterpret_cast<int32_t*>(ws + L.off_at);
        }
        g.q_stride = q_stride;
        g.out_stride = out_stride;
        g.qk_scale = qk_scale;
        g.v_scale = fixed ? c->v_scale : 1.0f;
        g.B = B;
        g.heads = heads;
        g.kv_heads = c->kv_heads;
        g.D = c->head_dim;
        g.pages = c->pages;
        g.page_size = c->page_size;
        g.width = table_width;
        g.window = window;
        g.mode = view.mode;
        g.splits = L.splits;
        wq::launch_paged_attention(g, act_dtype == WQ_BF16, (hipStream_t)stream);
        return after_launch(who);
    } catch (...) {
        return fail(WQ_ERR_HIP, "wq_paged_attention: unexpected exception");
    }
}

// ---------------------------------------------------------------------------
// the dense linear layer with an epilogue
// ---------------------------------------------------------------------------
namespace {
struct EpilogueLayout {
    bool split;  // dense_split.hip: one launch
    bool rows;   // otherwise 1..128 rows in one launch
    size_t off_gather, total;
};
EpilogueLayout epilogue_layout(int wbits, int M, int K, int N, bool act_order) {
    EpilogueLayout L{};
    L.split = wq::dense_split_supported(wbits, M, K, N);
    L.rows = !L.split && wq::dense_decode_supported(M, K);
    size_t o = L.split || L.rows ? 0 : round256(wq::dense_large_slab_bytes(M, K, N));
    L.off_gather = o;
    if (act_order) o += round256((size_t)M * K * 2);
    L.total = o;
    return L;
}

const char* epilogue_sizes(int wbits, int M, int K, int N) {
    if (M < 0 || K <= 0 || N <= 0) return "sizes must be positive (M >= 0)";
    if (M > MAX_PAIRS || K > (1 << 24) || N > (1 << 24)) return "M, K or N > 2^24";
    if (K % (wbits == 4 ? wq::WFmt<4>::KCHUNK : wq::WFmt<8>::KCHUNK)) return "K must be a multiple of 128 (int4) or 64 (int8)";
    if (N % 16) return "N must be a multiple of 16";
    if (!wq::dense_split_supported(wbits, M, K, N) && !wq::dense_decode_supported(M, K) && !wq::prefill_fits((size_t)M + 128, K)) return "more than 4 GiB of activations";
    if (M > 65535 * 64) return "more than 65535 * 64 rows";
    return nullptr;
}

wq_status dense_epilogue(int wbits, const void* d_x, int M, int K, int N, const void* d_w, const void* d_scales,
                         int group_size, const int32_t* d_k_perm, const wq_epilogue* e, void* d_y, int act_dtype,
                         void* d_ws, size_t ws_bytes, void* stream, const char* who) {
    WQ_REQUIRE(M >= 0 && K > 0 && N > 0, WQ_ERR_INVALID, "%s: bad sizes M %d K %d N %d", who, M, K, N);
    WQ_REQUIRE(act_dtype == WQ_F16 || act_dtype == WQ_BF16, WQ_ERR_INVALID, "%s: bad act dtype", who);
    if (wbits == 4) WQ_REQUIRE(act_dtype == WQ_F16, WQ_ERR_UNSUPPORTED, "%s: int4 path takes fp16 activations", who);
    const char* bad = epilogue_sizes(wbits, M, K, N);
    WQ_REQUIRE(!bad, WQ_ERR_UNSUPPORTED, "%s: %s", who, bad);
    if (wbits == 4)
        WQ_REQUIRE(group_size == 128 || group_size == -1, WQ_ERR_UNSUPPORTED, "%s: group_size %d", who, group_size);
    WQ_REQUIRE(e != nullptr && e->struct_size == sizeof(wq_epilogue), WQ_ERR_INVALID,
               "%s: epilogue is NULL or of another struct_size", who);
    WQ_REQUIRE(e->activation >= WQ_ACT_NONE && e->activation <= WQ_ACT_GELU_TANH, WQ_ERR_INVALID, "%s: activation %d",
               who, e->activation);
    const bool act_order = d_k_perm != nullptr;
    const EpilogueLayout L = epilogue_layout(wbits, M, K, N, act_order);
    WQ_REQUIRE(ws_bytes >= L.total, WQ_ERR_INVALID, "%s: workspace %zu < required %zu", who, ws_bytes, L.total);
    if (M == 0) return ok();
    const int64_t rs = e->d_residual ? e->residual_stride : N;
    WQ_REQUIRE(rs >= N && rs <= INT64_MAX / 4 / M, WQ_ERR_INVALID, "%s: residual row stride %lld (N %d)", who,
               (long long)rs, N);
    WQ_REQUIRE(rs % 8 == 0, WQ_ERR_UNSUPPORTED, "%s: the residual's row stride must be a multiple of 8", who);
    const int groups = (wbits == 4 && group_size == 128) ? K / 128 : 1;
    const Span8 in[6] = {{d_x, (int64_t)M * K * 2, "x"},
                         {d_w, (int64_t)N * K * wbits / 8, "w_packed"},
                         {d_scales, (int64_t)groups * N * 2, "scales"},
                         {d_k_perm, (int64_t)K * 4, "k_perm"},
                         {e->d_bias, (int64_t)N * 2, "bias"},
                         {e->d_residual, ((int64_t)(M - 1) * rs + N) * 2, "residual"}};
    const Span8 out[2] = {{d_y, (int64_t)M * N * 2, "y"}, {L.total ? d_ws : nullptr, (int64_t)L.total, "workspace"}};
    for (int i = 0; i < 6; ++i)
        if (in[i].p || i < 3) WQ_TRY(check_ptr(in[i].p, in[i].name));
    WQ_TRY(check_ptr(d_y, "y"));
    if (L.total) {
        WQ_TRY(check_ptr(d_ws, "workspace"));
        WQ_REQUIRE(reinterpret_cast<uintptr_t>(d_ws) % 256 == 0, WQ_ERR_INVALID, "%s: workspace not 256-byte aligned",
                   who);
    }
    // y may be the residual
    const bool in_place = e->d_residual == d_y && rs == N;
    WQ_TRY(apart(out, 2, in, 5, who));
    WQ_REQUIRE(in_place || !e->d_residual || !rows_overlap(d_y, (int64_t)N * 2, (int64_t)N * 2, e->d_residual, rs * 2,
                                                           (int64_t)N * 2, M),
               WQ_ERR_INVALID, "%s: y overlaps residual", who);
    WQ_REQUIRE(!spans_overlap(out[1], in[5]) && !spans_overlap(out[0], out[1]), WQ_ERR_INVALID,
               "%s: the workspace overlaps y or residual", who);
    int cur = -1;
    WQ_TRY(current_device(&cur));
    for (const Span8& a : in)
        if (a.p) WQ_TRY(check_dev(a.p, a.name, cur));
    for (const Span8& a : out)
        if (a.p) WQ_TRY(check_dev(a.p, a.name, cur));
    hipStream_t s = (hipStream_t)stream;
    const bool bf16 = act_dtype == WQ_BF16;
    uint8_t* ws = static_cast<uint8_t*>(d_ws);
    const uint16_t* x = static_cast<const uint16_t*>(d_x);
    if (act_order) {
        uint16_t* a1 = reinterpret_cast<uint16_t*>(ws + L.off_gather);
        wq::launch_gather_columns(x, d_k_perm, M, K, a1, s);
        WQ_TRY(after_launch(who));
        x = a1;
    }
    const wq::Epilogue ep{static_cast<const uint16_t*>(e->d_bias),
                          in_place ? nullptr : static_cast<const uint16_t*>(e->d_residual), rs, in_place,
                          e->activation};
    const uint8_t* w = static_cast<const uint8_t*>(d_w);
    const uint16_t* sc = static_cast<const uint16_t*>(d_scales);
    if (L.split) wq::launch_dense_split(wbits, bf16, x, M, K, N, w, sc, groups, static_cast<uint16_t*>(d_y), ep, s);
    else if (L.rows) wq::launch_dense_decode(wbits, bf16, x, M, K, N, w, sc, groups, static_cast<uint16_t*>(d_y), s, &ep);
    else
        wq::launch_dense_large(wbits, bf16, x, M, K, N, w, sc, groups, ep, reinterpret_cast<float*>(ws),
                               static_cast<uint16_t*>(d_y), s);
    return after_launch(who);
}
}  // namespace

size_t dense_epilogue_workspace_bytes(int wbits, int M, int K, int N, int act_order) {
    if ((wbits != 4 && wbits != 8) || M == 0 || epilogue_sizes(wbits, M, K, N)) return 0;
    return epilogue_layout(wbits, M, K, N, act_order != 0).total;
}

wq_status dense_w4a16_epilogue_gemm(const void* d_x, int M, int K, int N, const void* d_w_packed, const void* d_scales,
                                    int group_size, const int32_t* d_k_perm, const wq_epilogue* epilogue, void* d_y,
                                    int act_dtype, void* d_workspace, size_t workspace_bytes, void* stream) {
    try {
        return dense_epilogue(4, d_x, M, K, N, d_w_packed, d_scales, group_size, d_k_perm, epilogue, d_y, act_dtype,
                              d_workspace, workspace_bytes, stream, "dense_w4a16_epilogue_gemm");
    } catch (...) {
        return fail(WQ_ERR_HIP, "dense_w4a16_epilogue_gemm: unexpected exception");
    }
}

wq_status dense_w8a16_epilogue_gemm(const void* d_x, int M, int K, int N, const void* d_w_packed, const void* d_scales,
                                    const wq_epilogue* epilogue, void* d_y, int act_dtype, void* d_workspace,
                                    size_t workspace_bytes, void* stream) {
    try {
        return dense_epilogue(8, d_x, M, K, N, d_w_packed, d_scales, -1, nullptr, epilogue, d_y, act_dtype,
                              d_workspace, workspace_bytes, stream, "dense_w8a16_epilogue_gemm");
    } catch (...) {
        return fail(WQ_ERR_HIP, "dense_w8a16_epilogue_gemm: unexpected exception");
    }
}

// ---------------------------------------------------------------------------
wq_status wq_quantize_w8(const void* d_w, int64_t rows, int k, int dtype, int8_t* d_q, uint16_t* d_scales,
                         void* stream) {
    try {
        WQ_REQUIRE(rows >= 0 && k > 0, WQ_ERR_INVALID, "quantize_w8: bad sizes rows %lld k %d", (long long)rows, k);
        WQ_REQUIRE(dtype == WQ_F16 || dtype == WQ_BF16, WQ_ERR_INVALID, "quantize_w8: bad dtype %d", dtype);
        WQ_REQUIRE(k % 8 == 0, WQ_ERR_UNSUPPORTED, "quantize_w8: k %d not a multiple of 8", k);
        WQ_REQUIRE((rows + 3) / 4 <= 0x7fffffffLL, WQ_ERR_UNSUPPORTED, "quantize_w8: too many rows");
        if (rows == 0) return ok();
        WQ_TRY(check_ptr(d_w, "w"));
        WQ_TRY(check_ptr(d_q, "q"));
        WQ_TRY(check_ptr(d_scales, "scales"));
        WQ_TRY(check_dev(d_w, "w"));
        WQ_TRY(check_dev(d_q, "q"));
        WQ_TRY(check_dev(d_scales, "scales"));
        WQ_REQUIRE(reinterpret_cast<uintptr_t>(d_w) % 16 == 0 && reinterpret_cast<uintptr_t>(d_q) % 8 == 0,
                   WQ_ERR_INVALID, "quantize_w8: w must be 16-byte and q 8-byte aligned");
        wq::launch_quant_w8(static_cast<const uint16_t*>(d_w), rows, k, dtype == WQ_BF16, d_q, d_scales,
                            (hipStream_t)stream);
        return after_launch("wq_quantize_w8");
    } catch (...) {
        return fail(WQ_ERR_HIP, "quantize_w8: unexpected exception");
    }
}

// ---------------------------------------------------------------------------
// Offline packers
// ---------------------------------------------------------------------------
size_t wq_pack_w4_bytes(int E, int n_out, int k_in) {
    if (E <= 0 || n_out <= 0 || k_in <= 0 || n_out % 16 || k_in % 128) return 0;
    return (size_t)E * n_out * k_in / 2;
}

size_t wq_pack_w8_bytes(int E, int n_out, int k_in) {
    if (E <= 0 || n_out <= 0 || k_in <= 0 || n_out % 16 || k_in % 64) return 0;
    return (size_t)E * n_out * k_in;
}

// canonical row held by packed row p of expert e
static inline int logical_row(int p, int n_out, bool interleave, const int32_t* perm_e) {
    if (!interleave) return perm_e ? perm_e[p] : p;
    const int t = p / 16, j = t / 2, half = t % 2, within = p % 16;
    int lr = 16 * j + within;
    if (perm_e) lr = perm_e[lr];
    return half * (n_out / 2) + lr;
}

static wq_status check_row_perm(int E, int n, const int32_t* perm) {
    if (!perm) return WQ_OK;
    std::vector<char> seen((size_t)n);
    for (int e = 0; e < E; ++e) {
        std::fill(seen.begin(), seen.end(), 0);
        for (int i = 0; i < n; ++i) {
            const int32_t v = perm[(size_t)e * n + i];
            WQ_REQUIRE(v >= 0 && v < n && !seen[v], WQ_ERR_INVALID, "row_perm of expert %d is not a permutation", e);
            seen[v] = 1;
        }
    }
    return WQ_OK;
}

wq_status wq_pack_w4(int E, int n_out, int k_in, const int8_t* q, const uint16_t* scales, int group_size,
                     const int32_t* g_idx, const int32_t* row_perm, int flags, void* packed, uint16_t* scales_packed,
                     int32_t* k_perm) {
    try {
        WQ_REQUIRE(E > 0 && n_out > 0 && k_in > 0, WQ_ERR_INVALID, "pack_w4: bad sizes");
        const bool il = (flags & WQ_PACK_INTERLEAVE_GATE_UP) != 0;
        WQ_REQUIRE(n_out % (il ? 32 : 16) == 0, WQ_ERR_UNSUPPORTED, "pack_w4: n_out %d", n_out);
        WQ_REQUIRE(k_in % 128 == 0, WQ_ERR_UNSUPPORTED, "pack_w4: k_in %d not a multiple of 128", k_in);
        WQ_REQUIRE(group_size == 128 || group_size == -1, WQ_ERR_UNSUPPORTED, "pack_w4: group_size %d", group_size);
        WQ_REQUIRE(q && scales && packed && scales_packed, WQ_ERR_INVALID, "pack_w4: NULL buffer");
        WQ_REQUIRE(!g_idx || (group_size == 128 && k_perm), WQ_ERR_INVALID,
                   "pack_w4: act-order needs group_size 128 and a k_perm output");
        const int G = group_size == -1 ? 1 : k_in / group_size;
        WQ_TRY(check_row_perm(E, il ? n_out / 2 : n_out, row_perm));
        const int rows_perm = il ? n_out / 2 : n_out;
        // input-channel order: stable sort by group
        std::vector<int32_t> sig((size_t)E * k_in);
        for (int e = 0; e < E; ++e) {
            int32_t* s = sig.data() + (size_t)e * k_in;
            if (!g_idx) {
                for (int k = 0; k < k_in; ++k) s[k] = k;
                continue;
            }
            const int32_t* gi = g_idx + (size_t)e * k_in;
            std::vector<int> cnt(G, 0);
            for (int k = 0; k < k_in; ++k) {
                WQ_REQUIRE(gi[k] >= 0 && gi[k] < G, WQ_ERR_INVALID, "pack_w4: g_idx out of range (expert %d)", e);
                cnt[gi[k]]++;
            }
            for (int gg = 0; gg < G; ++gg)
                WQ_REQUIRE(cnt[gg] == group_size, WQ_ERR_UNSUPPORTED,
                           "pack_w4: act-order group %d of expert %d has %d channels, not %d", gg, e, cnt[gg],
                           group_size);
            std::vector<int> pos(G);
            for (int gg = 0; gg < G; ++gg) pos[gg] = gg * group_size;
            for (int k = 0; k < k_in; ++k) s[pos[gi[k]]++] = k;
        }
        // value range
        for (size_t i = 0, n = (size_t)E * n_out * k_in; i < n; ++i)
            WQ_REQUIRE(q[i] >= -8 && q[i] <= 7, WQ_ERR_INVALID, "pack_w4: code %d out of [-8, 7]", (int)q[i]);
        if (k_perm) std::memcpy(k_perm, sig.data(), sizeof(int32_t) * sig.size());

        const int C = k_in / 128;
        const size_t expert_bytes = (size_t)n_out * k_in / 2;
        uint8_t* out = static_cast<uint8_t*>(packed);
        parallel_for(E * (n_out / 16), [&](int job) {
            const int e = job / (n_out / 16), t = job % (n_out / 16);
            const int32_t* pe = row_perm ? row_perm + (size_t)e * rows_perm : nullptr;
            const int32_t* s = sig.data() + (size_t)e * k_in;
            for (int l = 0; l < 64; ++l) {
                const int p = t * 16 + (l & 15);
                const int lr = logical_row(p, n_out, il, pe);
                const int8_t* qr = q + ((size_t)e * n_out + lr) * k_in;
                for (int c = 0; c < C; ++c) {
                    uint32_t* dst = reinterpret_cast<uint32_t*>(out + (size_t)e * expert_bytes +
                                                                (((size_t)t * C + c) * 64 + l) * 16);
                    for (int st = 0; st < 4; ++st) {
                        uint32_t d = 0;
                        for (int j = 0; j < 8; ++j) {
                            const int kp = 128 * c + 32 * st + 8 * (l >> 4) + j;
                            const uint32_t u = (uint32_t)(qr[s[kp]] + 8);
                            d |= u << (4 * (j >> 1) + 16 * (j & 1));
                        }
                        dst[st] = d;
                    }
                }
            }
            if (t == 0) {
                for (int gg = 0; gg < G; ++gg)
                    for (int pp = 0; pp < n_out; ++pp)
                        scales_packed[((size_t)e * G + gg) * n_out + pp] =
                            scales[((size_t)e * G + gg) * n_out + logical_row(pp, n_out, il, pe)];
            }
        });
        return ok();
    } catch (...) {
        return fail(WQ_ERR_INVALID, "pack_w4: unexpected exception");
    }
}

wq_status wq_pack_w8(int E, int n_out, int k_in, const int8_t* q, const uint16_t* scales, const int32_t* row_perm,
                     int flags, void* packed, uint16_t* scales_packed) {
    try {
        WQ_REQUIRE(E > 0 && n_out > 0 && k_in > 0, WQ_ERR_INVALID, "pack_w8: bad sizes");
        const bool il = (flags & WQ_PACK_INTERLEAVE_GATE_UP) != 0;
        WQ_REQUIRE(n_out % (il ? 32 : 16) == 0, WQ_ERR_UNSUPPORTED, "pack_w8: n_out %d", n_out);
        WQ_REQUIRE(k_in % 64 == 0, WQ_ERR_UNSUPPORTED, "pack_w8: k_in %d not a multiple of 64", k_in);
        WQ_REQUIRE(q && scales && packed && scales_packed, WQ_ERR_INVALID, "pack_w8: NULL buffer");
        const int rows_perm = il ? n_out / 2 : n_out;
        WQ_TRY(check_row_perm(E, rows_perm, row_perm));
        const int C = k_in / 64;
        const size_t expert_bytes = (size_t)n_out * k_in;
        uint8_t* out = static_cast<uint8_t*>(packed);
        parallel_for(E * (n_out / 16), [&](int job) {
            const int e = job / (n_out / 16), t = job % (n_out / 16);
            const int32_t* pe = row_perm ? row_perm + (size_t)e * rows_perm : nullptr;
            for (int l = 0; l < 64; ++l) {
                const int p = t * 16 + (l & 15);
                const int lr = logical_row(p, n_out, il, pe);
                const int8_t* qr = q + ((size_t)e * n_out + lr) * k_in;
                for (int c = 0; c < C; ++c) {
                    uint8_t* dst = out + (size_t)e * expert_bytes + (((size_t)t * C + c) * 64 + l) * 16;
                    for (int st = 0; st < 2; ++st)
                        for (int j = 0; j < 8; ++j)
                            dst[8 * st + j] = (uint8_t)qr[64 * c + 32 * st + 8 * (l >> 4) + j];
                }
            }
            if (t == 0)
                for (int pp = 0; pp < n_out; ++pp)
                    scales_packed[(size_t)e * n_out + pp] = scales[(size_t)e * n_out + logical_row(pp, n_out, il, pe)];
        });
        return ok();
    } catch (...) {
        return fail(WQ_ERR_INVALID, "pack_w8: unexpected exception");
    }
}

size_t wq_pack_fp8_bytes(int E, int n_out, int k_in) {
    if (E <= 0 || n_out <= 0 || k_in <= 0 || n_out % 16 || k_in % wq::FP8_KCHUNK) return 0;
    return (size_t)E * n_out * k_in;
}

// E4M3 codes: tiles of 16 rows x 128 channels (2 KiB).  Lane l's MFMA operand
// is row l % 16, channels [32 (l / 16), +32) of the chunk; its first 16
// channels sit at bytes 16 l of the chunk and the other 16 at 1024 + 16 l, so
// each of a wave's two 128-bit loads reads one contiguous KiB
wq_status wq_pack_fp8(int E, int n_out, int k_in, const uint8_t* codes, const float* scales, const int32_t* row_perm,
                      int flags, void* packed, float* scales_packed) {
    try {
        WQ_REQUIRE(E > 0 && n_out > 0 && k_in > 0, WQ_ERR_INVALID, "pack_fp8: bad sizes");
        const bool il = (flags & WQ_PACK_INTERLEAVE_GATE_UP) != 0;
        WQ_REQUIRE(n_out % (il ? 32 : 16) == 0, WQ_ERR_UNSUPPORTED, "pack_fp8: n_out %d", n_out);
        WQ_REQUIRE(k_in % wq::FP8_KCHUNK == 0, WQ_ERR_UNSUPPORTED, "pack_fp8: k_in %d not a multiple of %d", k_in,
                   wq::FP8_KCHUNK);
        WQ_REQUIRE(codes && scales && packed && scales_packed, WQ_ERR_INVALID, "pack_fp8: NULL buffer");
        for (size_t i = 0, n = (size_t)E * n_out * k_in; i < n; ++i)
            WQ_REQUIRE((codes[i] & 0x7f) != 0x7f, WQ_ERR_INVALID, "pack_fp8: NaN code at %zu", i);
        for (size_t i = 0, n = (size_t)E * n_out; i < n; ++i)
            WQ_REQUIRE(std::isfinite(scales[i]), WQ_ERR_INVALID, "pack_fp8: non-finite scale at %zu", i);
        const int rows_perm = il ? n_out / 2 : n_out;
        WQ_TRY(check_row_perm(E, rows_perm, row_perm));
        const int C = k_in / wq::FP8_KCHUNK;
        const size_t expert_bytes = (size_t)n_out * k_in;
        uint8_t* out = static_cast<uint8_t*>(packed);
        parallel_for(E * (n_out / 16), [&](int job) {
            const int e = job / (n_out / 16), t = job % (n_out / 16);
            const int32_t* pe = row_perm ? row_perm + (size_t)e * rows_perm : nullptr;
            for (int l = 0; l < 64; ++l) {
                const int p = t * 16 + (l & 15);
                const uint8_t* qr = codes + ((size_t)e * n_out + logical_row(p, n_out, il, pe)) * k_in;
                for (int c = 0; c < C; ++c)
                    for (int h = 0; h < 2; ++h)
                        std::memcpy(out + (size_t)e * expert_bytes + ((size_t)t * C + c) * 2048 + 1024 * h + 16 * l,
                                    qr + (size_t)wq::FP8_KCHUNK * c + 32 * (l >> 4) + 16 * h, 16);
            }
            if (t == 0)
                for (int pp = 0; pp < n_out; ++pp)
                    scales_packed[(size_t)e * n_out + pp] = scales[(size_t)e * n_out + logical_row(pp, n_out, il, pe)];
        });
        return ok();
    } catch (...) {
        return fail(WQ_ERR_INVALID, "pack_fp8: unexpected exception");
    }
}

size_t wq_pack_sparse24_vals_bytes(int N, int K, int bits) {
    if (N <= 0 || K <= 0 || N % 16 || K % 256 || (bits != 4 && bits != 8)) return 0;
    return (size_t)N * K / 2 * bits / 8;
}

size_t wq_pack_sparse24_meta_bytes(int N, int K) {
    if (N <= 0 || K <= 0 || N % 16 || K % 256) return 0;
    return (size_t)N * K / 8;
}

wq_status wq_pack_sparse24(int N, int K, int bits, int group_size, const int8_t* vals, const uint8_t* idx,
                           const uint16_t* scales, void* vals_packed, void* meta_packed, uint16_t* scales_packed) {
    try {
        WQ_REQUIRE(N > 0 && K > 0, WQ_ERR_INVALID, "pack_sparse24: bad sizes");
        WQ_REQUIRE(bits == 4 || bits == 8, WQ_ERR_UNSUPPORTED, "pack_sparse24: bits %d (4 or 8)", bits);
        WQ_REQUIRE(group_size == 128 || group_size == -1, WQ_ERR_UNSUPPORTED, "pack_sparse24: group_size %d",
                   group_size);
        WQ_REQUIRE(N % 16 == 0 && K % 256 == 0, WQ_ERR_UNSUPPORTED, "pack_sparse24: need N %% 16 == 0, K %% 256 == 0");
        WQ_REQUIRE(vals && idx && scales && vals_packed && meta_packed && scales_packed, WQ_ERR_INVALID,
                   "pack_sparse24: NULL buffer");
        const size_t half = (size_t)N * K / 2;
        for (size_t i = 0; i < half; i += 2) {
            WQ_REQUIRE(bits == 8 || (vals[i] >= -8 && vals[i] <= 7 && vals[i + 1] >= -8 && vals[i + 1] <= 7),
                       WQ_ERR_INVALID, "pack_sparse24: code out of [-8, 7]");
            WQ_REQUIRE(idx[i] < idx[i + 1] && idx[i + 1] <= 3, WQ_ERR_INVALID,
                       "pack_sparse24: keep positions must be ascending in 0..3");
        }
        const int C = K / 256;
        uint8_t* vo = static_cast<uint8_t*>(vals_packed);
        uint8_t* mo = static_cast<uint8_t*>(meta_packed);
        parallel_for(N / 16, [&](int t) {
            for (int l = 0; l < 64; ++l) {
                const int n = t * 16 + (l & 15);
                const int8_t* vr = vals + (size_t)n * (K / 2);
                const uint8_t* ir = idx + (size_t)n * (K / 2);
                for (int c = 0; c < C; ++c) {
                    // lane l's values: 16 bytes (4-bit) or 32 bytes (8-bit) per chunk
                    uint8_t* vd = vo + (((size_t)t * C + c) * 64 + l) * (size_t)(4 * bits);
                    uint16_t* md = reinterpret_cast<uint16_t*>(mo + (((size_t)t * C + c) * 64 + l) * 8);
                    for (int st = 0; st < 4; ++st) {
                        const int g4 = (256 * c + 64 * st + 16 * (l >> 4)) / 4;  // first group of 4 of this lane
                        uint32_t d = 0;
                        uint32_t m = 0;
                        for (int b = 0; b < 4; ++b) {
                            for (int h = 0; h < 2; ++h) {
                                const int j = 2 * b + h;
                                const size_t v = (size_t)2 * (g4 + b) + h;
                                if (bits == 4) d |= (uint32_t)(vr[v] + 8) << (4 * (j >> 1) + 16 * (j & 1));
                                else vd[8 * st + j] = (uint8_t)vr[v];  // two's complement, natural order
                                m |= (uint32_t)ir[v] << (4 * b + 2 * h);
                            }
                        }
                        if (bits == 4) std::memcpy(vd + 4 * st, &d, 4);
                        md[st] = (uint16_t)m;
                    }
                }
            }
        });
        std::memcpy(scales_packed, scales, sizeof(uint16_t) * (size_t)(group_size == -1 ? 1 : K / 128) * N);
        return ok();
    } catch (...) {
        return fail(WQ_ERR_INVALID, "pack_sparse24: unexpected exception");
    }
}

}  // extern "C"
