// libmoe C ABI: host-side argument checks, then kernel launches on the
// caller's stream.  No call allocates memory or synchronises; invalid
// arguments return a negative status before anything is enqueued.
#include <stdio.h>
#include <string.h>

#include "internal.h"
#include "../../include/moe_probe.h"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace moe {
namespace {
thread_local char g_last_error[256] = "";
}

int fail(int status, const char* msg) {
    snprintf(g_last_error, sizeof g_last_error, "%s", msg);
    return status;
}

int hip_status(hipError_t e, const char* where) {
    if (e == hipSuccess) return MOE_OK;
    snprintf(g_last_error, sizeof g_last_error, "%s: %s", where, hipGetErrorString(e));
    return MOE_EHIP;
}

const char* last_error() { return g_last_error; }

}  // namespace moe

using moe::fail;
using moe::hip_status;

namespace {

int check_sizes(int B, int N, int k) {
    if (N < 1 || N > moe::kMaxExperts) return fail(MOE_EINVAL, "N must be in [1, 128]");
    if (k < 1 || k > N || k > moe::kMaxTopK) return fail(MOE_EINVAL, "k must be in [1, min(N, 16)]");
    if (B < 1) return fail(MOE_EINVAL, "B must be >= 1");
    if (B > moe::kMaxBatch) return fail(MOE_EUNSUPPORTED, "B > 128 is not supported");
    return MOE_OK;
}

hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

}  // namespace

MOE_API const char* moe_status_str(int status) {
    switch (status) {
        case MOE_OK: return "ok";
        case MOE_EINVAL: return "invalid argument";
        case MOE_EUNSUPPORTED: return "unsupported size";
        case MOE_EHIP: return "HIP runtime error";
        case MOE_EFULL: return "no free block (retry later)";
        default: return "unknown status";
    }
}

MOE_API const char* moe_last_error(void) { return moe::last_error(); }

MOE_API int moe_router_logits(const void* x, int x_dtype, const float* w_r, int B, int H, int N,
                              float* logits, void* stream) {
    if (!x || !w_r || !logits) return fail(MOE_EINVAL, "null pointer");
    if (x_dtype != MOE_DT_F32 && x_dtype != MOE_DT_BF16) return fail(MOE_EINVAL, "bad x_dtype");
    if (N < 1 || N > moe::kMaxExperts) return fail(MOE_EINVAL, "N must be in [1, 128]");
    if (B < 1) return fail(MOE_EINVAL, "B must be >= 1");
    if (B > moe::kMaxBatch) return fail(MOE_EUNSUPPORTED, "B > 128 is not supported");
    if (H < 8 || H % 8) return fail(MOE_EINVAL, "H must be a positive multiple of 8");
    return hip_status(moe::launch_router_logits(x, x_dtype, w_r, B, H, N, logits, as_stream(stream)),
                      "moe_router_logits");
}

MOE_API int moe_route_topk(const float* logits, int B, int N, int k, int renorm, int32_t* idx,
                           float* w, void* stream) {
    if (!logits || !idx || !w) return fail(MOE_EINVAL, "null pointer");
    int st = check_sizes(B, N, k);
    if (st) return st;
    return hip_status(moe::launch_route(logits, B, N, k, k, 1.0f, 0, renorm ? 1 : 0, idx, w,
                                        nullptr, nullptr, nullptr, as_stream(stream)),
                      "moe_route_topk");
}

MOE_API int moe_route_oea(const float* logits, int B, int N, int k0, float p, int k, int32_t* idx,
                          float* w, int32_t* n_base, uint32_t* sbase_mask, int32_t* T,
                          void* stream) {
    if (!logits || !idx || !w) return fail(MOE_EINVAL, "null pointer");
    int st = check_sizes(B, N, k);
    if (st) return st;
    if (k0 < 1 || k0 > k) return fail(MOE_EINVAL, "k0 must be in [1, k]");
    if (!(p > 0.0f)) return fail(MOE_EINVAL, "p must be > 0 (p >= 1 disables top-p)");
    return hip_status(moe::launch_route(logits, B, N, k, k0, p, 1, 1, idx, w, n_base, sbase_mask, T,
                                        as_stream(stream)),
                      "moe_route_oea");
}

MOE_API int moe_dispatch(const int32_t* idx, int B, int N, int k, int32_t* cnt, int32_t* offsets,
                         int32_t* perm, int32_t* active, int32_t* T, void* stream) {
    if (!idx || !cnt || !offsets || !perm || !active || !T) return fail(MOE_EINVAL, "null pointer");
    int st = check_sizes(B, N, k);
    if (st) return st;
    return hip_status(moe::launch_dispatch(idx, B, N, k, cnt, offsets, perm, active, T,
                                           as_stream(stream)),
                      "moe_dispatch");
}

MOE_API int moe_route_dispatch(const float* logits, int B, int N, int k, int mode, int k0, float p, int max_p,
                               int renorm, const int32_t* n_valid, const int32_t* k0_by_batch, int32_t* idx,
                               float* w, int32_t* n_base,
                               uint32_t* sbase_mask, int32_t* cnt, int32_t* offsets, int32_t* perm,
                               int32_t* active, int32_t* T, int32_t* sync, void* stream) {
    if (!logits || !idx || !w || !cnt || !offsets || !perm || !active || !T) return fail(MOE_EINVAL, "null pointer");
    int st = check_sizes(B, N, k);
    if (st) return st;
    if (mode != MOE_ROUTE_TOPK && mode != MOE_ROUTE_OEA && mode != MOE_ROUTE_PRUNED)
        return fail(MOE_EINVAL, "bad routing mode");
    if (mode != MOE_ROUTE_TOPK) {
        if (k0 < 1 || k0 > k) return fail(MOE_EINVAL, "k0 must be in [1, k]");
        if (!(p > 0.0f)) return fail(MOE_EINVAL, "p must be > 0 (p >= 1 disables top-p)");
        if (mode == MOE_ROUTE_OEA && (max_p < k0 || max_p > N)) return fail(MOE_EINVAL, "max_p must be in [k0, N]");
    }
    const bool oea_like = mode != MOE_ROUTE_TOPK;
    return hip_status(moe::launch_route_dispatch(logits, B, N, k, mode, k0, p, mode == MOE_ROUTE_OEA ? max_p : N,
                                                 renorm, n_valid, oea_like ? k0_by_batch : nullptr, idx, w,
                                                 oea_like ? n_base : nullptr,
                                                 oea_like ? sbase_mask : nullptr, cnt, offsets, perm, active, T,
                                                 sync, as_stream(stream)),
                      "moe_route_dispatch");
}

MOE_API int moe_router_route_dispatch(const void* x, int x_dtype, const float* w_r, int B, int H, int N, int k,
                                      int mode, int k0, float p, int max_p, int renorm, const int32_t* n_valid,
                                      const int32_t* k0_by_batch, float* logits, int32_t* idx, float* w,
                                      int32_t* n_base, uint32_t* sbase_mask, int32_t* cnt, int32_t* offsets,
                                      int32_t* perm, int32_t* active, int32_t* T, int32_t* sync, void* stream) {
    if (!x || !w_r || !logits || !idx || !w || !cnt || !offsets || !perm || !active || !T || !sync)
        return fail(MOE_EINVAL, "null pointer");
    if (x_dtype != MOE_DT_F32 && x_dtype != MOE_DT_BF16) return fail(MOE_EINVAL, "bad x_dtype");
    if (H < 8 || H % 8) return fail(MOE_EINVAL, "H must be a positive multiple of 8");
    int st = check_sizes(B, N, k);
    if (st) return st;
    if (mode != MOE_ROUTE_TOPK && mode != MOE_ROUTE_OEA && mode != MOE_ROUTE_PRUNED)
        return fail(MOE_EINVAL, "bad routing mode");
    if (mode != MOE_ROUTE_TOPK) {
        if (k0 < 1 || k0 > k) return fail(MOE_EINVAL, "k0 must be in [1, k]");
        if (!(p > 0.0f)) return fail(MOE_EINVAL, "p must be > 0 (p >= 1 disables top-p)");
        if (mode == MOE_ROUTE_OEA && (max_p < k0 || max_p > N)) return fail(MOE_EINVAL, "max_p must be in [k0, N]");
    }
    const bool oea_like = mode != MOE_ROUTE_TOPK;
    return hip_status(moe::launch_router_route_dispatch(x, x_dtype, w_r, B, H, N, k, mode, k0, p, max_p, renorm,
                                                        n_valid, oea_like ? k0_by_batch : nullptr, logits, idx, w,
                                                        oea_like ? n_base : nullptr, oea_like ? sbase_mask : nullptr,
                                                        cnt, offsets, perm, active, T, sync, as_stream(stream)),
                      "moe_router_route_dispatch");
}

namespace {

// Checks shared by both grouped-routing entry points.
int check_grouped(const moe::GroupedArgs& a, int score, int group_score, int max_n, int max_k, int max_b) {
    if (!a.logits || !a.idx || !a.w) return fail(MOE_EINVAL, "null pointer");
    if (a.logits_dtype != MOE_DT_F32 && a.logits_dtype != MOE_DT_BF16) return fail(MOE_EINVAL, "bad logits_dtype");
    if (reinterpret_cast<uintptr_t>(a.logits) % (a.logits_dtype == MOE_DT_F32 ? 4 : 2) != 0)
        return fail(MOE_EINVAL, "logits must be aligned to their element size");
    if (a.N < 1) return fail(MOE_EINVAL, "N must be >= 1");
    if (a.N > max_n) return fail(MOE_EUNSUPPORTED, "N above the limit of this entry point");
    if (a.k < 1 || a.k > a.N) return fail(MOE_EINVAL, "k must be in [1, N]");
    if (a.k > max_k) return fail(MOE_EUNSUPPORTED, "k above the limit of this entry point");
    if (a.B < 1) return fail(MOE_EINVAL, "B must be >= 1");
    if (a.B > max_b) return fail(MOE_EUNSUPPORTED, "B above the limit of this entry point");
    if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) return fail(MOE_EINVAL, "bad score function");
    if (group_score != MOE_GROUP_MAX && group_score != MOE_GROUP_TOP2) return fail(MOE_EINVAL, "bad group score");
    if (a.n_group < 1 || a.N % a.n_group) return fail(MOE_EINVAL, "n_group must divide N");
    if (a.n_group > moe::kMaxGroups) return fail(MOE_EUNSUPPORTED, "more than 64 groups are not supported");
    if (a.topk_group < 1 || a.topk_group > a.n_group) return fail(MOE_EINVAL, "topk_group must be in [1, n_group]");
    if (a.k > a.topk_group * (a.N / a.n_group)) return fail(MOE_EINVAL, "k exceeds the experts of topk_group groups");
    if (!(a.scale - a.scale == 0.0f)) return fail(MOE_EINVAL, "scale must be finite");
    return MOE_OK;
}

moe::GroupedArgs grouped_args(const void* logits, int logits_dtype, const float* bias, int B, int N, int k, int score,
                              int n_group, int topk_group, int group_score, int renorm, float scale,
                              const int32_t* n_valid, int32_t* idx, float* w) {
    moe::GroupedArgs a{};
    a.logits = logits; a.logits_dtype = logits_dtype; a.bias = bias;
    a.B = B; a.N = N; a.k = k;
    a.softmax = score == MOE_SCORE_SOFTMAX;
    a.n_group = n_group; a.topk_group = topk_group; a.group_top2 = group_score == MOE_GROUP_TOP2;
    a.renorm = renorm != 0; a.scale = scale;
    a.n_valid = n_valid; a.idx = idx; a.w = w;
    return a;
}

}  // namespace

MOE_API int moe_route_grouped(const void* logits, int logits_dtype, const float* bias, int B, int N, int k, int score,
                              int n_group, int topk_group, int group_score, int renorm, float scale,
                              const int32_t* n_valid, int32_t* idx, float* w, void* stream) {
    const moe::GroupedArgs a = grouped_args(logits, logits_dtype, bias, B, N, k, score, n_group, topk_group,
                                            group_score, renorm, scale, n_valid, idx, w);
    int st = check_grouped(a, score, group_score, moe::kMaxGroupedExperts, moe::kMaxGroupedTopK, moe::kMaxTokens);
    if (st) return st;
    return hip_status(moe::launch_route_grouped(a, as_stream(stream)), "moe_route_grouped");
}

MOE_API int moe_route_grouped_dispatch(const void* logits, int logits_dtype, const float* bias, int B, int N, int k,
                                       int score, int n_group, int topk_group, int group_score, int renorm,
                                       float scale, const int32_t* n_valid, int32_t* idx, float* w, int32_t* cnt,
                                       int32_t* offsets, int32_t* perm, int32_t* active, int32_t* T, int32_t* sync,
                                       void* stream) {
    moe::GroupedArgs a = grouped_args(logits, logits_dtype, bias, B, N, k, score, n_group, topk_group, group_score,
                                      renorm, scale, n_valid, idx, w);
    if (!cnt || !offsets || !perm || !active || !T || !sync) return fail(MOE_EINVAL, "null pointer");
    int st = check_grouped(a, score, group_score, moe::kMaxExperts, moe::kMaxTopK, moe::kMaxBatch);
    if (st) return st;
    a.cnt = cnt; a.offsets = offsets; a.perm = perm; a.active = active; a.T = T; a.sync = sync;
    return hip_status(moe::launch_route_grouped(a, as_stream(stream)), "moe_route_grouped_dispatch");
}

MOE_API size_t moe_ffn_workspace_bytes(int B, int k, int H, int I) {
    if (B < 1 || k < 1 || H < 1 || I < 1) return 0;
    return moe::ffn_workspace_bytes(B, k, H, I);
}

namespace {

// Checks shared by both expert-FFN entry points (everything but the workspace).
int check_ffn(const moe_expert_handle* table, int N, int H, int I, const void* x, int x_dtype, const int32_t* idx,
              const float* w, const int32_t* offsets, const int32_t* perm, const int32_t* active, const int32_t* T,
              int B, int k, float* y) {
    if (!table || !x || !idx || !w || !offsets || !perm || !active || !T || !y)
        return fail(MOE_EINVAL, "null pointer");
    int st = check_sizes(B, N, k);
    if (st) return st;
    if (x_dtype != MOE_DT_F32 && x_dtype != MOE_DT_BF16) return fail(MOE_EINVAL, "bad x_dtype");
    if (H < 32 || H % 32 || I < 32 || I % 32) return fail(MOE_EINVAL, "H and I must be positive multiples of 32");
    if (H > 16384 || I > 16384) return fail(MOE_EUNSUPPORTED, "H and I above 16384 are not supported");
    if (!moe::ffn_cost_fits(B, k, N, H, I)) return fail(MOE_EUNSUPPORTED, "B*k too large for H and I");
    if (reinterpret_cast<uintptr_t>(table) % 16 != 0) return fail(MOE_EINVAL, "handle table must be 16-byte aligned");
    return MOE_OK;
}

moe::FfnArgs ffn_args(const moe_expert_handle* table, int N, int H, int I, const void* x, int x_dtype,
                      const int32_t* idx, const float* w, const int32_t* offsets, const int32_t* perm,
                      const int32_t* active, const int32_t* T, int B, int k, float* y) {
    moe::FfnArgs a{};
    a.table = table;
    a.N = N; a.H = H; a.I = I; a.B = B; a.k = k;
    a.x = x; a.x_dtype = x_dtype;
    a.idx = idx; a.w = w; a.offsets = offsets; a.perm = perm; a.active = active; a.T = T;
    a.y = y;
    return a;
}

}  // namespace

MOE_API int moe_expert_ffn(const moe_expert_handle* table, int N, int H, int I, const void* x,
                           int x_dtype, const int32_t* idx, const float* w, const int32_t* offsets,
                           const int32_t* perm, const int32_t* active, const int32_t* T, int B,
                           int k, float* y, void* ws, size_t ws_bytes, void* stream) {
    if (!ws) return fail(MOE_EINVAL, "null pointer");
    int st = check_ffn(table, N, H, I, x, x_dtype, idx, w, offsets, perm, active, T, B, k, y);
    if (st) return st;
    if (ws_bytes < moe::ffn_workspace_bytes(B, k, H, I)) return fail(MOE_EINVAL, "workspace too small");
    if (reinterpret_cast<uintptr_t>(ws) % 256 != 0) return fail(MOE_EINVAL, "workspace must be 256-byte aligned");
    const moe::FfnArgs a = ffn_args(table, N, H, I, x, x_dtype, idx, w, offsets, perm, active, T, B, k, y);
    return hip_status(moe::launch_expert_ffn(a, ws, as_stream(stream)), "moe_expert_ffn");
}

MOE_API int moe_expert_ffn_noalloc(const moe_expert_handle* table, int N, int H, int I, const void* x,
                                   int x_dtype, const int32_t* idx, const float* w, const int32_t* offsets,
                                   const int32_t* perm, const int32_t* active, const int32_t* T, int B, int k,
                                   float* y, void* stream) {
    int st = check_ffn(table, N, H, I, x, x_dtype, idx, w, offsets, perm, active, T, B, k, y);
    if (st) return st;
    if (moe::ffn_workspace_bytes(B, k, H, I) > MOE_FFN_NOALLOC_WORKSPACE_BYTES)
        return fail(MOE_EUNSUPPORTED, "moe_ffn_workspace_bytes(B, k, H, I) exceeds the 32 MiB static workspace of "
                                      "moe_expert_ffn_noalloc");
    void* ws = nullptr;
    st = hip_status(moe::ffn_noalloc_workspace(&ws), "moe_expert_ffn_noalloc: static workspace lookup");
    if (st) return st;
    const moe::FfnArgs a = ffn_args(table, N, H, I, x, x_dtype, idx, w, offsets, perm, active, T, B, k, y);
    return hip_status(moe::launch_expert_ffn(a, ws, as_stream(stream)), "moe_expert_ffn_noalloc");
}

namespace {

bool misaligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }
int padded_rank(int r) { return (r + 15) / 16 * 16; }

// Checks shared by moe_lora_linear and moe_shared_ffn (everything but the
// weights, the tables and the workspace).
int check_proj(const moe::ProjArgs& a, int x_dtype, int y_dtype, bool any_table) {
    if (!a.x || !a.y) return fail(MOE_EINVAL, "null pointer");
    if (x_dtype != MOE_DT_F32 && x_dtype != MOE_DT_BF16) return fail(MOE_EINVAL, "bad x_dtype");
    if (y_dtype != MOE_DT_F32 && y_dtype != MOE_DT_BF16) return fail(MOE_EINVAL, "bad y_dtype");
    if (a.accumulate && y_dtype != MOE_DT_F32) return fail(MOE_EINVAL, "accumulating needs an fp32 y");
    if (a.B < 1) return fail(MOE_EINVAL, "B must be >= 1");
    if (a.B > moe::kMaxTokens) return fail(MOE_EUNSUPPORTED, "B above 2^20 is not supported");
    if (misaligned(a.x, 16) || misaligned(a.y, 16)) return fail(MOE_EINVAL, "x and y must be 16-byte aligned");
    if (any_table) {
        if (!a.adapter) return fail(MOE_EINVAL, "adapters need their token ids");
        if (a.n_adapters < 1) return fail(MOE_EINVAL, "n_adapters must be >= 1");
        if (a.max_rank < 16 || a.max_rank % 16) return fail(MOE_EINVAL, "max_rank must be a positive multiple of 16");
        if (a.max_rank > moe::kMaxLoraRank) return fail(MOE_EUNSUPPORTED, "max_rank above 256 is not supported");
    }
    return MOE_OK;
}

int check_workspace(const void* ws, size_t have, size_t need) {
    if (need == 0) return MOE_OK;
    if (!ws) return fail(MOE_EINVAL, "null workspace");
    if (have < need) return fail(MOE_EINVAL, "workspace too small");
    if (misaligned(ws, 256)) return fail(MOE_EINVAL, "workspace must be 256-byte aligned");
    return MOE_OK;
}

bool proj_sizes_ok(int B, int H, int O, int max_rank) {
    return B >= 1 && B <= moe::kMaxTokens && H >= 1 && H <= 16384 && O >= 1 && O <= 16384 && max_rank >= 0 &&
           max_rank <= moe::kMaxLoraRank;
}

}  // namespace

MOE_API int moe_lora_pack(const uint16_t* a, const uint16_t* b, int rank, int H, int O, void* dst_a, void* dst_b,
                          void* stream) {
    if (!a || !b || !dst_a || !dst_b) return fail(MOE_EINVAL, "null pointer");
    if (rank < 1) return fail(MOE_EINVAL, "rank must be >= 1");
    if (rank > moe::kMaxLoraRank) return fail(MOE_EUNSUPPORTED, "rank above 256 is not supported");
    if (H < 32 || H % 32) return fail(MOE_EINVAL, "H must be a positive multiple of 32");
    if (O < 16 || O % 16) return fail(MOE_EINVAL, "O must be a positive multiple of 16");
    if (H > 16384 || O > 16384) return fail(MOE_EUNSUPPORTED, "H and O above 16384 are not supported");
    if (misaligned(a, 16) || misaligned(dst_a, 16) || misaligned(dst_b, 16) || misaligned(b, 2))
        return fail(MOE_EINVAL, "a, dst_a and dst_b must be 16-byte aligned");
    return hip_status(moe::launch_lora_pack(a, b, rank, H, O, dst_a, dst_b, as_stream(stream)), "moe_lora_pack");
}

MOE_API int moe_lora_publish(moe_lora_handle* table, int i, const moe_lora_handle* h, void* stream) {
    if (!table || !h) return fail(MOE_EINVAL, "null pointer");
    if (i < 0) return fail(MOE_EINVAL, "adapter index must be >= 0");
    if (misaligned(table, 16)) return fail(MOE_EINVAL, "handle table must be 16-byte aligned");
    if (h->rank < 0 || h->rank % 16) return fail(MOE_EINVAL, "a handle's rank is the padded rank, a multiple of 16");
    if (h->rank > moe::kMaxLoraRank) return fail(MOE_EUNSUPPORTED, "rank above 256 is not supported");
    if (h->rank > 0) {
        if (!h->a || !h->b) return fail(MOE_EINVAL, "null adapter pointer");
        if (misaligned(h->a, 16) || misaligned(h->b, 16))
            return fail(MOE_EINVAL, "packed adapters must be 16-byte aligned");
        if (!(h->scale - h->scale == 0.0f)) return fail(MOE_EINVAL, "scale must be finite");
    }
    return hip_status(moe::launch_lora_publish(table, i, *h, as_stream(stream)), "moe_lora_publish");
}

MOE_API size_t moe_lora_workspace_bytes(int B, int H, int O, int max_rank, int x_dtype, int y_dtype) {
    (void)y_dtype;
    return proj_sizes_ok(B, H, O, max_rank) ? moe::lora_workspace_bytes(B, H, O, padded_rank(max_rank), x_dtype) : 0;
}

MOE_API int moe_lora_linear(const void* w, const moe_lora_handle* table, int n_adapters, int max_rank,
                            const int32_t* adapter, const void* x, int x_dtype, int B, int H, int O,
                            const int32_t* n_valid, void* y, int y_dtype, int accumulate, void* ws, size_t ws_bytes,
                            void* stream) {
    if (!w) return fail(MOE_EINVAL, "null pointer");
    moe::ProjArgs a{};
    a.w[0] = w; a.table[0] = table; a.adapter = table ? adapter : nullptr;
    a.n_adapters = n_adapters; a.max_rank = table ? max_rank : 0;
    a.x = x; a.x_kind = x_dtype == MOE_DT_F32 ? moe::kActF32 : moe::kActBf16; a.B = B; a.H = H; a.O = O;
    a.n_valid = n_valid; a.y = y; a.y_kind = y_dtype == MOE_DT_F32 ? moe::kActF32 : moe::kActBf16;
    a.accumulate = accumulate != 0;
    int st = check_proj(a, x_dtype, y_dtype, table != nullptr);
    if (st) return st;
    if (H < 32 || H % 32) return fail(MOE_EINVAL, "H must be a positive multiple of 32");
    if (O < 16 || O % 16) return fail(MOE_EINVAL, "O must be a positive multiple of 16");
    if (H > 16384 || O > 16384) return fail(MOE_EUNSUPPORTED, "H and O above 16384 are not supported");
    if (misaligned(w, 16) || misaligned(table, 16))
        return fail(MOE_EINVAL, "w and the handle table must be 16-byte aligned");
    st = check_workspace(ws, ws_bytes, moe_lora_workspace_bytes(B, H, O, a.max_rank, x_dtype, y_dtype));
    if (st) return st;
    return hip_status(moe::launch_lora_linear(a, ws, as_stream(stream)), "moe_lora_linear");
}

MOE_API size_t moe_shared_ffn_workspace_bytes(int B, int H, int I, int max_rank, int x_dtype, int y_dtype) {
    return proj_sizes_ok(B, H, I, max_rank)
               ? moe::shared_ffn_workspace_bytes(B, H, I, padded_rank(max_rank), x_dtype, y_dtype)
               : 0;
}

MOE_API int moe_shared_ffn(const moe_expert_handle* shared, const moe_lora_handle* t_gate,
                           const moe_lora_handle* t_up, const moe_lora_handle* t_down, int n_adapters, int max_rank,
                           const int32_t* adapter, const void* x, int x_dtype, int B, int H, int I,
                           const int32_t* n_valid, void* y, int y_dtype, int accumulate, void* ws, size_t ws_bytes,
                           void* stream) {
    if (!shared) return fail(MOE_EINVAL, "null pointer");
    if (shared->fmt != MOE_W_BF16) return fail(MOE_EUNSUPPORTED, "the shared expert's weights must be bf16");
    if (!shared->w_gate || !shared->w_up || !shared->w_down) return fail(MOE_EINVAL, "null weight pointer");
    if (misaligned(shared->w_gate, 16) || misaligned(shared->w_up, 16) || misaligned(shared->w_down, 16))
        return fail(MOE_EINVAL, "packed weights must be 16-byte aligned");
    const bool any = t_gate || t_up || t_down;
    moe::ProjArgs a{};
    a.w[0] = shared->w_gate; a.w[1] = shared->w_up;
    a.table[0] = t_gate; a.table[1] = t_up;
    a.adapter = any ? adapter : nullptr;
    a.n_adapters = n_adapters; a.max_rank = any ? max_rank : 0;
    a.x = x; a.x_kind = x_dtype == MOE_DT_F32 ? moe::kActF32 : moe::kActBf16; a.B = B; a.H = H; a.O = I;
    a.n_valid = n_valid; a.y = y; a.y_kind = y_dtype == MOE_DT_F32 ? moe::kActF32 : moe::kActBf16;
    a.accumulate = accumulate != 0;
    int st = check_proj(a, x_dtype, y_dtype, any);
    if (st) return st;
    if (H < 32 || H % 32 || I < 32 || I % 32) return fail(MOE_EINVAL, "H and I must be positive multiples of 32");
    if (H > 16384 || I > 16384) return fail(MOE_EUNSUPPORTED, "H and I above 16384 are not supported");
    if (misaligned(t_gate, 16) || misaligned(t_up, 16) || misaligned(t_down, 16))
        return fail(MOE_EINVAL, "handle tables must be 16-byte aligned");
    st = check_workspace(ws, ws_bytes, moe_shared_ffn_workspace_bytes(B, H, I, a.max_rank, x_dtype, y_dtype));
    if (st) return st;
    return hip_status(moe::launch_shared_ffn(a, shared->w_down, t_down, ws, as_stream(stream)), "moe_shared_ffn");
}

MOE_API int moe_handle_publish(moe_expert_handle* table, int e, const moe_expert_handle* h,
                               void* stream) {
    if (!table || !h) return fail(MOE_EINVAL, "null pointer");
    if (e < 0 || e >= moe::kMaxExperts) return fail(MOE_EINVAL, "expert index out of range");
    if (h->fmt != MOE_W_F32 && h->fmt != MOE_W_BF16 && h->fmt != MOE_W_INT4_G128)
        return fail(MOE_EINVAL, "bad weight format");
    if (!h->w_gate || !h->w_up || !h->w_down) return fail(MOE_EINVAL, "null weight pointer");
    if (h->fmt == MOE_W_INT4_G128 && (h->group != 128 || !h->s_gate || !h->s_up || !h->s_down))
        return fail(MOE_EINVAL, "INT4 handle needs group 128 and scale pointers");
    auto misaligned = [](const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; };
    if (misaligned(h->w_gate, 16) || misaligned(h->w_up, 16) || misaligned(h->w_down, 16))
        return fail(MOE_EINVAL, "packed weights must be 16-byte aligned");
    if (h->fmt == MOE_W_INT4_G128 && (misaligned(h->s_gate, 8) || misaligned(h->s_up, 8) || misaligned(h->s_down, 8)))
        return fail(MOE_EINVAL, "packed scales must be 8-byte aligned");
    return hip_status(moe::launch_handle_publish(table, e, *h, as_stream(stream)), "moe_handle_publish");
}

MOE_API int moe_quantize_int4_g128(const uint16_t* w, int rows, int cols, uint8_t* q,
                                   uint16_t* scales, void* stream) {
    if (!w || !q || !scales) return fail(MOE_EINVAL, "null pointer");
    if (rows < 1 || cols < 128 || cols % 128) return fail(MOE_EINVAL, "cols must be a positive multiple of 128");
    return hip_status(moe::launch_quantize_int4(w, rows, cols, q, scales, as_stream(stream)),
                      "moe_quantize_int4_g128");
}

MOE_API int moe_pack_weights(int fmt, const void* src, const uint16_t* src_scales, int rows, int cols,
                             void* dst, uint16_t* dst_scales, void* stream) {
    if (fmt != MOE_W_F32 && fmt != MOE_W_BF16 && fmt != MOE_W_INT4_G128) return fail(MOE_EINVAL, "bad weight format");
    if (!src || !dst) return fail(MOE_EINVAL, "null pointer");
    if (fmt == MOE_W_INT4_G128 && (!src_scales || !dst_scales)) return fail(MOE_EINVAL, "INT4 needs scale pointers");
    if (rows < 16 || rows % 16) return fail(MOE_EINVAL, "rows must be a positive multiple of 16");
    const int tc = moe::tile_cols(fmt);
    if (cols < tc || cols % tc) return fail(MOE_EINVAL, "cols must be a positive multiple of 16/32/128 (fp32/bf16/INT4)");
    if (static_cast<long>(rows) * cols > (1L << 31)) return fail(MOE_EUNSUPPORTED, "matrix above 2^31 elements");
    if (reinterpret_cast<uintptr_t>(src) % 16 || reinterpret_cast<uintptr_t>(dst) % 16)
        return fail(MOE_EINVAL, "src and dst must be 16-byte aligned");
    const size_t bytes = static_cast<size_t>(rows) * moe::weight_row_bytes(fmt, cols);
    const char* s0 = static_cast<const char*>(src);
    char* d0 = static_cast<char*>(dst);
    if (s0 < d0 + bytes && d0 < s0 + bytes) return fail(MOE_EINVAL, "src and dst overlap");
    return hip_status(moe::launch_pack_weights(fmt, src, src_scales, rows, cols, dst, dst_scales, as_stream(stream)),
                      "moe_pack_weights");
}

MOE_API int moe_hotness_ema(float* S, const int32_t* cnt, int N, float alpha, void* stream) {
    if (!S || !cnt) return fail(MOE_EINVAL, "null pointer");
    if (N < 1 || N > moe::kMaxExperts) return fail(MOE_EINVAL, "N must be in [1, 128]");
    if (!(alpha >= 0.0f && alpha <= 1.0f)) return fail(MOE_EINVAL, "alpha must be in [0, 1]");
    return hip_status(moe::launch_hotness_ema(S, cnt, N, alpha, as_stream(stream)), "moe_hotness_ema");
}

MOE_API int moe_expert_ffn_phase_events(const moe_expert_handle* table, int N, int H, int I, const void* x,
                                        int x_dtype, const int32_t* idx, const float* w, const int32_t* offsets,
                                        const int32_t* perm, const int32_t* active, const int32_t* T, int B, int k,
                                        float* y, void* ws, size_t ws_bytes, void* const* events, void* stream) {
    if (!events) return fail(MOE_EINVAL, "null events array");
    int st = check_ffn(table, N, H, I, x, x_dtype, idx, w, offsets, perm, active, T, B, k, y);
    if (st) return st;
    if (!ws) return fail(MOE_EINVAL, "null workspace");
    if (ws_bytes < moe::ffn_workspace_bytes(B, k, H, I)) return fail(MOE_EINVAL, "workspace too small");
    if (reinterpret_cast<uintptr_t>(ws) % 256 != 0) return fail(MOE_EINVAL, "workspace must be 256-byte aligned");
    hipEvent_t ev[4];
    for (int i = 0; i < 4; ++i) ev[i] = static_cast<hipEvent_t>(events[i]);
    const moe::FfnArgs a = ffn_args(table, N, H, I, x, x_dtype, idx, w, offsets, perm, active, T, B, k, y);
    return hip_status(moe::launch_expert_ffn(a, ws, as_stream(stream), ev), "moe_expert_ffn_phase_events");
}

MOE_API int moe_stream_read(const void* buf, size_t bytes, int waves_per_cu, uint32_t* out, void* stream) {
    if (!buf || !out) return fail(MOE_EINVAL, "null pointer");
    if (bytes < 16 || bytes % 16) return fail(MOE_EINVAL, "bytes must be a positive multiple of 16");
    if (waves_per_cu < 4 || waves_per_cu > 32 || waves_per_cu % 4)
        return fail(MOE_EINVAL, "waves_per_cu must be 4, 8, ..., 32");
    if (reinterpret_cast<uintptr_t>(buf) % 16 || reinterpret_cast<uintptr_t>(out) % 4)
        return fail(MOE_EINVAL, "buf must be 16-byte aligned");
    return hip_status(moe::launch_stream_read(buf, bytes, waves_per_cu, out, moe::device_cus(), as_stream(stream)),
                      "moe_stream_read");
}
