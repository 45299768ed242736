// ep_api.hip -- the exported C ABI: argument checks on the host, then launches.
// Every check happens before anything is enqueued, so an error code other
// than EP_ERR_HIP means the stream was not touched.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>
#include <mutex>

#include "ep.h"
#include "ep_internal.h"

// Device scratch of ep_layout_dispatch_noalloc: one copy per GPU (a file-scope
// __device__ array exists once in every device's memory), held until the
// process ends.  Host code never passes `scratch` itself to a kernel -- in
// host code the name stands for a host-side shadow, not a device address --
// but the pointer hipGetSymbolAddress returns for the current device.
static __device__ __align__(256) int32_t scratch[ep::kMaxLayoutWorkspaceBytes / 4];

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Shape checks shared by every entry point.
int check_problem(const ep_problem* p) {
    if (p == nullptr) return EP_ERR_ARG;
    if (p->num_tokens < 0 || p->hidden < 1 || p->num_topk < 1 || p->num_experts < 1 ||
        p->capacity < 0 || p->use_fp8 < 0 || p->use_fp8 > 2)
        return EP_ERR_ARG;
    if (p->num_experts > ep::kMaxExperts || p->num_topk > ep::kMaxTopk ||
        p->hidden > ep::kMaxHidden || p->hidden % 8 != 0 ||
        (p->use_fp8 && p->hidden % 128 != 0))
        return EP_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(p->num_tokens) * p->num_topk >= (int64_t{1} << 31) ||
        static_cast<int64_t>(p->num_experts) * p->capacity >= (int64_t{1} << 31))
        return EP_ERR_UNSUPPORTED;
    return EP_OK;
}

int64_t recv_rows(const ep_problem& p) {
    return p.capacity == 0 ? static_cast<int64_t>(p.num_tokens) * p.num_topk
                           : static_cast<int64_t>(p.num_experts) * p.capacity;
}

int check_layout_ptrs(const ep_problem& p, const ep_layout_t* lay, bool all) {
    if (lay == nullptr) return EP_ERR_ARG;
    const bool need_slots = static_cast<int64_t>(p.num_tokens) * p.num_topk > 0;
    if (need_slots && lay->slot_of == nullptr) return EP_ERR_ARG;
    if (!aligned4(lay->slot_of)) return EP_ERR_ALIGN;
    if (all) {
        if (lay->count == nullptr || lay->offset == nullptr || lay->status == nullptr)
            return EP_ERR_ARG;
        if (recv_rows(p) > 0 && lay->src_of_slot == nullptr) return EP_ERR_ARG;
        if (!aligned4(lay->count) || !aligned4(lay->offset) || !aligned4(lay->status) ||
            !aligned4(lay->src_of_slot))
            return EP_ERR_ALIGN;
    }
    return EP_OK;
}

int from_hip(hipError_t e) { return e == hipSuccess ? EP_OK : EP_ERR_HIP; }

// Device address of `scratch` on the current device, looked up once per
// device (with that device current) and kept.
constexpr int kMaxDevices = 64;
std::mutex g_scratch_mutex;
void* g_scratch_addr[kMaxDevices] = {};

hipError_t scratch_address(void** out) {
    int dev = -1;
    hipError_t err = hipGetDevice(&dev);
    if (err != hipSuccess) return err;
    if (dev < 0 || dev >= kMaxDevices) return hipErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(g_scratch_mutex);
    if (g_scratch_addr[dev] == nullptr) {
        void* ptr = nullptr;
        err = hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch));
        if (err != hipSuccess) return err;
        if (ptr == nullptr) return hipErrorInvalidSymbol;
        g_scratch_addr[dev] = ptr;
    }
    *out = g_scratch_addr[dev];
    return hipSuccess;
}

// Arguments of ep_layout_dispatch apart from the workspace.
int check_layout_dispatch_args(const ep_problem* prob, const int32_t* topk_idx,
                               const ep_layout_t* out, const void* x, void* recv_x,
                               void* recv_scales) {
    int rc = check_problem(prob);
    if (rc != EP_OK) return rc;
    rc = check_layout_ptrs(*prob, out, true);
    if (rc != EP_OK) return rc;
    if (static_cast<int64_t>(prob->num_tokens) * prob->num_topk > 0 && topk_idx == nullptr)
        return EP_ERR_ARG;
    if (!aligned16(topk_idx)) return EP_ERR_ALIGN;
    if (prob->num_tokens > 0) {
        if (x == nullptr || recv_x == nullptr) return EP_ERR_ARG;
        if (prob->use_fp8 && recv_scales == nullptr) return EP_ERR_ARG;
    }
    if (!aligned16(x) || !aligned16(recv_x) || (prob->use_fp8 && !aligned16(recv_scales)))
        return EP_ERR_ALIGN;
    return EP_OK;
}

// Shape and row pitch of a routing problem.
int check_routing(const ep_routing* rt) {
    if (rt == nullptr) return EP_ERR_ARG;
    if (rt->num_tokens < 0 || rt->num_experts < 1 || rt->num_topk < 1 || rt->num_groups < 1 ||
        rt->topk_groups < 1 || rt->num_seqs < 1 || rt->score < 0 || rt->score > 1 ||
        rt->normalize < 0 || rt->normalize > 1 || rt->choose_by_score < 0 ||
        rt->choose_by_score > 1 || !std::isfinite(rt->weight_scale))
        return EP_ERR_ARG;
    if (rt->num_experts > ep::kMaxExperts || rt->num_topk > ep::kMaxTopk ||
        rt->num_groups > ep::kMaxGroups || rt->num_seqs > ep::kMaxSeqs ||
        rt->num_tokens > ep::kMaxRouted || (rt->choose_by_score == 1 && rt->score != 1))
        return EP_ERR_UNSUPPORTED;
    if (rt->num_experts % rt->num_groups != 0 || rt->topk_groups > rt->num_groups ||
        rt->num_topk > rt->topk_groups * (rt->num_experts / rt->num_groups) ||
        rt->num_tokens % rt->num_seqs != 0)
        return EP_ERR_ARG;
    return EP_OK;
}

int check_logits(const ep_routing& rt, const void* logits, int bf16, int64_t stride) {
    if (bf16 < 0 || bf16 > 1 || stride < rt.num_experts) return EP_ERR_ARG;
    if (stride > (int64_t{1} << 31)) return EP_ERR_UNSUPPORTED;
    if (rt.num_tokens > 0 && logits == nullptr) return EP_ERR_ARG;
    if (reinterpret_cast<uintptr_t>(logits) % (bf16 ? 2 : 4) != 0) return EP_ERR_ALIGN;
    return EP_OK;
}

ep::RouteArgs route_args(const ep_routing& rt, const void* logits, int bf16, int64_t stride,
                         const void* d_logits, const void* per_expert) {
    ep::RouteArgs a;
    a.logits = logits;
    a.stride = stride;
    a.num_tokens = rt.num_tokens;
    a.num_experts = rt.num_experts;
    a.num_topk = rt.num_topk;
    a.num_groups = rt.num_groups;
    a.topk_groups = rt.topk_groups;
    a.num_seqs = rt.num_seqs;
    a.seq_len = rt.num_tokens / rt.num_seqs;
    a.scale = rt.weight_scale;
    a.bf16 = bf16 != 0;
    a.sigmoid = rt.score == 1;
    a.normalize = rt.normalize == 1;
    a.by_score = rt.choose_by_score == 1;
    const int el = bf16 ? 2 : 4;
    const ep::TokenShape shape = ep::token_shape(rt.num_experts, ep::kSixteenLanes);
    const int vpl = shape.vpl;
    const int group = rt.num_experts / rt.num_groups;
    const int lanes = group / vpl;
    a.group_lanes = shape.lpt == 16 && group % vpl == 0 &&
                            (lanes == 1 || lanes == 2 || lanes == 4 || lanes == 8)
                        ? lanes
                        : 0;
    const int piece = vpl * el < 16 ? vpl : 16 / el;  // elements per access
    const auto fits = [&](const void* p, int64_t pitch) {
        return rt.num_experts % piece == 0 && pitch % piece == 0 &&
               reinterpret_cast<uintptr_t>(p) % (piece * el) == 0;
    };
    a.pieces = fits(logits, stride);
    a.out_pieces = fits(d_logits, rt.num_experts);
    a.fours = rt.num_experts % 4 == 0 && aligned16(per_expert);
    return a;
}

}  // namespace

extern "C" {

int64_t ep_num_recv_rows(const ep_problem* prob) {
    if (check_problem(prob) != EP_OK) return -1;
    return recv_rows(*prob);
}

int64_t ep_layout_workspace_bytes(const ep_problem* prob) {
    if (check_problem(prob) != EP_OK) return -1;
    return ep::layout_workspace_bytes(*prob);
}

int ep_layout(const ep_problem* prob, const int32_t* topk_idx, const ep_layout_t* out,
              void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_problem(prob);
    if (rc != EP_OK) return rc;
    rc = check_layout_ptrs(*prob, out, true);
    if (rc != EP_OK) return rc;
    if (static_cast<int64_t>(prob->num_tokens) * prob->num_topk > 0 && topk_idx == nullptr)
        return EP_ERR_ARG;
    if (!aligned16(topk_idx)) return EP_ERR_ALIGN;
    if (workspace == nullptr ||
        static_cast<int64_t>(workspace_bytes) < ep::layout_workspace_bytes(*prob))
        return EP_ERR_ARG;
    if (!aligned16(workspace)) return EP_ERR_ALIGN;
    return from_hip(ep::launch_layout(*prob, topk_idx, *out, static_cast<int32_t*>(workspace),
                                      static_cast<hipStream_t>(stream)));
}

int ep_dispatch(const ep_problem* prob, const void* x, const ep_layout_t* layout, void* recv_x,
                void* recv_scales, void* stream) {
    int rc = check_problem(prob);
    if (rc != EP_OK) return rc;
    rc = check_layout_ptrs(*prob, layout, false);
    if (rc != EP_OK) return rc;
    if (prob->num_tokens > 0) {
        if (x == nullptr || recv_x == nullptr) return EP_ERR_ARG;
        if (prob->use_fp8 && recv_scales == nullptr) return EP_ERR_ARG;
    }
    if (!aligned16(x) || !aligned16(recv_x) || (prob->use_fp8 && !aligned16(recv_scales)))
        return EP_ERR_ALIGN;
    return from_hip(ep::launch_dispatch(*prob, x, layout->slot_of, recv_x,
                                        prob->use_fp8 ? recv_scales : nullptr,
                                        static_cast<hipStream_t>(stream)));
}

int ep_layout_dispatch(const ep_problem* prob, const int32_t* topk_idx, const ep_layout_t* out,
                       void* workspace, size_t workspace_bytes, const void* x, void* recv_x,
                       void* recv_scales, void* stream) {
    int rc = check_layout_dispatch_args(prob, topk_idx, out, x, recv_x, recv_scales);
    if (rc != EP_OK) return rc;
    if (workspace == nullptr ||
        static_cast<int64_t>(workspace_bytes) < ep::layout_workspace_bytes(*prob))
        return EP_ERR_ARG;
    if (!aligned16(workspace)) return EP_ERR_ALIGN;
    return from_hip(ep::launch_layout_dispatch(*prob, topk_idx, *out, workspace, x, recv_x,
                                               prob->use_fp8 ? recv_scales : nullptr,
                                               static_cast<hipStream_t>(stream)));
}

int ep_layout_dispatch_noalloc(const ep_problem* prob, const int32_t* topk_idx,
                               const ep_layout_t* out, const void* x, void* recv_x,
                               void* recv_scales, void* stream) {
    int rc = check_layout_dispatch_args(prob, topk_idx, out, x, recv_x, recv_scales);
    if (rc != EP_OK) return rc;
    if (ep::layout_workspace_bytes(*prob) > ep::kMaxLayoutWorkspaceBytes) return EP_ERR_UNSUPPORTED;
    void* ws = nullptr;
    const hipError_t err = scratch_address(&ws);
    if (err != hipSuccess) return EP_ERR_HIP;
    // The workspace needs no initialisation (the histogram kernel writes every
    // word it later reads), so the array's previous contents do not matter.
    return from_hip(ep::launch_layout_dispatch(*prob, topk_idx, *out, ws, x, recv_x,
                                               prob->use_fp8 ? recv_scales : nullptr,
                                               static_cast<hipStream_t>(stream)));
}

static_assert(EP_NOALLOC_SCRATCH_BYTES == ep::kMaxLayoutWorkspaceBytes,
              "ep.h states the size of the allocation-free entry point's device array");

int ep_combine(const ep_problem* prob, const void* expert_out, const ep_layout_t* layout,
               const float* topk_weights, void* y, void* stream) {
    int rc = check_problem(prob);
    if (rc != EP_OK) return rc;
    rc = check_layout_ptrs(*prob, layout, false);
    if (rc != EP_OK) return rc;
    if (prob->num_tokens > 0 && (expert_out == nullptr || topk_weights == nullptr || y == nullptr))
        return EP_ERR_ARG;
    if (!aligned16(expert_out) || !aligned16(y) || !aligned4(topk_weights)) return EP_ERR_ALIGN;
    return from_hip(ep::launch_combine(*prob, expert_out, layout->slot_of, topk_weights, y,
                                       static_cast<hipStream_t>(stream)));
}

int ep_e4m3_encode(const float* in, uint8_t* out, int64_t n, void* stream) {
    if (n < 0) return EP_ERR_ARG;
    if (n > 0 && (in == nullptr || out == nullptr)) return EP_ERR_ARG;
    if (!aligned4(in)) return EP_ERR_ALIGN;
    return from_hip(ep::launch_e4m3_encode(in, out, n, static_cast<hipStream_t>(stream)));
}

int ep_route(const ep_routing* rt, const void* logits, int logits_bf16, int64_t logits_stride,
             const float* expert_bias, const uint8_t* valid, int32_t* topk_idx,
             float* topk_weights, void* stream) {
    int rc = check_routing(rt);
    if (rc != EP_OK) return rc;
    rc = check_logits(*rt, logits, logits_bf16, logits_stride);
    if (rc != EP_OK) return rc;
    if (rt->num_tokens > 0 && (topk_idx == nullptr || topk_weights == nullptr)) return EP_ERR_ARG;
    if (!aligned4(expert_bias) || !aligned4(topk_idx) || !aligned4(topk_weights))
        return EP_ERR_ALIGN;
    const ep::RouteForward f = {expert_bias, valid, topk_idx, topk_weights};
    return from_hip(ep::launch_route(
        route_args(*rt, logits, logits_bf16, logits_stride, nullptr, expert_bias), f,
        static_cast<hipStream_t>(stream)));
}

int64_t ep_balance_workspace_bytes(const ep_routing* rt) {
    if (check_routing(rt) != EP_OK) return -1;
    return ep::balance_workspace_bytes(rt->num_tokens, rt->num_experts, rt->num_seqs);
}

int ep_balance_loss(const ep_routing* rt, const void* logits, int logits_bf16,
                    int64_t logits_stride, const int32_t* topk_idx, const uint8_t* valid,
                    float coef, int32_t* counts, float* mean_prob, int32_t* num_valid,
                    float* loss, void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_routing(rt);
    if (rc != EP_OK) return rc;
    rc = check_logits(*rt, logits, logits_bf16, logits_stride);
    if (rc != EP_OK) return rc;
    if (!std::isfinite(coef)) return EP_ERR_ARG;
    if (rt->num_tokens > 0 && topk_idx == nullptr) return EP_ERR_ARG;
    if (counts == nullptr || mean_prob == nullptr || num_valid == nullptr || loss == nullptr)
        return EP_ERR_ARG;
    if (workspace == nullptr ||
        static_cast<int64_t>(workspace_bytes) <
            ep::balance_workspace_bytes(rt->num_tokens, rt->num_experts, rt->num_seqs))
        return EP_ERR_ARG;
    if (!aligned4(topk_idx) || !aligned4(counts) || !aligned4(mean_prob) || !aligned4(num_valid) ||
        !aligned4(loss) || !aligned16(workspace))
        return EP_ERR_ALIGN;
    const ep::BalanceArgs b = {topk_idx, valid, coef, counts, mean_prob, num_valid, loss};
    return from_hip(ep::launch_balance(
        route_args(*rt, logits, logits_bf16, logits_stride, nullptr, nullptr), b, workspace,
        static_cast<hipStream_t>(stream)));
}

int ep_route_backward(const ep_routing* rt, const void* logits, int logits_bf16,
                      int64_t logits_stride, const int32_t* topk_idx, const float* d_weights,
                      const uint8_t* valid, float coef, const int32_t* counts,
                      const int32_t* num_valid, const float* d_loss, void* d_logits,
                      void* stream) {
    int rc = check_routing(rt);
    if (rc != EP_OK) return rc;
    rc = check_logits(*rt, logits, logits_bf16, logits_stride);
    if (rc != EP_OK) return rc;
    if (!std::isfinite(coef)) return EP_ERR_ARG;
    if (rt->num_tokens > 0) {
        if (d_logits == nullptr || (d_weights == nullptr && d_loss == nullptr)) return EP_ERR_ARG;
        if (d_weights != nullptr && topk_idx == nullptr) return EP_ERR_ARG;
        if (d_loss != nullptr && (counts == nullptr || num_valid == nullptr)) return EP_ERR_ARG;
    }
    if (!aligned4(topk_idx) || !aligned4(d_weights) || !aligned4(counts) || !aligned4(num_valid) ||
        !aligned4(d_loss) ||
        reinterpret_cast<uintptr_t>(d_logits) % (logits_bf16 ? 2 : 4) != 0)
        return EP_ERR_ALIGN;
    const ep::RouteBackward b = {topk_idx, d_weights, valid, coef, counts, num_valid, d_loss,
                                 d_logits};
    return from_hip(ep::launch_route_backward(
        route_args(*rt, logits, logits_bf16, logits_stride, d_logits, counts), b,
        static_cast<hipStream_t>(stream)));
}

int ep_expert_w4(const ep_problem* prob, const ep_expert_w4_t* mm, const void* rows,
                 const void* row_scales, const ep_layout_t* layout, const uint8_t* codes,
                 const uint8_t* scales, void* out, void* stream) {
    int rc = check_problem(prob);
    if (rc != EP_OK) return rc;
    if (mm == nullptr || layout == nullptr) return EP_ERR_ARG;
    if (mm->in_features < 1 || mm->out_features < 1 || mm->in_format < 0 || mm->in_format > 2 ||
        mm->activation < 0 || mm->activation > 1)
        return EP_ERR_ARG;
    if (mm->in_features > ep::kMaxHidden || mm->out_features > ep::kMaxHidden ||
        mm->in_features % (mm->in_format ? 128 : 32) != 0)
        return EP_ERR_UNSUPPORTED;
    if (layout->count == nullptr || (prob->capacity == 0 && layout->offset == nullptr))
        return EP_ERR_ARG;
    if (!aligned4(layout->count) || !aligned4(layout->offset)) return EP_ERR_ALIGN;
    if (prob->num_tokens > 0) {
        if (rows == nullptr || codes == nullptr || scales == nullptr || out == nullptr)
            return EP_ERR_ARG;
        if (mm->in_format && row_scales == nullptr) return EP_ERR_ARG;
    }
    if (!aligned16(rows) || !aligned16(codes) || !aligned16(scales) || !aligned16(out) ||
        (mm->in_format && !aligned16(row_scales)))
        return EP_ERR_ALIGN;
    return from_hip(ep::launch_expert_w4(*prob, *mm, rows, row_scales, *layout, codes, scales, out,
                                         static_cast<hipStream_t>(stream)));
}

const char* ep_strerror(int code) {
    switch (code) {
        case EP_OK: return "ok";
        case EP_ERR_ARG: return "invalid argument (size, null pointer or workspace too small)";
        case EP_ERR_UNSUPPORTED: return "problem size outside the supported envelope";
        case EP_ERR_ALIGN: return "pointer not aligned (data 16 bytes, int32/fp32 arrays 4 bytes)";
        case EP_ERR_HIP: return "HIP kernel launch failed";
        default: return "unknown status code";
    }
}

}  // extern "C"
