// ep_combine_backward.hip -- gradients of the combine, with dropout, in the expert
// rows and the routing weights.
//
//   g[t]            = kept ? dy[t] * f : 0          (f = 1 / (1 - p))
//   d_expert_out[s] = w[t, j] g[t]                  s the receive row of entry (t, j)
//   d_weights[t, j] = <g[t], expert_out[s]>
//
// A workgroup takes a token.  A lane holds VPL 16-byte pieces of dy with the
// dropped channels zeroed, made once for all k entries, and goes through the
// entries: each expert row is read once, each gradient row written once.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ep_dropout_dev.h"
#include "ep_internal.h"
#include "ep_norm_dev.h"

namespace ep {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kMaxThreads = 1024;

template <int VPL>
__global__ __launch_bounds__(kMaxThreads) void combine_backward_kernel(
        const u32x4* __restrict__ dy, const u32x4* __restrict__ eo, int nvec, int k,
        const int32_t* __restrict__ slot_of, int64_t R, const float* __restrict__ weights,
        DropArgs drop, u32x4* __restrict__ deo, float* __restrict__ dw) {
    __shared__ float s_part[kMaxThreads / kWave][kMaxTopk];
    const int t = blockIdx.x;
    const int32_t* slots = slot_of + static_cast<int64_t>(t) * k;
    const int wave = threadIdx.x / kWave;
    u32x4 g[VPL];
#pragma unroll
    for (int u = 0; u < VPL; ++u) {
        const int v = threadIdx.x + u * blockDim.x;
        g[u] = u32x4{0, 0, 0, 0};
        if (v >= nvec) continue;
        g[u] = __builtin_nontemporal_load(dy + static_cast<int64_t>(t) * nvec + v);
        const uint32_t kept = dropout::keep8(drop, t, v);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            g[u][i] &= (kept >> (2 * i) & 1 ? 0xffffu : 0u) | (kept >> (2 * i + 1) & 1 ? 0xffff0000u : 0u);
    }
    for (int j = 0; j < k; ++j) {
        const int32_t slot = slots[j];
        float sum = 0.0f;
        if (slot >= 0 && slot < R) {
            const float w = weights[static_cast<int64_t>(t) * k + j];
#pragma unroll
            for (int u = 0; u < VPL; ++u) {
                const int v = threadIdx.x + u * blockDim.x;
                if (v >= nvec) continue;
                const int64_t at = static_cast<int64_t>(slot) * nvec + v;
                u32x4 e = u32x4{0, 0, 0, 0}, d;
                if (dw != nullptr) e = __builtin_nontemporal_load(eo + at);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t gi = g[u][i];
                    const float lo = bf16_lo(gi) * drop.factor, hi = bf16_hi(gi) * drop.factor;
                    sum = fmaf(lo, bf16_lo(e[i]), sum);
                    sum = fmaf(hi, bf16_hi(e[i]), sum);
                    d[i] = pack_bf16(lo * w, hi * w);
                }
                __builtin_nontemporal_store(d, deo + at);
            }
        }
        if (dw != nullptr) {
            sum = norm::wave_sum(sum);
            if (threadIdx.x % kWave == 0) s_part[wave][j] = sum;
        }
    }
    if (dw == nullptr) return;
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < k) {
        float sum = 0.0f;
        for (int i = 0; i < static_cast<int>(blockDim.x) / kWave; ++i) sum += s_part[i][threadIdx.x];
        dw[static_cast<int64_t>(t) * k + threadIdx.x] = sum;
    }
}

}  // namespace

hipError_t launch_combine_backward(const ep_problem& p, const void* dy, const void* expert_out,
                                   const int32_t* slot_of, const float* topk_weights,
                                   const DropArgs& drop, void* d_expert_out, float* d_weights,
                                   hipStream_t stream) {
    const int T = p.num_tokens;
    if (T == 0) return hipSuccess;
    const int64_t R = p.capacity == 0 ? static_cast<int64_t>(T) * p.num_topk
                                      : static_cast<int64_t>(p.num_experts) * p.capacity;
    const int nvec = p.hidden / 8;
    int threads = kWave;
    while (threads < kMaxThreads && nvec > 4 * threads) threads *= 2;
    const auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(T), dim3(threads), 0, stream, static_cast<const u32x4*>(dy),
                           static_cast<const u32x4*>(expert_out), nvec, p.num_topk, slot_of, R,
                           topk_weights, drop, static_cast<u32x4*>(d_expert_out), d_weights);
    };
    const int vpl = (nvec + threads - 1) / threads;
    if (vpl == 1)
        go(combine_backward_kernel<1>);
    else if (vpl == 2)
        go(combine_backward_kernel<2>);
    else if (vpl <= 4)
        go(combine_backward_kernel<4>);
    else
        go(combine_backward_kernel<8>);
    return hipGetLastError();
}

}  // namespace ep
