// ep_quant.hip -- token rows to 8-bit integer receive rows (ep_dispatch_i8), and
// receive rows to 8-bit integers (inside ep_expert_i8).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ep_internal.h"
#include "ep_quant_dev.h"

namespace ep {
namespace {

using quant::Row;
using quant::u32x2;
using quant::u32x4;

constexpr int kMaxThreads = 1024;

// A workgroup per token: its row is read and quantised once however large k is.
// The stores bound it: 8192 tokens, H 4096, top-6: 42 us, 6.4 TB/s.  A decode batch of 128
// tokens, H 7168, top-8 takes the GPU 5.1 us, one piece per lane.
template <int VPL>
__global__ __launch_bounds__(kMaxThreads) void dispatch_i8_kernel(
        const u32x4* __restrict__ x, int nvec, int k, const int32_t* __restrict__ slot_of, int64_t R,
        u32x2* __restrict__ recv_q, float* __restrict__ recv_scales) {
    __shared__ float s_part[kMaxThreads / kWave];
    const int64_t t = blockIdx.x;
    const int32_t* slots = slot_of + t * k;
    Row<VPL> row;
    row.load(x + t * nvec, nvec, s_part);
    for (int j = 0; j < k; ++j) {
        const int32_t slot = slots[j];
        if (slot < 0 || slot >= R) continue;
        row.store(recv_q + static_cast<int64_t>(slot) * nvec, nvec);
        if (threadIdx.x == 0) recv_scales[slot] = row.scale;
    }
}

// Rows that an entry fills: those before offset[E], or the first count[e] of
// expert e's.  A workgroup takes rows gridDim apart; with a capacity blockIdx.y
// is the expert.  1024 rows of K 2048 among 32768: 5.0 us, in front of products of 570.
template <int VPL>
__global__ __launch_bounds__(kMaxThreads) void quant_rows_kernel(
        const u32x4* __restrict__ rows, int nvec, const int32_t* __restrict__ count,
        const int32_t* __restrict__ offset, int E, int capacity, int64_t R, u32x2* __restrict__ q,
        float* __restrict__ scales) {
    __shared__ float s_part[2][kMaxThreads / kWave];
    int64_t first = 0, n;
    if (capacity > 0) {
        first = static_cast<int64_t>(blockIdx.y) * capacity;
        n = min(count[blockIdx.y], capacity);
    } else {
        n = min(static_cast<int64_t>(offset[E]), R);
    }
    int turn = 0;
    for (int64_t i = blockIdx.x; i < n; i += gridDim.x, turn ^= 1) {
        const int64_t r = first + i;
        Row<VPL> row;
        row.load(rows + r * nvec, nvec, s_part[turn]);
        row.store(q + r * nvec, nvec);
        if (threadIdx.x == 0) scales[r] = row.scale;
    }
}

// Lanes of a row: as few as hold it with `most` pieces each, or with eight where a workgroup
// does not hold it with two (512 tokens, H 20480, top-8: 20.6 us, with three of eight used 22.5).
int lanes_of(int nvec, int most) {
    if (nvec > 2 * kMaxThreads) most = 8;
    const int lanes = (nvec + most - 1) / most;
    const int threads = (lanes + kWave - 1) / kWave * kWave;
    return threads < kMaxThreads ? threads : kMaxThreads;
}

}  // namespace

hipError_t launch_dispatch_i8(const ep_problem& p, const void* x, const int32_t* slot_of,
                              void* recv_q, float* recv_scales, hipStream_t stream) {
    const int T = p.num_tokens;
    if (T == 0) return hipSuccess;
    const int64_t R = p.capacity == 0 ? static_cast<int64_t>(T) * p.num_topk
                                      : static_cast<int64_t>(p.num_experts) * p.capacity;
    const int nvec = p.hidden / 8;
    const int threads = lanes_of(nvec, T < 1024 ? 1 : 2);
    const auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(T), dim3(threads), 0, stream, static_cast<const u32x4*>(x),
                           nvec, p.num_topk, slot_of, R, static_cast<u32x2*>(recv_q), recv_scales);
    };
    const int vpl = (nvec + threads - 1) / threads;
    if (vpl == 1)
        go(dispatch_i8_kernel<1>);
    else if (vpl == 2)
        go(dispatch_i8_kernel<2>);
    else
        go(dispatch_i8_kernel<8>);
    return hipGetLastError();
}

hipError_t launch_quant_rows(const ep_problem& p, int K, const void* rows,
                             const ep_layout_t& layout, int8_t* q, float* scales,
                             hipStream_t stream) {
    const int64_t entries = static_cast<int64_t>(p.num_tokens) * p.num_topk;
    const int64_t R = p.capacity == 0 ? entries : static_cast<int64_t>(p.num_experts) * p.capacity;
    if (entries == 0) return hipSuccess;
    const int nvec = K / 8;
    const int threads = lanes_of(nvec, 2);
    // a workgroup per row, up to 2^20; with a capacity twice as many per expert as it has rows
    // in the mean, up to 1024
    dim3 grid;
    if (p.capacity > 0) {
        int64_t per = 2 * (entries / p.num_experts) + 1;
        if (per > p.capacity) per = p.capacity;
        if (per > 1024) per = 1024;
        grid = dim3(static_cast<unsigned>(per), p.num_experts);
    } else {
        grid = dim3(static_cast<unsigned>(R < (1 << 20) ? R : 1 << 20));
    }
    const auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(threads), 0, stream, static_cast<const u32x4*>(rows),
                           nvec, layout.count, layout.offset, p.num_experts, p.capacity, R,
                           reinterpret_cast<u32x2*>(q), scales);
    };
    const int vpl = (nvec + threads - 1) / threads;
    if (vpl == 1)
        go(quant_rows_kernel<1>);
    else if (vpl == 2)
        go(quant_rows_kernel<2>);
    else
        go(quant_rows_kernel<8>);
    return hipGetLastError();
}

}  // namespace ep
