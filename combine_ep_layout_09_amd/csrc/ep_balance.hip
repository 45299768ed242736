// ep_balance.hip -- the balance loss of a routing with its per-expert counts.
//
//   p[t, e]   probability of expert e for token t (softmax, or sigmoid scores
//             over their sum)
//   c[s, e]   entries of sequence s's tokens that name expert e
//   P[s, e]   mean of p[t, e] over the n_s tokens of the sequence
//   loss = coef / B * sum_s sum_e E / (k n_s) c[s, e] P[s, e]
//
// First kernel: a workgroup per run of consecutive tokens of one sequence, one
// pass of its 16 waves where the batch allows (64 tokens at up to 256 experts:
// about a workgroup per CU), adds its tokens' probabilities per expert in
// registers, its entries in an LDS histogram, and writes both as one row of
// partial sums.  Second kernel: the rows are added in order, in fp64.  Up to
// kOneGroup partial sums one workgroup does it, and the loss with them; above
// that many, of which the last to finish adds their parts of the loss, in
// order.  No sum depends on the order in which workgroups run.  16384 x 256 fp32
// in four sequences: the call 14.5 us (8.6 and 7.0 us for the kernels in a trace,
// which times each alone), with a third kernel for the parts 16.2; with one
// workgroup for all 65536 partial sums 38.  65536 tokens in one sequence: 27.6 us,
// 2.4 TB/s; 2^18: 66.7, 4.0 TB/s.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ep_internal.h"
#include "ep_route_dev.h"

namespace ep {
namespace {

using namespace route;

constexpr int kSum = 1024;     // threads of the first kernel
constexpr int kFinish = 1024;  // and of the second
constexpr int64_t kMostGroups = kFinish;  // workgroups of the second: a thread adds each part
// Experts up to which 16 lanes take a token: at 512, where a lane would hold 32,
// 16000 tokens take 24.7 us with 16 lanes, 23.5 with 64, 256 tokens 12.5 and 9.9.
constexpr int kSixteen = 256;
constexpr int kRowsWanted = 256;
// Passes of a workgroup: a lane adds one fp32 probability per pass, and those of
// equal tokens all round the same way (2048 passes of 17 equal experts: the means were
// off by 221 units of 2^-24, with 32 by 12).  Longer sequences get more workgroups; their rows are added in fp64.
constexpr int64_t kMostPasses = 32;
constexpr int64_t kOneGroup = 8192;

struct Geometry {
    int runs;        // runs of tokens per sequence
    int run_tokens;  // tokens per run
    int64_t probs, hist, live, part, done, bytes;  // workspace offsets and size
};

Geometry geometry(int T, int E, int B) {
    Geometry g;
    const int64_t len = T / B;
    const int64_t pass = kSum / token_shape(E, kSixteen).lpt;  // tokens of a workgroup's pass
    int64_t runs = (kRowsWanted + B - 1) / B;
    const int64_t most = (len + pass - 1) / pass;
    const int64_t least = (most + kMostPasses - 1) / kMostPasses;
    if (runs < least) runs = least;
    if (runs > most) runs = most;
    if (runs < 1) runs = 1;
    g.run_tokens = static_cast<int>((len + runs - 1) / runs);
    g.runs = g.run_tokens ? static_cast<int>((len + g.run_tokens - 1) / g.run_tokens) : 1;
    const auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
    const int64_t rows = static_cast<int64_t>(B) * g.runs;
    g.probs = 0;
    g.hist = up(g.probs + rows * E * 4);
    g.live = up(g.hist + rows * E * 4);
    g.part = up(g.live + rows * 4);
    g.done = g.part + kMostGroups * 8;
    g.bytes = up(g.done + 4);
    return g;
}

template <int LPT, int VPL, bool BF16>
__global__ __launch_bounds__(kSum) void balance_sum_kernel(RouteArgs a, const int32_t* topk_idx,
                                                           const uint8_t* valid, int runs,
                                                           int run_tokens, float* probs,
                                                           int32_t* hist, int32_t* live_rows,
                                                           uint32_t* done) {
    constexpr int kTokens = kSum / LPT;
    constexpr int kWidth = LPT * VPL;
    constexpr int kSel = kMaxTopk > LPT ? kMaxTopk / LPT : 1;
    constexpr int kWaves = kSum / kWave;
    __shared__ float sums[kWaves][kWidth];
    __shared__ int32_t counts[kWidth];
    __shared__ int32_t live_count;
    const int lane = threadIdx.x % LPT;
    const Experts own = spread<LPT, VPL, BF16>(lane);
    const int slot = threadIdx.x / LPT;
    const int wave = threadIdx.x / kWave;
    const int E = a.num_experts, k = a.num_topk;
    const int64_t seq = blockIdx.x / runs;
    const int run = blockIdx.x % runs;
    const int begin = run * run_tokens;
    const int end = min(begin + run_tokens, a.seq_len);
    const int64_t t0 = seq * a.seq_len;
    for (int e = threadIdx.x; e < kWidth; e += kSum) counts[e] = 0;
    if (threadIdx.x == 0) live_count = 0;
    __syncthreads();

    float acc[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) acc[i] = 0.0f;
    int mine = 0;
    for (int base = begin; base < end; base += kTokens) {  // the same count for every wave
        const int at = base + slot;
        const bool inside = at < end;
        const int64_t t = inside ? t0 + at : t0;
        float x[VPL], z[VPL], slope[VPL], total, top;
        load_logits<VPL, BF16>(a.logits, t * a.stride, inside ? E : 0, own, a.pieces, x);
        int ids[kSel];
#pragma unroll
        for (int q = 0; q < kSel; ++q) {
            const int j = q * LPT + lane;
            ids[q] = inside && j < k ? topk_idx[t * k + j] : -1;
        }
        const bool live = inside && (valid == nullptr || valid[t] != 0);
        if (live && lane == 0) ++mine;
#pragma unroll
        for (int q = 0; q < kSel; ++q)
            if (live && ids[q] >= 0 && ids[q] < E) atomicAdd(&counts[ids[q]], 1);
        scores<LPT, VPL>(x, a.sigmoid, z, slope, total, top);
        const float r = live && total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) acc[i] += z[i] * r;
    }
    // the wave's tokens (4 with 16 lanes each), then the waves in order
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        if constexpr (LPT == 16) {
            uint2 p = swap16(__float_as_uint(acc[i]));
            acc[i] = __uint_as_float(p.x) + __uint_as_float(p.y);
            p = swap32(__float_as_uint(acc[i]));
            acc[i] = __uint_as_float(p.x) + __uint_as_float(p.y);
        }
        if (LPT == 64 || threadIdx.x % kWave < 16) sums[wave][expert<VPL, BF16>(own, i)] = acc[i];
    }
    if (mine) atomicAdd(&live_count, mine);
    __syncthreads();
    const int64_t out = static_cast<int64_t>(blockIdx.x) * E;
    for (int e = threadIdx.x; e < E; e += kSum) {
        float s = 0.0f;
#pragma unroll
        for (int q = 0; q < kWaves; ++q) s += sums[q][e];
        probs[out + e] = s;
        hist[out + e] = counts[e];
    }
    if (threadIdx.x == 0) live_rows[blockIdx.x] = live_count;
    if (blockIdx.x == 0 && threadIdx.x == 0) *done = 0;  // for the second kernel
}

// Sum over the workgroup of one double per thread, in thread 0.
__device__ __forceinline__ double group_sum(double v, double* lds) {
#pragma unroll
    for (int d = kWave / 2; d > 0; d /= 2) v += __shfl_down(v, d, kWave);
    if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = v;
    __syncthreads();
    v = threadIdx.x < kFinish / kWave ? lds[threadIdx.x] : 0.0;
#pragma unroll
    for (int d = kFinish / kWave / 2; d > 0; d /= 2) v += __shfl_down(v, d, kWave);
    return v;
}

// Outputs are the (sequence, expert) pairs in order.  A workgroup takes `cols`
// of them at a time (a power of two, 32 to kFinish), kFinish / cols threads
// each adding every kFinish / cols-th row of partial sums.  Every workgroup
// writes its part of the loss; the one that is last to count itself in `done`
// adds them in order.
__global__ __launch_bounds__(kFinish) void balance_mean_kernel(
    int E, int cols, int runs, int64_t outputs, const float* probs, const int32_t* hist,
    const int32_t* live_rows, int32_t* counts, float* mean_prob, int32_t* num_valid, double* part,
    uint32_t* done, double factor, float* loss) {
    __shared__ double sum_s[kFinish];
    __shared__ int32_t sum_c[kFinish], sum_n[kFinish];
    const int col = threadIdx.x % cols, slice = threadIdx.x / cols, slices = kFinish / cols;
    double term = 0.0;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * cols; base < outputs;
         base += static_cast<int64_t>(gridDim.x) * cols) {
        const uint32_t o = static_cast<uint32_t>(base) + col;  // B * E is at most 2^30
        const int64_t seq = o / static_cast<uint32_t>(E);
        const int e = static_cast<int>(o % static_cast<uint32_t>(E));
        double s = 0.0;
        int c = 0, n = 0;
        if (o < outputs) {
            const int64_t row = seq * runs;
#pragma unroll 16
            for (int r = slice; r < runs; r += slices) {
                s += static_cast<double>(probs[(row + r) * E + e]);
                c += hist[(row + r) * E + e];
                n += live_rows[row + r];
            }
        }
        if (slices > 1) {
            __syncthreads();
            sum_s[threadIdx.x] = s;
            sum_c[threadIdx.x] = c;
            sum_n[threadIdx.x] = n;
            __syncthreads();
        }
        if (slice == 0 && o < outputs) {
            for (int q = 1; q < slices; ++q) {
                s += sum_s[q * cols + col];
                c += sum_c[q * cols + col];
                n += sum_n[q * cols + col];
            }
            const double mean = n ? s / n : 0.0;
            counts[o] = c;
            mean_prob[o] = static_cast<float>(mean);
            if (n) term += mean * c / n;
            if (e == 0) num_valid[seq] = n;
        }
    }
    __syncthreads();
    double p = group_sum(term, sum_s);
    if (gridDim.x > 1) {
        __shared__ bool last;
        if (threadIdx.x == 0) {
            __hip_atomic_store(&part[blockIdx.x], p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            last = __hip_atomic_fetch_add(done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
                   gridDim.x - 1;
        }
        __syncthreads();
        if (!last) return;
        p = threadIdx.x < gridDim.x ? __hip_atomic_load(&part[threadIdx.x], __ATOMIC_RELAXED,
                                                        __HIP_MEMORY_SCOPE_AGENT)
                                    : 0.0;
        p = group_sum(p, sum_s);
    }
    if (threadIdx.x == 0) loss[0] = static_cast<float>(p * factor);
}

template <int LPT, int VPL>
void launch_sum(const RouteArgs& a, const BalanceArgs& b, const Geometry& g, char* ws,
                hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(a.num_seqs) * g.runs);
    float* probs = reinterpret_cast<float*>(ws + g.probs);
    int32_t* hist = reinterpret_cast<int32_t*>(ws + g.hist);
    int32_t* live = reinterpret_cast<int32_t*>(ws + g.live);
    uint32_t* done = reinterpret_cast<uint32_t*>(ws + g.done);
    if (a.bf16)
        hipLaunchKernelGGL((balance_sum_kernel<LPT, VPL, true>), grid, dim3(kSum), 0, stream, a,
                           b.topk_idx, b.valid, g.runs, g.run_tokens, probs, hist, live, done);
    else
        hipLaunchKernelGGL((balance_sum_kernel<LPT, VPL, false>), grid, dim3(kSum), 0, stream, a,
                           b.topk_idx, b.valid, g.runs, g.run_tokens, probs, hist, live, done);
}

}  // namespace

int64_t balance_workspace_bytes(int num_tokens, int num_experts, int num_seqs) {
    return geometry(num_tokens, num_experts, num_seqs).bytes;
}

hipError_t launch_balance(const RouteArgs& a, const BalanceArgs& b, void* workspace,
                          hipStream_t stream) {
    const Geometry g = geometry(a.num_tokens, a.num_experts, a.num_seqs);
    char* ws = static_cast<char*>(workspace);
    const TokenShape s = token_shape(a.num_experts, kSixteen);
    if (s.lpt == 16) {
        switch (s.vpl) {
            case 1: launch_sum<16, 1>(a, b, g, ws, stream); break;
            case 2: launch_sum<16, 2>(a, b, g, ws, stream); break;
            case 4: launch_sum<16, 4>(a, b, g, ws, stream); break;
            case 8: launch_sum<16, 8>(a, b, g, ws, stream); break;
            default: launch_sum<16, 16>(a, b, g, ws, stream); break;
        }
    } else if (s.vpl == 8) {
        launch_sum<64, 8>(a, b, g, ws, stream);
    } else {
        launch_sum<64, 16>(a, b, g, ws, stream);
    }
    double* part = reinterpret_cast<double*>(ws + g.part);
    const int64_t outputs = static_cast<int64_t>(a.num_seqs) * a.num_experts;
    // One workgroup up to kOneGroup partial sums (4096 of them: 4.5 us, 6.4 with
    // many; 16384: 10.1 and 7.1); above that 32 outputs and 32 slices of rows per
    // workgroup (256 rows of 256 outputs: 8.6 us, with 64 outputs 12.4).
    const bool one = outputs * g.runs <= kOneGroup;
    int cols = 32;
    while (one && cols < kFinish && cols < outputs) cols *= 2;
    int64_t groups = one ? 1 : (outputs + cols - 1) / cols;
    groups = groups < kMostGroups ? groups : kMostGroups;
    const double factor = static_cast<double>(b.coef) / a.num_seqs * a.num_experts / a.num_topk;
    hipLaunchKernelGGL(balance_mean_kernel, dim3(static_cast<unsigned>(groups)), dim3(kFinish), 0,
                       stream, a.num_experts, cols, g.runs, outputs,
                       reinterpret_cast<float*>(ws + g.probs),
                       reinterpret_cast<int32_t*>(ws + g.hist),
                       reinterpret_cast<int32_t*>(ws + g.live), b.counts, b.mean_prob, b.num_valid,
                       part, reinterpret_cast<uint32_t*>(ws + g.done), factor, b.loss);
    return hipGetLastError();
}

}  // namespace ep
