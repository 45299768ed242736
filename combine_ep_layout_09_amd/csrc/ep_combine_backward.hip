// ep_combine_backward.hip -- gradients of the combine, with dropout, in the expert
// rows and the routing weights.
//
//   g[t]            = kept ? dy[t] * f : 0          (f = 1 / (1 - p))
//   d_expert_out[s] = kept ? w[t, j] g[t] : 0       s the receive row of entry (t, j)
//   d_weights[t, j] = <g[t], expert_out[s]>         over the kept channels
//
// Dropped channels are selected out of all three: the output does not depend on what
// is there, so that an infinite weight or expert row there leaves no 0 * inf.
//
// A workgroup takes a token.  A lane holds VPL 16-byte pieces of dy with the
// dropped channels zeroed, made once for all k entries.  Entries are taken in batches of
// KB: the loads of their expert rows are issued together, with no branches, and
// the mask is made while they are under way.  Each expert row is read once,
// each gradient row written once.
//
// Memory bounds it, as many bytes written as read: 4096 tokens, H 7168, top-8, p 0.1:
// 184 to 205 us by box, 5.0 to 5.4 TB/s; the loads alone take 111, the stores alone 116.  Fewer lanes
// with more pieces each (VPL 2 to 7: 199 to 208), batches of 512 to 2048 tokens a launch
// (203 to 225) and stores that stay in the caches (207) were slower.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ep_dropout_dev.h"
#include "ep_internal.h"

namespace ep {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kMaxThreads = 1024;

template <int CTRL>
__device__ __forceinline__ float moved(float v) {
    return __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_update_dpp(
        0, static_cast<int>(__float_as_uint(v)), CTRL, 0xf, 0xf, false)));
}

// One step of wave_sums: each lane keeps one value of a pair, by bit BIT of its
// number, and gives the other to the lane across, which keeps that.
template <int N, int BIT, int CTRL>
__device__ __forceinline__ void halve(float (&v)[8], int lane) {
    const bool odd = lane >> BIT & 1;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const float keep = odd ? v[2 * i + 1] : v[2 * i], give = odd ? v[2 * i] : v[2 * i + 1];
        v[i] = keep + moved<CTRL>(give);
    }
}

// Sums over a wave of eight values per lane, in a third of the instructions that eight
// sums take: lane l returns the sum of value (l / 8 & 1) + 2 (l / 4 & 1) + 4 (l / 2 & 1).
__device__ __forceinline__ float wave_sums(float (&v)[8]) {
    const int lane = threadIdx.x % kWave;
    halve<8, 3, 0x140>(v, lane);  // lane ^ 15
    halve<4, 2, 0x141>(v, lane);  // lane ^ 7
    halve<2, 1, 0x1b>(v, lane);   // lane ^ 3
    float s = v[0] + moved<0xb1>(v[0]);  // lane ^ 1
    s += __shfl_xor(s, 16, kWave);
    return s + __shfl_xor(s, 32, kWave);
}

template <int VPL, int KB, bool WIDE>
__global__ __launch_bounds__(kMaxThreads) void combine_backward_kernel(
        const u32x4* __restrict__ dy, const u32x4* __restrict__ eo, int nvec, int k,
        const int32_t* __restrict__ slot_of, int64_t R, const float* __restrict__ weights,
        DropArgs drop, u32x4* __restrict__ deo, float* __restrict__ dw) {
    __shared__ float s_part[kMaxThreads / kWave][kMaxTopk];
    const int t = blockIdx.x;
    const int32_t* slots = slot_of + static_cast<int64_t>(t) * k;
    const float* w = weights + static_cast<int64_t>(t) * k;
    const int wave = threadIdx.x / kWave;
    // WIDE: rows of more than two pieces per lane, a part after the other.  (512 tokens, H 16392,
    // top-8: 61 us; a lane with eight pieces, which do not fit its registers, 203; H 65536, top-4
    // 118 and 232; eight entries at a time 63 and 129.)
    for (int v0 = 0; v0 < nvec; v0 += VPL * blockDim.x) {
        int v[VPL];  // lanes past the end redo the last piece, and add and store nothing
        bool here[VPL];
        u32x4 dyv[VPL];
        float g[VPL][8];
        uint32_t pass[VPL][4];  // ones at the kept channels' halves of a piece's words
#pragma unroll
        for (int u = 0; u < VPL; ++u) {
            const int at = v0 + threadIdx.x + u * blockDim.x;
            here[u] = at < nvec;
            v[u] = min(at, nvec - 1);
            dyv[u] = __builtin_nontemporal_load(dy + static_cast<int64_t>(t) * nvec + v[u]);
        }
        for (int j0 = 0; j0 < k; j0 += KB) {
            bool ok[KB];
            float wj[KB];
            int64_t row[KB];
            u32x4 e[KB][VPL];
#pragma unroll
            for (int jj = 0; jj < KB; ++jj) {
                const int j = j0 + jj;
                const int32_t slot = j < k ? slots[j] : -1;
                ok[jj] = slot >= 0 && slot < R;
                wj[jj] = ok[jj] ? w[j] : 0.0f;
                // an entry without a slot loads row 0, whose products are dropped
                row[jj] = static_cast<int64_t>(ok[jj] ? slot : 0) * nvec;
            }
            if (dw != nullptr) {
#pragma unroll
                for (int jj = 0; jj < KB; ++jj)
#pragma unroll
                    for (int u = 0; u < VPL; ++u)
                        e[jj][u] = __builtin_nontemporal_load(eo + row[jj] + v[u]);
            } else {
#pragma unroll
                for (int jj = 0; jj < KB; ++jj)
#pragma unroll
                    for (int u = 0; u < VPL; ++u) e[jj][u] = u32x4{0, 0, 0, 0};
            }
            __builtin_amdgcn_sched_barrier(0);  // all loads first
            if (j0 == 0) {
#pragma unroll
                for (int u = 0; u < VPL; ++u) {
                    const uint32_t kept = here[u] ? dropout::keep8(drop, t, v[u]) : 0u;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t word = dyv[u][i / 2];
                        const float f = (i % 2 == 0 ? bf16_lo(word) : bf16_hi(word)) * drop.factor;
                        g[u][i] = kept >> i & 1 ? f : 0.0f;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        pass[u][i] = (kept >> 2 * i & 1 ? 0xffffu : 0u) | (kept >> 2 * i & 2 ? 0xffff0000u : 0u);
                }
            }
            float sums[8];
#pragma unroll
            for (int jj = 0; jj < 8; ++jj) sums[jj] = 0.0f;
#pragma unroll
            for (int jj = 0; jj < KB; ++jj) {
#pragma unroll
                for (int u = 0; u < VPL; ++u) {
                    u32x4 d;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float lo = g[u][2 * i], hi = g[u][2 * i + 1];
                        const uint32_t word = e[jj][u][i] & pass[u][i];
                        sums[jj] = fmaf(lo, bf16_lo(word), sums[jj]);
                        sums[jj] = fmaf(hi, bf16_hi(word), sums[jj]);
                        d[i] = pack_bf16(lo * wj[jj], hi * wj[jj]) & pass[u][i];
                    }
                    if (ok[jj] && here[u]) __builtin_nontemporal_store(d, deo + row[jj] + v[u]);
                }
                if (!ok[jj]) sums[jj] = 0.0f;
            }
            if (dw != nullptr) {
                const float sum = wave_sums(sums);
                const int lane = threadIdx.x % kWave;
                const int j = j0 + (lane >> 3 & 1) + (lane >> 1 & 2) + (lane << 1 & 4);
                if (lane < 16 && lane % 2 == 0 && j < k && j - j0 < KB)
                    s_part[wave][j] = WIDE && v0 > 0 ? s_part[wave][j] + sum : sum;
            }
        }
        if (!WIDE) break;
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
    // Two pieces per lane where a row is more than two waves' and there are fewer than
    // 2048 tokens, from five entries on: half the waves, each with twice as much in flight (517 tokens,
    // H 4096, top-6: 12.7 us with one piece, 10.2 with two; 1000, H 2048: 11.4 and
    // 10.0; 1000, H 4096, top-8: 26.9 and 25.8; but 2000, H 4096, top-6: 42.3 and 43.5).
    const int k = p.num_topk;
    const int parts = (nvec + 2 * kMaxThreads - 1) / (2 * kMaxThreads);
    const int vpl = nvec > kMaxThreads || (T < 2048 && nvec > 2 * kWave && k >= 5) ? 2 : 1;
    const int lanes = (nvec + vpl * parts - 1) / (vpl * parts);
    const int threads = (lanes + kWave - 1) / kWave * kWave;
    const auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(T), dim3(threads), 0, stream, static_cast<const u32x4*>(dy),
                           static_cast<const u32x4*>(expert_out), nvec, k, slot_of, R,
                           topk_weights, drop, static_cast<u32x4*>(d_expert_out), d_weights);
    };
    if (parts > 1)
        go(combine_backward_kernel<2, 4, true>);
    else if (vpl == 2 && k <= 4)
        go(combine_backward_kernel<2, 4, false>);
    else if (vpl == 2 && k <= 6)
        go(combine_backward_kernel<2, 6, false>);
    else if (vpl == 2)
        go(combine_backward_kernel<2, 8, false>);
    else if (k <= 2)
        go(combine_backward_kernel<1, 2, false>);
    else if (k <= 4)
        go(combine_backward_kernel<1, 4, false>);
    else if (k <= 6)
        go(combine_backward_kernel<1, 6, false>);
    else
        go(combine_backward_kernel<1, 8, false>);
    return hipGetLastError();
}

}  // namespace ep
