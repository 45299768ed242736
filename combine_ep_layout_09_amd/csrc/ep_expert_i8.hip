// ep_expert_i8.hip -- the experts' products with 8-bit integer weights on the
// dispatched rows.
//
//   y[r, n] = (sum_k q[r, k] w[e, n, k]) * row_scale[r] * scale[e, n]
//
// for the rows r of expert e; optionally the gated activation
// silu(y[r, n]) * y[r, N + n]; one rounding to bf16.  The sums are exact: 65536
// products of at most 2^14 stay below 2^31, so they do not depend on the order
// or on how the channels are split.
//
// The channels of an MFMA may be taken in any order if both operands agree.
// Lane l multiplies row l % 16 and the 16 channels, 16 bytes, at piece l / 16 of
// a chunk of 64: codes are used as they lie in memory.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ep_device.h"
#include "ep_expert_dev.h"
#include "ep_internal.h"

namespace ep {
namespace {

using namespace expert;

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

constexpr int kTiles = 4;            // 16-row weight tiles of a wave
constexpr int kRows = 16 * kTiles;   // weight rows of a wave
constexpr int kStep = 128;           // channels of a step: two chunks
constexpr int kRedRow = kRows + 4;   // words

struct Args {
    const uint8_t* rows;      // int8 [R, K]
    const float* row_scales;  // [R]
    const int32_t* count;
    const uint8_t* weights;   // int8 [E, n2, K]
    const float* scales;      // [E, n2]
    uint16_t* out;            // bf16 [R, N]
    int64_t num_rows;         // R
    int32_t num_experts, capacity, K, N;
};

__device__ __forceinline__ i32x4 mfma(const u32x4& a, const u32x4& b, const i32x4& c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a),
                                                 __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

__device__ __forceinline__ float scaled(int32_t sum, float row, float channel) {
    return static_cast<float>(sum) * row * channel;
}

// One step's operands of a wave.
struct Stage {
    u32x4 w[2][kTiles];
    u32x4 x[2];
};

// Few rows per expert: the weights are the traffic and are read once.  A
// workgroup takes 64 weight rows of one expert against up to 16 rows; its WAVES
// waves take steps of 128 channels in turns and add their sums in LDS.  A load
// covers 8 weight rows x 128 bytes, whole cache lines that are not kept; two
// chunks change places across lanes afterwards (pair_chunks).  GATED: tiles 0, 1 are
// rows n of the gate half and tiles 2, 3 rows N + n.
template <int WAVES, bool GATED>
__global__ __launch_bounds__(WAVES* kWave, 4) void expert_i8_kernel(Args a) {
    constexpr int kThreads = WAVES * kWave;
    constexpr int MC = 16;
    constexpr int kOut = GATED ? kRows / 2 : kRows;  // outputs per workgroup
    __shared__ __attribute__((aligned(16))) int32_t red[WAVES][MC][kRedRow];

    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r16 = lane % 16, group = lane / 16;
    const uint32_t K = a.K;
    const int N = a.N;
    const int n0 = blockIdx.x * kOut;
    const int here = N - n0 < kOut ? N - n0 : kOut;  // outputs of this workgroup

    const Found f = find_tile<MC>(a, [](uint32_t) { return blockIdx.z * gridDim.y + blockIdx.y; });
    if (f.expert < 0) return;
    const int m0 = f.tile * MC;
    const int rows_here = f.count - m0 < MC ? f.count - m0 : MC;
    if (rows_here <= 0) return;
    const int64_t row0 = f.start + m0;

    const int64_t w_row = static_cast<int64_t>(f.expert) * (GATED ? 2 * N : N) + n0;
    const int64_t up_row = w_row + (GATED ? N : 0);
    const auto w_view = view(a.weights + w_row * K, here * K);
    const auto up_view = view(a.weights + up_row * K, here * K);
    const auto x_view = view(a.rows + row0 * K, rows_here * K);
    const uint32_t w_col = lane / 8 % 2 * 64 + group * 16, x_col = group * 16;

    i32x4 acc[kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) acc[t] = i32x4{0, 0, 0, 0};

    const auto load = [&](uint32_t c, Stage& s) {  // channels c .. c + 127; zeros past the end
        const uint32_t at = c + w_col < K ? lane % 8 * K + w_col : kNowhere;
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                s.w[i][t] = load16<true>(t * 16 < kOut ? w_view : up_view,
                                         at + (t * 16 % kOut + i * 8) * K, c);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            s.x[h] = load16<false>(x_view, c + h * 64 + x_col < K ? r16 * K + x_col : kNowhere,
                                   c + h * 64);
    };
    Stage s;
    uint32_t c = wave * kStep;
    load(c, s);
    while (c < K) {
#pragma unroll
        for (int t = 0; t < kTiles; ++t) pair_chunks(s.w[0][t], s.w[1][t]);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int t = 0; t < kTiles; ++t) acc[t] = mfma(s.w[h][t], s.x[h], acc[t]);
        c += WAVES * kStep;
        if (c < K) load(c, s);
    }

    // lane l holds weight rows 4 * (l / 16) .. + 3 of a tile against row l % 16
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
        *reinterpret_cast<i32x4*>(&red[wave][r16][t * 16 + group * 4]) = acc[t];
    __syncthreads();
    for (int i = threadIdx.x; i < rows_here * kOut; i += kThreads) {
        const int m = i / kOut, n = i % kOut;
        if (n >= here) continue;
        int32_t sum = 0, up_sum = 0;
#pragma unroll
        for (int v = 0; v < WAVES; ++v) {
            sum += red[v][m][n];
            if constexpr (GATED) up_sum += red[v][m][kRows / 2 + n];
        }
        const float row_scale = a.row_scales[row0 + m];
        float y = scaled(sum, row_scale, a.scales[w_row + n]);
        if constexpr (GATED) y = y / (1.0f + expf(-y)) * scaled(up_sum, row_scale, a.scales[up_row + n]);
        a.out[(row0 + m) * N + n0 + n] = static_cast<uint16_t>(f32_to_bf16_rne(y));
    }
}

template <int WAVES, bool GATED>
void launch_few(const Args& a, int64_t tiles, hipStream_t stream) {
    const int outs = GATED ? kRows / 2 : kRows;
    const int64_t y = tiles < 32768 ? tiles : 32768;
    const dim3 grid((a.N + outs - 1) / outs, static_cast<unsigned>(y),
                    static_cast<unsigned>((tiles + y - 1) / y));
    hipLaunchKernelGGL((expert_i8_kernel<WAVES, GATED>), grid, dim3(WAVES * kWave), 0, stream, a);
}

int64_t padded(int64_t bytes) { return (bytes + 255) / 256 * 256; }

int64_t recv_rows(const ep_problem& p) {
    return p.capacity == 0 ? static_cast<int64_t>(p.num_tokens) * p.num_topk
                           : static_cast<int64_t>(p.num_experts) * p.capacity;
}

}  // namespace

int64_t expert_i8_workspace_bytes(const ep_problem& p, const ep_expert_i8_t& mm) {
    if (mm.in_format != 0) return 0;
    const int64_t R = recv_rows(p);
    return padded(R * mm.in_features) + padded(R * 4);
}

hipError_t launch_expert_i8(const ep_problem& p, const ep_expert_i8_t& mm, const void* rows,
                            const float* row_scales, const ep_layout_t& layout,
                            const int8_t* weights, const float* scales, void* out,
                            void* workspace, hipStream_t stream) {
    const int64_t entries = static_cast<int64_t>(p.num_tokens) * p.num_topk;
    const int64_t held = static_cast<int64_t>(p.num_experts) * p.capacity;
    const int64_t filled = p.capacity > 0 && held < entries ? held : entries;
    if (filled == 0) return hipSuccess;
    Args a;
    a.num_rows = recv_rows(p);
    if (mm.in_format == 0) {
        auto* q = static_cast<int8_t*>(workspace);
        auto* s = reinterpret_cast<float*>(q + padded(a.num_rows * mm.in_features));
        const hipError_t err = launch_quant_rows(p, mm.in_features, rows, layout, q, s, stream);
        if (err != hipSuccess) return err;
        rows = q;
        row_scales = s;
    }
    a.rows = static_cast<const uint8_t*>(rows);
    a.row_scales = row_scales;
    a.count = layout.count;
    a.weights = reinterpret_cast<const uint8_t*>(weights);
    a.scales = scales;
    a.out = static_cast<uint16_t*>(out);
    a.num_experts = p.num_experts;
    a.capacity = p.capacity;
    a.K = mm.in_features;
    a.N = mm.out_features;
    // Row tiles: no more than one per expert that can have rows, plus one per
    // full tile.
    const int64_t experts = p.num_experts < filled ? p.num_experts : filled;
    const int64_t tiles = experts + filled / 16;
    if (mm.activation == 1)
        launch_few<4, true>(a, tiles, stream);
    else
        launch_few<4, false>(a, tiles, stream);
    return hipGetLastError();
}

}  // namespace ep
