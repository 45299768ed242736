// ep_expert_w4.hip -- the experts' products with 4-bit weights on the
// dispatched rows.
//
//   y[r, n] = sum_k x[r, k] * e2m1(code[e, n, k]) * 2^(scale[e, n, k / 32] - 127)
//
// for the rows r of expert e, summed in fp32; optionally the gated activation
// silu(y[r, n]) * y[r, N + n]; one rounding to bf16.
//
// A decode batch gives each expert a handful of rows, so the weights, 17/32
// byte each, are the traffic and every one should be read once.  A workgroup
// takes 64 weight rows of one expert against up to 16 * MT rows; its four
// waves split the input channels in turns of 128 and add their sums in LDS, in
// wave order.  Weights and rows meet in bf16 MFMA: every E2M1 value times a
// power of two is a bf16, and v_cvt_scalef32_pk_bf16_fp4 makes two of them
// from one byte, so the products are those of the formula and only the sum
// rounds.  (The MFMA that takes E2M1 itself keeps fewer bits of its partial
// sums than fp32: 3e-5 of the result on random data.)
//
// The channels of an MFMA may be taken in any order if both operands agree.
// Lane l holds weight row l % 16 and the 16 bytes, 32 channels, one scale, at
// block l / 16 of the 128: a wave reads the codes as they lie in memory, row
// by row, and needs neither a shuffle nor LDS.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ep_internal.h"
#include "ep_device.h"

namespace ep {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kTiles = 4;            // 16-row weight tiles per workgroup
constexpr int kRows = 16 * kTiles;   // weight rows per workgroup
constexpr int kStep = 128;           // channels per wave and step
constexpr int kSegment = 8192;       // channels whose scales LDS holds at a time
constexpr int kSegSteps = kSegment / kStep;
constexpr int kScaleRow = kSegment / 32 + 4;  // bytes; a step's four scales of 16
                                              // consecutive rows are in 16 banks
constexpr int kRowScaleRow = kSegSteps + 1;   // floats
constexpr int kRedRow = kRows + 4;            // floats

struct Args {
    const uint8_t* rows;      // bf16 or E4M3FN [R, K]
    const void* row_scales;   // fp32 or UE8M0 [R, K / 128]
    const int32_t* count;
    const int32_t* offset;
    const uint8_t* codes;     // [E, n2, K / 2]
    const uint8_t* scales;    // [E, n2, K / 32]
    uint16_t* out;            // bf16 [R, N]
    int64_t tiles;            // row tiles at most
    int64_t num_rows;         // R
    int32_t num_experts, capacity, K, N;
};

union Frag {
    uint32_t u[4];
    u32x4 w;
    bf16x8 v;
};

__device__ __forceinline__ float exponent_value(uint32_t byte) {
    // 2^(byte - 127); byte 0 is the subnormal 2^-127, 255 is NaN
    return byte == 0 ? __uint_as_float(0x00400000u)
                     : byte == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float(byte << 23);
}

// Eight codes of one word -> bf16, scaled by the power of two in s's exponent
// field (field 0 stands for 2^-127, 255 gives NaN: the UE8M0 values).
__device__ __forceinline__ bf16x8 weights8(uint32_t w, float s) {
    Frag f;
    f.u[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
    f.u[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
    f.u[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
    f.u[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
    return f.v;
}

// Eight E4M3FN codes -> bf16, exact.
__device__ __forceinline__ bf16x8 rows8(uint32_t lo, uint32_t hi) {
    Frag f;
    f.u[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false));
    f.u[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true));
    f.u[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false));
    f.u[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true));
    return f.v;
}

// Bounded view of `bytes` bytes at p: loads past its end give 0 and touch
// nothing.  p and bytes are the same in every lane.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t view(const void* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00020000);
}
constexpr uint32_t kNowhere = 0x7fffff00u;  // past the end of every view
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t at, uint32_t step) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at, step, 0));
}

// Rows of expert e: their number, and the first one in *start.
__device__ __forceinline__ int expert_rows(const Args& a, int e, int64_t* start) {
    int64_t s, n = a.count[e];
    if (a.capacity > 0) {
        s = static_cast<int64_t>(e) * a.capacity;
        n = n < a.capacity ? n : a.capacity;
    } else {
        // a layout of another problem must not lead outside the rows
        s = a.offset[e];
        s = s < 0 ? 0 : s;
        n = n < a.num_rows - s ? n : a.num_rows - s;
    }
    *start = s;
    return n > 0 ? static_cast<int>(n) : 0;
}

// The expert and row tile number `want` names: experts with rows, in order,
// each with one tile per MC rows.
template <int THREADS, int MC>
struct Finder {
    int first[THREADS / kWave];   // tiles of each wave's experts
    int expert, tile;

    __device__ __forceinline__ void find(const Args& a, int64_t want) {
        const int per = (a.num_experts + THREADS - 1) / THREADS;
        const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
        const int e0 = threadIdx.x * per;
        int tiles = 0;
        int64_t s;
        for (int i = 0; i < per; ++i)
            if (e0 + i < a.num_experts) tiles += (expert_rows(a, e0 + i, &s) + MC - 1) / MC;
        int before = tiles;
#pragma unroll
        for (int d = 1; d < kWave; d *= 2) {
            const int v = __shfl_up(before, d, kWave);
            if (lane >= d) before += v;
        }
        if (lane == kWave - 1) first[wave] = before;
        if (threadIdx.x == 0) expert = -1;
        __syncthreads();
        int64_t at = before - tiles;
        for (int w = 0; w < wave; ++w) at += first[w];
        if (want >= at && want < at + tiles) {
            for (int i = 0; i < per; ++i) {
                const int n = (expert_rows(a, e0 + i, &s) + MC - 1) / MC;
                if (want < at + n) {
                    expert = e0 + i;
                    tile = static_cast<int>(want - at);
                    break;
                }
                at += n;
            }
        }
        __syncthreads();
    }
};

// One step's operands of a wave.
template <int MT, bool FP8>
struct Stage {
    u32x4 w[kTiles];
    u32x4 x[MT][FP8 ? 2 : 4];
};

// Few rows per expert.  FP8: rows are E4M3FN with one scale per 128 channels
// (UE8: a UE8M0 byte, else fp32), which multiplies the step's sum.  GATED:
// tiles 0, 1 are rows n of the gate half and tiles 2, 3 rows N + n.
//
// WAVES waves take the steps of a segment in turns.  Each keeps the loads of
// its next step in flight while it multiplies the present one.  The scales,
// scattered bytes in memory, are read once, whole rows at a time, into LDS.
template <int WAVES, int MT, bool FP8, bool UE8, bool GATED>
__global__ __launch_bounds__(WAVES* kWave, MT == 1 ? 4 : MT == 2 ? 3 : 2) void expert_w4_kernel(Args a) {
    constexpr int kThreads = WAVES * kWave;
    constexpr int MC = 16 * MT;
    constexpr int kOut = GATED ? kRows / 2 : kRows;  // outputs per workgroup
    constexpr int kScaleBytes = kRows * kScaleRow;
    constexpr int kRowScaleBytes = FP8 ? MC * kRowScaleRow * 4 : 0;
    constexpr int kRedBytes = WAVES * MC * kRedRow * 4;
    constexpr int kBytes =
        kScaleBytes + kRowScaleBytes > kRedBytes ? kScaleBytes + kRowScaleBytes : kRedBytes;
    __shared__ Finder<kThreads, MC> finder;
    __shared__ __attribute__((aligned(16))) uint8_t lds[kBytes];
    uint8_t(*lds_scale)[kScaleRow] = reinterpret_cast<uint8_t(*)[kScaleRow]>(lds);
    float(*lds_row)[kRowScaleRow] =
        reinterpret_cast<float(*)[kRowScaleRow]>(lds + kScaleBytes);
    float(*red)[MC][kRedRow] = reinterpret_cast<float(*)[MC][kRedRow]>(lds);

    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r16 = lane % 16, group = lane / 16;
    const int K = a.K, N = a.N;
    const int blocks = K / 32;
    const int n0 = blockIdx.x * kOut;
    const int here = N - n0 < kOut ? N - n0 : kOut;  // outputs of this workgroup

    for (int64_t tile = blockIdx.y; tile < a.tiles; tile += gridDim.y) {
        finder.find(a, tile);
        const int e = __builtin_amdgcn_readfirstlane(finder.expert);
        if (e < 0) break;  // tiles are in order: no later one has rows either
        int64_t start;
        const int count = expert_rows(a, e, &start);
        const int m0 = __builtin_amdgcn_readfirstlane(finder.tile) * MC;
        const int rows_here = count - m0 < MC ? count - m0 : MC;

        const int64_t w_row = static_cast<int64_t>(e) * (GATED ? 2 * N : N) + n0;
        const uint32_t w_pitch = K / 2;
        const uint32_t x_pitch = K * (FP8 ? 1 : 2);
        const auto w_view = view(a.codes + w_row * w_pitch, here * w_pitch);
        const auto up_view = view(a.codes + (w_row + (GATED ? N : 0)) * w_pitch, here * w_pitch);
        const auto x_view = view(a.rows + (start + m0) * x_pitch, rows_here * x_pitch);
        uint32_t w_at[kOut / 16], x_at[MT];
#pragma unroll
        for (int t = 0; t < kOut / 16; ++t)
            w_at[t] = t * 16 + r16 < here ? (t * 16 + r16) * w_pitch + group * 16 : kNowhere;
#pragma unroll
        for (int m = 0; m < MT; ++m)
            x_at[m] = m * 16 + r16 < rows_here
                          ? (m * 16 + r16) * x_pitch + group * (FP8 ? 32 : 64)
                          : kNowhere;

        f32x4 acc[kTiles][MT];
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[t][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

        const auto load = [&](int c, Stage<MT, FP8>& s) {
            const bool has = c * 4 + group < blocks;
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
                const uint32_t at = w_at[t % (kOut / 16)];
                s.w[t] = load16(GATED && t >= 2 ? up_view : w_view, has ? at : kNowhere, c * 64);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < (FP8 ? 2 : 4); ++i)
                    s.x[m][i] = load16(x_view, has ? x_at[m] : kNowhere,
                                       c * (FP8 ? 128 : 256) + i * 16);
        };
        const auto multiply = [&](int c, const Stage<MT, FP8>& s) {  // c within the segment
            float sf[kTiles];
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
                sf[t] = __uint_as_float(
                    static_cast<uint32_t>(lds_scale[t * 16 + r16][c * 4 + group]) << 23);
            f32x4 part[kTiles][MT];
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    part[t][m] = FP8 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : acc[t][m];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                __builtin_amdgcn_sched_barrier(0);  // or every operand is made at once
                bf16x8 xf[MT];
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    if constexpr (FP8) {
                        const u32x4 v = s.x[m][i / 2];
                        xf[m] = i % 2 == 0 ? rows8(v.x, v.y) : rows8(v.z, v.w);
                    } else {
                        Frag f;
                        f.w = s.x[m][i];
                        xf[m] = f.v;
                    }
                }
#pragma unroll
                for (int t = 0; t < kTiles; ++t) {
                    const bf16x8 wf = weights8(s.w[t][i], sf[t]);
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        part[t][m] =
                            __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, xf[m], part[t][m], 0, 0, 0);
                }
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const float xs = FP8 ? lds_row[m * 16 + r16][c] : 1.0f;
#pragma unroll
                for (int t = 0; t < kTiles; ++t) {
                    if constexpr (FP8) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            acc[t][m][i] = fmaf(xs, part[t][m][i], acc[t][m][i]);
                    } else {
                        acc[t][m] = part[t][m];
                    }
                }
            }
        };

        for (int seg = 0; seg * kSegment < K; ++seg) {
            const int c0 = seg * kSegSteps;
            int steps = (K - seg * kSegment + kStep - 1) / kStep;
            steps = steps < kSegSteps ? steps : kSegSteps;
            Stage<MT, FP8> s0, s1;
            int c = wave;
            load(c0 + c, s0);
            if (seg > 0) __syncthreads();  // the scales before are done with
            // weight scales: 16 bytes of four rows, or one word of one row, per lane
            const int seg_blocks = blocks - c0 * 4 < kSegment / 32 ? blocks - c0 * 4 : kSegment / 32;
            const auto scale_row = [&](int r) {
                const int half = GATED ? r / kOut : 0;
                int n = GATED ? r % kOut : r;
                n = n < here ? n : here - 1;
                return a.scales + (w_row + n + static_cast<int64_t>(half) * N) * blocks + c0 * 4;
            };
            if (K % 512 == 0) {
                for (int r = wave * 4 + group; r < kRows; r += WAVES * 4)
                    if (r16 * 16 < seg_blocks) {
                        const u32x4 v = *reinterpret_cast<const u32x4*>(scale_row(r) + r16 * 16);
                        uint32_t* to = reinterpret_cast<uint32_t*>(&lds_scale[r][r16 * 16]);
                        to[0] = v.x, to[1] = v.y, to[2] = v.z, to[3] = v.w;
                    }
            } else {
                for (int r = wave; r < kRows; r += WAVES)
                    for (int b = lane; b < (seg_blocks + 3) / 4 * 4; b += kWave)
                        lds_scale[r][b] = b < seg_blocks ? scale_row(r)[b] : 0;
            }
            if constexpr (FP8) {
                for (int i = threadIdx.x; i < MC * kSegSteps; i += kThreads) {
                    const int m = i / kSegSteps, q = i % kSegSteps;
                    float v = 0.0f;
                    if (m < rows_here && q < steps) {
                        const int64_t at = (start + m0 + m) * (K / 128) + c0 + q;
                        v = UE8 ? exponent_value(static_cast<const uint8_t*>(a.row_scales)[at])
                                : static_cast<const float*>(a.row_scales)[at];
                    }
                    lds_row[m][q] = v;
                }
            }
            __syncthreads();
            // Steps past the end load nothing, but the loads are issued all the
            // same: a branch around them would make the wait for the present
            // step's operands one for the next step's too.
            for (; c < steps; c += 2 * WAVES) {
                load(c0 + c + WAVES, s1);
                multiply(c, s0);
                load(c0 + c + 2 * WAVES, s0);
                if (c + WAVES < steps) multiply(c + WAVES, s1);
            }
        }
        __syncthreads();  // the scales are done with: their LDS takes the sums

        // lane l holds weight rows 4 * (l / 16) .. + 3 of a tile against row l % 16
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int m = 0; m < MT; ++m)
                *reinterpret_cast<f32x4*>(&red[wave][m * 16 + r16][t * 16 + group * 4]) = acc[t][m];
        __syncthreads();
        for (int i = threadIdx.x; i < rows_here * kOut; i += kThreads) {
            const int m = i / kOut, n = i % kOut;
            if (n < here) {
                float y = 0.0f, up = 0.0f;
#pragma unroll
                for (int v = 0; v < WAVES; ++v) {
                    y += red[v][m][n];
                    if constexpr (GATED) up += red[v][m][kRows / 2 + n];
                }
                if constexpr (GATED) y = y / (1.0f + expf(-y)) * up;
                a.out[(start + m0 + m) * N + n0 + n] = static_cast<uint16_t>(f32_to_bf16_rne(y));
            }
        }
        __syncthreads();
    }
}

template <int WAVES, int MT>
void launch_rows(const Args& a, int format, bool gated, dim3 grid, hipStream_t stream) {
    constexpr int kThreads = WAVES * kWave;
    const auto go = [&](auto* kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, a);
    };
    if (format == 0)
        gated ? go(expert_w4_kernel<WAVES, MT, false, false, true>)
              : go(expert_w4_kernel<WAVES, MT, false, false, false>);
    else if (format == 1)
        gated ? go(expert_w4_kernel<WAVES, MT, true, false, true>)
              : go(expert_w4_kernel<WAVES, MT, true, false, false>);
    else
        gated ? go(expert_w4_kernel<WAVES, MT, true, true, true>)
              : go(expert_w4_kernel<WAVES, MT, true, true, false>);
}

}  // namespace

hipError_t launch_expert_w4(const ep_problem& p, const ep_expert_w4_t& mm, const void* rows,
                            const void* row_scales, const ep_layout_t& layout,
                            const uint8_t* codes, const uint8_t* scales, void* out,
                            hipStream_t stream) {
    const int64_t entries = static_cast<int64_t>(p.num_tokens) * p.num_topk;
    const int64_t held = static_cast<int64_t>(p.num_experts) * p.capacity;
    const int64_t filled = p.capacity > 0 && held < entries ? held : entries;
    if (filled == 0) return hipSuccess;
    const bool gated = mm.activation == 1;
    const int outs = gated ? kRows / 2 : kRows;
    Args a;
    a.rows = static_cast<const uint8_t*>(rows);
    a.row_scales = row_scales;
    a.count = layout.count;
    a.offset = layout.offset;
    a.codes = codes;
    a.scales = scales;
    a.out = static_cast<uint16_t*>(out);
    a.num_rows = p.capacity > 0 ? held : entries;
    a.num_experts = p.num_experts;
    a.capacity = p.capacity;
    a.K = mm.in_features;
    a.N = mm.out_features;
    // Row tiles: no more than one per expert that can have rows, plus one per
    // full tile.
    const int64_t experts = p.num_experts < filled ? p.num_experts : filled;
    const int64_t mean = filled / experts;
    const int mt = mean > 24 ? 4 : mean > 8 ? 2 : 1;
    a.tiles = experts + filled / (16 * mt);
    const dim3 grid((mm.out_features + outs - 1) / outs,
                    static_cast<unsigned>(a.tiles < 32768 ? a.tiles : 32768));
    switch (mt) {
        case 1: launch_rows<4, 1>(a, mm.in_format, gated, grid, stream); break;
        case 2: launch_rows<4, 2>(a, mm.in_format, gated, grid, stream); break;
        default: launch_rows<4, 4>(a, mm.in_format, gated, grid, stream); break;
    }
    return hipGetLastError();
}

}  // namespace ep
