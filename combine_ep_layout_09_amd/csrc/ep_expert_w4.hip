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

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kTiles = 4;            // 16-row weight tiles per workgroup
constexpr int kRows = 16 * kTiles;   // weight rows per workgroup
constexpr int kStep = 128;           // channels per wave and step

struct Args {
    const uint8_t* rows;      // bf16 or E4M3FN [R, K]
    const void* row_scales;   // fp32 or UE8M0 [R, K / 128]
    const int32_t* count;
    const int32_t* offset;
    const uint8_t* codes;     // [E, n2, K / 2]
    const uint8_t* scales;    // [E, n2, K / 32]
    uint16_t* out;            // bf16 [R, N]
    int64_t items;            // row tiles * n_blocks
    int64_t num_rows;         // R
    int32_t num_experts, capacity, K, N, n_blocks;
};

union Frag {
    uint32_t u[4];
    bf16x8 v;
};

__device__ __forceinline__ float exponent_value(uint32_t byte) {
    // 2^(byte - 127); byte 0 is the subnormal 2^-127, 255 is NaN
    return byte == 0 ? __uint_as_float(0x00400000u)
                     : byte == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float(byte << 23);
}

// Eight codes of one word -> bf16, scaled by the power of two s carries.
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

__device__ __forceinline__ int clamp_count(const Args& a, int e, int64_t* start) {
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

// The expert and row tile of each item: experts with rows, in order, each with
// one tile per MC rows.
template <int MC>
struct Finder {
    int first[kWaves];   // tiles of the experts of the waves before
    int expert, tile;

    __device__ __forceinline__ void find(const Args& a, int64_t want) {
        const int per = (a.num_experts + kThreads - 1) / kThreads;
        const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
        const int e0 = threadIdx.x * per;
        int tiles = 0;
        int64_t s;
        for (int i = 0; i < per; ++i)
            if (e0 + i < a.num_experts) tiles += (clamp_count(a, e0 + i, &s) + MC - 1) / MC;
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
                const int n = (clamp_count(a, e0 + i, &s) + MC - 1) / MC;
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

// FP8: rows are E4M3FN with one scale per 128 channels (UE8: a UE8M0 byte,
// else fp32), which multiplies the step's sum.  GATED: tiles 0, 1 are rows n
// of the gate half and tiles 2, 3 rows N + n.  WORD: K % 128 == 0, so a step's
// four scale bytes are one aligned word.
template <int MT, bool FP8, bool UE8, bool GATED, bool WORD>
__global__ __launch_bounds__(kThreads) void expert_w4_kernel(Args a) {
    constexpr int MC = 16 * MT;
    constexpr int kOut = GATED ? kRows / 2 : kRows;  // outputs per workgroup
    __shared__ Finder<MC> finder;
    __shared__ float red[kWaves][MC][kRows];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int r16 = lane % 16, group = lane / 16;
    const int K = a.K, N = a.N;
    const int blocks = K / 32;

    for (int64_t item = blockIdx.x; item < a.items; item += gridDim.x) {
        finder.find(a, item / a.n_blocks);
        const int e = finder.expert;
        if (e < 0) break;  // items are in order: no later one has rows either
        int64_t start;
        const int count = clamp_count(a, e, &start);
        const int m0 = finder.tile * MC;
        const int n0 = static_cast<int>(item % a.n_blocks) * kOut;

        const int n2 = GATED ? 2 * N : N;
        const uint8_t* w[kTiles];
        const uint8_t* sc[kTiles];
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            int n = GATED ? n0 + (t % 2) * 16 + r16 : n0 + t * 16 + r16;
            n = n < N ? n : N - 1;  // rows past the end read the last one, unused
            if (GATED && t >= 2) n += N;
            const int64_t row = static_cast<int64_t>(e) * n2 + n;
            w[t] = a.codes + row * (K / 2) + group * 16;
            sc[t] = a.scales + row * blocks;
        }
        const uint8_t* x[MT];
        int64_t xrow[MT];
        bool in[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            in[m] = m0 + m * 16 + r16 < count;
            xrow[m] = start + m0 + (in[m] ? m * 16 + r16 : 0);
            x[m] = a.rows + xrow[m] * K * (FP8 ? 1 : 2) + group * (FP8 ? 32 : 64);
        }

        f32x4 acc[kTiles][MT];
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[t][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

        const int steps = (K + kStep - 1) / kStep;
        for (int c = wave; c < steps; c += kWaves) {
            const bool has = WORD || c * 4 + group < blocks;
            uint4 q[kTiles];
            uint32_t s[kTiles];
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
                q[t] = make_uint4(0, 0, 0, 0);
                s[t] = 127;
                if (has) {
                    q[t] = *reinterpret_cast<const uint4*>(w[t] + static_cast<int64_t>(c) * 64);
                    if constexpr (WORD)
                        s[t] = (*reinterpret_cast<const uint32_t*>(sc[t] + c * 4) >> (8 * group)) &
                               0xffu;
                    else
                        s[t] = sc[t][c * 4 + group];
                }
            }
            uint4 xv[MT][FP8 ? 2 : 4];
            float xs[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                xs[m] = 0.0f;
#pragma unroll
                for (int i = 0; i < (FP8 ? 2 : 4); ++i) {
                    xv[m][i] = make_uint4(0, 0, 0, 0);
                    if (has && in[m])
                        xv[m][i] = *reinterpret_cast<const uint4*>(
                            x[m] + static_cast<int64_t>(c) * (FP8 ? 128 : 256) + i * 16);
                }
                if constexpr (FP8) {
                    if (in[m]) {
                        const int64_t at = xrow[m] * (K / 128) + c;
                        xs[m] = UE8 ? exponent_value(static_cast<const uint8_t*>(a.row_scales)[at])
                                    : static_cast<const float*>(a.row_scales)[at];
                    }
                }
            }
            float sf[kTiles];
#pragma unroll
            for (int t = 0; t < kTiles; ++t) sf[t] = __uint_as_float(s[t] << 23);
            f32x4 part[kTiles][MT];
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    part[t][m] = FP8 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : acc[t][m];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                bf16x8 xf[MT];
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    if constexpr (FP8) {
                        const uint4 v = xv[m][i / 2];
                        xf[m] = i % 2 == 0 ? rows8(v.x, v.y) : rows8(v.z, v.w);
                    } else {
                        Frag f;
                        f.u[0] = xv[m][i].x, f.u[1] = xv[m][i].y;
                        f.u[2] = xv[m][i].z, f.u[3] = xv[m][i].w;
                        xf[m] = f.v;
                    }
                }
#pragma unroll
                for (int t = 0; t < kTiles; ++t) {
                    const uint32_t word = i == 0 ? q[t].x : i == 1 ? q[t].y : i == 2 ? q[t].z : q[t].w;
                    const bf16x8 wf = weights8(word, sf[t]);
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        part[t][m] =
                            __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, xf[m], part[t][m], 0, 0, 0);
                }
            }
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    if constexpr (FP8) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            acc[t][m][i] = fmaf(xs[m], part[t][m][i], acc[t][m][i]);
                    } else {
                        acc[t][m] = part[t][m];
                    }
                }
        }

        // lane l holds weight rows 4 * (l / 16) .. + 3 of a tile against row l % 16
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int m = 0; m < MT; ++m)
                *reinterpret_cast<f32x4*>(&red[wave][m * 16 + r16][t * 16 + group * 4]) = acc[t][m];
        __syncthreads();
        for (int i = threadIdx.x; i < MC * kOut; i += kThreads) {
            const int m = i / kOut, n = i % kOut;
            if (m0 + m < count && n0 + n < N) {
                float y = 0.0f, up = 0.0f;
#pragma unroll
                for (int v = 0; v < kWaves; ++v) {
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

template <int MT, bool FP8, bool UE8, bool GATED>
void launch_word(const Args& a, unsigned grid, hipStream_t stream) {
    if (a.K % kStep == 0)
        hipLaunchKernelGGL((expert_w4_kernel<MT, FP8, UE8, GATED, true>), dim3(grid),
                           dim3(kThreads), 0, stream, a);
    else if constexpr (!FP8)
        hipLaunchKernelGGL((expert_w4_kernel<MT, FP8, UE8, GATED, false>), dim3(grid),
                           dim3(kThreads), 0, stream, a);
}

template <int MT>
void launch_rows(const Args& a, int format, bool gated, unsigned grid, hipStream_t stream) {
    if (format == 0) {
        if (gated)
            launch_word<MT, false, false, true>(a, grid, stream);
        else
            launch_word<MT, false, false, false>(a, grid, stream);
    } else if (format == 1) {
        if (gated)
            launch_word<MT, true, false, true>(a, grid, stream);
        else
            launch_word<MT, true, false, false>(a, grid, stream);
    } else {
        if (gated)
            launch_word<MT, true, true, true>(a, grid, stream);
        else
            launch_word<MT, true, true, false>(a, grid, stream);
    }
}

}  // namespace

hipError_t launch_expert_w4(const ep_problem& p, const ep_expert_w4_t& mm, const void* rows,
                            const void* row_scales, const ep_layout_t& layout,
                            const uint8_t* codes, const uint8_t* scales, void* out,
                            hipStream_t stream) {
    const int64_t entries = static_cast<int64_t>(p.num_tokens) * p.num_topk;
    const int64_t held = static_cast<int64_t>(p.num_experts) * p.capacity;
    const int64_t num_rows = p.capacity > 0 ? held : entries;
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
    a.num_rows = num_rows;
    a.num_experts = p.num_experts;
    a.capacity = p.capacity;
    a.K = mm.in_features;
    a.N = mm.out_features;
    a.n_blocks = (mm.out_features + outs - 1) / outs;
    // Row tiles: no more than one per expert that can have rows, plus one per
    // full tile.
    const int64_t experts = p.num_experts < filled ? p.num_experts : filled;
    const int64_t mean = filled / experts;
    const int mt = mean > 24 ? 4 : mean > 8 ? 2 : 1;
    a.items = (experts + filled / (16 * mt)) * a.n_blocks;
    const unsigned grid = static_cast<unsigned>(a.items < (1 << 24) ? a.items : (1 << 24));
    switch (mt) {
        case 1: launch_rows<1>(a, mm.in_format, gated, grid, stream); break;
        case 2: launch_rows<2>(a, mm.in_format, gated, grid, stream); break;
        default: launch_rows<4>(a, mm.in_format, gated, grid, stream); break;
    }
    return hipGetLastError();
}

}  // namespace ep
