// ep_expert_w4.hip -- the experts' products with 4-bit weights on the
// dispatched rows.
//
//   y[r, n] = sum_k x[r, k] * e2m1(code[e, n, k]) * 2^(scale[e, n, k / 32] - 127)
//
// for the rows r of expert e, summed in fp32; optionally the gated activation
// silu(y[r, n]) * y[r, N + n]; one rounding to bf16.
//
// Weights and rows meet in bf16 MFMA: every E2M1 value times a power of two is
// a bf16, and v_cvt_scalef32_pk_bf16_fp4 makes two of them from one byte at the
// rate of any other instruction, so the products are those of the formula and
// only the sums round.  (The MFMA that takes E2M1 itself keeps fewer bits of
// its partial sums than fp32: 3e-5 of the result on random data.)
//
// The channels of an MFMA may be taken in any order if both operands agree.
// Lane l multiplies weight row l % 16 and the 32 channels, 16 bytes of codes
// and one scale, at block l / 16 of a chunk of 128: codes are used as they lie
// in memory.
//
// Two kernels.  A decode batch gives each expert a handful of rows, so the
// weights, 17/32 byte each, are the traffic and should be read once, at the
// memory's rate: expert_w4_kernel.  With many rows per expert the matrix cores
// and the rows' own traffic count as well: expert_w4_tile_kernel.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ep_internal.h"
#include "ep_device.h"
#include "ep_expert_dev.h"

namespace ep {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
using namespace expert;

constexpr int kTiles = 4;            // 16-row weight tiles of a wave
constexpr int kRows = 16 * kTiles;   // weight rows of a wave
constexpr int kStep = 128;           // channels of a chunk
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
    const uint8_t* codes;     // [E, n2, K / 2]
    const uint8_t* scales;    // [E, n2, K / 32]
    uint16_t* out;            // bf16 [R, N]
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

// One step's operands of a wave: two chunks of 128 channels.
template <bool FP8>
struct Stage {
    u32x4 w[2][kTiles];
    u32x4 x[2][FP8 ? 2 : 4];
};

// Few rows per expert.  A workgroup takes 64 weight rows of one expert against
// up to 16 rows; its WAVES waves take pairs of chunks in turns and add
// their sums in LDS, in wave order.  FP8: rows are E4M3FN with one scale per 128
// channels (UE8: a UE8M0 byte, else fp32), which multiplies the chunk's sum.
// GATED: tiles 0, 1 are rows n of the gate half and tiles 2, 3 rows N + n.
// WORDS: K % 128 == 0, so rows of scales are whole words.
//
// What bounds it is how the codes are read.  A load covers 8 rows x 128 bytes:
// whole cache lines, so they need not be kept for another wave (non-temporal),
// which this memory rewards: reading alone reaches 7.0 TB/s so, 6.2 with 64-byte
// pieces of 16 rows, the MFMA's own layout, or when the lines are kept.  Pairing
// two chunks across lanes afterwards costs 1.5 instructions per word.  The
// scales, scattered bytes in memory, come once, whole rows at a time, to LDS.
// Loads two steps ahead, or more waves, were slower: what is in flight then
// outgrows the caches.  256 experts, K 7168, N 2048 gated, 4 FP8 rows each: 595 to
// 603 us, 6.6 TB/s (696 with 64-byte pieces, 640 with the lines kept); K 2048, N 7168,
// bf16 rows: 344 to 359 us, 5.6 TB/s; 8 experts of one token: 25.4 us, 4.9 TB/s.
template <int WAVES, bool FP8, bool UE8, bool GATED, bool WORDS>
__global__ __launch_bounds__(WAVES* kWave, 4) void expert_w4_kernel(Args a) {
    constexpr int kThreads = WAVES * kWave;
    constexpr int MC = 16;
    constexpr int kOut = GATED ? kRows / 2 : kRows;  // outputs per workgroup
    constexpr int kScaleBytes = kRows * kScaleRow;
    constexpr int kRowScaleBytes = FP8 ? MC * kRowScaleRow * 4 : 0;
    constexpr int kRedBytes = WAVES * MC * kRedRow * 4;
    constexpr int kBytes =
        kScaleBytes + kRowScaleBytes > kRedBytes ? kScaleBytes + kRowScaleBytes : kRedBytes;
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

    const Found f = find_tile<MC>(a, [](uint32_t) { return blockIdx.z * gridDim.y + blockIdx.y; });
    const int e = f.expert;
    if (e < 0) return;
    const int64_t start = f.start;
    const int m0 = f.tile * MC;
    const int rows_here = f.count - m0 < MC ? f.count - m0 : MC;
    if (rows_here <= 0) return;

    const int64_t w_row = static_cast<int64_t>(e) * (GATED ? 2 * N : N) + n0;
    const uint32_t w_pitch = K / 2;
    const uint32_t x_pitch = K * (FP8 ? 1 : 2);
    const auto w_view = view(a.codes + w_row * w_pitch, here * w_pitch);
    const auto up_view = view(a.codes + (w_row + (GATED ? N : 0)) * w_pitch, here * w_pitch);
    const auto s_view = view(a.scales + w_row * blocks, here * blocks);
    const auto up_s_view = view(a.scales + (w_row + (GATED ? N : 0)) * blocks, here * blocks);
    const auto x_view = view(a.rows + (start + m0) * x_pitch, rows_here * x_pitch);
    const int half = lane / 8 % 2;
    const uint32_t w_at = lane % 8 * w_pitch + half * 64 + group * 16;
    const uint32_t x_at = r16 * x_pitch + group * (FP8 ? 32 : 64);

    f32x4 acc[kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const auto load = [&](int p, Stage<FP8>& s) {  // chunks 2p and 2p + 1
        const uint32_t at = p * 8 + half * 4 + group < blocks ? w_at : kNowhere;
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                s.w[i][t] = load16<true>(t * 16 < kOut ? w_view : up_view,
                                         at + (t * 16 % kOut + i * 8) * w_pitch, p * 128);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bool has = p * 8 + h * 4 + group < blocks;
#pragma unroll
            for (int i = 0; i < (FP8 ? 2 : 4); ++i)
                s.x[h][i] = load16<false>(x_view, has ? x_at : kNowhere,
                                          (2 * p + h) * (FP8 ? 128 : 256) + i * 16);
        }
    };
    const auto multiply = [&](int c, const u32x4(&w)[kTiles],
                              const u32x4(&x)[FP8 ? 2 : 4]) {  // c within the segment
        float sf[kTiles];
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
            sf[t] = __uint_as_float(
                static_cast<uint32_t>(lds_scale[t * 16 + r16][c * 4 + group]) << 23);
        f32x4 part[kTiles];
#pragma unroll
        for (int t = 0; t < kTiles; ++t) part[t] = FP8 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : acc[t];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __builtin_amdgcn_sched_barrier(0);  // or every operand is made at once
            bf16x8 xf;
            if constexpr (FP8) {
                const u32x4 v = x[i / 2];
                xf = i % 2 == 0 ? rows8(v.x, v.y) : rows8(v.z, v.w);
            } else {
                Frag f;
                f.w = x[i];
                xf = f.v;
            }
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
                part[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(weights8(w[t][i], sf[t]), xf,
                                                                  part[t], 0, 0, 0);
        }
        const float xs = FP8 ? lds_row[r16][c] : 1.0f;
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            if constexpr (FP8) {
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[t][i] = fmaf(xs, part[t][i], acc[t][i]);
            } else {
                acc[t] = part[t];
            }
        }
    };

    for (int seg = 0; seg * kSegment < K; ++seg) {
        const int c0 = seg * kSegSteps;
        int steps = (K - seg * kSegment + kStep - 1) / kStep;
        steps = steps < kSegSteps ? steps : kSegSteps;
        // The segment's scales: a word of one row per lane where rows are
        // whole words.  Their loads go first, so that waiting for them does
        // not wait for the first step's operands.
        constexpr int kMine = kRows / WAVES;
        const int seg_blocks = blocks - c0 * 4 < kSegment / 32 ? blocks - c0 * 4 : kSegment / 32;
        uint32_t scale[kMine];
        if constexpr (WORDS) {
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                const int r = wave * kMine + i;
                scale[i] = __builtin_amdgcn_raw_buffer_load_b32(
                    r < kOut ? s_view : up_s_view, lane * 4 < seg_blocks && r % kOut < here ? lane * 4 : kNowhere,
                    (r % kOut) * blocks + c0 * 4, 0);
            }
        }
        constexpr int kRowMine = FP8 ? MC * kSegSteps / kThreads : 1;
        float row_scale[kRowMine];
        if constexpr (FP8) {
#pragma unroll
            for (int i = 0; i < kRowMine; ++i) {
                const int m = wave + i * WAVES;  // lane: the step
                const int64_t at = (start + m0 + m) * (K / 128) + c0 + lane;
                row_scale[i] = 0.0f;
                if (m < rows_here && lane < steps)
                    row_scale[i] =
                        UE8 ? exponent_value(static_cast<const uint8_t*>(a.row_scales)[at])
                            : static_cast<const float*>(a.row_scales)[at];
            }
        }
        Stage<FP8> s;
        int p = wave;
        load(c0 / 2 + p, s);  // past the end of the channels it loads nothing
        if (seg > 0) __syncthreads();  // the scales before are done with
        if constexpr (WORDS) {
#pragma unroll
            for (int i = 0; i < kMine; ++i)
                *reinterpret_cast<uint32_t*>(&lds_scale[wave * kMine + i][lane * 4]) = scale[i];
        } else {
            // bytes, 64 of a row per load, four rows on their way at a time (one
            // after the other K 4192, N 167 took 23.5 us); 0 past the row's end
#pragma unroll 1
            for (int i = 0; i < kMine; i += 4) {
                uint8_t v[4][kSegment / 32 / kWave];
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int q = 0; q < kSegment / 32 / kWave; ++q) {
                        const int r = wave * kMine + i + j, b = q * kWave + lane;
                        v[j][q] = __builtin_amdgcn_raw_buffer_load_b8(
                            r < kOut ? s_view : up_s_view,
                            b < seg_blocks && r % kOut < here ? b : kNowhere,
                            (r % kOut) * blocks + c0 * 4, 0);
                    }
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int q = 0; q < kSegment / 32 / kWave; ++q)
                        lds_scale[wave * kMine + i + j][q * kWave + lane] = v[j][q];
            }
        }
        if constexpr (FP8) {
#pragma unroll
            for (int i = 0; i < kRowMine; ++i) lds_row[wave + i * WAVES][lane] = row_scale[i];
        }
        __syncthreads();
        while (2 * p < steps) {
#pragma unroll
            for (int t = 0; t < kTiles; ++t) pair_chunks(s.w[0][t], s.w[1][t]);
            multiply(2 * p, s.w[0], s.x[0]);
            if (2 * p + 1 < steps) multiply(2 * p + 1, s.w[1], s.x[1]);
            p += WAVES;
            if (2 * p < steps) load(c0 / 2 + p, s);
        }
    }
    __syncthreads();  // the scales are done with: their LDS takes the sums

    // lane l holds weight rows 4 * (l / 16) .. + 3 of a tile against row l % 16
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
        *reinterpret_cast<f32x4*>(&red[wave][r16][t * 16 + group * 4]) = acc[t];
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
}

// Many rows per expert: a workgroup takes 256 weight rows, 64 per wave, against
// up to 16 * MT rows.  The rows' operands are the same for the four waves: each
// chunk of 128 channels passes through LDS, as bf16, once for all of them,
// loaded two chunks ahead; the weights' next pair of chunks is in flight as
// well.  GATED: a wave's tiles 0, 1 are gate and 2, 3 up of the same 32 outputs.
// bf16 rows have 32-row tiles where an expert mostly has one, whose codes are read
// once (not kept: 48.5 us, kept 51.6, at 24 rows each), and 64-row tiles where
// several read them (128 rows each: kept 124, not 127).  FP8 rows have 32-row tiles
// at any number of rows, and their codes are never kept, which pays for few rows
// only (64 experts, K 4096, N 1408 gated: 24 rows each 90 to 96 us, kept 100 to 103;
// 64: 204, kept 187; 128: 342, kept 309; 512: 1184, kept 965).
// 64 skewed experts, 48 rows each in the mean, K 4096, N 1408 gated, bf16: 127 to
// 133 us (242 with the other kernel).  Matrix instructions are a third of that, their
// operands' conversion another; memory alone would take 61 at the rate that reading
// reaches.  128 rows each, 256 experts, K 7168, N 2048 gated: 2.25 ms, 854 TFLOP/s;
// FP8 3.38 ms, 569 TFLOP/s: a tile of 32 rows converts the codes again for each.
constexpr int kTileSegment = 4096;                 // channels of weight scales in LDS
constexpr int kTileScaleRow = kTileSegment / 32 + 4;  // bytes
constexpr int kTileRow = kStep * 2 + 16;           // bytes of a row's chunk in LDS

template <int MT, bool FP8, bool UE8, bool GATED, bool WORDS>
__global__ __launch_bounds__(256, 2) void expert_w4_tile_kernel(Args a) {
    constexpr int MC = 16 * MT;
    constexpr int kOut = GATED ? kRows / 2 : kRows;  // outputs per wave
    constexpr int kPieces = FP8 ? 8 : 16;            // 16-byte pieces of a row's chunk
    constexpr int kMine = MC * kPieces / 256;        // pieces per thread
    __shared__ __attribute__((aligned(16))) uint8_t lds_x[2][MC][kTileRow];
    __shared__ float lds_row[2][MC];
    __shared__ uint32_t lds_scale[4 * kRows][kTileScaleRow / 4];

    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r16 = lane % 16, group = lane / 16;
    const int K = a.K, N = a.N;
    const int blocks = K / 32;
    const int steps = (K + kStep - 1) / kStep;
    // Workgroups go round the 8 XCDs in turn.  Each XCD takes a run of items
    // (row tile, output block), so that its L2 serves one tile's rows to that
    // tile's blocks, and one expert's weights to that expert's tiles.
    const uint32_t n_blocks = (N + 4 * kOut - 1) / (4 * kOut);
    const uint64_t id = static_cast<uint64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
    uint32_t block = 0;
    const Found f = find_tile<MC>(a, [&](uint32_t tiles) {
        const uint64_t items = static_cast<uint64_t>(tiles) * n_blocks;
        const uint64_t run = (items + 7) / 8;
        const uint64_t item = id % 8 * run + id / 8;
        if (id / 8 >= run || item >= items) return 0xffffffffu;
        block = static_cast<uint32_t>(item % n_blocks);
        return static_cast<uint32_t>(item / n_blocks);
    });
    if (f.expert < 0) return;
    const int n0 = (block * 4 + wave) * kOut;
    const int left = N - n0 < kOut ? N - n0 : kOut;
    const int here = left > 0 ? left : 0;  // outputs of this wave
    const int m0 = f.tile * MC;
    const int rows_here = f.count - m0 < MC ? f.count - m0 : MC;
    if (rows_here <= 0) return;
    const int64_t row0 = f.start + m0;

    const int64_t w_row = static_cast<int64_t>(f.expert) * (GATED ? 2 * N : N) + (here ? n0 : 0);
    const uint32_t w_pitch = K / 2;
    const uint32_t x_pitch = K * (FP8 ? 1 : 2);
    const auto w_view = view(a.codes + w_row * w_pitch, here * w_pitch);
    const auto up_view = view(a.codes + (w_row + (GATED ? N : 0)) * w_pitch, here * w_pitch);
    const auto x_view = view(a.rows + row0 * x_pitch, rows_here * x_pitch);
    const int half = lane / 8 % 2;
    const uint32_t w_at = lane % 8 * w_pitch + half * 64 + group * 16;

    f32x4 acc[kTiles][MT];
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[t][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    u32x4 next_w[2][kTiles];
    const auto load_w = [&](int p) {  // chunks 2p and 2p + 1; nothing past the end
        const uint32_t at = p * 8 + half * 4 + group < blocks ? w_at : kNowhere;
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                next_w[i][t] = load16<MT == 2>(t * 16 < kOut ? w_view : up_view,
                                             at + (t * 16 % kOut + i * 8) * w_pitch, p * 128);
    };
    // A chunk's rows on their way to LDS: even and odd chunks have a set each,
    // loaded two chunks ahead.
    struct Ahead {
        u32x4 x[kMine];
        float row;
    };
    const auto load_x = [&](Ahead& s, int c) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int at = threadIdx.x + i * 256;
            const int m = at / kPieces, q = at % kPieces;
            const bool has = c * 4 + q / (kPieces / 4) < blocks;
            s.x[i] = load16<false>(x_view, has ? m * x_pitch + q * 16 : kNowhere, c * kPieces * 16);
        }
        if constexpr (FP8) {
            const int m = threadIdx.x;
            s.row = 0.0f;
            if (m < rows_here && c < steps) {
                const int64_t at = (row0 + m) * (K / kStep) + c;
                s.row = UE8 ? exponent_value(static_cast<const uint8_t*>(a.row_scales)[at])
                            : static_cast<const float*>(a.row_scales)[at];
            }
        }
    };
    const auto store_x = [&](const Ahead& s, int buf) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int at = threadIdx.x + i * 256;
            const int m = at / kPieces, q = at % kPieces;
            if constexpr (FP8) {
                Frag lo, hi;
                lo.v = rows8(s.x[i].x, s.x[i].y);
                hi.v = rows8(s.x[i].z, s.x[i].w);
                *reinterpret_cast<u32x4*>(&lds_x[buf][m][q * 32]) = lo.w;
                *reinterpret_cast<u32x4*>(&lds_x[buf][m][q * 32 + 16]) = hi.w;
            } else {
                *reinterpret_cast<u32x4*>(&lds_x[buf][m][q * 16]) = s.x[i];
            }
        }
        if constexpr (FP8) {
            if (threadIdx.x < MC) lds_row[buf][threadIdx.x] = s.row;
        }
    };
    // The wave's own rows of weight scales.  16 bytes of eight rows per load
    // where every piece lies whole in a row, else a word of two rows.
    const auto scale_view = [&](int r) {
        return view(a.scales + (w_row + (r < kOut ? 0 : N)) * blocks, here * blocks);
    };
    const auto stage_scales = [&](int first_block) {
        constexpr int n_words = kTileSegment / 32 / 4;
        if (WORDS && K % (16 * 32) == 0) {
            u32x4 v[kRows / 8];
#pragma unroll
            for (int i = 0; i < kRows / 8; ++i) {
                const int n = (i * 8 + lane / 8) % kOut, b = first_block + lane % 8 * 16;
                v[i] = load16<false>(scale_view(i * 8), b < blocks ? n * blocks + b : kNowhere, 0);
            }
#pragma unroll
            for (int i = 0; i < kRows / 8; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    lds_scale[wave * kRows + i * 8 + lane / 8][lane % 8 * 4 + k] = v[i][k];
            return;
        }
#pragma unroll 4
        for (int i = 0; i < kRows * n_words / kWave; ++i) {
            const int r = i * 2 + lane / n_words, q = lane % n_words;
            const int n = r % kOut, b = first_block + q * 4;
            const uint32_t at = n * blocks + b;
            const auto from = scale_view(i * 2);
            uint32_t v = 0;
            if constexpr (WORDS) {
                v = __builtin_amdgcn_raw_buffer_load_b32(from, b < blocks ? at : kNowhere, 0, 0);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    v |= static_cast<uint32_t>(__builtin_amdgcn_raw_buffer_load_b8(
                             from, b + k < blocks ? at + k : kNowhere, 0, 0))
                         << (8 * k);
            }
            lds_scale[wave * kRows + r][q] = v;
        }
    };
    const auto multiply = [&](int c, const u32x4(&w)[kTiles], int buf) {
        float sf[kTiles];
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            const uint32_t word = lds_scale[wave * kRows + t * 16 + r16][c % (kTileSegment / kStep)];
            sf[t] = __uint_as_float((word >> (8 * group) & 0xffu) << 23);
        }
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
                Frag x;
                x.w = *reinterpret_cast<const u32x4*>(&lds_x[buf][m * 16 + r16][group * 64 + i * 16]);
                xf[m] = x.v;
            }
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
                const bf16x8 wf = weights8(w[t][i], sf[t]);
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    part[t][m] =
                        __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, xf[m], part[t][m], 0, 0, 0);
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const float xs = FP8 ? lds_row[buf][m * 16 + r16] : 1.0f;
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

    Ahead even, odd;
    load_x(even, 0);
    stage_scales(0);
    load_w(0);
    load_x(odd, 1);
    store_x(even, 0);
    load_x(even, 2);
    u32x4 w[2][kTiles];
    for (int p = 0; 2 * p < steps; ++p) {
        const int c = 2 * p;
        // a segment's rows of scales are this wave's own: no barrier
        if (c > 0 && c % (kTileSegment / kStep) == 0) stage_scales(c * 4);
        __syncthreads();
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            w[0][t] = next_w[0][t];
            w[1][t] = next_w[1][t];
            pair_chunks(w[0][t], w[1][t]);
        }
        load_w(p + 1);
        __builtin_amdgcn_s_setprio(1);  // over the workgroup that loads
        multiply(c, w[0], 0);
        __builtin_amdgcn_s_setprio(0);
        store_x(odd, 1);
        load_x(odd, c + 3);
        __syncthreads();
        __builtin_amdgcn_s_setprio(1);
        if (c + 1 < steps) multiply(c + 1, w[1], 1);
        __builtin_amdgcn_s_setprio(0);
        store_x(even, 0);
        load_x(even, c + 4);
    }

    // lane l holds outputs 4 * (l / 16) .. + 3 of a tile for row l % 16
#pragma unroll
    for (int t = 0; t < kOut / 16; ++t)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int n = t * 16 + group * 4;
            if (m * 16 + r16 >= rows_here) continue;
            uint16_t* to = a.out + (row0 + m * 16 + r16) * N + n0 + n;
            uint32_t y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float v = acc[t][m][i];
                if constexpr (GATED) v = v / (1.0f + expf(-v)) * acc[t + kOut / 16][m][i];
                y[i] = f32_to_bf16_rne(v);
            }
            if (N % 4 == 0) {
                if (n < here)
                    *reinterpret_cast<uint2*>(to) = make_uint2(y[0] | y[1] << 16, y[2] | y[3] << 16);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n + i < here) to[i] = static_cast<uint16_t>(y[i]);
            }
        }
}

// The kernel of WAVES waves for few rows (MT 1), or (WAVES 0) the one for many.
template <int WAVES, int MT, bool FP8, bool UE8, bool GATED, bool WORDS>
void launch_one(const Args& a, dim3 grid, hipStream_t stream) {
    if constexpr (WAVES == 0)
        hipLaunchKernelGGL((expert_w4_tile_kernel<MT, FP8, UE8, GATED, WORDS>), grid, dim3(256), 0,
                           stream, a);
    else
        hipLaunchKernelGGL((expert_w4_kernel<WAVES, FP8, UE8, GATED, WORDS>), grid,
                           dim3(WAVES * kWave), 0, stream, a);
}

template <int WAVES, int MT, bool GATED>
void launch_format(const Args& a, int format, dim3 grid, hipStream_t stream) {
    static_assert(WAVES == 0 || MT == 1, "a few-row tile has 16 rows");
    if constexpr (MT < 4) {
        if (format == 1) return launch_one<WAVES, MT, true, false, GATED, true>(a, grid, stream);
        if (format == 2) return launch_one<WAVES, MT, true, true, GATED, true>(a, grid, stream);
    }
    if (a.K % kStep == 0)
        launch_one<WAVES, MT, false, false, GATED, true>(a, grid, stream);
    else
        launch_one<WAVES, MT, false, false, GATED, false>(a, grid, stream);
}

template <int WAVES, int MT>
void launch_rows(const Args& a, int format, bool gated, int64_t tiles, hipStream_t stream) {
    const int outs = (gated ? kRows / 2 : kRows) * (WAVES == 0 ? 4 : 1);
    const int64_t blocks = (a.N + outs - 1) / outs;
    dim3 grid;
    if (WAVES == 0) {  // a row of ids whose length 8 divides
        const int64_t items = (tiles * blocks + 7) / 8 * 8;
        const int64_t x = items < (1 << 20) ? items : 1 << 20;
        grid = dim3(static_cast<unsigned>(x), static_cast<unsigned>((items + x - 1) / x));
    } else {
        const int64_t y = tiles < 32768 ? tiles : 32768;
        grid = dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(y),
                    static_cast<unsigned>((tiles + y - 1) / y));
    }
    if (gated)
        launch_format<WAVES, MT, true>(a, format, grid, stream);
    else
        launch_format<WAVES, MT, false>(a, format, grid, stream);
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
    Args a;
    a.rows = static_cast<const uint8_t*>(rows);
    a.row_scales = row_scales;
    a.count = layout.count;
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
    const auto tiles = [&](int mc) { return experts + filled / mc; };
    // By the mean rows of an expert, measured at 64 experts, K 4096, N 1408:
    // bf16 rows 8: 44 us with the few-row kernel, 47 with 32-row tiles; 12: 51,
    // 48; 24: 90, 51 and 63 with 64-row tiles; 48 (skewed): 140 and 134; 128: 146
    // and 126.  FP8 rows, whose 64-row tile does not fit the registers: 12: 42,
    // 51; 48 (skewed): 234, 155.
    // Few-row kernel: two waves where four would have less than four steps each
    // (K 2048, 256 experts: 343 us against 403; K 7168: 589 against 587).
    // The many-row kernel gives 256 weight rows of a row tile to one workgroup, so
    // with few of those most CUs idle and the few-row kernel's smaller pieces win.
    // K 4096, bf16: 58 workgroups of 32 rows 28 us against 12 with the few-row
    // kernel, 116: 29 and 27, 232: 30 and 41; 40 of 64 rows: 37 and 26, 160: 40 and
    // 68; FP8: 58: 33 and 11, 72: 31 and 22, 232: 33 and 34, 288: 48 and 53.
    const bool fp8 = mm.in_format != 0;
    const int64_t blocks = (mm.out_features * (gated ? 2 : 1) + 4 * kRows - 1) / (4 * kRows);
    const auto many = [&](int rows, int mc) {
        return mean > rows && tiles(mc) * blocks > (fp8 ? 200 : 120);
    };
    if (!fp8 && many(40, 64))
        launch_rows<0, 4>(a, mm.in_format, gated, tiles(64), stream);
    else if (many(fp8 ? 16 : 8, 32))
        launch_rows<0, 2>(a, mm.in_format, gated, tiles(32), stream);
    else if (a.K < 4 * 4 * 2 * kStep)
        launch_rows<2, 1>(a, mm.in_format, gated, tiles(16), stream);
    else
        launch_rows<4, 1>(a, mm.in_format, gated, tiles(16), stream);
    return hipGetLastError();
}

}  // namespace ep
