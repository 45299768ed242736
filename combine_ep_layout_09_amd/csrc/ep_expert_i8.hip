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

#include <type_traits>

#include "ep_device.h"
#include "ep_expert_dev.h"
#include "ep_internal.h"

namespace ep {
namespace {

using namespace expert;

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));

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

// silu(v) = v / (1 + exp(-v)) with the hardware's exponential and reciprocal: a division
// and expf for each of a tile's outputs took a sixth of the many-row kernel's time.  Besides
// a few roundings of fp32, the exponent's rounded product and constant cost the exponential,
// and so silu below zero, a relative error of up to 1.3 |v| 2^-24: 2^-17 at v = -100, far
// below bf16's half step of 2^-8.
__device__ __forceinline__ float silu(float v) {
    return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.44269504f));
}

// The same for v below kFar.  The reciprocal returns no subnormal values: from 2^126 on, v
// below -87.3, it would be 0, where silu is still 2^-119.  So the exponential is
// taken 2^-32 smaller (the 1 is nothing beside it), which leaves its reciprocal normal down
// to v = -109, and the product then as much smaller, which rounds to fp32's subnormals.
constexpr float kFar = -44.0f;
__device__ __forceinline__ float silu_far(float v) {
    return v * __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(v * -1.44269504f - 32.0f)) * 0x1p-32f;
}

// One step's operands of a wave.
struct Stage {
    u32x4 w[2][kTiles];
    u32x4 x[2];
};

// Few rows per expert: the weights are the traffic and are read once.  A
// workgroup takes 64 weight rows of one expert against up to 16 rows; its WAVES
// waves take steps of 128 channels in turns and add their sums in LDS.  A load
// covers 8 weight rows x 128 bytes; two chunks change places across lanes afterwards
// (pair_chunks).  ONCE: K is a multiple of 128, so that these are whole cache lines, which
// are not kept; else two steps share lines, and not keeping them would read
// those twice (17 tokens over 32 experts, K 2672, N 7117: 86 us, not kept 101; decode batch, K 2048,
// N 7168: 568, kept 628).  GATED: tiles 0, 1 are
// rows n of the gate half and tiles 2, 3 rows N + n.
//
// Reading the weights bounds it.  128 tokens over 256 experts, top-8: K 7168, N 2048
// gated 1065 to 1070 us, 6.9 TB/s; K 2048, N 7168 560 to 572, 6.5 TB/s, 16 steps for
// four waves; one token, K 7168, N 2048 gated: 40 us, 5.9 TB/s.  Two waves take 37 there but
// 141 where four take 123 (64 experts of 8 rows, K 4096, N 1408 gated), and 18
// where four take 12 (32 of 6, K 4096, N 167).
template <int WAVES, bool GATED, bool ONCE>
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

    const Found f = find_tile<MC>(a, [](uint32_t) { return blockIdx.y; });
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
                s.w[i][t] = load16<ONCE>(t * 16 < kOut ? w_view : up_view,
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
        if constexpr (GATED)
            y = (y < kFar ? silu_far(y) : silu(y)) * scaled(up_sum, row_scale, a.scales[up_row + n]);
        a.out[(row0 + m) * N + n0 + n] = static_cast<uint16_t>(f32_to_bf16_rne(y));
    }
}

// Many rows per expert: a workgroup of eight waves takes 256 weight rows (GATED: 128
// of the gate and the 128 of up that belong to them) against up to 64 XT rows, a wave
// 128 of the former against 16 XT of the latter.  Stages of 128 channels pass
// through LDS, written by the loads themselves.
//
// A stage's row is 128 bytes, eight pieces; piece q of row r lies at place
// q ^ (r % 8), so that the 16 rows a fragment takes the same piece of are in
// different banks.  A load instruction fills 1 KB of LDS in lane order, eight
// rows, so its lanes fetch the pieces in that order.
//
// What is in flight bounds the loads, so LDS holds as much as fits: three stages of
// weights and, at XT = 4, two of rows, 160 KB in all.  Weights, which mostly come
// from HBM, are loaded two stages ahead, rows, which other workgroups of the XCD
// read as well, one.  (Loads alone at XT 2, 8192 skewed tokens over 64 experts: 721 us one
// stage ahead, 515 two.)  ONCE: up to XT 2 weights are not kept in the caches, which is
// faster where an expert has one row tile (64 experts, K 4096, N 1408 gated, 24 rows each: 134 us,
// kept 145; 64 rows 148 and 152), unless two stages share cache lines (K 3872, no multiple of
// 128, N 535 gated, 21 rows each of 256 experts: 233, not kept 271).  Where an expert has
// several, either side is ahead by case: 8 experts of 250 rows, K 4096, N 1408 gated 37.4, kept
// 39.8, 32 of 250 121 and 125, but 16 of 200, not gated, 41.7 and 38.5, 32 of 237 with as
// large a capacity, K 7168, N 946, 77.8 and 71.9.
//
// That batch, K 4096, N 1408 gated: 540 to 590 us by box, 1.9 to 2.1 POP/s; 49152 rows of one expert
// 2.35 POP/s; an 8192^3 int8 library product 2.06.  LDS and the matrix cores bound it
// together: fragments and stages take LDS as many cycles as the products take them, which
// are busy for 47 % of the time, at 2.0 to 2.1 GHz (435 us without loads, 449 without
// products).  4096 tokens over 256 experts, K 7168, N 2048 gated: 1463 to 1512 us, 5.2 to 5.4 TB/s
// with rows and outputs, 5.0 to 5.1 of weights.  Slower were matrix instructions of 32 x 32 x 32 (625 where this
// took 566), a stage through registers (648 where this took 596) and four waves of
// 128 x 128 (637 where this took 600).
constexpr int kTileWaves = 8;
constexpr int kTileW = 256;  // weight rows of a workgroup
constexpr int kTileGroup = 8;

template <bool ONCE>  // not kept in the caches
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t from, u32x4* to, uint32_t at,
                                         uint32_t step) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        from, reinterpret_cast<__attribute__((address_space(3))) void*>(reinterpret_cast<uintptr_t>(to)),
        16, at, step, 0, ONCE ? 2 : 0);
}

template <int XT, bool GATED, bool ONCE>
__global__ __launch_bounds__(kTileWaves* kWave, 2) void expert_i8_tile_kernel(Args a) {
    constexpr int MC = 64 * XT;
    constexpr int kOut = GATED ? kTileW / 2 : kTileW;  // outputs of a workgroup
    constexpr int WT = 8;                              // 16-row weight tiles of a wave
    constexpr int WB = 3, XB = XT == 4 ? 2 : 3;        // stages held
    __shared__ u32x4 s_w[WB * kTileW * 8];
    __shared__ u32x4 s_x[XB * MC * 8];

    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r16 = lane % 16, group = lane / 16;
    const uint32_t K = a.K;
    const int N = a.N;
    // Workgroups go round the 8 XCDs in turn.  Each XCD takes a run of items
    // (row tile, output block), so that its L2 serves one expert's weights to that
    // expert's tiles and one tile's rows to that tile's blocks.  Up to kTileGroup row
    // tiles of an expert take a block in turn before the next block: the weights,
    // the larger part, are then read by all of them at about the same time.
    const uint32_t n_blocks = (N + kOut - 1) / kOut;
    const uint64_t id = static_cast<uint64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
    uint32_t block = 0;
    Found f = find_tile<MC>(a, [&](uint32_t tiles) {
        const uint64_t items = static_cast<uint64_t>(tiles) * n_blocks;
        const uint64_t run = (items + 7) / 8;
        const uint64_t item = id % 8 * run + id / 8;
        if (id / 8 >= run || item >= items) return 0xffffffffu;
        block = static_cast<uint32_t>(item % n_blocks);
        return static_cast<uint32_t>(item / n_blocks);
    });
    if (f.expert < 0) return;
    {
        const int first = f.tile / kTileGroup * kTileGroup, left = (f.count + MC - 1) / MC - first;
        const uint32_t held = left < kTileGroup ? left : kTileGroup;
        const uint32_t item = (f.tile - first) * n_blocks + block;
        f.tile = first + item % held;
        block = item / held;
    }
    const int n0 = block * kOut;
    const int here = N - n0 < kOut ? N - n0 : kOut;
    const int m0 = f.tile * MC;
    const int rows_here = f.count - m0 < MC ? f.count - m0 : MC;
    if (rows_here <= 0) return;
    const int64_t row0 = f.start + m0;

    // Loads: wave i fills weight rows 32 i .. 32 i + 31 and rows 8 XT i .. of a
    // stage.  GATED: of each 128 weight rows 64 are gate and 64 up.
    const int64_t w_row = static_cast<int64_t>(f.expert) * (GATED ? 2 * N : N) + n0;
    const bool up = GATED && wave % 4 >= 2;
    const auto w_view = view(a.weights + (w_row + (up ? N : 0)) * K, here * K);
    const auto x_view = view(a.rows + row0 * K, rows_here * K);
    const uint32_t piece = (lane % 8 ^ lane / 8) * 16;
    const uint32_t w_first = (GATED ? wave / 4 * 64 + wave % 2 * 32 : wave * 32) + lane / 8;
    const uint32_t w_at = w_first * K + piece;
    const uint32_t x_at = (wave * 8 * XT + lane / 8) * K + piece;
    // channels c .. c + 127; zeros past the end, where nothing is read
    const auto load_w = [&](uint32_t c, int buf) {
        const bool has = c + piece < K;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            load_lds<ONCE>(w_view, &s_w[(buf * kTileW + wave * 32 + i * 8) * 8],
                     has ? w_at + i * 8 * K : kNowhere, c);
    };
    const auto load_x = [&](uint32_t c, int buf) {
        const bool has = c + piece < K;
#pragma unroll
        for (int i = 0; i < XT; ++i)
            load_lds<false>(x_view, &s_x[(buf * MC + wave * 8 * XT + i * 8) * 8],
                     has ? x_at + i * 8 * K : kNowhere, c);
    };

    // Products.  A wave multiplies those of its 16-row tiles that hold rows; waves
    // 0-3 take the first half of the rows, so that every SIMD has one wave of each half.
    const int w_half = wave % 2, x_group = wave / 2;
    const int tiles_here = (rows_here + 15) / 16 - x_group * XT;  // not positive: none
    const int place = r16 * 8 + (group ^ r16 % 8);  // of chunk 0; chunk 1: place ^ 4
    i32x4 acc[WT][XT];
#pragma unroll
    for (int t = 0; t < WT; ++t)
#pragma unroll
        for (int m = 0; m < XT; ++m) acc[t][m] = i32x4{0, 0, 0, 0};
    struct Frags {
        u32x4 w[WT], x[XT];
    };
    const auto fetch = [&](auto active, Frags& f, int w_buf, int x_buf, int h) {  // chunk h of a stage
        constexpr int M = decltype(active)::value;
        if constexpr (M == 0) return;
        const u32x4* w = &s_w[(w_buf * kTileW + w_half * 128) * 8];
        const u32x4* x = &s_x[(x_buf * MC + x_group * 16 * XT) * 8];
#pragma unroll
        for (int m = 0; m < M; ++m) f.x[m] = x[m * 128 + (place ^ 4 * h)];
#pragma unroll
        for (int t = 0; t < WT; ++t) f.w[t] = w[t * 128 + (place ^ 4 * h)];
    };
    const auto multiply = [&](auto active, const Frags& f) {
#pragma unroll
        for (int t = 0; t < WT; ++t)
#pragma unroll
            for (int m = 0; m < decltype(active)::value; ++m) acc[t][m] = mfma(f.w[t], f.x[m], acc[t][m]);
    };

    // The scales that the products take at the end, one per thread.
    float scale = 0.0f;
    {
        const int i = threadIdx.x % kTileW;
        const int n = GATED ? i / 128 * 64 + i % 64 : i;
        if (threadIdx.x < kTileW) {
            if (n < here) scale = a.scales[w_row + (GATED && i % 128 >= 64 ? N : 0) + n];
        } else if (i < rows_here) {
            scale = a.row_scales[row0 + i];
        }
    }
    // A wave's loads end in order: waiting until only the newest are left waits for
    // a stage's own.  Where every wave has waited, all of the stage is in LDS, and
    // the buffers that the waves are done with are free.  (A barrier that does not wait
    // for the loads behind it, which __syncthreads does.)
    constexpr int kAhead = XB == 3 ? 4 + XT : 4;  // loads of the stage ahead
    const auto stage_ready = [&] {
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(kAhead, 7, 0));
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    load_x(0, 0);
    load_w(0, 0);
    load_x(kStep, 1);
    load_w(kStep, 1);
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(4 + XT, 7, 15));
    if constexpr (XB == 3) load_x(2 * kStep, 2);
    load_w(2 * kStep, 2);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    // Each chunk's fragments are fetched while the chunk before is multiplied.  One
    // loop for each number of a wave's tiles, with the same barriers.
    const auto all_stages = [&](auto active) {
        int w_buf = 0, x_buf = 0;
        Frags even, odd;
        fetch(active, even, 0, 0, 0);
        for (uint32_t c = 0; c < K; c += kStep) {
            const int w_next = w_buf == WB - 1 ? 0 : w_buf + 1;
            const int x_next = x_buf == XB - 1 ? 0 : x_buf + 1;
            fetch(active, odd, w_buf, x_buf, 1);
            __builtin_amdgcn_sched_barrier(0);
            multiply(active, even);
            __builtin_amdgcn_sched_barrier(0);
            stage_ready();  // the next one; this one's buffers are free
            load_x(c + XB * kStep, x_buf);
            load_w(c + WB * kStep, w_buf);
            fetch(active, even, w_next, x_next, 0);
            __builtin_amdgcn_sched_barrier(0);
            multiply(active, odd);
            __builtin_amdgcn_sched_barrier(0);
            w_buf = w_next;
            x_buf = x_next;
        }
    };
    if (tiles_here >= XT)
        all_stages(std::integral_constant<int, XT>{});
    else if (XT > 3 && tiles_here == 3)
        all_stages(std::integral_constant<int, XT < 3 ? XT : 3>{});
    else if (XT > 2 && tiles_here == 2)
        all_stages(std::integral_constant<int, XT < 2 ? XT : 2>{});
    else if (XT > 1 && tiles_here == 1)
        all_stages(std::integral_constant<int, 1>{});
    else
        all_stages(std::integral_constant<int, 0>{});
    __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);  // loads of nothing, but into LDS
    __syncthreads();
    float* s_scale = reinterpret_cast<float*>(s_x);  // of the weight rows, then of the rows
    s_scale[threadIdx.x] = scale;
    __syncthreads();

    // Outputs change places in LDS, so that a row's leave together, 16 bytes a lane, at
    // whatever address: an odd N has rows of any alignment.  Lane l holds outputs 4 * (l / 16) .. + 3
    // of a tile for row l % 16; piece q (8 outputs) of row r lies at place q ^ (r % 16).
    // All rows at once, or those of waves 0-3 and of 4-7 in turn where they do not fit.
    constexpr int OT = GATED ? WT / 2 : WT;
    constexpr int kPieces = kOut / 8;
    constexpr int kTurns = MC * kOut * 2 > static_cast<int>(sizeof(s_w)) ? 2 : 1;
    constexpr int kTurnRows = MC / kTurns;
    uint2* s_out = reinterpret_cast<uint2*>(s_w);
    const float* w_scale = &s_scale[w_half * 128 + group * 4];
#pragma unroll
    for (int turn = 0; turn < kTurns; ++turn) {
        if (turn > 0) __syncthreads();
        if (x_group / (4 / kTurns) == turn) {
#pragma unroll
            for (int m = 0; m < XT; ++m) {
                if (m >= tiles_here) break;
                const int r = (x_group * XT + m) * 16 + r16;
                const float row_scale = s_scale[kTileW + r];
                // Gates far below zero hardly occur: outputs are made as if there were none, and
                // those of a wave that has some once more (600 tokens over 8 experts, top-6, K 256,
                // N 1408: 12.2 us, without the far ones 11.9, a choice for each output 12.8).
                float low = 0.0f;
                const auto put = [&](auto activation) {
#pragma unroll
                    for (int t = 0; t < OT; ++t) {
                        const int n = (w_half * OT + t) * 16 + group * 4;
                        float y[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            y[i] = scaled(acc[t][m][i], row_scale, w_scale[t * 16 + i]);
                            if constexpr (GATED) {
                                low = fminf(low, y[i]);
                                y[i] = activation(y[i]) *
                                       scaled(acc[t + OT][m][i], row_scale, w_scale[(t + OT) * 16 + i]);
                            }
                        }
                        const int at = (r - turn * kTurnRows) * kPieces + (n / 8 ^ r16);
                        s_out[at * 2 + n / 4 % 2] =
                            make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
                    }
                };
                put([](float v) { return silu(v); });
                if constexpr (GATED) {
                    if (__ballot(low < kFar) != 0)
                        put([](float v) { return v < kFar ? silu_far(v) : silu(v); });
                }
            }
        }
        __syncthreads();
        const int rows_now = rows_here - turn * kTurnRows < kTurnRows ? rows_here - turn * kTurnRows : kTurnRows;
        for (int i = threadIdx.x; i < rows_now * kPieces; i += kTileWaves * kWave) {
            const int r = i / kPieces, q = i % kPieces;
            const u32x4 v = reinterpret_cast<const u32x4*>(s_w)[r * kPieces + (q ^ r % 16)];
            uint16_t* to = a.out + (row0 + turn * kTurnRows + r) * N + n0 + q * 8;
            if (q * 8 + 8 <= here) {
                *reinterpret_cast<u32x4_at2*>(to) = v;
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (q * 8 + k < here) to[k] = static_cast<uint16_t>(v[k / 2] >> (16 * (k % 2)));
            }
        }
    }
}

template <int XT, bool GATED, bool ONCE>
void launch_many(const Args& a, int64_t tiles, hipStream_t stream) {
    const int outs = GATED ? kTileW / 2 : kTileW;
    const int64_t blocks = (a.N + outs - 1) / outs;
    const int64_t items = (tiles * blocks + 7) / 8 * 8;  // a row of ids whose length 8 divides
    const int64_t x = items < (1 << 20) ? items : 1 << 20;
    const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>((items + x - 1) / x));
    hipLaunchKernelGGL((expert_i8_tile_kernel<XT, GATED, ONCE>), grid, dim3(kTileWaves * kWave), 0,
                       stream, a);
}

// Where this kernel is taken there are fewer than 2000 tiles: 1024 experts of a mean of 12
// rows, or 512 workgroups.
template <int WAVES, bool GATED, bool ONCE>
void launch_few(const Args& a, int64_t tiles, hipStream_t stream) {
    const int outs = GATED ? kRows / 2 : kRows;
    const dim3 grid((a.N + outs - 1) / outs, static_cast<unsigned>(tiles));
    hipLaunchKernelGGL((expert_i8_kernel<WAVES, GATED, ONCE>), grid, dim3(WAVES * kWave), 0, stream, a);
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
    const int64_t mean = filled / experts;
    const auto tiles = [&](int64_t mc) {
        const int64_t most = experts + filled / mc;
        const int64_t held_tiles = p.num_experts * ((p.capacity + mc - 1) / mc);
        return p.capacity > 0 && held_tiles < most ? held_tiles : most;
    };
    // Few rows: up to a mean of 12 (64 experts, K 4096, N 1408 gated, rows each, us:
    //   rows   8    12   16   24   48   64   75   96   112  121  128
    //   few    122  135  168  231  379
    //   XT 1   127  137  128  140  139  163  192
    //   XT 2   128  138  129  142  140  146  153  156  168  183  215
    //   XT 4                                 162  162  177  172  180),
    // and where the CUs hold all of the few-row kernel's workgroups at once (32 experts of 25
    // rows, N 167: 246 of them 14 us, XT 1 22; 8 of 16, K 2048, N 1024: 256, 9 and 15;
    // 32 of 100, N 167: 696, 35 and 24).
    // Of the many-row kernel's tiles those whose rounds over 256 CUs cost the least; a
    // workgroup of XT 1, 2, 4 takes as 10, 12, 16 do (8 experts of 250 rows, K 4096, N 704 gated, one
    // round each: 29, 35 and 49 us; of 1000 rows two rounds of XT 2 68, one of XT 4 53; 32 of 237,
    // K 7120, N 946: two rounds of XT 1 169, one of XT 2 121, of XT 4 148, half of its CUs idle).
    // Half a tile per expert is taken to be empty.
    const int64_t rows2 = static_cast<int64_t>(a.N) * (mm.activation == 1 ? 2 : 1);
    const auto rounds = [&](int64_t mc) {
        int64_t n = experts / 2 + filled / mc;
        if (n < experts) n = experts;
        if (n > tiles(mc)) n = tiles(mc);
        return (n * ((rows2 + kTileW - 1) / kTileW) + 255) / 256;
    };
    const int64_t cost1 = 10 * rounds(64), cost2 = 12 * rounds(128), cost4 = 16 * rounds(256);
    const auto go = [&](auto gated, auto once) {
        constexpr bool kGated = decltype(gated)::value, kOnce = decltype(once)::value;
        if (mean <= 12 || tiles(16) * ((rows2 + kRows - 1) / kRows) <= 512)
            launch_few<4, kGated, kOnce>(a, tiles(16), stream);
        else if (cost1 <= cost2 && cost1 <= cost4)
            launch_many<1, kGated, kOnce>(a, tiles(64), stream);
        else if (cost2 <= cost4)
            launch_many<2, kGated, kOnce>(a, tiles(128), stream);
        else
            launch_many<4, kGated, false>(a, tiles(256), stream);
    };
    const auto go_once = [&](auto once) {
        if (mm.activation == 1)
            go(std::true_type{}, once);
        else
            go(std::false_type{}, once);
    };
    if (a.K % kStep == 0)
        go_once(std::true_type{});
    else
        go_once(std::false_type{});
    return hipGetLastError();
}

}  // namespace ep
