// ep_norm.hip -- layer norm of token rows and its backward pass.
//
//   y  = (x - m) r w + b,   m = mean(x),  r = 1 / sqrt(mean((x - m)^2) + eps)
//   dx = r (a - mean(a) - n mean(a n)) + skip,   n = (x - m) r,  a = dy w
//   dw = sum_t dy n,   db = sum_t dy
//
// Rows are moved in 16-byte pieces of P channels (8 bf16 or 4 fp32), at any
// alignment that the element type allows.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ep_internal.h"
#include "ep_norm_dev.h"

namespace ep {
namespace {

using namespace norm;

constexpr int kMaxThreads = 1024;

// Workgroups in rows of 2^20, since a dimension of a grid has to stay below 2^32
// threads.
__device__ __forceinline__ int64_t block_number() {
    return static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
}
dim3 grid_of(int64_t blocks) {
    const int64_t x = blocks < (1 << 20) ? blocks : 1 << 20;
    return dim3(static_cast<unsigned>(x), static_cast<unsigned>((blocks + x - 1) / x));
}

// A group of L lanes (a multiple of 64 that divides the workgroup) takes B rows,
// which it holds in registers between the statistics and the output: x is read
// once, and m is known before the squares of x - m are added.  B rows share each
// load of weight and bias, which as fp32 are four times the bytes of a bf16 row: from
// 4096 rows on two, which leaves one row per group where rows are few.
//
// Memory bounds it: 16384 x 7168 bf16 85 us, 5.5 TB/s (a 4 GiB copy: 4.8), 94 with one
// row per load of weight and bias, 103 with rows kept in the caches as well; 77 without
// weight and bias.  One wave per row with both in LDS took 96: four waves per SIMD
// are too few for a load, three passes over the row and a store in turn.
template <bool XB, bool WB, int VPL, int B>
__global__ __launch_bounds__(kMaxThreads) void norm_kernel(NormArgs a, int L) {
    typedef Piece<XB> X;
    typedef typename X::T T;
    constexpr int P = X::P;
    __shared__ float s_part[2][B][kMaxThreads / kWave];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int waves = L / kWave, group = wave / waves, wave0 = group * waves;
    const int l = threadIdx.x - group * L;
    const int64_t t0 = (block_number() * (blockDim.x / L) + group) * B;
    X x[B][VPL];
#pragma unroll
    for (int b = 0; b < B; ++b) {
        const auto row = row_view<T>(a.x, t0 + b, a.x_stride, a.hidden, t0 + b < a.num_tokens);
#pragma unroll
        for (int u = 0; u < VPL; ++u) x[b][u].load(row, (l + u * L) * P, a.hidden);
    }
    // Registers: between its uses a row is kept as it came, not as fp32 values.
    const auto as_it_came = [&] {
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
            for (int u = 0; u < VPL; ++u) asm volatile("" : "+v"(x[b][u].v));
    };
    float m[B], r[B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
        m[b] = 0.0f;
#pragma unroll
        for (int u = 0; u < VPL; ++u)
#pragma unroll
            for (int i = 0; i < P; ++i) m[b] += x[b][u].at(i);
    }
    group_sums(m, s_part[0], wave0, waves, wave);
    as_it_came();
#pragma unroll
    for (int b = 0; b < B; ++b) {
        m[b] /= a.hidden;
        r[b] = 0.0f;
#pragma unroll
        for (int u = 0; u < VPL; ++u) {
            const int left = a.hidden - (l + u * L) * P;  // channels from this piece on
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float d = i < left ? x[b][u].at(i) - m[b] : 0.0f;
                r[b] = fmaf(d, d, r[b]);
            }
        }
    }
    group_sums(r, s_part[1], wave0, waves, wave);
    as_it_came();
#pragma unroll
    for (int b = 0; b < B; ++b) {
        r[b] = 1.0f / sqrtf(r[b] / a.hidden + a.eps);
        if (l == 0 && a.mean != nullptr && t0 + b < a.num_tokens) {
            a.mean[t0 + b] = m[b];
            a.rstd[t0 + b] = r[b];
        }
    }
#pragma unroll
    for (int u = 0; u < VPL; ++u) {
        const int c = (l + u * L) * P;
        float w[P], p[P], y[P];
        load_params<P, WB>(a.weight, c, a.hidden, 1.0f, w);
        load_params<P, WB>(a.bias, c, a.hidden, 0.0f, p);
#pragma unroll
        for (int b = 0; b < B; ++b) {
#pragma unroll
            for (int i = 0; i < P; ++i) y[i] = fmaf((x[b][u].at(i) - m[b]) * r[b], w[i], p[i]);
            X::store(row_view<T>(a.y, t0 + b, a.hidden, a.hidden, t0 + b < a.num_tokens), c, a.hidden,
                     y);
        }
    }
}

// The whole backward pass in one reading of the rows.  A group of L lanes takes
// B rows at a time, a lane V pieces of each at the same channels all along, so
// that its sums for the gradients of weight and bias stay in registers: V P of each.
// The next rows are loaded before these ones' sums are joined.  A workgroup's groups
// join their sums in LDS, a single group's leave as they are: one part of both gradients
// (norm_join_kernel).
//
// Memory bounds it: 4096 x 7168 bf16 with d_skip 49.5 us for both kernels, 4.75 TB/s of what the
// call has to move and 7 % more in parts (a single group's sums through LDS as well: 52); 86 with
// the rows read a second time for the sums over tokens.  1999 x 1409 fp32: 12.9 us for both, which by
// themselves take 10.6 and 3.8: starts and ends, 7.1 of bytes.  More than 8192 bf16 channels leave
// CUs without a workgroup (norm_parts): 4096 x 12288 98 us, 4.1 TB/s, 4096 x 16384 137, 3.9.

// Sums of B pairs of values over the lanes of a group; parts: B pairs per wave.
template <int B>
__device__ __forceinline__ void pair_sums(float (&c1)[B], float (&c2)[B],
                                          float (*parts)[2 * B], int wave0, int waves,
                                          int wave) {
    float v[2 * B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
        v[2 * b] = wave_sum(c1[b]);
        v[2 * b + 1] = wave_sum(c2[b]);
    }
    if (waves > 1) {
        const int lane = threadIdx.x % kWave;
        if (lane < 2 * B) {
            float own = v[0];
#pragma unroll
            for (int i = 1; i < 2 * B; ++i) own = lane == i ? v[i] : own;
            parts[wave][lane] = own;
        }
        __syncthreads();
        // lane i of a row of 16 takes wave i's values
        const bool has = lane % 16 < waves;
#pragma unroll
        for (int i = 0; i < 2 * B; ++i) v[i] = has ? parts[wave0 + lane % 16][i] : 0.0f;
#pragma unroll
        for (int i = 0; i < 2 * B; ++i) v[i] = row16_sum(v[i]);
    }
#pragma unroll
    for (int b = 0; b < B; ++b) {
        c1[b] = v[2 * b];
        c2[b] = v[2 * b + 1];
    }
}

template <bool XB, bool WB, int V, int B>
__global__ __launch_bounds__(kMaxThreads) void norm_grad_kernel(NormGradArgs a, int L, float* parts) {
    typedef Piece<XB> X;
    constexpr int P = X::P;
    __shared__ float s_part[2][kMaxThreads / kWave][2 * B];
    __shared__ __attribute__((aligned(16))) float s_sum[2][V][P / 4][kMaxThreads][4];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int waves = L / kWave, group = wave / waves, wave0 = group * waves;
    const int l = threadIdx.x - group * L, groups = blockDim.x / L;
    const int64_t step = static_cast<int64_t>(gridDim.x) * groups * B;
    float w[V][P], dw[V][P], db[V][P];
#pragma unroll
    for (int u = 0; u < V; ++u) {
        const int c = (l + u * L) * P;
        load_params<P, WB>(a.weight, c, a.hidden, 1.0f, w[u]);
#pragma unroll
        for (int i = 0; i < P; ++i) dw[u][i] = db[u][i] = 0.0f;
    }
    struct Rows {
        X x[B][V], g[B][V], s[B][V];
        float m[B], r[B];
    };
    typedef typename X::T T;
    const auto load = [&](Rows& q, int64_t t0) {
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const bool there = t0 + b < a.num_tokens;
            const int64_t t = there ? t0 + b : 0;
            q.m[b] = there ? a.mean[t] : 0.0f;
            q.r[b] = there ? a.rstd[t] : 0.0f;
            const auto xv = row_view<T>(a.x, t, a.x_stride, a.hidden, there);
            const auto gv = row_view<T>(a.dy, t, a.dy_stride, a.hidden, there);
            const auto sv = row_view<T>(a.d_skip, t, a.hidden, a.hidden, there);
#pragma unroll
            for (int u = 0; u < V; ++u) {
                q.x[b][u].load(xv, (l + u * L) * P, a.hidden);
                q.g[b][u].load(gv, (l + u * L) * P, a.hidden);
                q.s[b][u].load(sv, (l + u * L) * P, a.hidden);
            }
        }
    };
    // Two pieces of bf16 rows leave no registers for rows ahead.
    constexpr bool kAhead = !(XB && V == 2);
    Rows now, next;
    int64_t t0 = (static_cast<int64_t>(blockIdx.x) * groups + group) * B;
    // every group of the workgroup takes as many turns, for the barriers
    const int64_t first = static_cast<int64_t>(blockIdx.x) * groups * B;
    if constexpr (kAhead) load(now, t0);
    int turn = 0;
#pragma unroll 1
    for (int64_t at = first; at < a.num_tokens; at += step, t0 += step, turn ^= 1) {
        if constexpr (kAhead)
            load(next, t0 + step);
        else
            load(now, t0);
        float c1[B], c2[B];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            c1[b] = c2[b] = 0.0f;
#pragma unroll
            for (int u = 0; u < V; ++u)
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const float g = now.g[b][u].at(i), v = g * w[u][i];
                    const float n = (now.x[b][u].at(i) - now.m[b]) * now.r[b];
                    c1[b] += v;
                    c2[b] = fmaf(v, n, c2[b]);
                    db[u][i] += g;
                    dw[u][i] = fmaf(g, n, dw[u][i]);
                }
            __builtin_amdgcn_sched_barrier(0);  // one row's values at a time: registers
        }
        pair_sums(c1, c2, s_part[turn], wave0, waves, wave);
        // what was made of the rows is made again, not kept: registers
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
            for (int u = 0; u < V; ++u) asm volatile("" : "+v"(now.x[b][u].v), "+v"(now.g[b][u].v));
#pragma unroll
        for (int b = 0; b < B; ++b) {
            if (t0 + b >= a.num_tokens) continue;
            const float a1 = c1[b] / a.hidden, a2 = c2[b] / a.hidden;
            const auto dx = row_view<T>(a.dx, t0 + b, a.hidden, a.hidden, true);
#pragma unroll
            for (int u = 0; u < V; ++u) {
                const int c = (l + u * L) * P;
                float d[P];
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const float n = (now.x[b][u].at(i) - now.m[b]) * now.r[b];
                    d[i] = fmaf(now.r[b], fmaf(-n, a2, now.g[b][u].at(i) * w[u][i] - a1),
                                now.s[b][u].at(i));
                }
                X::store(dx, c, a.hidden, d);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (kAhead) now = next;
    }
    if (a.d_weight == nullptr && a.d_bias == nullptr) return;
    if (groups == 1 && gridDim.x > 1) {  // the lanes' sums are the part
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const auto part = view(parts + (static_cast<int64_t>(blockIdx.x) * 2 + which) * a.hidden,
                                   a.hidden * 4);
#pragma unroll
            for (int u = 0; u < V; ++u)
#pragma unroll
                for (int i = 0; i < P; i += 4) {
                    const auto word = [&](int j) {
                        return __float_as_uint(which == 0 ? dw[u][i + j] : db[u][i + j]);
                    };
                    __builtin_amdgcn_raw_buffer_store_b128(u32x4{word(0), word(1), word(2), word(3)},
                                                           part, ((l + u * L) * P + i) * 4, 0, 0);
                }
        }
        return;
    }
    // Through LDS, to this workgroup's part, or, where it is the only one, to the gradient
    // itself.
#pragma unroll
    for (int which = 0; which < 2; ++which)
#pragma unroll
        for (int u = 0; u < V; ++u)
#pragma unroll
            for (int i = 0; i < P; ++i)
                s_sum[which][u][i / 4][threadIdx.x][i % 4] = which == 0 ? dw[u][i] : db[u][i];
    __syncthreads();
#pragma unroll
    for (int u = 0; u < V; ++u) {
        const int c0 = u * L * P, end = min(L * P, a.hidden - c0);
        for (int c = threadIdx.x; c < end; c += blockDim.x) {
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                float sum = 0.0f;
                for (int q = 0; q < groups; ++q) sum += s_sum[which][u][c % P / 4][q * L + c / P][c % 4];
                if (gridDim.x == 1)
                    store_param<WB>(which == 0 ? a.d_weight : a.d_bias, c0 + c, sum);
                else
                    parts[(static_cast<int64_t>(blockIdx.x) * 2 + which) * a.hidden + c0 + c] = sum;
            }
        }
    }
}

// Rows longer than 2048 pieces, whose sums over tokens do not fit the registers.
// Gradient of the rows: a workgroup, of 512 or 1024 lanes at these lengths, takes a row,
// reads it once for the two means and once more for dx.
template <bool XB, bool WB>
__global__ __launch_bounds__(kMaxThreads) void norm_rows_kernel(NormGradArgs a) {
    typedef Piece<XB> X;
    constexpr int P = X::P;
    __shared__ float s_part[2][kMaxThreads / kWave];
    const int l = threadIdx.x, L = blockDim.x;
    const int64_t t = block_number();
    const bool there = t < a.num_tokens;
    typedef typename X::T T;
    const int H = a.hidden;
    const int64_t at = there ? t : 0;
    const auto xr = row_view<T>(a.x, t, a.x_stride, H, there);
    const auto gr = row_view<T>(a.dy, t, a.dy_stride, H, there);
    const float m = a.mean[at], r = a.rstd[at];
    float c1 = 0.0f, c2 = 0.0f;
    for (int c = l * P; c < H; c += L * P) {
        X x, g;
        x.template load<0>(xr, c, H);
        g.template load<0>(gr, c, H);
        float w[P];
        load_params<P, WB>(a.weight, c, H, 1.0f, w);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float v = g.at(i) * w[i];  // 0 behind the row's end
            c1 += v;
            c2 = fmaf(v, (x.at(i) - m) * r, c2);
        }
    }
    c1 = workgroup_sum(c1, s_part[0]) / a.hidden;
    c2 = workgroup_sum(c2, s_part[1]) / a.hidden;
    const auto out = row_view<T>(a.dx, t, H, H, there);
    const auto skip = row_view<T>(a.d_skip, t, H, H, there);
    for (int c = l * P; c < H; c += L * P) {
        X x, g, s;
        x.load(xr, c, H);
        g.load(gr, c, H);
        s.load(skip, c, H);
        float w[P], d[P];
        load_params<P, WB>(a.weight, c, H, 1.0f, w);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float n = (x.at(i) - m) * r;
            d[i] = fmaf(r, fmaf(-n, c2, g.at(i) * w[i] - c1), s.at(i));
        }
        X::store(out, c, H, d);
    }
}

// Sums over a run of rows for the gradients of weight and bias: a workgroup takes
// 64 P channels, its waves the rows of the run in turns, joined in wave order.
constexpr int kColumnWaves = 4;
template <bool XB>
__global__ __launch_bounds__(kColumnWaves* kWave) void norm_columns_kernel(NormGradArgs a, int run,
                                                                           float* parts) {
    typedef Piece<XB> X;
    constexpr int P = X::P;
    __shared__ float s_sum[kColumnWaves][2][kWave * P];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int c0 = blockIdx.x * kWave * P, c = c0 + lane * P;
    const int64_t first = static_cast<int64_t>(blockIdx.y) * run;
    const int64_t end = min(first + run, static_cast<int64_t>(a.num_tokens));
    float dw[P], db[P];
#pragma unroll
    for (int i = 0; i < P; ++i) dw[i] = db[i] = 0.0f;
    for (int64_t t = first + wave; t < end; t += kColumnWaves) {
        X x, g;
        x.load(row_view<typename X::T>(a.x, t, a.x_stride, a.hidden, true), c, a.hidden);
        g.load(row_view<typename X::T>(a.dy, t, a.dy_stride, a.hidden, true), c, a.hidden);
        const float m = a.mean[t], r = a.rstd[t];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            db[i] += g.at(i);
            dw[i] = fmaf(g.at(i), (x.at(i) - m) * r, dw[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
        s_sum[wave][0][lane * P + i] = dw[i];
        s_sum[wave][1][lane * P + i] = db[i];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * kWave * P; i += kColumnWaves * kWave) {
        const int which = i / (kWave * P), at = i % (kWave * P);
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kColumnWaves; ++w) s += s_sum[w][which][at];
        if (c0 + at < a.hidden)
            parts[(static_cast<int64_t>(blockIdx.y) * 2 + which) * a.hidden + c0 + at] = s;
    }
}

// The parts [n][2][H] of the runs, added: 64 sums per workgroup, the parts taken
// by its waves in turns.
constexpr int kJoinWaves = 16;
template <bool WB>
__global__ __launch_bounds__(kJoinWaves* kWave) void norm_join_kernel(const float* parts, int n, int H,
                                                                      void* dw, void* db) {
    __shared__ float s_sum[kJoinWaves][kWave];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int i = blockIdx.x * kWave + lane;  // of 2 H
    float s = 0.0f;
    if (i < 2 * H) {
        const float* from = parts + i;
        // eight parts on their way at a time
        for (int p = wave; p < n; p += 8 * kJoinWaves) {
            float v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const int at = p + q * kJoinWaves;
                v[q] = at < n ? from[static_cast<int64_t>(at) * 2 * H] : 0.0f;
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) s += v[q];
        }
    }
    s_sum[wave][lane] = s;
    __syncthreads();
    if (wave != 0 || i >= 2 * H) return;
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWaves; ++w) s += s_sum[w][lane];
    store_param<WB>(i < H ? dw : db, i < H ? i : i - H, s);
}

// Lanes per row: as few as hold the row with at most `most` pieces each, more
// where there are too few rows to fill the GPU.
int lanes_per_row(int pieces, int most, int64_t tokens) {
    int L = kWave;
    while (L < kMaxThreads && pieces > most * L) L *= 2;
    while (L < kMaxThreads && L < pieces && tokens * (L / kWave) < 2048) L *= 2;
    return L;
}

template <bool XB, bool WB, int B>
void launch_norm_rows(const NormArgs& a, int pieces, int L, hipStream_t stream) {
    const int threads = L < 256 ? 256 : L;
    const int rows = threads / L * B;
    const dim3 grid = grid_of((a.num_tokens + rows - 1) / rows);
    const auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(threads), 0, stream, a, L);
    };
    switch ((pieces + L - 1) / L) {
        case 1: go(norm_kernel<XB, WB, 1, B>); break;
        case 2: go(norm_kernel<XB, WB, 2, B>); break;
        case 3: go(norm_kernel<XB, WB, 3, B>); break;
        case 4: go(norm_kernel<XB, WB, 4, B>); break;
        case 5: go(norm_kernel<XB, WB, 5, B>); break;
        case 6: go(norm_kernel<XB, WB, 6, B>); break;
        case 7: go(norm_kernel<XB, WB, 7, B>); break;
        case 8: go(norm_kernel<XB, WB, 8, B>); break;
        default:  // fp32 rows of more than 32768 channels
            if constexpr (!XB && B == 1) go(norm_kernel<XB, WB, 16, 1>);
    }
}

template <bool XB, bool WB>
void launch_norm_types(const NormArgs& a, hipStream_t stream) {
    const int pieces = (a.hidden + Piece<XB>::P - 1) / Piece<XB>::P;
    const int L = lanes_per_row(pieces, 8, a.num_tokens);
    if (a.num_tokens >= 4096 && pieces <= 8 * L)
        launch_norm_rows<XB, WB, 2>(a, pieces, L, stream);
    else
        launch_norm_rows<XB, WB, 1>(a, pieces, L, stream);
}

template <bool WB>
void launch_join(const NormGradArgs& a, const float* parts, int n, hipStream_t stream) {
    hipLaunchKernelGGL((norm_join_kernel<WB>), dim3((2 * a.hidden + kWave - 1) / kWave),
                       dim3(kJoinWaves * kWave), 0, stream, parts, n, a.hidden, a.d_weight, a.d_bias);
}

template <bool XB, bool WB>
hipError_t launch_norm_grad_types(const NormGradArgs& a, void* workspace, hipStream_t stream) {
    const int P = Piece<XB>::P;
    const int pieces = (a.hidden + P - 1) / P;
    const bool params = a.d_weight != nullptr || a.d_bias != nullptr;
    float* parts = static_cast<float*>(workspace);
    const int most = a.num_tokens > 0 ? norm_parts(a.num_tokens, a.hidden) : 0;
    int n = 0;  // parts written
    bool joined = false;
    if (a.num_tokens > 0 && pieces <= 2 * kMaxThreads) {
        const int lanes = (pieces <= kMaxThreads ? pieces : (pieces + 1) / 2);
        const int L = (lanes + kWave - 1) / kWave * kWave;
        const int groups = kMaxThreads / L;
        const auto go = [&](auto kernel, int rows) {  // rows of a group's turn
            const int each = groups * rows, turns = (a.num_tokens + each - 1) / each;
            // Few rows: one workgroup, whose sums are the gradients (one row of 7168: 9.7 us,
            // 12.3 with a second launch; four turns of two rows: 19 and 11.5).  Without them there is no
            // second launch to save (four rows: 6.5, by one workgroup 9.6).
            // Otherwise as many workgroups as take their turns in the time of the fullest: a last turn
            // of a few would leave as many parts (264 x 6712 fp32: 132 workgroups 16.2 us, 256 19.3;
            // 6278 x 4096 bf16: 242 45.1, 256 48.0).
            const int rounds = (turns + most - 1) / most;
            n = turns <= 2 && params ? 1 : (turns + rounds - 1) / rounds;
            hipLaunchKernelGGL(kernel, dim3(n), dim3(groups * L), 0, stream, a, L, parts);
            if (n == 1) joined = true;
        };
        if (pieces <= kMaxThreads)
            go(norm_grad_kernel<XB, WB, 1, 2>, 2);
        else
            go(norm_grad_kernel<XB, WB, 2, 1>, 1);
    } else if (a.num_tokens > 0) {
        hipLaunchKernelGGL((norm_rows_kernel<XB, WB>), grid_of(a.num_tokens),
                           dim3(lanes_per_row(pieces, 8, a.num_tokens)), 0, stream, a);
        if (params) {
            const int run = (a.num_tokens + most - 1) / most;
            n = (a.num_tokens + run - 1) / run;
            hipLaunchKernelGGL((norm_columns_kernel<XB>), dim3((pieces + kWave - 1) / kWave, n),
                               dim3(kColumnWaves * kWave), 0, stream, a, run, parts);
        }
    }
    if (params && !joined) launch_join<WB>(a, parts, n, stream);
    return hipGetLastError();
}

}  // namespace

// Partial sums of the gradients of weight and bias: at most one per CU, and at
// most 2^21 channels of them (16 MB).  As many workgroups make them at most, with those sums or
// without: 170 for rows of 12288 channels, 128 for 16384.
int norm_parts(int num_tokens, int hidden) {
    int n = 256;
    if (n > (1 << 21) / hidden) n = (1 << 21) / hidden;
    return n < num_tokens ? n : num_tokens;
}

int64_t norm_workspace_bytes(int num_tokens, int hidden) {
    const int64_t n = norm_parts(num_tokens, hidden);
    return (n * 2 * hidden * 4 + 255) / 256 * 256;
}

hipError_t launch_norm(const NormArgs& a, bool x_bf16, bool w_bf16, hipStream_t stream) {
    if (a.num_tokens == 0) return hipSuccess;
    if (x_bf16 && w_bf16) launch_norm_types<true, true>(a, stream);
    if (x_bf16 && !w_bf16) launch_norm_types<true, false>(a, stream);
    if (!x_bf16 && w_bf16) launch_norm_types<false, true>(a, stream);
    if (!x_bf16 && !w_bf16) launch_norm_types<false, false>(a, stream);
    return hipGetLastError();
}

hipError_t launch_norm_grad(const NormGradArgs& a, bool x_bf16, bool w_bf16, void* workspace,
                            hipStream_t stream) {
    if (x_bf16 && w_bf16) return launch_norm_grad_types<true, true>(a, workspace, stream);
    if (x_bf16) return launch_norm_grad_types<true, false>(a, workspace, stream);
    if (w_bf16) return launch_norm_grad_types<false, true>(a, workspace, stream);
    return launch_norm_grad_types<false, false>(a, workspace, stream);
}

}  // namespace ep
