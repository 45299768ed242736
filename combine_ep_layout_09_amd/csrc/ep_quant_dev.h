// ep_quant_dev.h -- rows as 8-bit integers with one scale per row.
//
//   scale = amax / 127,  q = round-to-nearest-even(fl(x / scale))
//
// both quotients IEEE fp32.  A workgroup holds a row, VPL 16-byte pieces of 8
// bf16 channels per lane.
#pragma once

#include "ep_dispatch_dev.h"

namespace ep {
namespace quant {

using dispatch::u32x2;
using dispatch::u32x4;

// Codes of the 8 channels of a piece (scale == 0: all codes 0; x finite).
//
// One reciprocal per piece instead of a division per channel: r = fl(1 / scale) and
// p = fl(x r) carry two roundings, so p lies within 3 * 2^-24 |q| < 2^-15 of the
// quotient q.  Where p is further than that from the middle between two integers,
// both round to the same one.  A channel next to a middle, and every
// channel when r is not finite (scale below 2^-128), takes the division, in a branch a wave
// enters only when one of its lanes needs it.  |q| < 127.5: the scale's own rounding
// moves the largest quotient by 2^-24 of it, or, where the scale is subnormal, by
// 2^-10, since the smallest bf16 magnitude over 127 is more than 512 fp32 units.
__device__ __forceinline__ u32x2 codes8(const u32x4& w, float scale) {
    u32x2 q = {0, 0};
    if (scale == 0.0f) return q;
    const float f[8] = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y),
                        bf16_lo(w.z), bf16_hi(w.z), bf16_lo(w.w), bf16_hi(w.w)};
    const float r = 1.0f / scale;
    const bool r_ok = __float_as_uint(r) < 0x7f800000u;
    // Added to 1.5 * 2^23, a value rounds to an integer whose two's complement is
    // in the sum's low bits.
    constexpr float kInt = 0x1.8p23f;
    float s[8], far = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float p = f[i] * r;
        s[i] = p + kInt;
        far = fmaxf(far, fabsf(p - (s[i] - kInt)));
    }
    const bool divide = !r_ok || far >= 0.5f - 0x1p-15f;
    if (__ballot(divide) != 0 && divide) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = f[i] / scale + kInt;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const auto b = [&](int i) { return __float_as_uint(s[4 * h + i]); };
        const uint32_t lo = __builtin_amdgcn_perm(b(1), b(0), 0x0c0c0400u);
        const uint32_t hi = __builtin_amdgcn_perm(b(3), b(2), 0x04000c0cu);
        q[h] = lo | hi;
    }
    return q;
}

// Largest of non-negative values over the workgroup's waves; parts: one float per wave.
__device__ __forceinline__ float workgroup_max(float v, float* parts) {
    v = dispatch::row16_max(v);
    const auto lane = [&](int i) {
        return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), i));
    };
    v = fmaxf(fmaxf(lane(0), lane(16)), fmaxf(lane(32), lane(48)));
    const int waves = blockDim.x / kWave;
    if (waves == 1) return v;
    if (threadIdx.x % kWave == 0) parts[threadIdx.x / kWave] = v;
    __syncthreads();
    for (int i = 0; i < waves; ++i) v = fmaxf(v, parts[i]);
    return v;
}

// A row of nvec pieces: lane i holds the pieces i, i + blockDim.x, ...
template <int VPL>
struct Row {
    u32x2 q[VPL];
    float scale;

    __device__ __forceinline__ void load(const u32x4* __restrict__ row, int nvec, float* parts) {
        u32x4 x[VPL];
        float top = 0.0f;
#pragma unroll
        for (int u = 0; u < VPL; ++u) {
            // lanes past the end redo the last piece
            x[u] = row[min(static_cast<int>(threadIdx.x + u * blockDim.x), nvec - 1)];
            top = fmaxf(top, dispatch::absmax8(x[u]));
        }
        scale = workgroup_max(top, parts) / 127.0f;
#pragma unroll
        for (int u = 0; u < VPL; ++u) q[u] = codes8(x[u], scale);
    }
    __device__ __forceinline__ void store(u32x2* __restrict__ to, int nvec) const {
#pragma unroll
        for (int u = 0; u < VPL; ++u) {
            const int v = threadIdx.x + u * blockDim.x;
            if (v < nvec) __builtin_nontemporal_store(q[u], to + v);
        }
    }
};

}  // namespace quant
}  // namespace ep
