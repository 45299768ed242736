// ep_norm_dev.h -- device-side helpers of the layer norm kernels.
#pragma once

#include <type_traits>

#include "ep_device.h"

namespace ep {
namespace norm {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Rows are accessed through bounded views (any alignment): words past the end of
// the row read as 0 and are not written.  A row of an odd number of bf16 channels
// ends within a word, which counts as past the end: its last channel is moved by
// itself.  kOnce: not kept in the caches.
constexpr int kOnce = 2;

// The last of H channels, for the piece of P from channel c on that holds it:
// its word of the piece, or -1 (also where H is even).
__device__ __forceinline__ int odd_word(int c, int H, int P) {
    const int at = H - 1 - c;
    return H % 2 == 1 && at >= 0 && at < P ? at / 2 : -1;
}

// 16 bytes of a row: P channels from c on, 0 behind the row's end.
template <bool BF16>
struct Piece;

template <>
struct Piece<true> {
    typedef uint16_t T;
    static constexpr int P = 8;
    u32x4 v;
    template <int AUX = kOnce>
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t row, int c, int H) {
        v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(row, c * 2, 0, AUX));
        if (H % 2 == 1) {
            const uint32_t last = __builtin_amdgcn_raw_buffer_load_b16(row, (H - 1) * 2, 0, 0);
            const int word = odd_word(c, H, P);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = word == i ? last : v[i];
        }
    }
    __device__ __forceinline__ float at(int i) const {
        return i % 2 == 0 ? bf16_lo(v[i / 2]) : bf16_hi(v[i / 2]);
    }
    static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t row, int c, int H,
                                                 const float (&f)[P]) {
        const u32x4 o = {pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                         pack_bf16(f[6], f[7])};
        __builtin_amdgcn_raw_buffer_store_b128(o, row, c * 2, 0, kOnce);
        if (H % 2 == 1) {
            const int word = odd_word(c, H, P);
            uint32_t last = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) last = word == i ? o[i] : last;
            if (word >= 0)
                __builtin_amdgcn_raw_buffer_store_b16(static_cast<uint16_t>(last), row, (H - 1) * 2, 0, 0);
        }
    }
};

template <>
struct Piece<false> {
    typedef float T;
    static constexpr int P = 4;
    u32x4 v;
    template <int AUX = kOnce>
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t row, int c, int) {
        v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(row, c * 4, 0, AUX));
    }
    __device__ __forceinline__ float at(int i) const { return __uint_as_float(v[i]); }
    static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t row, int c, int,
                                                 const float (&f)[P]) {
        const u32x4 o = {__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                         __float_as_uint(f[3])};
        __builtin_amdgcn_raw_buffer_store_b128(o, row, c * 4, 0, kOnce);
    }
};

// View of row t of [T, H] rows `stride` elements apart; empty where there is no such
// row or no such tensor.
template <class T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_view(const void* p, int64_t t, int64_t stride,
                                                           int H, bool there) {
    return view(static_cast<const T*>(p) + (there ? t * stride : 0),
                there && p != nullptr ? H * sizeof(T) : 0);
}

// P channels of a per-channel parameter; `otherwise` where there is no such tensor.
template <int P, bool BF16>
__device__ __forceinline__ void load_params(const void* p, int c, int H, float otherwise,
                                            float (&f)[P]) {
    if (p == nullptr) {
#pragma unroll
        for (int i = 0; i < P; ++i) f[i] = otherwise;
        return;
    }
    const auto v = view(p, H * (BF16 ? 2 : 4));
    if constexpr (BF16 && P == 4) {
        u32x2 w = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(v, c * 2, 0, 0));
        if (H % 2 == 1) {
            const uint32_t last = __builtin_amdgcn_raw_buffer_load_b16(v, (H - 1) * 2, 0, 0);
            const int word = odd_word(c, H, P);
#pragma unroll
            for (int i = 0; i < 2; ++i) w[i] = word == i ? last : w[i];
        }
#pragma unroll
        for (int i = 0; i < P; ++i) f[i] = i % 2 == 0 ? bf16_lo(w[i / 2]) : bf16_hi(w[i / 2]);
    } else {
        constexpr int Q = Piece<BF16>::P;
        Piece<BF16> q;
#pragma unroll
        for (int k = 0; k < P / Q; ++k) {
            q.template load<0>(v, c + k * Q, H);
#pragma unroll
            for (int i = 0; i < Q; ++i) f[k * Q + i] = q.at(i);
        }
    }
}

template <bool BF16>
__device__ __forceinline__ void store_param(void* p, int c, float v) {
    if (p == nullptr) return;
    if (BF16)
        static_cast<__bf16*>(p)[c] = static_cast<__bf16>(v);
    else
        static_cast<float*>(p)[c] = v;
}

// Sum over the lanes of a row of 16, in every lane, by rotation.
__device__ __forceinline__ float row16_sum(float v) {
    const auto turned = [&](auto i) {
        return __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_update_dpp(
            0, static_cast<int>(__float_as_uint(v)), 0x120 + decltype(i)::value, 0xf, 0xf, false)));
    };
    v += turned(std::integral_constant<int, 8>{});
    v += turned(std::integral_constant<int, 4>{});
    v += turned(std::integral_constant<int, 2>{});
    v += turned(std::integral_constant<int, 1>{});
    return v;
}

// Sum over the lanes of a wave, in every lane.
__device__ __forceinline__ float wave_sum(float v) {
    v = row16_sum(v);
    const auto lane = [&](int i) {
        return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), i));
    };
    return (lane(0) + lane(16)) + (lane(32) + lane(48));
}

// Sum over the workgroup's waves; parts: one float per wave, not used since the last
// barrier.
__device__ __forceinline__ float workgroup_sum(float v, float* parts) {
    v = wave_sum(v);
    if (threadIdx.x % kWave == 0) parts[threadIdx.x / kWave] = v;
    __syncthreads();
    float s = 0.0f;
    for (int i = 0; i < static_cast<int>(blockDim.x) / kWave; ++i) s += parts[i];
    return s;
}

// Sums of B values over the `waves` waves from wave0 on, which call it together with the
// whole workgroup; parts: B floats per wave of the workgroup, not used since the last barrier.
template <int B>
__device__ __forceinline__ void group_sums(float (&v)[B], float (*parts)[16], int wave0, int waves,
                                           int wave) {
#pragma unroll
    for (int b = 0; b < B; ++b) v[b] = wave_sum(v[b]);
    if (waves == 1) return;
    if (threadIdx.x % kWave == 0) {
#pragma unroll
        for (int b = 0; b < B; ++b) parts[b][wave] = v[b];
    }
    __syncthreads();
#pragma unroll
    for (int b = 0; b < B; ++b) {
        v[b] = 0.0f;
        for (int i = 0; i < waves; ++i) v[b] += parts[b][wave0 + i];
    }
}

}  // namespace norm
}  // namespace ep
