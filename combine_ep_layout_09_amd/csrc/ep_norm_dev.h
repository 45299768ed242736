// ep_norm_dev.h -- device-side helpers of the layer norm kernels.
#pragma once

#include <type_traits>

#include "ep_device.h"

namespace ep {
namespace norm {

// Sixteen and eight bytes at any address that two-byte elements may have.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
typedef u32x2 u32x2_at2 __attribute__((aligned(2)));
// 16 bytes of a row: P channels from c on, 0 behind the row's end.  Through a
// bounded view of a row that P divides: no lane has to ask where the row ends.
template <bool BF16>
struct Piece;

template <>
struct Piece<true> {
    typedef uint16_t T;
    static constexpr int P = 8;
    static __device__ __forceinline__ u32x4 pack(const float (&f)[P]) {
        return u32x4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                     pack_bf16(f[6], f[7])};
    }
    u32x4 v;
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t row, int c) {
        v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(row, c * sizeof(T), 0, 0));
    }
    static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t row, int c,
                                                 const float (&f)[P]) {
        __builtin_amdgcn_raw_buffer_store_b128(pack(f), row, c * sizeof(T), 0, 0);
    }
    __device__ __forceinline__ void load(const T* row, int c, int H) {
        v = u32x4{0, 0, 0, 0};
        if (c + P <= H) {
            v = *reinterpret_cast<const u32x4_at2*>(row + c);
        } else {
            // a row of uneven length: at most one piece of it
            for (int i = 0; c + i < H; ++i) {
                const uint32_t e = static_cast<uint32_t>(row[c + i]) << (16 * (i & 1));
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] |= q == i / 2 ? e : 0u;
            }
        }
    }
    __device__ __forceinline__ float at(int i) const {
        return i % 2 == 0 ? bf16_lo(v[i / 2]) : bf16_hi(v[i / 2]);
    }
    static __device__ __forceinline__ void store(T* row, int c, int H, const float (&f)[P]) {
        const u32x4 o = pack(f);
        if (c + P <= H) {
            *reinterpret_cast<u32x4_at2*>(row + c) = o;
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (c + i < H) row[c + i] = static_cast<T>(o[i / 2] >> (16 * (i & 1)));
        }
    }
};

template <>
struct Piece<false> {
    typedef float T;
    typedef u32x4 u32x4_at4 __attribute__((aligned(4)));
    static constexpr int P = 4;
    static __device__ __forceinline__ u32x4 pack(const float (&f)[P]) {
        return u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                     __float_as_uint(f[3])};
    }
    u32x4 v;
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t row, int c) {
        v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(row, c * sizeof(T), 0, 0));
    }
    static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t row, int c,
                                                 const float (&f)[P]) {
        __builtin_amdgcn_raw_buffer_store_b128(pack(f), row, c * sizeof(T), 0, 0);
    }
    __device__ __forceinline__ void load(const T* row, int c, int H) {
        v = u32x4{0, 0, 0, 0};
        if (c + P <= H) {
            v = *reinterpret_cast<const u32x4_at4*>(row + c);
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i) v[i] = c + i < H ? __float_as_uint(row[c + i]) : 0u;
        }
    }
    __device__ __forceinline__ float at(int i) const { return __uint_as_float(v[i]); }
    static __device__ __forceinline__ void store(T* row, int c, int H, const float (&f)[P]) {
        if (c + P <= H) {
            *reinterpret_cast<u32x4_at4*>(row + c) = pack(f);
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (c + i < H) row[c + i] = f[i];
        }
    }
};

// P channels of a per-channel parameter, `otherwise` where there is none.
template <int P, bool BF16>
__device__ __forceinline__ void load_params(const void* p, int c, int H, float otherwise,
                                            float (&f)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) f[i] = otherwise;
    if (p == nullptr) return;
    if constexpr (BF16) {
        const uint16_t* from = static_cast<const uint16_t*>(p) + c;
        if (c + P <= H) {
            if constexpr (P == 8) {
                const u32x4 v = *reinterpret_cast<const u32x4_at2*>(from);
#pragma unroll
                for (int i = 0; i < P; ++i) f[i] = i % 2 == 0 ? bf16_lo(v[i / 2]) : bf16_hi(v[i / 2]);
            } else {
                const u32x2 v = *reinterpret_cast<const u32x2_at2*>(from);
#pragma unroll
                for (int i = 0; i < P; ++i) f[i] = i % 2 == 0 ? bf16_lo(v[i / 2]) : bf16_hi(v[i / 2]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (c + i < H) f[i] = bf16_lo(from[i]);
        }
    } else {
        const float* from = static_cast<const float*>(p);
        Piece<false> v;
#pragma unroll
        for (int q = 0; q < P / 4; ++q) {
            v.load(from, c + 4 * q, H);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[4 * q + i] = v.at(i);
        }
    }
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

// Sum over the `waves` waves from wave0 on, which call it together with the
// whole workgroup; parts: one float per wave of the workgroup, not used since the
// last barrier.
__device__ __forceinline__ float group_sum(float v, float* parts, int wave0, int waves, int wave) {
    v = wave_sum(v);
    if (waves == 1) return v;
    if (threadIdx.x % kWave == 0) parts[wave] = v;
    __syncthreads();
    float s = 0.0f;
    for (int i = 0; i < waves; ++i) s += parts[wave0 + i];
    return s;
}

}  // namespace norm
}  // namespace ep
