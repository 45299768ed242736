// ep_route_dev.h -- device helpers of the routing kernels (gfx950, wave64).
//
// A token is handled by LPT consecutive lanes of one wave (16 or 64), each
// holding VPL experts, LPT * VPL >= E.  Where the order of the experts matters
// a lane's are consecutive, so the lowest lane with a value also holds the
// lowest expert index; elsewhere they lie in pieces of up to 16 bytes spread so
// that the lanes of a token access consecutive memory.  Reductions leave their result
// in every lane of the token and combine in a fixed order.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ep_device.h"
#include "ep_internal.h"

namespace ep {
namespace route {

constexpr int kThreads = 256;

// Lane permutations: rotate by N inside each row of 16 lanes.
template <int N>
__device__ __forceinline__ uint32_t row_ror(uint32_t v) {
    return static_cast<uint32_t>(
        __builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x120 + N, 0xf, 0xf, true));
}

// Value of lane N of each row of 16 lanes, in every lane of it.
template <int N>
__device__ __forceinline__ uint32_t row_bcast(uint32_t v) {
    return static_cast<uint32_t>(
        __builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x150 + N, 0xf, 0xf, true));
}

// All lanes of an aligned run of 2^S: after S - 1, run it with S.  Lane i meets
// a lane of the other half of its run.
template <int S>
__device__ __forceinline__ uint32_t other_half(uint32_t v) {
    constexpr int ctrl = S == 1 ? 0xb1      // quad_perm 1, 0, 3, 2
                         : S == 2 ? 0x4e    // quad_perm 2, 3, 0, 1
                         : S == 3 ? 0x141   // mirrored in 8 lanes
                                  : 0x140;  // mirrored in 16 lanes
    return static_cast<uint32_t>(
        __builtin_amdgcn_update_dpp(0, static_cast<int>(v), ctrl, 0xf, 0xf, true));
}

// LDS that one wave writes and reads needs no barrier, but the compiler has to
// keep the order.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The two halves of a pairwise exchange: {rows 0, 0, 2, 2} and {1, 1, 3, 3}
// for 16, {lanes 0-31 twice} and {lanes 32-63 twice} for 32.
__device__ __forceinline__ uint2 swap16(uint32_t v) {
    auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return make_uint2(r[0], r[1]);
}
__device__ __forceinline__ uint2 swap32(uint32_t v) {
    auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return make_uint2(r[0], r[1]);
}

template <int LPT>
__device__ __forceinline__ uint32_t token_max(uint32_t v) {
    v = max(v, row_ror<8>(v));
    v = max(v, row_ror<4>(v));
    v = max(v, row_ror<2>(v));
    v = max(v, row_ror<1>(v));
    if constexpr (LPT == 64) {
        uint2 p = swap16(v);
        v = max(p.x, p.y);
        p = swap32(v);
        v = max(p.x, p.y);
    }
    return v;
}

// Sum and maximum of floats.  Every lane adds the same pairs: x + y == y + x.
template <int LPT>
__device__ __forceinline__ float token_sum(float f) {
    f += __uint_as_float(row_ror<8>(__float_as_uint(f)));
    f += __uint_as_float(row_ror<4>(__float_as_uint(f)));
    f += __uint_as_float(row_ror<2>(__float_as_uint(f)));
    f += __uint_as_float(row_ror<1>(__float_as_uint(f)));
    if constexpr (LPT == 64) {
        uint2 p = swap16(__float_as_uint(f));
        f = __uint_as_float(p.x) + __uint_as_float(p.y);
        p = swap32(__float_as_uint(f));
        f = __uint_as_float(p.x) + __uint_as_float(p.y);
    }
    return f;
}

template <int LPT>
__device__ __forceinline__ float token_fmax(float f) {
    f = fmaxf(f, __uint_as_float(row_ror<8>(__float_as_uint(f))));
    f = fmaxf(f, __uint_as_float(row_ror<4>(__float_as_uint(f))));
    f = fmaxf(f, __uint_as_float(row_ror<2>(__float_as_uint(f))));
    f = fmaxf(f, __uint_as_float(row_ror<1>(__float_as_uint(f))));
    if constexpr (LPT == 64) {
        uint2 p = swap16(__float_as_uint(f));
        f = fmaxf(__uint_as_float(p.x), __uint_as_float(p.y));
        p = swap32(__float_as_uint(f));
        f = fmaxf(__uint_as_float(p.x), __uint_as_float(p.y));
    }
    return f;
}

// Value held by lane J (0 .. LPT-1) of this lane's token.
template <int LPT, int J>
__device__ __forceinline__ uint32_t token_bcast(uint32_t v) {
    if constexpr (LPT == 64)
        return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), J));
    else
        return row_bcast<J>(v);
}

// Sum over the lanes of this lane's token up to and with this one.
template <int LPT>
__device__ __forceinline__ int token_prefix(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // row_shr 1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
    if constexpr (LPT == 64) {
        v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast 15
        v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row_bcast 31
    }
    return v;
}

// Lowest lane of this lane's token for which `p` holds (p holds for one at
// least).
template <int LPT>
__device__ __forceinline__ int token_first(bool p, int wave_lane) {
    const uint64_t b = __ballot(p);
    if constexpr (LPT == 64) return __ffsll(static_cast<unsigned long long>(b)) - 1;
    const uint32_t mine = static_cast<uint32_t>(b >> (wave_lane & ~15)) & 0xffffu;
    return __ffs(static_cast<int>(mine)) - 1;
}

__device__ __forceinline__ bool finite(float x) {
    return __builtin_isfinite(x);
}

// Order-preserving map of a finite float to an integer > 0; -0 and +0 agree.
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t k) {
    return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}

// The larger of two numbers, without the quieting of NaN that fmaxf adds.
__device__ __forceinline__ float larger(float x, float y) {
    return __builtin_amdgcn_fmed3f(x, y, __builtin_inff());
}

// exp(x) for x <= 0: 2^t with t = x log2(e) rounded, times 1 + the rounding's
// part.  v_exp_f32 is good to one unit in the last place, so the result is to
// about two, in half the instructions of a library exponential.  It gives 0 for
// results below 2^-126, the smallest normal number (x below -87.3): v_exp_f32 does.
// Below -150 the bound keeps the rounding's part finite.
__device__ __forceinline__ float exp_neg(float x) {
    constexpr float kLog2e = 1.44269504088896340736f;
    constexpr float kLog2eRest = static_cast<float>(1.44269504088896340736 - kLog2e);
    constexpr float kLn2 = 0.693147180559945309417f;
    x = fmaxf(x, -150.0f);
    const float t = x * kLog2e;
    const float rest = fmaf(x, kLog2eRest, fmaf(x, kLog2e, -t));
    const float e = __builtin_amdgcn_exp2f(t);
    return fmaf(e, rest * kLn2, e);
}

// sigma(x) and sigma(-x), both to full relative precision: with
// t = exp(-|x|), the larger of the two is 1 / (1 + t), the smaller t times it.
struct Sigmoids {
    float pos, neg;
};
__device__ __forceinline__ Sigmoids sigmoids(float x) {
    const float t = exp_neg(-fabsf(x));
    const float r = __builtin_amdgcn_rcpf(1.0f + t);  // one unit in the last place
    const float s = t * r;
    return x >= 0.0f ? Sigmoids{r, s} : Sigmoids{s, r};
}

// fp32(sigma(x)), from a value of sigma(x) good to about 2^-46.  The choice
// compares keys made of it, and two fp32 units, which sigmoids() is good to,
// would decide between close ones at random: with t = exp(-|x|) = 2^n exp(f ln 2),
// |f| <= 1/2, the exponential is its series to f^12 (rest below 2^-52), the
// quotient two Newton steps from the hardware's reciprocal.  46 instructions a
// value, most of them fp64.
__device__ __forceinline__ float sigmoid_rounded(float x) {
    const double y = -fabs(static_cast<double>(x)) * 1.44269504088896340736;
    const double v = fmax(y, -1000.0);  // exp is 0 in fp32 long before, and n stays an int
    const double n = rint(v);
    const double f = (v - n) * 0.693147180559945309417;
    constexpr double kSeries[13] = {1.0,         1.0,          1.0 / 2,       1.0 / 6,     1.0 / 24,
                                    1.0 / 120,   1.0 / 720,    1.0 / 5040,    1.0 / 40320, 1.0 / 362880,
                                    1.0 / 3628800, 1.0 / 39916800, 1.0 / 479001600};
    double p = kSeries[12];
#pragma unroll
    for (int i = 11; i >= 0; --i) p = fma(p, f, kSeries[i]);
    const double t = ldexp(p, static_cast<int>(n));
    const double d = 1.0 + t;
    double r = __builtin_amdgcn_rcp(d);
    r = fma(fma(-d, r, 1.0), r, r);
    r = fma(fma(-d, r, 1.0), r, r);
    return static_cast<float>(x >= 0.0f ? r : t * r);
}

// Elements of a piece: 16 bytes, or all that a lane holds.
template <int VPL, bool BF16>
constexpr int kPiece = VPL < (BF16 ? 8 : 4) ? VPL : (BF16 ? 8 : 4);

// The experts of a lane: register i is expert first + (i / W) * step + i % W
// with W = kPiece.
struct Experts {
    int first, step;
};
template <int LPT, int VPL, bool BF16>
__device__ __forceinline__ Experts spread(int lane) {
    return {lane * kPiece<VPL, BF16>, LPT * kPiece<VPL, BF16>};
}
template <int VPL, bool BF16>
__device__ __forceinline__ int expert(const Experts& x, int i) {
    return x.first + i / kPiece<VPL, BF16> * x.step + i % kPiece<VPL, BF16>;
}

// A lane's logits of a row of n, NaN (an expert that is off) past the end.
// `piece` is the host's word that rows may be read in aligned pieces that do
// not straddle the row's end.
template <int VPL, bool BF16>
__device__ __forceinline__ void load_logits(const void* base, int64_t row_start, int n,
                                            const Experts& at, bool piece, float (&x)[VPL]) {
    const float nan = __uint_as_float(0x7fc00000u);
    constexpr int W = kPiece<VPL, BF16>;
    if constexpr (BF16) {
        const uint16_t* p = static_cast<const uint16_t*>(base) + row_start;
        if (W > 1 && piece) {
#pragma unroll
            for (int i = 0; i < VPL; i += W) {
                const int e = at.first + i / W * at.step;
                const bool in = e < n;
                uint32_t w[W > 1 ? W / 2 : 1];
#pragma unroll
                for (int q = 0; q < W / 2; ++q) w[q] = 0x7fc07fc0u;
                if (in) {
                    if constexpr (W == 8) {
                        const uint4 v = *reinterpret_cast<const uint4*>(p + e);
                        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
                    } else if constexpr (W == 4) {
                        const uint2 v = *reinterpret_cast<const uint2*>(p + e);
                        w[0] = v.x, w[1] = v.y;
                    } else if constexpr (W == 2) {
                        w[0] = *reinterpret_cast<const uint32_t*>(p + e);
                    }
                }
#pragma unroll
                for (int q = 0; q < W / 2; ++q) {
                    x[i + 2 * q] = bf16_lo(w[q]);
                    x[i + 2 * q + 1] = bf16_hi(w[q]);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const int e = expert<VPL, BF16>(at, i);
                x[i] = e < n ? __uint_as_float(static_cast<uint32_t>(p[e]) << 16) : nan;
            }
        }
    } else {
        const float* p = static_cast<const float*>(base) + row_start;
        if (W > 1 && piece) {
#pragma unroll
            for (int i = 0; i < VPL; i += W) {
                const int e = at.first + i / W * at.step;
                const bool in = e < n;
#pragma unroll
                for (int q = 0; q < W; ++q) x[i + q] = nan;
                if (in) {
                    if constexpr (W == 4) {
                        const float4 v = *reinterpret_cast<const float4*>(p + e);
                        x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
                    } else if constexpr (W == 2) {
                        const float2 v = *reinterpret_cast<const float2*>(p + e);
                        x[i] = v.x, x[i + 1] = v.y;
                    }
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const int e = expert<VPL, BF16>(at, i);
                x[i] = e < n ? p[e] : nan;
            }
        }
    }
}

// Where even the largest logit is below this, sigma(x) is exp(x) to 2e-9.
constexpr float kSmallScore = -20.0f;

// Unnormalised scores of a token's experts: z[i] / (sum of z over the token)
// are its probabilities; 0 for experts that are off.  Softmax: exp(x - max).
// Sigmoid: sigma(x), or for a row of small scores exp(x - max), which keeps it
// from vanishing.
// slope[i] is d log z / dx of the score: 1, or sigma(-x).  m is the largest
// logit.
template <int LPT, int VPL>
__device__ __forceinline__ void scores(const float (&x)[VPL], bool sigmoid, float (&z)[VPL],
                                       float (&slope)[VPL], float& total, float& m) {
    m = -3.402823466e38f;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        m = larger(m, finite(x[i]) ? x[i] : m);
    m = token_fmax<LPT>(m);
    // no branch per expert: what an expert that is off computes is dropped
    if (sigmoid && m > kSmallScore) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const Sigmoids g = sigmoids(x[i]);
            z[i] = finite(x[i]) ? g.pos : 0.0f;
            slope[i] = finite(x[i]) ? g.neg : 1.0f;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const float v = exp_neg(x[i] - m);
            z[i] = finite(x[i]) ? v : 0.0f;
            slope[i] = 1.0f;  // below -20 sigma(-x) rounds to 1
        }
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) s += z[i];
    total = token_sum<LPT>(s);
}

// One logit, or NaN where the entry is absent.
template <bool BF16>
__device__ __forceinline__ float logit_at(const void* base, int64_t row_start, int e, bool there) {
    if (!there) return __uint_as_float(0x7fc00000u);
    if constexpr (BF16)
        return __uint_as_float(
            static_cast<uint32_t>(static_cast<const uint16_t*>(base)[row_start + e]) << 16);
    else
        return static_cast<const float*>(base)[row_start + e];
}

// Weights of a token's entries before the scale: entry q * LPT + lane has the
// logit xe[q] (NaN: absent, weight 0).  m and total are the maximum and the
// exp sum of the whole row, for softmax weights that are not normalised over
// the entries.
template <int LPT, int SEL>
__device__ __forceinline__ void entry_weights(const float (&xe)[SEL], const RouteArgs& a, float m,
                                              float total, float (&w)[SEL]) {
    if (a.normalize) {
        float top = -3.402823466e38f, s = 0.0f;
#pragma unroll
        for (int q = 0; q < SEL; ++q)
            if (finite(xe[q])) top = fmaxf(top, xe[q]);
        top = token_fmax<LPT>(top);
        const bool sigmoid = a.sigmoid && top > kSmallScore;
#pragma unroll
        for (int q = 0; q < SEL; ++q) {
            w[q] = 0.0f;
            if (q * LPT < a.num_topk && finite(xe[q]))
                w[q] = sigmoid ? sigmoids(xe[q]).pos : exp_neg(xe[q] - top);
            s += w[q];
        }
        s = token_sum<LPT>(s);
        const float r = s > 0.0f ? 1.0f / s : 0.0f;
#pragma unroll
        for (int q = 0; q < SEL; ++q) w[q] *= r;
    } else {
        const float r = 1.0f / total;
#pragma unroll
        for (int q = 0; q < SEL; ++q) {
            w[q] = 0.0f;
            if (q * LPT < a.num_topk && finite(xe[q]))
                w[q] = a.sigmoid ? sigmoids(xe[q]).pos : exp_neg(xe[q] - m) * r;
        }
    }
}

// A lane's part of a dense row of n gradients in the logits' type, rounded to
// nearest even.
template <int VPL, bool BF16>
__device__ __forceinline__ void store_logits(void* base, int64_t row_start, int n,
                                             const Experts& at, bool piece, const float (&v)[VPL]) {
    constexpr int W = kPiece<VPL, BF16>;
    if constexpr (BF16) {
        uint16_t* p = static_cast<uint16_t*>(base) + row_start;
        uint32_t h[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) h[i] = f32_to_bf16_rne(v[i]);
        if (W > 1 && piece) {
#pragma unroll
            for (int i = 0; i < VPL; i += W) {
                const int e = at.first + i / W * at.step;
                if (e >= n) continue;
                if constexpr (W == 8)
                    *reinterpret_cast<uint4*>(p + e) =
                        make_uint4(h[i] | h[i + 1] << 16, h[i + 2] | h[i + 3] << 16,
                                   h[i + 4] | h[i + 5] << 16, h[i + 6] | h[i + 7] << 16);
                else if constexpr (W == 4)
                    *reinterpret_cast<uint2*>(p + e) =
                        make_uint2(h[i] | h[i + 1] << 16, h[i + 2] | h[i + 3] << 16);
                else if constexpr (W == 2)
                    *reinterpret_cast<uint32_t*>(p + e) = h[i] | h[i + 1] << 16;
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const int e = expert<VPL, BF16>(at, i);
                if (e < n) p[e] = static_cast<uint16_t>(h[i]);
            }
        }
    } else {
        float* p = static_cast<float*>(base) + row_start;
        if (W > 1 && piece) {
#pragma unroll
            for (int i = 0; i < VPL; i += W) {
                const int e = at.first + i / W * at.step;
                if (e >= n) continue;
                if constexpr (W == 4)
                    *reinterpret_cast<float4*>(p + e) =
                        make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                else if constexpr (W == 2)
                    *reinterpret_cast<float2*>(p + e) = make_float2(v[i], v[i + 1]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const int e = expert<VPL, BF16>(at, i);
                if (e < n) p[e] = v[i];
            }
        }
    }
}

}  // namespace route
}  // namespace ep
