// ep_route.hip -- the choice of experts from gate logits, and the gradient of
// the logits from the routing weights and the balance loss.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ep_internal.h"
#include "ep_route_dev.h"

namespace ep {
namespace {

using namespace route;

// ---------------------------------------------------------------- the choice

// The score of a group: the sum of its two largest keys' values, an expert that
// is off (key 0) counting as -FLT_MAX.  fp64 holds the sum of two fp32 values
// closely enough that only equal sums of equal terms tie.
__device__ __forceinline__ double group_score(uint32_t m1, uint32_t m2, bool single) {
    const double low = -3.4028234663852886e38;
    double s = m1 ? static_cast<double>(order_value(m1)) : low;
    if (!single) s += m2 ? static_cast<double>(order_value(m2)) : low;
    return s;
}

template <int S>
__device__ __forceinline__ void merge_half(uint32_t& m1, uint32_t& m2) {
    const uint32_t o1 = other_half<S>(m1), o2 = other_half<S>(m2);
    m2 = max(min(m1, o1), max(m2, o2));
    m1 = max(m1, o1);
}

// How many lanes of the row of 16 hold a better group than this one, when a
// group is 2^S lanes (so 2^S times the number of better groups).
template <int S, int N>
__device__ __forceinline__ int better_lanes(double s, int lane) {
    if constexpr (N >= 16) {
        return 0;
    } else {
        const uint64_t u = __builtin_bit_cast(uint64_t, s);
        const uint64_t lo = row_ror<N>(static_cast<uint32_t>(u));
        const uint64_t hi = row_ror<N>(static_cast<uint32_t>(u >> 32));
        const double o = __builtin_bit_cast(double, hi << 32 | lo);
        // row_ror moves lane i - N to lane i, so it is a lower one from lane N on
        const bool better = o > s || (o == s && lane >= N);
        return (better ? 1 : 0) + better_lanes<S, N + (1 << S)>(s, lane);
    }
}

// Groups of 2^S lanes of a 16-lane token: two-largest by pairwise exchanges,
// then each lane meets one lane of every other group.
template <int S, int VPL>
__device__ __forceinline__ bool lane_group_kept(const uint32_t (&key)[VPL], int lane,
                                                const RouteArgs& a) {
    uint32_t m1 = 0, m2 = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        m2 = max(m2, min(m1, key[i]));
        m1 = max(m1, key[i]);
    }
    if constexpr (S >= 1) merge_half<1>(m1, m2);
    if constexpr (S >= 2) merge_half<2>(m1, m2);
    if constexpr (S >= 3) merge_half<3>(m1, m2);
    // lanes past the last group are below every score
    const double s = lane * VPL < a.num_experts ? group_score(m1, m2, VPL << S == 1) : -1.0e300;
    return better_lanes<S, 1 << S>(s, lane) < a.topk_groups;
}

// Words of LDS for a lane's run of VPL keys: 16-byte accesses of 8 lanes meet 32
// banks.
template <int VPL>
constexpr int kRun = VPL >= 8 ? VPL + 4 : VPL;

// A lane's run of VPL keys in LDS.
template <int VPL>
__device__ __forceinline__ void read_run(const uint32_t* from, uint32_t (&to)[VPL]) {
    if constexpr (VPL >= 4) {
#pragma unroll
        for (int i = 0; i < VPL; i += 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(from + i);
            to[i] = v.x, to[i + 1] = v.y, to[i + 2] = v.z, to[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) to[i] = from[i];
    }
}

// Keys of experts outside the token's best topk_groups groups become 0 (off).
// A group is kept if fewer than topk_groups groups are better; equal scores go
// to the lower index.  Groups that are 1, 2, 4 or 8 whole lanes of a 16-lane
// token are handled in registers; others in LDS, which has the keys in runs:
// `split` lanes take a group each, score it, and switch it off if it is not kept:
// one lane, or with 64 lanes a token a power of two (1024 experts in 8 groups,
// 16000 tokens: 27 us, with one lane each 60).
template <int LPT, int VPL>
__device__ __forceinline__ void limit_groups(uint32_t (&key)[VPL], uint32_t* keys, double* score,
                                             int lane, const RouteArgs& a) {
    const int gs = a.num_experts / a.num_groups;
    if (LPT == 16 && a.group_lanes > 0) {
        bool kept;
        if (a.group_lanes == 1)
            kept = lane_group_kept<0, VPL>(key, lane, a);
        else if (a.group_lanes == 2)
            kept = lane_group_kept<1, VPL>(key, lane, a);
        else if (a.group_lanes == 4)
            kept = lane_group_kept<2, VPL>(key, lane, a);
        else
            kept = lane_group_kept<3, VPL>(key, lane, a);
#pragma unroll
        for (int i = 0; i < VPL; ++i) key[i] = kept ? key[i] : 0u;
        return;
    }
    const auto key_of = [&](int e) -> uint32_t& { return keys[e / VPL * kRun<VPL> + e % VPL]; };
    int split = 1;
    while (LPT == 64 && split < 16 && 2 * split * a.num_groups <= LPT) split *= 2;
    const int part = lane % split, step = LPT / split;
    for (int g = lane / split; g < a.num_groups; g += step) {
        uint32_t m1 = 0, m2 = 0;
        for (int i = part; i < gs; i += split) {
            const uint32_t k = key_of(g * gs + i);
            m2 = max(m2, min(m1, k));
            m1 = max(m1, k);
        }
        if (split >= 2) merge_half<1>(m1, m2);
        if (split >= 4) merge_half<2>(m1, m2);
        if (split >= 8) merge_half<3>(m1, m2);
        if (split >= 16) merge_half<4>(m1, m2);
        score[g] = group_score(m1, m2, gs == 1);
    }
    wave_sync();
    for (int g = lane / split; g < a.num_groups; g += step) {
        const double s = score[g];
        int better = 0;
        for (int h = 0; h < a.num_groups; ++h) {
            const double o = score[h];
            better += (o > s || (o == s && h < g)) ? 1 : 0;
        }
        if (better >= a.topk_groups)
            for (int i = part; i < gs; i += split) key_of(g * gs + i) = 0;
    }
    wave_sync();
    read_run<VPL>(&keys[lane * kRun<VPL>], key);
}

// One launch, a token per LPT lanes; logits are read in pieces that lie
// consecutively over a token's lanes (with each lane reading its own run of
// experts, 16384 x 256 fp32 took 16.6 us, so 11.1).  The k best keys are taken
// one after the other: every lane keeps the best of its own keys, a reduction
// over the token's lanes finds the best of all, and the lowest lane that holds it
// goes on to its next.  Entry j goes to lane j % LPT through LDS; the weights are
// then computed with one lane per entry from the logits themselves (the bias only
// steers the choice).  16384 x 256 fp32, 4 of 8 groups: 9.9 us, 1.7 TB/s; 700
// instructions per wave are a half of it, the read before them the other.
//
// BY_SCORE: keys are sigma(logit) + bias instead of logit + bias.  16384 x 256, 4 of
// 8 groups, with a bias: 14.8 us a call in a graph, by logits 10.1; the scores in
// fp64 are the difference.
template <int LPT, int VPL, bool BF16, bool BY_SCORE>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteArgs a, const float* bias,
                                                         const uint8_t* valid, int32_t* topk_idx,
                                                         float* topk_weights) {
    constexpr int kTokens = kThreads / LPT;
    constexpr int kSel = kMaxTopk > LPT ? kMaxTopk / LPT : 1;
    __shared__ __attribute__((aligned(16))) uint32_t lds_keys[kTokens][LPT * kRun<VPL>];
    __shared__ double lds_score[kTokens][kMaxGroups];
    __shared__ int lds_chosen[kTokens][kMaxTopk];
    const int lane = threadIdx.x % LPT;
    const int slot = threadIdx.x / LPT;
    const int wave_lane = threadIdx.x % kWave;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kTokens + slot;
    const bool inside = t < a.num_tokens;
    const int E = a.num_experts;
    const int64_t row = (inside ? t : 0) * a.stride;

    const Experts from = spread<LPT, VPL, BF16>(lane);
    float x[VPL], more[VPL] = {};
    load_logits<VPL, BF16>(a.logits, row, inside ? E : 0, from, a.pieces, x);
    if (bias != nullptr) {
        if (kPiece<VPL, BF16> >= 4 && a.fours) {
#pragma unroll
            for (int i = 0; i + 3 < VPL; i += 4) {
                const int e = expert<VPL, BF16>(from, i);
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (e < E) v = *reinterpret_cast<const float4*>(bias + e);
                more[i] = v.x, more[i + 1] = v.y, more[i + 2] = v.z, more[i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const int e = expert<VPL, BF16>(from, i);
                more[i] = e < E ? bias[e] : 0.0f;
            }
        }
    }
    const bool live = inside && (valid == nullptr || valid[t] != 0);
    float m = 0.0f, total = 1.0f;
    if (!a.sigmoid && !a.normalize) {
        float z[VPL], slope[VPL];
        scores<LPT, VPL>(x, false, z, slope, total, m);
    }
    uint32_t key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const float v = (BY_SCORE ? sigmoid_rounded(x[i]) : x[i]) + more[i];
        const bool on = finite(v) && (!BY_SCORE || finite(x[i]));  // logit + bias is not if x is not
        key[i] = on ? order_key(v) : 0u;
    }
    if constexpr (VPL > kPiece<VPL, BF16>) {  // to consecutive experts, through LDS
#pragma unroll
        for (int i = 0; i < VPL; i += 4) {  // kPiece is 4 or 8 here
            const int e = expert<VPL, BF16>(from, i);
            *reinterpret_cast<uint4*>(&lds_keys[slot][e / VPL * kRun<VPL> + e % VPL]) =
                make_uint4(key[i], key[i + 1], key[i + 2], key[i + 3]);
        }
        wave_sync();
        read_run<VPL>(&lds_keys[slot][lane * kRun<VPL>], key);
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) lds_keys[slot][lane * kRun<VPL> + i] = key[i];
        wave_sync();
    }
    if (a.num_groups > 1) limit_groups<LPT, VPL>(key, lds_keys[slot], lds_score[slot], lane, a);

    // The k best pairs of (key, lane); lane j keeps pair j.  The lane that gave a
    // pair goes on to its largest key below that.  It finds it by unsigned
    // distance (keys at or above wrap round to more than the distance of 0), or
    // with 16 keys or more the token's lanes find it together from LDS (16384 tokens
    // of 256 experts: 7.8 us against 8.4; of 64, 4 keys a lane: 4.8 against 4.6).
    // Lanes of groups that are off still have keys in LDS, but are never first.
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) best = max(best, key[i]);
    if (!live) best = 0;
    uint32_t top[kSel];
    int owner[kSel];
#pragma unroll
    for (int q = 0; q < kSel; ++q) {
        top[q] = 0;
        owner[q] = 0;
#pragma unroll 1
        for (int j = 0; j < LPT && q * LPT + j < a.num_topk; ++j) {
            const uint32_t now = token_max<LPT>(best);
            const int first = token_first<LPT>(best == now, wave_lane);
            top[q] = lane == j ? now : top[q];
            owner[q] = lane == j ? first : owner[q];
            if constexpr (VPL >= 16) {
                uint32_t next = 0;
#pragma unroll
                for (int i = 0; i < VPL; i += LPT) {
                    const uint32_t k =
                        i + lane < VPL ? lds_keys[slot][first * kRun<VPL> + i + lane] : 0u;
                    next = max(next, k < now ? k : 0u);
                }
                next = token_max<LPT>(next);
                best = lane == first ? next : best;
            } else if (lane == first && now != 0) {
                const uint32_t below = best - 1;
                uint32_t gap = below;
#pragma unroll
                for (int i = 0; i < VPL; ++i) gap = min(gap, below - key[i]);
                best = below - gap;
            }
        }
    }
    // A pair stands for every expert of its lane with that key, in their order:
    // entries are the pairs' experts one after the other, up to k.
    int before = 0;  // entries of the pairs before this lane's
#pragma unroll
    for (int q = 0; q < kSel; ++q) {
        if (q > 0 && q * LPT >= a.num_topk) continue;
        const bool there = q * LPT + lane < a.num_topk;
        uint32_t mask = 0;
        if (there && top[q] != 0) {
            uint32_t held[VPL];
            read_run<VPL>(&lds_keys[slot][owner[q] * kRun<VPL>], held);
#pragma unroll
            for (int i = 0; i < VPL; ++i) mask |= held[i] == top[q] ? 1u << i : 0u;
        }
        const int entries = there ? (mask == 0 ? 1 : __popc(mask)) : 0;
        const int to = before + token_prefix<LPT>(entries);
        if (there) {
            int at = to - entries;
            if (mask == 0 && at < a.num_topk) lds_chosen[slot][at] = -1;
            for (; mask != 0 && at < a.num_topk; ++at, mask &= mask - 1)
                lds_chosen[slot][at] = owner[q] * VPL + __ffs(static_cast<int>(mask)) - 1;
        }
        if (q + 1 < kSel) before = static_cast<int>(token_bcast<LPT, LPT - 1>(to));
    }
    wave_sync();
    int sel[kSel];
#pragma unroll
    for (int q = 0; q < kSel; ++q)
        sel[q] = q * LPT + lane < a.num_topk ? lds_chosen[slot][q * LPT + lane] : -1;

    float xe[kSel], w[kSel];
#pragma unroll
    for (int q = 0; q < kSel; ++q) xe[q] = logit_at<BF16>(a.logits, row, sel[q], sel[q] >= 0);
    entry_weights<LPT, kSel>(xe, a, m, total, w);
    if (inside) {
#pragma unroll
        for (int q = 0; q < kSel; ++q) {
            const int j = q * LPT + lane;
            if (j < a.num_topk) {
                topk_idx[t * a.num_topk + j] = sel[q];
                topk_weights[t * a.num_topk + j] = a.scale * w[q];
            }
        }
    }
}

// -------------------------------------------------------------- the gradient

// Entry j of the token (lane j % LPT, register j / LPT) to every lane: those of
// the same expert add it to their sum, in the order of j, and stay responsible
// for the expert only if no earlier entry names it.
template <int LPT, int SEL, int J>
__device__ __forceinline__ void join_entries(const int (&e)[SEL], const float (&part)[SEL], int k,
                                             int lane, float (&sum)[SEL], bool (&mine)[SEL]) {
    if constexpr (J < kMaxTopk) {
        if (J >= k) return;
        const int ej = static_cast<int>(
            token_bcast<LPT, J % LPT>(static_cast<uint32_t>(e[J / LPT])));
        const float pj =
            __uint_as_float(token_bcast<LPT, J % LPT>(__float_as_uint(part[J / LPT])));
#pragma unroll
        for (int q = 0; q < SEL; ++q) {
            if (J == 0) sum[q] = 0.0f;
            if (ej == e[q]) {
                sum[q] += pj;
                if (J < q * LPT + lane) mine[q] = false;
            }
        }
        join_entries<LPT, SEL, J + 1>(e, part, k, lane, sum, mine);
    }
}

// d_logits of a token = the balance loss's part, dense, plus the weights'
// part, which is dense only for weights that were not normalised over the
// chosen experts of a softmax.
//   p = probabilities, A_e = coef d_loss E / (B k n^2) count_e:
//     p_e (A_e - sum_i A_i p_i) slope_e
// Counts enter as their (exact) distance from the first expert's: adding a
// constant to A changes nothing, and the difference keeps the digits that
// A_e - sum A p would cancel.  16384 x 256 fp32, both parts: 12.0 us, 3.0 TB/s
// (16.0 with each lane reading and writing a run of experts).  Entries that
// name one expert twice are added up in their order by the first of them, so
// no order of atomics matters.
template <int LPT, int VPL, bool BF16>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(
    RouteArgs a, const int32_t* topk_idx, const float* d_weights, const uint8_t* valid, float factor,
    const int32_t* counts, const int32_t* num_valid, const float* d_loss, void* d_logits) {
    constexpr int kTokens = kThreads / LPT;
    constexpr int kSel = kMaxTopk > LPT ? kMaxTopk / LPT : 1;
    constexpr int W = kPiece<VPL, BF16>;
    __shared__ __attribute__((aligned(16))) float add[kTokens][LPT * VPL];
    const int lane = threadIdx.x % LPT;
    const int slot = threadIdx.x / LPT;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kTokens + slot;
    const bool inside = t < a.num_tokens;
    const int E = a.num_experts, k = a.num_topk;
    const Experts own = spread<LPT, VPL, BF16>(lane);
    const int64_t row = (inside ? t : 0) * a.stride;

    // What a token needs of its own is read first, none of it waiting for another
    // load but the entries' logits.
    const bool loss = d_loss != nullptr;
    const bool spread_weights = d_weights != nullptr && !a.sigmoid && !a.normalize;
    float x[VPL], dx[VPL];
    load_logits<VPL, BF16>(a.logits, row, inside ? E : 0, own, a.pieces, x);
    int e[kSel];
    float xe[kSel], g[kSel];
#pragma unroll
    for (int q = 0; q < kSel; ++q) {
        const int j = q * LPT + lane;
        e[q] = -1;
        g[q] = 0.0f;
        if (d_weights != nullptr && inside && j < k) {
            e[q] = topk_idx[t * k + j];
            g[q] = d_weights[t * k + j];
        }
    }
    const bool live = inside && (valid == nullptr || valid[t] != 0);
#pragma unroll
    for (int q = 0; q < kSel; ++q) {
        if (!live || e[q] < 0 || e[q] >= E) e[q] = -1;
        xe[q] = logit_at<BF16>(a.logits, row, e[q], e[q] >= 0);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) dx[i] = 0.0f;
    float m = 0.0f, total = 1.0f;
    float p[VPL], slope[VPL];
    if (loss || spread_weights) {
        scores<LPT, VPL>(x, a.sigmoid, p, slope, total, m);
        const float r = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) p[i] *= r;
    }
    if (loss) {
        const uint32_t seq = static_cast<uint32_t>(inside ? t : 0) / static_cast<uint32_t>(a.seq_len);
        const int32_t* c = counts + static_cast<int64_t>(seq) * E;
        const int32_t c0 = c[0];
        int32_t ci[VPL];
        if (W >= 4 && a.fours) {
#pragma unroll
            for (int i = 0; i + 3 < VPL; i += 4) {
                const int at = expert<VPL, BF16>(own, i);
                int4 v = make_int4(0, 0, 0, 0);
                if (at < E) v = *reinterpret_cast<const int4*>(c + at);
                ci[i] = v.x, ci[i + 1] = v.y, ci[i + 2] = v.z, ci[i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const int at = expert<VPL, BF16>(own, i);
                ci[i] = at < E ? c[at] : 0;
            }
        }
        const float n = static_cast<float>(max(num_valid[seq], 1));
        const float f = factor * d_loss[0] / n / n;
        float d[VPL], dot = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            d[i] = static_cast<float>(ci[i] - c0);
            dot += d[i] * p[i];
        }
        dot = token_sum<LPT>(dot);
#pragma unroll
        for (int i = 0; i < VPL; ++i) dx[i] = f * (p[i] * (d[i] - dot) * slope[i]);
    }
    if (d_weights != nullptr) {
        float w[kSel], part[kSel];
        float gw = 0.0f;
#pragma unroll
        for (int q = 0; q < kSel; ++q) {
            if (!finite(xe[q])) e[q] = -1;
            g[q] = e[q] >= 0 ? a.scale * g[q] : 0.0f;
        }
        entry_weights<LPT, kSel>(xe, a, m, total, w);
#pragma unroll
        for (int q = 0; q < kSel; ++q) gw += g[q] * w[q];
        gw = token_sum<LPT>(gw);
#pragma unroll
        for (int q = 0; q < kSel; ++q) {
            part[q] = 0.0f;
            if (q * LPT < k && e[q] >= 0) {
                const float neg = a.sigmoid ? sigmoids(xe[q]).neg : 1.0f;
                part[q] = w[q] * (a.normalize ? g[q] - gw : g[q]) * neg;
            }
        }
        if (spread_weights) {
#pragma unroll
            for (int i = 0; i < VPL; ++i) dx[i] -= p[i] * gw;
        }
        float sum[kSel];
        bool mine[kSel];
#pragma unroll
        for (int q = 0; q < kSel; ++q) {
            mine[q] = e[q] >= 0;
            sum[q] = part[q];
        }
        // Every entry leaves its number at its expert: one that finds another's
        // there shares the expert, which routing itself never gives.
        float* to = add[slot];
#pragma unroll
        for (int q = 0; q < kSel; ++q)
            if (mine[q]) to[e[q]] = __int_as_float(q * LPT + lane);
        wave_sync();
        bool shared = false;
#pragma unroll
        for (int q = 0; q < kSel; ++q)
            if (mine[q]) shared |= __float_as_int(to[e[q]]) != q * LPT + lane;
        if (__any(shared)) join_entries<LPT, kSel, 0>(e, part, k, lane, sum, mine);
        wave_sync();
#pragma unroll
        for (int i = 0; i < VPL; ++i) to[expert<VPL, BF16>(own, i)] = 0.0f;
        wave_sync();
#pragma unroll
        for (int q = 0; q < kSel; ++q)
            if (mine[q]) to[e[q]] = sum[q];
        wave_sync();
#pragma unroll
        for (int i = 0; i < VPL; ++i) dx[i] += to[expert<VPL, BF16>(own, i)];
    }
    if (inside) {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (!(live && finite(x[i]))) dx[i] = 0.0f;
        store_logits<VPL, BF16>(d_logits, t * E, E, own, a.out_pieces, dx);
    }
}

template <int LPT, int VPL, bool BF16>
void launch_one(const RouteArgs& a, const RouteForward* f, const RouteBackward* b,
                hipStream_t stream) {
    constexpr int kTokens = kThreads / LPT;
    const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(a.num_tokens) + kTokens - 1) /
                                                kTokens);
    if (f != nullptr) {
        if (a.by_score)
            hipLaunchKernelGGL((route_kernel<LPT, VPL, BF16, true>), dim3(grid), dim3(kThreads), 0,
                               stream, a, f->bias, f->valid, f->topk_idx, f->topk_weights);
        else
            hipLaunchKernelGGL((route_kernel<LPT, VPL, BF16, false>), dim3(grid), dim3(kThreads), 0,
                               stream, a, f->bias, f->valid, f->topk_idx, f->topk_weights);
    } else {
        const float factor = b->coef * static_cast<float>(a.num_experts) /
                             (static_cast<float>(a.num_seqs) * static_cast<float>(a.num_topk));
        hipLaunchKernelGGL((route_backward_kernel<LPT, VPL, BF16>), dim3(grid), dim3(kThreads), 0,
                           stream, a, b->topk_idx, b->d_weights, b->valid, factor, b->counts,
                           b->num_valid, b->d_loss, b->d_logits);
    }
}

template <bool BF16>
hipError_t launch(const RouteArgs& a, const RouteForward* f, const RouteBackward* b,
                  hipStream_t stream) {
    if (a.num_tokens == 0) return hipSuccess;
    const TokenShape s = token_shape(a.num_experts, kSixteenLanes);
    if (s.lpt == 16) {
        switch (s.vpl) {
            case 1: launch_one<16, 1, BF16>(a, f, b, stream); break;
            case 2: launch_one<16, 2, BF16>(a, f, b, stream); break;
            case 4: launch_one<16, 4, BF16>(a, f, b, stream); break;
            case 8: launch_one<16, 8, BF16>(a, f, b, stream); break;
            case 16: launch_one<16, 16, BF16>(a, f, b, stream); break;
            default: launch_one<16, 32, BF16>(a, f, b, stream); break;
        }
    } else {
        launch_one<64, 16, BF16>(a, f, b, stream);
    }
    return hipGetLastError();
}

}  // namespace

// 16 lanes a token up to `most` experts, so that four tokens share each of a
// wave's reductions; 64 lanes above.
TokenShape token_shape(int num_experts, int most) {
    const int lpt = num_experts <= most ? 16 : 64;
    int vpl = 1;
    while (lpt * vpl < num_experts) vpl *= 2;
    return {lpt, vpl};
}

hipError_t launch_route(const RouteArgs& a, const RouteForward& f, hipStream_t stream) {
    return a.bf16 ? launch<true>(a, &f, nullptr, stream) : launch<false>(a, &f, nullptr, stream);
}

hipError_t launch_route_backward(const RouteArgs& a, const RouteBackward& b, hipStream_t stream) {
    return a.bf16 ? launch<true>(a, nullptr, &b, stream) : launch<false>(a, nullptr, &b, stream);
}

}  // namespace ep
