// ep_dropout_dev.h -- dropout's mask, made where it is needed and never stored.
//
// Philox4x32 with ten rounds (Salmon, Moraes, Dror and Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", 2011): four words from a counter of four words
// and a key of two.  A round multiplies two of the counter's words by constants and
// mixes the halves of the products with the other two and the key, which moves on
// by two more constants.  Element (t, c) takes word c % 4 at the counter
// {c / 4, t, offset}, so that any kernel makes the same mask, however it splits
// the rows.
#pragma once

#include "ep_device.h"
#include "ep_internal.h"

namespace ep {
namespace dropout {

// Bit i: channel 8 v + i of token t is kept.  Two counters at a time, the rounds as
// a loop: unrolled they make the combine's own loop over its pieces too long to be
// unrolled, and its pieces leave the registers (4096 tokens, H 7168, top-8: 114 us instead of
// 85, with no dropout in either).
__device__ __forceinline__ uint32_t keep8(const DropArgs& d, int t, int v) {
    if (d.border == 0) return 0xffu;
    const uint64_t seed = d.rng[0], offset = d.rng[1];
    uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
    uint32_t c[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        c[h][0] = static_cast<uint32_t>(2 * v + h);
        c[h][1] = static_cast<uint32_t>(t);
        c[h][2] = static_cast<uint32_t>(offset);
        c[h][3] = static_cast<uint32_t>(offset >> 32);
    }
#pragma unroll 1
    for (int i = 0; i < 10; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint64_t p0 = static_cast<uint64_t>(c[h][0]) * 0xD2511F53u;
            const uint64_t p1 = static_cast<uint64_t>(c[h][2]) * 0xCD9E8D57u;
            c[h][0] = static_cast<uint32_t>(p1 >> 32) ^ c[h][1] ^ k0;
            c[h][2] = static_cast<uint32_t>(p0 >> 32) ^ c[h][3] ^ k1;
            c[h][1] = static_cast<uint32_t>(p1);
            c[h][3] = static_cast<uint32_t>(p0);
        }
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    uint32_t kept = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) kept |= c[h][i] >= d.border ? 1u << (4 * h + i) : 0u;
    return kept;
}

}  // namespace dropout
}  // namespace ep
