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

__device__ __forceinline__ void philox(uint32_t (&c)[4], uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t p0 = static_cast<uint64_t>(c[0]) * 0xD2511F53u;
        const uint64_t p1 = static_cast<uint64_t>(c[2]) * 0xCD9E8D57u;
        c[0] = static_cast<uint32_t>(p1 >> 32) ^ c[1] ^ k0;
        c[2] = static_cast<uint32_t>(p0 >> 32) ^ c[3] ^ k1;
        c[1] = static_cast<uint32_t>(p1);
        c[3] = static_cast<uint32_t>(p0);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
}

// Bit i: channel 8 v + i of token t is kept.
__device__ __forceinline__ uint32_t keep8(const DropArgs& d, int t, int v) {
    if (d.border == 0) return 0xffu;
    const uint64_t seed = d.rng[0], offset = d.rng[1];
    uint32_t kept = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t c[4] = {static_cast<uint32_t>(2 * v + h), static_cast<uint32_t>(t),
                         static_cast<uint32_t>(offset), static_cast<uint32_t>(offset >> 32)};
        philox(c, static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32));
#pragma unroll
        for (int i = 0; i < 4; ++i) kept |= c[i] >= d.border ? 1u << (4 * h + i) : 0u;
    }
    return kept;
}

}  // namespace dropout
}  // namespace ep
