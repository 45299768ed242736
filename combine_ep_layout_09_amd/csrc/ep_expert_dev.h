// ep_expert_dev.h -- what the experts' product kernels share: loads through bounded
// views, the exchange of lanes that lets weights be loaded as whole cache lines,
// and the search for a workgroup's expert and rows.
#pragma once

#include "ep_device.h"

namespace ep {
namespace expert {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kNowhere = 0x7fffff00u;  // past the end of every view
template <bool ONCE>  // not kept in the caches
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t at, uint32_t step) {
    return __builtin_bit_cast(u32x4,
                              __builtin_amdgcn_raw_buffer_load_b128(r, at, step, ONCE ? 2 : 0));
}

// a: rows 0-7, b: rows 8-15 of a weight tile, lane l of a row of 16 lanes
// holding row l % 8 and, below lane 8, the first chunk, from lane 8 on, the
// second one.  Afterwards a is the first chunk and b the second one, lane l
// holding row l: lanes 8-15 of a and 0-7 of b change places.
__device__ __forceinline__ void pair_chunks(u32x4& a, u32x4& b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int x = static_cast<int>(a[i]), y = static_cast<int>(b[i]);
        a[i] = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(x, y, 0x128, 0xf, 0xc, false));
        b[i] = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(y, x, 0x128, 0xf, 0x3, false));
    }
}

// Inclusive sum over the lanes of a wave, stopping at `top` (v at most top,
// top below 2^31).
__device__ __forceinline__ uint32_t wave_scan(uint32_t v, uint32_t top) {
    const auto step = [&](auto shifted) { v = min(v + static_cast<uint32_t>(shifted), top); };
    const auto now = [&]() { return static_cast<int>(v); };
    step(__builtin_amdgcn_update_dpp(0, now(), 0x111, 0xf, 0xf, false));  // row_shr 1
    step(__builtin_amdgcn_update_dpp(0, now(), 0x112, 0xf, 0xf, false));
    step(__builtin_amdgcn_update_dpp(0, now(), 0x114, 0xf, 0xf, false));
    step(__builtin_amdgcn_update_dpp(0, now(), 0x118, 0xf, 0xf, false));
    step(__builtin_amdgcn_update_dpp(0, now(), 0x142, 0xa, 0xf, false));  // row_bcast 15
    step(__builtin_amdgcn_update_dpp(0, now(), 0x143, 0xc, 0xf, false));  // row_bcast 31
    return v;
}

// The expert, rows and row tile that number pick(number of tiles) names: experts
// with rows, in order, each with one tile per MC rows; expert -1 if there are
// fewer.
// Every wave finds it by itself, a lane per run of experts, so no wave waits
// for another; contiguous rows start where the counts before them end.
struct Found {
    int expert, count, tile;
    int64_t start;
};
template <int MC, class Args, class Pick>
__device__ __forceinline__ Found find_tile(const Args& a, Pick pick) {
    const int lane = threadIdx.x % kWave;
    const int per = (a.num_experts + kWave - 1) / kWave;
    // Counts of another problem's layout must not lead outside the rows: all
    // sums stop at the number of rows (and of tiles).
    const uint32_t most = static_cast<uint32_t>(a.capacity > 0 ? a.capacity : a.num_rows);
    const uint32_t top_rows = static_cast<uint32_t>(a.num_rows), top_tiles = 0x40000000u;
    const auto count_of = [&](int e) {
        const int n = e < a.num_experts ? a.count[e] : 0;
        return n < 0 ? 0u : min(static_cast<uint32_t>(n), most);
    };
    const auto tiles_of = [](uint32_t n) { return (n + MC - 1) / MC; };
    uint32_t rows = 0, tiles = 0;
    for (int i = 0; i < per; ++i) {
        const uint32_t n = count_of(lane * per + i);
        rows = min(rows + n, top_rows);
        tiles = min(tiles + tiles_of(n), top_tiles);
    }
    // sums up to and with this lane
    const uint32_t rows_to = wave_scan(rows, top_rows);
    const uint32_t tiles_to = wave_scan(tiles, top_tiles);
    const uint32_t want = pick(__builtin_amdgcn_readlane(tiles_to, kWave - 1));
    const uint64_t beyond = __ballot(tiles_to > want);
    Found f{-1, 0, 0, 0};
    if (beyond == 0) return f;
    const int owner = __ffsll(static_cast<unsigned long long>(beyond)) - 1;
    uint32_t at = 0, row = 0;
    if (owner > 0) {
        at = __builtin_amdgcn_readlane(tiles_to, owner - 1);
        row = __builtin_amdgcn_readlane(rows_to, owner - 1);
    }
    for (int i = 0; i < per; ++i) {
        const uint32_t n = __builtin_amdgcn_readfirstlane(count_of(owner * per + i));
        if (want - at < tiles_of(n)) {
            f.expert = owner * per + i;
            f.tile = static_cast<int>(want - at);
            f.start = a.capacity > 0 ? static_cast<int64_t>(f.expert) * a.capacity : row;
            f.count = static_cast<int>(a.capacity > 0 ? n : min(n, top_rows - row));
            break;
        }
        at += tiles_of(n);
        row = min(row + n, top_rows);
    }
    return f;
}

}  // namespace expert
}  // namespace ep
