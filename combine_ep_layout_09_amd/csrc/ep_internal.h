// ep_internal.h -- launch helpers behind the libep C ABI (not exported).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ep.h"

namespace ep {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopk = 32;
constexpr int kMaxHidden = 65536;
constexpr int kMaxGroups = 64;
constexpr int kMaxSeqs = 1 << 20;
constexpr int kMaxRouted = 1 << 25;  // tokens: 64 lanes each stay below 2^32 threads
constexpr int kMaxRowed = 1 << 21;   // tokens: 1024 lanes each stay below 2^32 threads

// Workgroup width (a multiple of 64, at most 1024) and number of column tiles
// that cover a row of nvec 16-byte pieces with vpl pieces per lane.
struct TileShape {
    int threads;
    int tiles;
};
TileShape row_tile_shape(int nvec, int vpl);

// Dispatch launch shape: pieces per lane and the (token, column tile) grid's
// tile width and count.
struct DispatchShape {
    int vpl;
    TileShape tile;
};
DispatchShape dispatch_shape(int nvec, int T, bool fp8);

// Partition of the T*k routing entries into layout blocks.
struct LayoutGeometry {
    int64_t entries;   // T*k
    int32_t chunk;     // entries per block, a multiple of 256
    int32_t blocks;    // >= 1
    bool single_pass;  // one kernel, no workspace traffic
};

LayoutGeometry layout_geometry(const ep_problem& p);
LayoutGeometry layout_geometry_two_pass(const ep_problem& p);
int64_t layout_workspace_bytes(const ep_problem& p);

// Largest layout workspace of any supported problem (E = kMaxExperts): two
// tables of 64 rows by (E + 1) int32, rounded up to 256 bytes.  The
// allocation-free entry point keeps a device array of this size.
constexpr int64_t kMaxLayoutWorkspaceBytes = ((2 * 64 * (kMaxExperts + 1) * 4 + 255) / 256) * 256;

// Small routing tables (T*k entries): ep_layout and ep_layout_dispatch handle
// them in one kernel in which every workgroup reads the whole table, as long
// as the id visits of all workgroups together stay below kFusedMaxVisits.
constexpr int kFusedMaxEntries = 8192;
constexpr int64_t kFusedMaxVisits = int64_t{1} << 23;

// Mid-size tables (kFusedMaxEntries < T*k <= kWholeMaxEntries, LDS for E):
// ep_layout is one kernel in which every workgroup reads the whole table.
constexpr int kWholeMaxEntries = 65536;
constexpr int kWholeMinExperts = 32;
bool layout_whole_fits(const ep_problem& p);
hipError_t launch_layout(const ep_problem& p, const int32_t* topk_idx, const ep_layout_t& out,
                         int32_t* workspace, hipStream_t stream);
// The histogram kernel alone, with the per-block expert prefixes the ranking
// dispatch kernel of ep_layout_dispatch reads (two tables in the workspace);
// also zeroes status[1].
hipError_t launch_layout_tables(const ep_problem& p, const int32_t* topk_idx,
                                const LayoutGeometry& g, int32_t* workspace, int32_t* status,
                                hipStream_t stream);
hipError_t launch_dispatch(const ep_problem& p, const void* x, const int32_t* slot_of,
                           void* recv_x, void* recv_scales, hipStream_t stream);
hipError_t launch_layout_dispatch(const ep_problem& p, const int32_t* topk_idx,
                                  const ep_layout_t& out, void* workspace, const void* x,
                                  void* recv_x, void* recv_scales, hipStream_t stream);
// Prefill-sized tables: layout and dispatch in one launch of one workgroup
// per CU (ncu CUs), each holding its share of the rows in registers.  fits()
// says whether the problem takes that form.
bool layout_dispatch_persistent_fits(const ep_problem& p, int ncu);
hipError_t launch_layout_dispatch_persistent(const ep_problem& p, const int32_t* topk_idx,
                                             const ep_layout_t& out, const void* x, void* recv_x,
                                             void* recv_scales, int ncu, hipStream_t stream);
hipError_t launch_combine(const ep_problem& p, const void* expert_out, const int32_t* slot_of,
                          const float* topk_weights, void* y, hipStream_t stream);

// Routing (gate logits): the problem as the kernels take it.  `pieces` /
// `out_pieces`: rows of the logits / of the dense gradient can be accessed in
// aligned pieces of min(experts per lane, 16 bytes' worth) elements;
// `fours`: the bias (or rows of counts) in aligned groups of four.  `group_lanes`:
// lanes of a token that a group of experts fills exactly, 0 if it does not.
struct RouteArgs {
    const void* logits;
    int64_t stride;  // elements between rows of the logits
    int32_t num_tokens, num_experts, num_topk, num_groups, topk_groups;
    int32_t num_seqs, seq_len;
    float scale;
    int32_t group_lanes;
    bool bf16, sigmoid, normalize, pieces, out_pieces, fours, by_score;
};
// Lanes per token and experts per lane of the routing kernels.
struct TokenShape {
    int lpt, vpl;
};
// Experts up to which 16 lanes take a token: 16000 x 512 fp32, choice 11.9 us with
// 16 lanes, 15.7 with 64, gradient 19.5 and 21.1.
constexpr int kSixteenLanes = 512;
TokenShape token_shape(int num_experts, int most);
struct RouteForward {
    const float* bias;
    const uint8_t* valid;
    int32_t* topk_idx;
    float* topk_weights;
};
struct RouteBackward {
    const int32_t* topk_idx;
    const float* d_weights;
    const uint8_t* valid;
    float coef;
    const int32_t* counts;
    const int32_t* num_valid;
    const float* d_loss;
    void* d_logits;
};
hipError_t launch_route(const RouteArgs& a, const RouteForward& f, hipStream_t stream);
hipError_t launch_route_backward(const RouteArgs& a, const RouteBackward& b, hipStream_t stream);

struct BalanceArgs {
    const int32_t* topk_idx;
    const uint8_t* valid;
    float coef;
    int32_t* counts;
    float* mean_prob;
    int32_t* num_valid;
    float* loss;
};
int64_t balance_workspace_bytes(int num_tokens, int num_experts, int num_seqs);
hipError_t launch_balance(const RouteArgs& a, const BalanceArgs& b, void* workspace,
                          hipStream_t stream);

hipError_t launch_expert_w4(const ep_problem& p, const ep_expert_w4_t& mm, const void* rows,
                            const void* row_scales, const ep_layout_t& layout,
                            const uint8_t* codes, const uint8_t* scales, void* out,
                            hipStream_t stream);

// Layer norm: rows of x (and dy) a pitch apart, everything else dense.
struct NormArgs {
    const void* x;
    int64_t x_stride;  // elements
    const void* weight;
    const void* bias;
    void* y;
    float* mean;
    float* rstd;
    int32_t num_tokens, hidden;
    float eps;
};
struct NormGradArgs {
    const void* x;
    const void* dy;
    int64_t x_stride, dy_stride;
    const void* weight;
    const float* mean;
    const float* rstd;
    const void* d_skip;
    void* dx;
    void* d_weight;
    void* d_bias;
    int32_t num_tokens, hidden;
};
int norm_parts(int num_tokens, int hidden);
int64_t norm_workspace_bytes(int num_tokens, int hidden);
hipError_t launch_norm(const NormArgs& a, bool x_bf16, bool w_bf16, hipStream_t stream);
hipError_t launch_norm_grad(const NormGradArgs& a, bool x_bf16, bool w_bf16, void* workspace,
                            hipStream_t stream);

// Dropout of the combine: kept where the word is at least `border`, times `factor`.
struct DropArgs {
    const uint64_t* rng;  // {seed, offset}
    uint32_t border;      // 0: nothing is dropped, rng is not read
    float factor;
};
hipError_t launch_combine_dropout(const ep_problem& p, const void* expert_out,
                                  const int32_t* slot_of, const float* topk_weights,
                                  const void* residual, const DropArgs& drop, void* y,
                                  hipStream_t stream);
hipError_t launch_combine_backward(const ep_problem& p, const void* dy, const void* expert_out,
                                   const int32_t* slot_of, const float* topk_weights,
                                   const DropArgs& drop, void* d_expert_out, float* d_weights,
                                   hipStream_t stream);

hipError_t launch_dispatch_i8(const ep_problem& p, const void* x, const int32_t* slot_of,
                              void* recv_q, float* recv_scales, hipStream_t stream);
// 8-bit rows and their scales of the receive rows that an entry fills.
hipError_t launch_quant_rows(const ep_problem& p, int K, const void* rows,
                             const ep_layout_t& layout, int8_t* q, float* scales,
                             hipStream_t stream);
int64_t expert_i8_workspace_bytes(const ep_problem& p, const ep_expert_i8_t& mm);
hipError_t launch_expert_i8(const ep_problem& p, const ep_expert_i8_t& mm, const void* rows,
                            const float* row_scales, const ep_layout_t& layout,
                            const int8_t* weights, const float* scales, void* out,
                            void* workspace, hipStream_t stream);
hipError_t launch_e4m3_encode(const float* in, uint8_t* out, int64_t n, hipStream_t stream);

}  // namespace ep
