// Declarations shared by the operators of a layer whose experts are resident
// (route, rows to experts and back, products grouped by expert) and of linear
// products with 4-bit weights.
#pragma once

#include "dense.cuh"

namespace pe {
namespace dense {

// ---- route

struct RouteArgs {
    const float* logits;
    int64_t ld;
    int32_t* ids;      // [tokens, k]
    float* weights;    // [tokens, k]
    int32_t* offsets;  // [experts + 1]
    int32_t* place;    // [tokens, k]
    int32_t* counts;   // [route_chunks(tokens)][experts]: entries of each chunk of tokens
    int tokens, experts, k;
};
constexpr int kMaxGroups = 1024;  // experts of a route, groups of a product
constexpr int kMostTopK = 32;
int route_chunks(int tokens);
cudaError_t launch_route_tokens(const RouteArgs& a, cudaStream_t st);

struct RouteBwdArgs {
    const float *dweights, *weights;
    const int32_t* ids;
    float* dlogits;
    int tokens, experts, k;
};
cudaError_t launch_route_bwd(const RouteBwdArgs& a, cudaStream_t st);

// ---- rows to experts and back

struct RowsArgs {
    const int32_t* place;  // [tokens, k]; entries outside [0, rows) are left out
    const void *x, *y, *res;
    int64_t ld_x, ld_y, ld_res;
    const float* weights;  // [tokens, k] or NULL: 1
    void* out;
    float* dweights;
    int tokens, k, rows, hidden;
};
// out[place] = weight * x
cudaError_t launch_expand(const RowsArgs& a, int elem, cudaStream_t st);
// out[t] = sum of weight * y[place] + res
cudaError_t launch_combine(const RowsArgs& a, int elem, cudaStream_t st);
// out[place] = weight * x (x: the gradient of the sum), dweights = <x, y[place]>
cudaError_t launch_combine_bwd(const RowsArgs& a, int elem, cudaStream_t st);

// ---- products grouped by expert

// Rows offsets[g] .. offsets[g + 1] - 1 belong to group g; what decreases or
// leaves [0, rows] is clamped.  Features lie along the MMA's M.
enum GroupKind {
    GROUP_ROWS = 0,      // out[r, f] = sum_k w[g][f, k] x[r, k]  (w_mn: w[g][k, f])
    GROUP_GATED = 1,     // the same with gate and up rows of w, act(gate) * up; optionally both kept, in fp32
    GROUP_GATED_BWD = 2, // dh as GROUP_ROWS, then the gradients of gate and up, and h, from what was kept
    GROUP_WEIGHTS = 3,   // out[g][m, n] = sum over the group's rows of w[r, m] x[r, n]
};
struct Grouped {
    const int32_t* offsets;
    int groups, rows;
    const void* w;   // GROUP_WEIGHTS: [rows, M], row pitch ld_w; else [groups][.., ..] contiguous
    int64_t ld_w;
    int w_mn;
    const void* x;   // [rows, K], GROUP_WEIGHTS: [rows, N]
    int64_t ld_x;
    int features;    // result columns (M); GROUP_GATED: w has twice as many rows
    int depth;       // K (GROUP_WEIGHTS: N)
    Epi e;           // out, act, keep, gu, h; rows and columns are the kernel's
};
cudaError_t launch_grouped(const Grouped& p, GroupKind kind, int elem, uint32_t* err, cudaStream_t st,
                           const WaitLimits* limits = nullptr);

// ---- 4-bit weights

enum W4Format { W4_INT4 = 0, W4_MXFP4 = 1, W4_NVFP4 = 2 };
constexpr int w4_group(int fmt) { return fmt == W4_INT4 ? 128 : fmt == W4_MXFP4 ? 32 : 16; }
struct W4Args {
    const void* x;
    int64_t ld_x;
    const void* codes;   // [N, K / 2]
    const void* scales;  // [N, ceil(K / group)]
    const float* tensor_scale;
    int M, N, K, fmt;
    Epi e;
};
// Rows that the kernel streaming into registers takes, and the one that decodes
// into shared memory; above, the weights are unpacked first.
constexpr int kW4Stream = 16, kW4Rows = 128;
cudaError_t launch_w4(const W4Args& a, int elem, cudaStream_t st);
cudaError_t launch_w4_tc(const W4Args& a, int elem, uint32_t* err, cudaStream_t st, const WaitLimits* limits = nullptr);
// w [N, K] of the element type = codes times scales, without the tensor's
cudaError_t launch_w4_unpack(const W4Args& a, void* w, int elem, cudaStream_t st);

}  // namespace dense
}  // namespace pe
