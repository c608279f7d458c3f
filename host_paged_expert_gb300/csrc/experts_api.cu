// C ABI of the operators of a layer whose experts are resident, and of linear
// products with 4-bit weights: checks of arguments, workspaces, and the order
// of their kernels.
#include <stdio.h>

#include "dense_args.h"
#include "experts.cuh"

using namespace pe;
using namespace pe::dense;

namespace {

cudaStream_t stream_of(void* s) { return static_cast<cudaStream_t>(s); }
bool entries_fit(int64_t tokens, int64_t k) { return tokens * k <= INT32_MAX; }

}  // namespace

// ---- route

extern "C" size_t pe_route_workspace(int32_t tokens, int32_t experts) {
    if (tokens <= 0 || experts <= 0 || route_chunks(tokens) == 1) return 0;  // one block needs none
    return up256(sizeof(int32_t) * (size_t)route_chunks(tokens) * experts);
}

extern "C" pe_status pe_route(const float* logits, int64_t logits_stride, int32_t* ids, float* weights, int32_t* offsets,
                              int32_t* place, void* workspace, size_t workspace_bytes, int32_t tokens, int32_t top_k,
                              int32_t experts, void* stream) {
    if (tokens < 0 || experts < 1 || top_k < 1 || top_k > experts)
        return bad("pe_route: top_k must be between 1 and experts, tokens not negative");
    if (experts > kMaxGroups || top_k > kMostTopK) return bad("pe_route: more than 1024 experts or top_k above 32", PE_ERR_RANGE);
    if (tokens > PE_MAX_ROWS || !entries_fit(tokens, top_k)) return bad("pe_route: more than 2^31 - 1 entries, or PE_MAX_ROWS tokens", PE_ERR_RANGE);
    if (!offsets || (tokens && (!logits || !ids || !weights || !place))) return bad("pe_route: NULL pointer");
    if (!whole(logits) || !whole(ids) || !whole(weights) || !whole(offsets) || !whole(place))
        return bad("pe_route: pointers must be 4-byte aligned");
    if (tokens == 0) return done(cudaMemsetAsync(offsets, 0, sizeof(int32_t) * (size_t)(experts + 1), stream_of(stream)));
    if (logits_stride < experts || logits_stride >= (int64_t(1) << 36)) return bad("pe_route: the logits' row pitch must be at least experts");
    const size_t need = pe_route_workspace(tokens, experts);
    if (workspace_bytes < need || (need && !workspace)) return bad("pe_route: workspace too small");
    if (!aligned(workspace)) return bad("pe_route: the workspace must be 16-byte aligned");
    RouteArgs a = {logits, logits_stride, ids, weights, offsets, place, static_cast<int32_t*>(workspace), tokens, experts, top_k};
    return done(launch_route_tokens(a, stream_of(stream)));
}

extern "C" pe_status pe_route_backward(const float* dweights, const float* weights, const int32_t* ids, float* dlogits,
                                       int32_t tokens, int32_t top_k, int32_t experts, void* stream) {
    if (tokens < 0 || experts < 1 || top_k < 1 || top_k > experts)
        return bad("pe_route_backward: top_k must be between 1 and experts, tokens not negative");
    if (experts > kMaxGroups || top_k > kMostTopK) return bad("pe_route_backward: more than 1024 experts or top_k above 32", PE_ERR_RANGE);
    if (tokens > PE_MAX_ROWS || !entries_fit(tokens, top_k)) return bad("pe_route_backward: more than 2^31 - 1 entries, or PE_MAX_ROWS tokens", PE_ERR_RANGE);
    if (tokens == 0) return PE_OK;
    if (!dweights || !weights || !ids || !dlogits) return bad("pe_route_backward: NULL pointer");
    if (!whole(dweights) || !whole(weights) || !whole(ids)) return bad("pe_route_backward: pointers must be 4-byte aligned");
    if (!aligned(dlogits)) return bad("pe_route_backward: dlogits must be 16-byte aligned");
    return done(launch_route_bwd({dweights, weights, ids, dlogits, tokens, experts, top_k}, stream_of(stream)));
}

// ---- rows to experts and back

namespace {

// What the three calls check alike; PE_OK with nothing to do is up to them.
pe_status rows_ok(const char* name, int32_t tokens, int32_t top_k, int32_t rows, int32_t hidden, int32_t elem) {
    static thread_local char msg[160];
    auto say = [&](const char* what, pe_status st) {
        snprintf(msg, sizeof msg, "%s: %s", name, what);
        return bad(msg, st);
    };
    if (!is_elem(elem)) return say("elem must be PE_ELEM_BF16 or PE_ELEM_F16", PE_ERR_INVALID);
    if (tokens < 0 || rows < 0 || top_k < 1 || hidden < 8 || hidden % 8)
        return say("hidden must be a positive multiple of 8, top_k positive, tokens and rows not negative", PE_ERR_INVALID);
    if (hidden > kMaxFeatures) return say("more than 2^24 features", PE_ERR_RANGE);
    if (tokens > PE_MAX_ROWS || rows > PE_MAX_ROWS || !entries_fit(tokens, top_k))
        return say("more than PE_MAX_ROWS tokens or rows, or 2^31 - 1 entries", PE_ERR_RANGE);
    return PE_OK;
}

}  // namespace

extern "C" pe_status pe_expand_rows(const void* x, int64_t x_stride, const int32_t* place, void* out, int32_t tokens,
                                    int32_t top_k, int32_t rows, int32_t hidden, int32_t elem, void* stream) {
    if (pe_status s = rows_ok("pe_expand_rows", tokens, top_k, rows, hidden, elem)) return s;
    if (tokens == 0 || rows == 0) return PE_OK;
    if (!x || !place || !out) return bad("pe_expand_rows: NULL pointer");
    if (!aligned(x) || !aligned(out) || !whole(place)) return bad("pe_expand_rows: pointers must be 16-byte aligned, place 4-byte aligned");
    if (!pitch_ok(x_stride, hidden, 2)) return bad("pe_expand_rows: x's row pitch must be a multiple of 8 and at least hidden");
    RowsArgs a = {};
    a.place = place;
    a.x = x;
    a.ld_x = x_stride;
    a.out = out;
    a.tokens = tokens;
    a.k = top_k;
    a.rows = rows;
    a.hidden = hidden;
    return done(launch_expand(a, elem, stream_of(stream)));
}

extern "C" pe_status pe_combine_rows(const void* y, int64_t y_stride, const int32_t* place, const float* weights,
                                     const void* residual, int64_t residual_stride, void* out, int32_t tokens,
                                     int32_t top_k, int32_t rows, int32_t hidden, int32_t elem, void* stream) {
    if (pe_status s = rows_ok("pe_combine_rows", tokens, top_k, rows, hidden, elem)) return s;
    if (tokens == 0) return PE_OK;
    if ((rows && !y) || !place || !out) return bad("pe_combine_rows: NULL pointer");
    if (!aligned(y) || !aligned(residual) || !aligned(out) || !whole(place) || !whole(weights))
        return bad("pe_combine_rows: pointers must be 16-byte aligned, place and weights 4-byte aligned");
    if ((rows && !pitch_ok(y_stride, hidden, 2)) || (residual && !pitch_ok(residual_stride, hidden, 2)))
        return bad("pe_combine_rows: row pitches must be multiples of 8 and at least hidden");
    RowsArgs a = {};
    a.place = place;
    a.y = y;
    a.ld_y = y_stride;
    a.res = residual;
    a.ld_res = residual_stride;
    a.weights = weights;
    a.out = out;
    a.tokens = tokens;
    a.k = top_k;
    a.rows = rows;
    a.hidden = hidden;
    return done(launch_combine(a, elem, stream_of(stream)));
}

extern "C" pe_status pe_combine_rows_backward(const void* dout, int64_t dout_stride, const void* y, int64_t y_stride,
                                              const int32_t* place, const float* weights, void* dy, float* dweights,
                                              int32_t tokens, int32_t top_k, int32_t rows, int32_t hidden, int32_t elem,
                                              void* stream) {
    if (pe_status s = rows_ok("pe_combine_rows_backward", tokens, top_k, rows, hidden, elem)) return s;
    if (tokens == 0) return PE_OK;
    if (!dout || !place || !weights || (rows && (!dy || (dweights && !y)))) return bad("pe_combine_rows_backward: NULL pointer");
    if (!aligned(dout) || !aligned(y) || !aligned(dy) || !whole(place) || !whole(weights) || !whole(dweights))
        return bad("pe_combine_rows_backward: pointers must be 16-byte aligned, place, weights and dweights 4-byte aligned");
    if (!pitch_ok(dout_stride, hidden, 2) || (rows && dweights && !pitch_ok(y_stride, hidden, 2)))
        return bad("pe_combine_rows_backward: row pitches must be multiples of 8 and at least hidden");
    RowsArgs a = {};
    a.place = place;
    a.x = dout;
    a.ld_x = dout_stride;
    a.y = y;
    a.ld_y = y_stride;
    a.weights = weights;
    a.out = dy;
    a.dweights = dweights;
    a.tokens = tokens;
    a.k = top_k;
    a.rows = rows;
    a.hidden = hidden;
    return done(dweights ? launch_combine_bwd(a, elem, stream_of(stream)) : launch_expand(a, elem, stream_of(stream)));
}

// ---- products grouped by expert

namespace {

pe_status grouped_ok(const char* name, int32_t rows, int32_t groups, int32_t a, int32_t b, const int32_t* offsets, int32_t elem) {
    static thread_local char msg[160];
    auto say = [&](const char* what, pe_status st) {
        snprintf(msg, sizeof msg, "%s: %s", name, what);
        return bad(msg, st);
    };
    if (!is_elem(elem)) return say("elem must be PE_ELEM_BF16 or PE_ELEM_F16", PE_ERR_INVALID);
    if (rows < 0 || groups < 1 || a < 8 || a % 8 || b < 8 || b % 8)
        return say("features must be positive multiples of 8, groups positive, rows not negative", PE_ERR_INVALID);
    if (groups > kMaxGroups) return say("more than 1024 groups", PE_ERR_RANGE);
    if (a > kMaxFeatures || b > kMaxFeatures || (int64_t)a * b > (int64_t(1) << 36)) return say("more than 2^24 features, or 2^36 weights of a group", PE_ERR_RANGE);
    if (rows > PE_MAX_ROWS) return say("more than PE_MAX_ROWS rows", PE_ERR_RANGE);
    if (rows && !offsets) return say("NULL pointer", PE_ERR_INVALID);
    if (!whole(offsets)) return say("offsets must be 4-byte aligned", PE_ERR_INVALID);
    return PE_OK;
}

// w [groups][features][depth] (mn: [groups][depth][features]) against x's rows
Grouped product(const void* w, int w_mn, const void* x, int64_t ld_x, const int32_t* offsets, int rows, int groups,
                int features, int depth) {
    Grouped p = {};
    p.offsets = offsets;
    p.groups = groups;
    p.rows = rows;
    p.w = w;
    p.w_mn = w_mn;
    p.x = x;
    p.ld_x = ld_x;
    p.features = features;
    p.depth = depth;
    return p;
}
// out [groups][m][n] = sum over a group's rows of a[r, m] b[r, n]
Grouped gradient(const void* a, int64_t ld_a, const void* b, int64_t ld_b, const int32_t* offsets, int rows, int groups, int m,
                 int n, void* out) {
    Grouped p = product(a, 1, b, ld_b, offsets, rows, groups, m, n);
    p.ld_w = ld_a;
    p.e.out = out;
    return p;
}

}  // namespace

extern "C" pe_status pe_grouped_linear(const void* x, int64_t x_stride, const void* weight, const int32_t* offsets, void* out,
                                       int32_t rows, int32_t groups, int32_t in_features, int32_t out_features, int32_t elem,
                                       void* stream) {
    if (pe_status s = grouped_ok("pe_grouped_linear", rows, groups, in_features, out_features, offsets, elem)) return s;
    if (rows == 0) return PE_OK;
    if (!x || !weight || !out) return bad("pe_grouped_linear: NULL pointer");
    if (!aligned(x) || !aligned(weight) || !aligned(out)) return bad("pe_grouped_linear: pointers must be 16-byte aligned");
    if (!pitch_ok(x_stride, in_features, 2)) return bad("pe_grouped_linear: x's row pitch must be a multiple of 8 and at least in_features");
    uint32_t* err = nullptr;
    if (cudaError_t e = error_word(&err)) return done(e);
    Grouped p = product(weight, 0, x, x_stride, offsets, rows, groups, out_features, in_features);
    p.e.out = out;
    p.e.ld_out = out_features;
    return done(launch_grouped(p, GROUP_ROWS, elem, err, stream_of(stream)));
}

extern "C" pe_status pe_grouped_linear_backward(const void* dy, int64_t dy_stride, const void* x, int64_t x_stride,
                                                const void* weight, const int32_t* offsets, void* dx, void* dweight,
                                                int32_t rows, int32_t groups, int32_t in_features, int32_t out_features,
                                                int32_t elem, void* stream) {
    if (pe_status s = grouped_ok("pe_grouped_linear_backward", rows, groups, in_features, out_features, offsets, elem)) return s;
    cudaStream_t st = stream_of(stream);
    if (rows == 0)
        return done(dweight ? cudaMemsetAsync(dweight, 0, 2 * (size_t)groups * in_features * out_features, st) : cudaSuccess);
    if (!dy || (dx && !weight) || (dweight && !x)) return bad("pe_grouped_linear_backward: NULL pointer");
    if (!aligned(dy) || !aligned(x) || !aligned(weight) || !aligned(dx) || !aligned(dweight))
        return bad("pe_grouped_linear_backward: pointers must be 16-byte aligned");
    if (!pitch_ok(dy_stride, out_features, 2) || (dweight && !pitch_ok(x_stride, in_features, 2)))
        return bad("pe_grouped_linear_backward: row pitches must be multiples of 8 and at least the row's length");
    uint32_t* err = nullptr;
    cudaError_t e = error_word(&err);
    if (!e && dx) {
        Grouped p = product(weight, 1, dy, dy_stride, offsets, rows, groups, in_features, out_features);
        p.e.out = dx;
        p.e.ld_out = in_features;
        e = launch_grouped(p, GROUP_ROWS, elem, err, st);
    }
    if (!e && dweight)
        e = launch_grouped(gradient(dy, dy_stride, x, x_stride, offsets, rows, groups, out_features, in_features, dweight),
                           GROUP_WEIGHTS, elem, err, st);
    return done(e);
}

extern "C" size_t pe_grouped_ffn_workspace(int32_t rows, int32_t intermediate) { return pe_gated_ffn_workspace(rows, intermediate); }

extern "C" pe_status pe_grouped_ffn(const void* x, int64_t x_stride, const void* w13, const void* w2, const int32_t* offsets,
                                    void* out, void* keep, int32_t act, void* workspace, size_t workspace_bytes, int32_t rows,
                                    int32_t groups, int32_t hidden, int32_t intermediate, int32_t elem, void* stream) {
    if (pe_status s = grouped_ok("pe_grouped_ffn", rows, groups, hidden, intermediate, offsets, elem)) return s;
    if (!is_act(act)) return bad("pe_grouped_ffn: unknown activation");
    if (rows == 0) return PE_OK;
    if (!x || !w13 || !w2 || !out) return bad("pe_grouped_ffn: NULL pointer");
    if (workspace_bytes < pe_grouped_ffn_workspace(rows, intermediate) || !workspace) return bad("pe_grouped_ffn: workspace too small");
    if (!aligned(x) || !aligned(w13) || !aligned(w2) || !aligned(out) || !aligned(keep) || !aligned(workspace))
        return bad("pe_grouped_ffn: pointers must be 16-byte aligned");
    if (!pitch_ok(x_stride, hidden, 2)) return bad("pe_grouped_ffn: x's row pitch must be a multiple of 8 and at least hidden");
    cudaStream_t st = stream_of(stream);
    uint32_t* err = nullptr;
    cudaError_t e = error_word(&err);
    if (!e) {
        Grouped p = product(w13, 0, x, x_stride, offsets, rows, groups, intermediate, hidden);
        p.e.act = act;
        // h is rounded to 16 bits, the type that the second product's MMA takes; what is
        // kept is not (16 bits would add as much again to the gradients' error)
        p.e.out = workspace;
        p.e.ld_out = intermediate;
        p.e.keep = keep;
        p.e.ld_keep = 2 * (int64_t)intermediate;
        e = launch_grouped(p, GROUP_GATED, elem, err, st);
    }
    if (!e) {
        Grouped p = product(w2, 0, workspace, intermediate, offsets, rows, groups, hidden, intermediate);
        p.e.out = out;
        p.e.ld_out = hidden;
        e = launch_grouped(p, GROUP_ROWS, elem, err, st);
    }
    return done(e);
}

extern "C" size_t pe_grouped_ffn_backward_workspace(int32_t rows, int32_t intermediate) {
    return pe_gated_ffn_backward_workspace(rows, intermediate);
}

extern "C" pe_status pe_grouped_ffn_backward(const void* dy, int64_t dy_stride, const void* x, int64_t x_stride,
                                             const void* w13, const void* w2, const void* keep, const int32_t* offsets,
                                             int32_t act, void* dx, void* dw13, void* dw2, void* workspace,
                                             size_t workspace_bytes, int32_t rows, int32_t groups, int32_t hidden,
                                             int32_t intermediate, int32_t elem, void* stream) {
    if (pe_status s = grouped_ok("pe_grouped_ffn_backward", rows, groups, hidden, intermediate, offsets, elem)) return s;
    if (!is_act(act)) return bad("pe_grouped_ffn_backward: unknown activation");
    cudaStream_t st = stream_of(stream);
    const size_t wbytes = 2 * (size_t)groups * hidden * intermediate;
    if (rows == 0) {
        cudaError_t e = dw13 ? cudaMemsetAsync(dw13, 0, 2 * wbytes, st) : cudaSuccess;
        if (!e && dw2) e = cudaMemsetAsync(dw2, 0, wbytes, st);
        return done(e);
    }
    if (!dy || !w2 || !keep || (dx && !w13) || (dw13 && !x)) return bad("pe_grouped_ffn_backward: NULL pointer");
    if (workspace_bytes < pe_grouped_ffn_backward_workspace(rows, intermediate) || !workspace)
        return bad("pe_grouped_ffn_backward: workspace too small");
    if (!aligned(dy) || !aligned(x) || !aligned(w13) || !aligned(w2) || !aligned(keep) || !aligned(dx) || !aligned(dw13) ||
        !aligned(dw2) || !aligned(workspace))
        return bad("pe_grouped_ffn_backward: pointers must be 16-byte aligned");
    if (!pitch_ok(dy_stride, hidden, 2) || (dw13 && !pitch_ok(x_stride, hidden, 2)))
        return bad("pe_grouped_ffn_backward: row pitches must be multiples of 8 and at least hidden");
    uint32_t* err = nullptr;
    cudaError_t e = error_word(&err);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    void* dgu = ws;
    void* h = ws + up256(4 * (size_t)rows * intermediate);
    const int64_t I2 = 2 * (int64_t)intermediate;
    // dg, du and h are rounded to 16 bits for the next products' MMAs, as in pe_gated_ffn_backward
    if (!e) {
        Grouped p = product(w2, 1, dy, dy_stride, offsets, rows, groups, intermediate, hidden);
        p.e.act = act;
        p.e.gu = keep;
        p.e.ld_keep = I2;
        p.e.out = dgu;
        p.e.ld_out = I2;
        p.e.h = dw2 ? h : nullptr;
        e = launch_grouped(p, GROUP_GATED_BWD, elem, err, st);
    }
    if (!e && dx) {
        Grouped p = product(w13, 1, dgu, I2, offsets, rows, groups, hidden, (int)I2);
        p.e.out = dx;
        p.e.ld_out = hidden;
        e = launch_grouped(p, GROUP_ROWS, elem, err, st);
    }
    if (!e && dw13)
        e = launch_grouped(gradient(dgu, I2, x, x_stride, offsets, rows, groups, (int)I2, hidden, dw13), GROUP_WEIGHTS, elem, err, st);
    if (!e && dw2)
        e = launch_grouped(gradient(dy, dy_stride, h, intermediate, offsets, rows, groups, hidden, intermediate, dw2), GROUP_WEIGHTS,
                           elem, err, st);
    return done(e);
}

// ---- 4-bit weights

extern "C" size_t pe_linear_four_bit_workspace(int32_t rows, int32_t in_features, int32_t out_features) {
    if (rows <= kW4Rows || in_features <= 0 || out_features <= 0) return 0;
    return up256(2 * (size_t)in_features * out_features);
}

extern "C" pe_status pe_linear_four_bit(const void* x, int64_t x_stride, const void* codes, const void* scales,
                                        const float* tensor_scale, int32_t format, const void* bias, const void* residual,
                                        int64_t residual_stride, void* out, int32_t out_elem, int32_t act, void* workspace,
                                        size_t workspace_bytes, int32_t rows, int32_t in_features, int32_t out_features,
                                        int32_t elem, void* stream) {
    const int fmt = format == PE_INT4_GPTQ ? W4_INT4 : format == PE_MXFP4 ? W4_MXFP4 : format == PE_NVFP4 ? W4_NVFP4 : -1;
    if (fmt < 0) return bad("pe_linear_four_bit: the format must be int4, MXFP4 or NVFP4", PE_ERR_UNSUPPORTED_DTYPE);
    if (!is_elem(elem)) return bad("pe_linear_four_bit: elem must be PE_ELEM_BF16 or PE_ELEM_F16");
    if (out_elem != elem && out_elem != PE_ELEM_F32) return bad("pe_linear_four_bit: out_elem must be elem or PE_ELEM_F32");
    if (!is_act(act)) return bad("pe_linear_four_bit: unknown activation");
    if (rows < 0 || out_features < 1 || in_features < 32 || in_features % 32)
        return bad("pe_linear_four_bit: in_features must be a positive multiple of 32, out_features positive");
    if (in_features > kMaxFeatures || out_features > kMaxFeatures) return bad("pe_linear_four_bit: more than 2^24 features", PE_ERR_RANGE);
    if (rows > PE_MAX_ROWS) return bad("pe_linear_four_bit: more than PE_MAX_ROWS rows", PE_ERR_RANGE);
    if (rows == 0) return PE_OK;
    if (!x || !codes || !scales || !out || (fmt == W4_NVFP4 && !tensor_scale)) return bad("pe_linear_four_bit: NULL pointer");
    if (!aligned(x) || !aligned(codes) || !aligned(scales) || !aligned(bias) || !aligned(residual) || !aligned(out))
        return bad("pe_linear_four_bit: pointers must be 16-byte aligned");
    if (!whole(tensor_scale)) return bad("pe_linear_four_bit: tensor_scale must be 4-byte aligned");
    if (!pitch_ok(x_stride, in_features, 2)) return bad("pe_linear_four_bit: x's row pitch must be a multiple of 8 and at least in_features");
    if (residual && !(out_features % 8 ? residual_stride == out_features : pitch_ok(residual_stride, out_features, 2)))
        return bad("pe_linear_four_bit: residual's row pitch must be a multiple of 8 and at least out_features "
                   "(contiguous if out_features is no multiple of 8)");
    const size_t need = pe_linear_four_bit_workspace(rows, in_features, out_features);
    if (workspace_bytes < need || (need && !workspace)) return bad("pe_linear_four_bit: workspace too small");
    if (!aligned(workspace)) return bad("pe_linear_four_bit: the workspace must be 16-byte aligned");
    cudaStream_t st = stream_of(stream);
    W4Args a = {};
    a.x = x;
    a.ld_x = x_stride;
    a.codes = codes;
    a.scales = scales;
    a.tensor_scale = tensor_scale;
    a.M = rows;
    a.N = out_features;
    a.K = in_features;
    a.fmt = fmt;
    a.e.act = act;
    a.e.rows = rows;
    a.e.cols = out_features;
    a.e.vec = out_features % 8 == 0;
    a.e.out = out;
    a.e.ld_out = out_features;
    a.e.out_f32 = out_elem == PE_ELEM_F32;
    a.e.bias = bias;
    a.e.res = residual;
    a.e.ld_res = residual_stride;
    if (rows <= kW4Stream) return done(launch_w4(a, elem, st));
    uint32_t* err = nullptr;
    cudaError_t e = error_word(&err);
    if (rows <= kW4Rows) return done(e ? e : launch_w4_tc(a, elem, err, st));
    if (!e) e = launch_w4_unpack(a, workspace, elem, st);
    if (!e) {
        Product p = {};
        p.a = x;
        p.lda = x_stride;
        p.b = workspace;
        p.ldb = in_features;
        p.M = rows;
        p.N = out_features;
        p.K = in_features;
        p.e = a.e;
        p.e.factor = tensor_scale;
        e = launch_product(p, fmt == W4_NVFP4 ? EPI_SCALED : EPI_LINEAR, elem, CHAIN_NONE, err, st);
    }
    return done(e);
}

// ---- self-test

extern "C" pe_status pe_selftest_experts_waits(uint32_t poll_limit, void* scratch, size_t scratch_bytes, uint32_t* out_words) {
    if (!out_words || !scratch || poll_limit == 0) return bad("pe_selftest_experts_waits: NULL pointer or no polls");
    if (scratch_bytes < PE_SELFTEST_EXPERTS_BYTES || !aligned(scratch, 256))
        return bad("pe_selftest_experts_waits: scratch too small or not 256-byte aligned");
    // operands and scales are zeros; one group; a word of its own for each run
    constexpr int R = 1000, N = 256, K = 1024, T = 32, K4 = 4096;  // a tail of rows, more blocks than stages
    constexpr int kTileRows = 128;
    constexpr size_t kOperand = 2 * (size_t)K * K, kRuns = 12;
    static_assert(2 * R * N <= (int)kOperand && T * K4 * 2 <= (int)kOperand && 512 + kOperand + 4 * N * K <= PE_SELFTEST_EXPERTS_BYTES, "the scratch holds them");
    uint8_t* base = static_cast<uint8_t*>(scratch);
    uint32_t* words = reinterpret_cast<uint32_t*>(base);
    int32_t* offsets = reinterpret_cast<int32_t*>(base + 256);
    uint8_t *ops = base + 512, *out = ops + kOperand;
    const int32_t ends[2] = {0, R};
    cudaError_t e = cudaMemset(scratch, 0, PE_SELFTEST_EXPERTS_BYTES);
    if (!e) e = cudaMemcpy(offsets, ends, sizeof ends, cudaMemcpyHostToDevice);
    // one role gives up at once, the others after poll_limit polls
    const WaitLimits gives_up[3] = {{poll_limit, 0, poll_limit}, {poll_limit, poll_limit, 0}, {0, poll_limit, poll_limit}};
    for (size_t i = 0; !e && i < kRuns; ++i) {
        const WaitLimits* limits = &gives_up[i % 3];
        if (i < 9) {
            const GroupKind kind = i < 3 ? GROUP_ROWS : i < 6 ? GROUP_GATED : GROUP_WEIGHTS;
            // rows in no group past K, the operands' ends
            Grouped p = kind == GROUP_WEIGHTS ? gradient(ops, N, ops, N, offsets, R, 1, N, N, out)
                                              : product(ops, 0, ops, K, offsets, N, 1, kind == GROUP_GATED ? N / 2 : N, K);
            p.e.out = out;
            p.e.ld_out = N;
            e = launch_grouped(p, kind, PE_ELEM_BF16, words + i, 0, limits);
        } else {
            W4Args a = {};
            a.x = ops;
            a.ld_x = K4;
            a.codes = ops;
            a.scales = ops;
            a.M = T;
            a.N = kTileRows;
            a.K = K4;
            a.e.rows = T;
            a.e.cols = kTileRows;
            a.e.vec = 1;
            a.e.out = out;
            a.e.ld_out = kTileRows;
            e = launch_w4_tc(a, PE_ELEM_BF16, words + i, 0, limits);
        }
    }
    if (!e) e = cudaDeviceSynchronize();
    if (!e) e = cudaMemcpy(out_words, words, kRuns * sizeof(uint32_t), cudaMemcpyDeviceToHost);
    return done(e);
}
