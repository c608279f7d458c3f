// C ABI of the dense operators: checks of arguments, workspaces, and the
// order of their kernels.
#include <mutex>

#include "dense.cuh"
#include "pe_internal.h"

namespace pe {
namespace dense {
namespace {

constexpr int kMaxDevices = 64;
constexpr int kMaxNormHidden = 32768;
constexpr int kMaxFeatures = 1 << 24;

__device__ uint32_t g_dense_err;

std::mutex g_mu;
uint32_t* g_err_ptr[kMaxDevices] = {};

// Device address of the error word on the current device, looked up once.
cudaError_t error_word(uint32_t** out) {
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(g_mu);
    if (!g_err_ptr[dev]) {
        void* p = nullptr;
        if (cudaError_t e = cudaGetSymbolAddress(&p, g_dense_err)) return e;
        g_err_ptr[dev] = static_cast<uint32_t*>(p);
    }
    *out = g_err_ptr[dev];
    return cudaSuccess;
}

pe_status bad(const char* msg, pe_status st = PE_ERR_INVALID) {
    set_thread_error(msg);
    return st;
}
pe_status done(cudaError_t e) {
    if (!e) return PE_OK;
    return bad(cudaGetErrorString(e), PE_ERR_CUDA);
}

bool aligned(const void* p, int to = 16) { return reinterpret_cast<uintptr_t>(p) % to == 0; }
// what is read and written one element at a time
bool whole(const float* p) { return aligned(p, sizeof(float)); }
bool is_elem(int e) { return e == PE_ELEM_BF16 || e == PE_ELEM_F16; }
bool is_act(int a) { return a >= PE_ACT_NONE && a <= PE_ACT_RELU; }
bool pitch_ok(int64_t ld, int64_t row, int bytes) { return ld >= row && ld * bytes % 16 == 0 && ld < (int64_t(1) << 36); }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }

Product make(const void* a, int64_t lda, int a_mn, const void* b, int64_t ldb, int b_mn, int M, int N, int K) {
    Product p = {};
    p.a = a;
    p.lda = lda;
    p.a_mn = a_mn;
    p.b = b;
    p.ldb = ldb;
    p.b_mn = b_mn;
    p.M = M;
    p.N = N;
    p.K = K;
    p.e.rows = M;
    p.e.cols = N;
    p.e.vec = N % 8 == 0;
    return p;
}

int pad8(int n) { return (n + 7) / 8 * 8; }

}  // namespace
}  // namespace dense
}  // namespace pe

using namespace pe;
using namespace pe::dense;

extern "C" pe_status pe_dense_error(uint32_t* word) {
    if (!word) return bad("pe_dense_error: NULL pointer");
    uint32_t* p = nullptr;
    cudaError_t e = error_word(&p);
    if (!e) e = cudaDeviceSynchronize();
    if (!e) e = cudaMemcpy(word, p, sizeof(uint32_t), cudaMemcpyDeviceToHost);
    return done(e);
}

extern "C" pe_status pe_selftest_dense_waits(uint32_t poll_limit, void* scratch, size_t scratch_bytes, uint32_t* out12) {
    if (!out12 || !scratch || poll_limit == 0) return bad("pe_selftest_dense_waits: NULL pointer or no polls");
    if (scratch_bytes < PE_SELFTEST_DENSE_BYTES || !aligned(scratch, 256))
        return bad("pe_selftest_dense_waits: scratch too small or not 256-byte aligned");
    // operands and scales are zeros; a word of its own for each run
    constexpr int M = 256, KB = 16, kOperands = M * KB * 128;
    uint8_t* base = static_cast<uint8_t*>(scratch);
    uint32_t* words = reinterpret_cast<uint32_t*>(base);
    uint8_t *ab = base + 256, *out = ab + kOperands;
    static_assert(256 + kOperands + 2 * M * M <= PE_SELFTEST_DENSE_BYTES, "the scratch holds operands and result");
    cudaError_t e = cudaMemset(scratch, 0, PE_SELFTEST_DENSE_BYTES);
    // one role gives up at once, the others after poll_limit polls
    const WaitLimits gives_up[3] = {{poll_limit, 0, poll_limit}, {poll_limit, poll_limit, 0}, {0, poll_limit, poll_limit}};
    for (int i = 0; !e && i < 12; ++i) {
        const bool fp8 = i / 6 != 0, split = i / 3 % 2 != 0;
        const int k = KB * (fp8 ? 128 : 64), m = split ? 64 : M, n = split ? 128 : M;
        Product p = make(ab, k, 0, ab, k, 0, m, n, k);
        if (fp8) p.a_scale = p.b_scale = reinterpret_cast<const float*>(ab);
        p.e.out = out;
        p.e.ld_out = n;
        e = split ? launch_split(p, EPI_LINEAR, PE_ELEM_BF16, {64, 2}, CHAIN_NONE, words + i, 0, &gives_up[i % 3])
                  : launch_pairs(&p, 1, EPI_LINEAR, PE_ELEM_BF16, 256, words + i, 0, &gives_up[i % 3]);
    }
    if (!e) e = cudaDeviceSynchronize();
    if (!e) e = cudaMemcpy(out12, words, 12 * sizeof(uint32_t), cudaMemcpyDeviceToHost);
    return done(e);
}

extern "C" pe_status pe_rms_norm(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                                 const void* weight, float eps, void* y, void* sum, void* codes, float* scales,
                                 float* rstd, int32_t rows, int32_t hidden, int32_t elem, void* stream) {
    if (!is_elem(elem)) return bad("pe_rms_norm: elem must be PE_ELEM_BF16 or PE_ELEM_F16");
    if (rows < 0 || hidden < 8 || hidden % 8) return bad("pe_rms_norm: hidden must be a positive multiple of 8, rows not negative");
    if (hidden > kMaxNormHidden) return bad("pe_rms_norm: hidden above 32768", PE_ERR_RANGE);
    if (rows > PE_MAX_ROWS) return bad("pe_rms_norm: more than PE_MAX_ROWS rows", PE_ERR_RANGE);
    if (rows == 0) return PE_OK;
    if (!x || !weight) return bad("pe_rms_norm: NULL pointer");
    if (!codes != !scales) return bad("pe_rms_norm: codes and scales go together");
    if (!aligned(x) || !aligned(residual) || !aligned(weight) || !aligned(y) || !aligned(sum) || !aligned(codes))
        return bad("pe_rms_norm: pointers must be 16-byte aligned");
    if (!whole(scales) || !whole(rstd)) return bad("pe_rms_norm: scales and rstd must be 4-byte aligned");
    if (!pitch_ok(x_stride, hidden, 2) || (residual && !pitch_ok(residual_stride, hidden, 2)))
        return bad("pe_rms_norm: row pitches must be multiples of 8 and at least hidden");
    NormArgs a = {x, residual, weight, x_stride, residual_stride, eps, y, sum, codes, scales, rstd, rows, hidden};
    return done(launch_rms_norm(a, elem, static_cast<cudaStream_t>(stream)));
}

extern "C" size_t pe_rms_norm_backward_workspace(int32_t rows, int32_t hidden) {
    if (rows <= 0 || hidden <= 0) return 0;
    return up256(sizeof(float) * (size_t)norm_bwd_blocks(rows) * hidden);
}

extern "C" pe_status pe_rms_norm_backward(const void* dy, int64_t dy_stride, const void* dsum, int64_t dsum_stride,
                                          const void* sum, int64_t sum_stride, const void* weight, const float* rstd,
                                          void* dx, void* dweight, void* workspace, size_t workspace_bytes,
                                          int32_t rows, int32_t hidden, int32_t elem, void* stream) {
    if (!is_elem(elem)) return bad("pe_rms_norm_backward: elem must be PE_ELEM_BF16 or PE_ELEM_F16");
    if (rows < 0 || hidden < 8 || hidden % 8)
        return bad("pe_rms_norm_backward: hidden must be a positive multiple of 8, rows not negative");
    if (hidden > kMaxNormHidden) return bad("pe_rms_norm_backward: hidden above 32768", PE_ERR_RANGE);
    if (rows > PE_MAX_ROWS) return bad("pe_rms_norm_backward: more than PE_MAX_ROWS rows", PE_ERR_RANGE);
    if (!dweight || (rows && (!dy || !sum || !weight || !rstd || !dx))) return bad("pe_rms_norm_backward: NULL pointer");
    const size_t need = pe_rms_norm_backward_workspace(rows, hidden);
    if (workspace_bytes < need || (need && !workspace)) return bad("pe_rms_norm_backward: workspace too small");
    if (!aligned(dy) || !aligned(dsum) || !aligned(sum) || !aligned(weight) || !aligned(dx) || !aligned(workspace))
        return bad("pe_rms_norm_backward: pointers must be 16-byte aligned");
    if (!whole(rstd) || !aligned(dweight, 2)) return bad("pe_rms_norm_backward: rstd must be 4-byte, dweight 2-byte aligned");
    if (rows && (!pitch_ok(dy_stride, hidden, 2) || !pitch_ok(sum_stride, hidden, 2) ||
                 (dsum && !pitch_ok(dsum_stride, hidden, 2))))
        return bad("pe_rms_norm_backward: row pitches must be multiples of 8 and at least hidden");
    NormBwdArgs a = {dy,   dsum, sum,     weight, dy_stride,                       dsum_stride, sum_stride,
                     rstd, dx,   dweight, static_cast<float*>(workspace), rows,        hidden};
    return done(launch_rms_norm_bwd(a, elem, static_cast<cudaStream_t>(stream)));
}

extern "C" pe_status pe_linear(const void* x, int64_t x_stride, const float* x_scale, const void* weight,
                               const float* w_scale, const void* bias, const void* residual, int64_t residual_stride,
                               void* out, int32_t out_elem, void* keep, int32_t act, int32_t rows, int32_t in_features,
                               int32_t out_features, int32_t elem, void* stream) {
    if (!is_elem(elem)) return bad("pe_linear: elem must be PE_ELEM_BF16 or PE_ELEM_F16");
    if (out_elem != elem && out_elem != PE_ELEM_F32) return bad("pe_linear: out_elem must be elem or PE_ELEM_F32");
    if (!is_act(act)) return bad("pe_linear: unknown activation");
    if (!x_scale != !w_scale) return bad("pe_linear: x_scale and w_scale go together");
    const int bytes = x_scale ? 1 : 2;
    if (rows < 0 || out_features < 1 || in_features < 16 / bytes || in_features * (int64_t)bytes % 16)
        return bad("pe_linear: in_features must be a positive multiple of 8 (of 16 for E4M3), out_features positive");
    if (in_features > kMaxFeatures || out_features > kMaxFeatures) return bad("pe_linear: more than 2^24 features", PE_ERR_RANGE);
    if (rows > PE_MAX_ROWS) return bad("pe_linear: more than PE_MAX_ROWS rows", PE_ERR_RANGE);
    if (rows == 0) return PE_OK;
    if (!x || !weight || !out) return bad("pe_linear: NULL pointer");
    if (!aligned(x) || !aligned(weight) || !aligned(bias) || !aligned(residual) || !aligned(out) || !aligned(keep))
        return bad("pe_linear: pointers must be 16-byte aligned");
    if (!whole(x_scale) || !whole(w_scale)) return bad("pe_linear: scales must be 4-byte aligned");
    if (!pitch_ok(x_stride, in_features, bytes)) return bad("pe_linear: x's row pitch must be a multiple of 16 bytes and at least in_features");
    if (residual && !(out_features % 8 ? residual_stride == out_features : pitch_ok(residual_stride, out_features, 2)))
        return bad("pe_linear: residual's row pitch must be a multiple of 8 and at least out_features "
                   "(contiguous if out_features is no multiple of 8)");
    uint32_t* err = nullptr;
    if (cudaError_t e = error_word(&err)) return done(e);
    Product p = make(x, x_stride, 0, weight, in_features, 0, rows, out_features, in_features);
    p.a_scale = x_scale;
    p.b_scale = w_scale;
    p.e.act = act;
    p.e.out = out;
    p.e.ld_out = out_features;
    p.e.out_f32 = out_elem == PE_ELEM_F32;
    p.e.bias = bias;
    p.e.res = residual;
    p.e.ld_res = residual_stride;
    p.e.keep = keep;
    p.e.ld_keep = out_features;
    return done(launch_product(p, EPI_LINEAR, elem, CHAIN_NONE, err, static_cast<cudaStream_t>(stream)));
}

namespace {
// pe_linear_backward's workspace: dz with rows padded to 8 elements, then the
// column sums' partials, whose room goes by the sizes alone (the chunk that
// the kernel takes is a matter of speed, and no caller's).
size_t dz_bytes(int rows, int n) { return up256(2 * (size_t)rows * pad8(n)); }
}  // namespace

extern "C" size_t pe_linear_backward_workspace(int32_t rows, int32_t out_features, int32_t act) {
    if (rows <= 0 || out_features <= 0 || !is_act(act)) return 0;
    const size_t dz = act != PE_ACT_NONE || out_features % 8 ? dz_bytes(rows, out_features) : 0;
    return dz + up256(sizeof(float) * (((size_t)rows + kSumRows - 1) / kSumRows) * out_features);
}

extern "C" pe_status pe_linear_backward(const void* dy, int64_t dy_stride, const void* x, int64_t x_stride,
                                        const void* weight, const void* keep, int32_t act, void* dx, void* dweight,
                                        void* dbias, void* workspace, size_t workspace_bytes, int32_t rows,
                                        int32_t in_features, int32_t out_features, int32_t elem, void* stream) {
    if (!is_elem(elem)) return bad("pe_linear_backward: elem must be PE_ELEM_BF16 or PE_ELEM_F16");
    if (!is_act(act)) return bad("pe_linear_backward: unknown activation");
    if (rows < 0 || out_features < 1 || in_features < 8 || in_features % 8)
        return bad("pe_linear_backward: in_features must be a positive multiple of 8, out_features positive");
    if (in_features > kMaxFeatures || out_features > kMaxFeatures)
        return bad("pe_linear_backward: more than 2^24 features", PE_ERR_RANGE);
    if (rows > PE_MAX_ROWS) return bad("pe_linear_backward: more than PE_MAX_ROWS rows", PE_ERR_RANGE);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (rows == 0) {
        cudaError_t e = dweight ? cudaMemsetAsync(dweight, 0, 2 * (size_t)out_features * in_features, st) : cudaSuccess;
        if (!e && dbias) e = cudaMemsetAsync(dbias, 0, 2 * (size_t)out_features, st);
        return done(e);
    }
    if (!dy || (dx && !weight) || (dweight && !x) || (act != PE_ACT_NONE && !keep))
        return bad("pe_linear_backward: NULL pointer");
    const size_t need = pe_linear_backward_workspace(rows, out_features, act);
    if (workspace_bytes < need || !workspace) return bad("pe_linear_backward: workspace too small");
    if (!aligned(dy) || !aligned(x) || !aligned(weight) || !aligned(keep) || !aligned(dx) || !aligned(dweight) || !aligned(workspace))
        return bad("pe_linear_backward: pointers must be 16-byte aligned");
    if (!aligned(dbias, 2)) return bad("pe_linear_backward: dbias must be 2-byte aligned");
    const bool odd = out_features % 8 != 0;
    if (!(odd ? dy_stride == out_features : pitch_ok(dy_stride, out_features, 2)))
        return bad("pe_linear_backward: dy's row pitch must be a multiple of 8 and at least out_features "
                   "(contiguous if out_features is no multiple of 8)");
    if (dweight && !pitch_ok(x_stride, in_features, 2))
        return bad("pe_linear_backward: x's row pitch must be a multiple of 8 and at least in_features");
    uint32_t* err = nullptr;
    cudaError_t e = error_word(&err);
    // dz, unless it is dy itself
    const bool own_dz = act != PE_ACT_NONE || odd;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const void* dz = own_dz ? ws : dy;
    const int64_t ld_dz = own_dz ? pad8(out_features) : dy_stride;
    if (!e && (dbias || (own_dz && (dx || dweight)))) {
        ActBwdArgs a = {};
        a.dy = dy;
        a.ld_dy = dy_stride;
        a.z = act == PE_ACT_NONE ? nullptr : keep;
        a.ld_z = out_features;
        a.dz = own_dz ? ws : nullptr;
        a.ld_dz = ld_dz;
        a.db = dbias;
        a.partial = reinterpret_cast<float*>(ws + (own_dz ? dz_bytes(rows, out_features) : 0));
        a.act = act;
        a.rows = rows;
        a.cols = out_features;
        e = launch_act_bwd(a, elem, st);
    }
    Product p[2];
    int n = 0;
    if (dx) {
        p[n] = make(dz, ld_dz, 0, weight, in_features, 1, rows, in_features, out_features);
        p[n].e.out = dx;
        p[n++].e.ld_out = in_features;
    }
    if (dweight) {
        p[n] = make(dz, ld_dz, 1, x, x_stride, 1, out_features, in_features, rows);
        p[n].e.out = dweight;
        p[n++].e.ld_out = in_features;
    }
    if (!e) e = launch_products(p, n, elem, err, st);
    return done(e);
}

extern "C" size_t pe_gated_ffn_workspace(int32_t rows, int32_t intermediate) {
    if (rows <= 0 || intermediate <= 0) return 0;
    return up256(2 * (size_t)rows * intermediate);
}

extern "C" pe_status pe_gated_ffn(const void* x, int64_t x_stride, const void* w13, const void* w2,
                                  const void* residual, int64_t residual_stride, void* out, void* keep, int32_t act,
                                  void* workspace, size_t workspace_bytes, int32_t rows, int32_t hidden,
                                  int32_t intermediate, int32_t elem, void* stream) {
    if (!is_elem(elem)) return bad("pe_gated_ffn: elem must be PE_ELEM_BF16 or PE_ELEM_F16");
    if (!is_act(act)) return bad("pe_gated_ffn: unknown activation");
    if (rows < 0 || hidden < 8 || hidden % 8 || intermediate < 8 || intermediate % 8)
        return bad("pe_gated_ffn: hidden and intermediate must be positive multiples of 8");
    if (hidden > kMaxFeatures || intermediate > kMaxFeatures) return bad("pe_gated_ffn: more than 2^24 features", PE_ERR_RANGE);
    if (rows > PE_MAX_ROWS) return bad("pe_gated_ffn: more than PE_MAX_ROWS rows", PE_ERR_RANGE);
    if (rows == 0) return PE_OK;
    if (!x || !w13 || !w2 || !out) return bad("pe_gated_ffn: NULL pointer");
    if (workspace_bytes < pe_gated_ffn_workspace(rows, intermediate) || !workspace) return bad("pe_gated_ffn: workspace too small");
    if (!aligned(x) || !aligned(w13) || !aligned(w2) || !aligned(residual) || !aligned(out) || !aligned(keep) || !aligned(workspace))
        return bad("pe_gated_ffn: pointers must be 16-byte aligned");
    if (!pitch_ok(x_stride, hidden, 2) || (residual && !pitch_ok(residual_stride, hidden, 2)))
        return bad("pe_gated_ffn: row pitches must be multiples of 8 and at least hidden");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint32_t* err = nullptr;
    cudaError_t e = error_word(&err);
    if (!e) {
        Product p = make(x, x_stride, 0, w13, hidden, 0, rows, 2 * intermediate, hidden);
        p.e.cols = intermediate;
        p.e.act = act;
        // h is rounded to 16 bits, the type that the second product's MMA takes
        p.e.out = workspace;
        p.e.ld_out = intermediate;
        p.e.keep = keep;
        p.e.ld_keep = 2 * (int64_t)intermediate;
        e = launch_product(p, EPI_GATED, elem, CHAIN_NONE, err, st);
    }
    if (!e) {
        Product p = make(workspace, intermediate, 0, w2, intermediate, 0, rows, hidden, intermediate);
        p.e.out = out;
        p.e.ld_out = hidden;
        p.e.res = residual;
        p.e.ld_res = residual_stride;
        e = launch_product(p, EPI_LINEAR, elem, CHAIN_AFTER, err, st);
    }
    return done(e);
}

extern "C" size_t pe_gated_ffn_backward_workspace(int32_t rows, int32_t intermediate) {
    if (rows <= 0 || intermediate <= 0) return 0;
    return up256(4 * (size_t)rows * intermediate) + up256(2 * (size_t)rows * intermediate);
}

extern "C" pe_status pe_gated_ffn_backward(const void* dy, int64_t dy_stride, const void* x, int64_t x_stride,
                                           const void* w13, const void* w2, const void* keep, int32_t act, void* dx,
                                           void* dw13, void* dw2, void* workspace, size_t workspace_bytes, int32_t rows,
                                           int32_t hidden, int32_t intermediate, int32_t elem, void* stream) {
    if (!is_elem(elem)) return bad("pe_gated_ffn_backward: elem must be PE_ELEM_BF16 or PE_ELEM_F16");
    if (!is_act(act)) return bad("pe_gated_ffn_backward: unknown activation");
    if (rows < 0 || hidden < 8 || hidden % 8 || intermediate < 8 || intermediate % 8)
        return bad("pe_gated_ffn_backward: hidden and intermediate must be positive multiples of 8");
    if (hidden > kMaxFeatures || intermediate > kMaxFeatures)
        return bad("pe_gated_ffn_backward: more than 2^24 features", PE_ERR_RANGE);
    if (rows > PE_MAX_ROWS) return bad("pe_gated_ffn_backward: more than PE_MAX_ROWS rows", PE_ERR_RANGE);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const size_t wbytes = 2 * (size_t)hidden * intermediate;
    if (rows == 0) {
        cudaError_t e = dw13 ? cudaMemsetAsync(dw13, 0, 2 * wbytes, st) : cudaSuccess;
        if (!e && dw2) e = cudaMemsetAsync(dw2, 0, wbytes, st);
        return done(e);
    }
    if (!dy || !w2 || !keep || (dx && !w13) || (dw13 && !x)) return bad("pe_gated_ffn_backward: NULL pointer");
    if (workspace_bytes < pe_gated_ffn_backward_workspace(rows, intermediate) || !workspace)
        return bad("pe_gated_ffn_backward: workspace too small");
    if (!aligned(dy) || !aligned(x) || !aligned(w13) || !aligned(w2) || !aligned(keep) || !aligned(dx) || !aligned(dw13) ||
        !aligned(dw2) || !aligned(workspace))
        return bad("pe_gated_ffn_backward: pointers must be 16-byte aligned");
    if (!pitch_ok(dy_stride, hidden, 2) || (dw13 && !pitch_ok(x_stride, hidden, 2)))
        return bad("pe_gated_ffn_backward: row pitches must be multiples of 8 and at least hidden");
    uint32_t* err = nullptr;
    cudaError_t e = error_word(&err);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    void* dgu = ws;
    void* h = ws + up256(4 * (size_t)rows * intermediate);
    const int64_t I2 = 2 * (int64_t)intermediate;
    // dg, du and h are rounded to 16 bits, the type that the next products' MMAs
    // take, and so were the kept gate and up, half the memory of fp32: together
    // the gradients are off by twice their own rounding (bf16: 3.5e-3 instead
    // of 1.7e-3 in the 2-norm), independent per element.
    if (!e) {
        Product p = make(dy, dy_stride, 0, w2, intermediate, 1, rows, intermediate, hidden);
        p.e.act = act;
        p.e.gu = keep;
        p.e.ld_keep = I2;
        p.e.out = dgu;
        p.e.ld_out = I2;
        p.e.h = dw2 ? h : nullptr;
        e = launch_product(p, EPI_GATED_BWD, elem, CHAIN_NONE, err, st);
    }
    Product p[3];
    int n = 0;
    if (dx) {
        p[n] = make(dgu, I2, 0, w13, hidden, 1, rows, hidden, (int)I2);
        p[n].e.out = dx;
        p[n++].e.ld_out = hidden;
    }
    if (dw13) {
        p[n] = make(dgu, I2, 1, x, x_stride, 1, (int)I2, hidden, rows);
        p[n].e.out = dw13;
        p[n++].e.ld_out = hidden;
    }
    if (dw2) {
        p[n] = make(dy, dy_stride, 1, h, intermediate, 1, hidden, intermediate, rows);
        p[n].e.out = dw2;
        p[n++].e.ld_out = intermediate;
    }
    if (!e) e = launch_products(p, n, elem, err, st);
    return done(e);
}
