// RMS norm with the residual's addition and an 8-bit output, its backward
// pass, and the activation's backward pass with its column sums.  All of them
// are bound by HBM: each element is read and written once, in 16-byte
// vectors, and held in registers in between.
#include "dense.cuh"

namespace pe {
namespace dense {
namespace {

__device__ __forceinline__ float warp_total(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over the block, the same on every thread (and in the same order on
// every run).  red: 32 floats of shared memory, free again on return.
__device__ __forceinline__ float block_total(float v, float* red) {
    const int warps = blockDim.x >> 5;
    v = warp_total(v);
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.f;
    for (int i = 0; i < warps; ++i) t += red[i];
    __syncthreads();
    return t;
}

// The larger of two magnitudes; NaN wins, so that a NaN reaches the scale.
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// One block per row, NV vectors of 8 elements per thread.  The norm is taken
// of the fp32 sum, before it is rounded for the residual stream.
template <typename E, int NV>
__global__ void __launch_bounds__(1024) rms_norm_kernel(const NormArgs a) {
    __shared__ float red[32];
    const int row = blockIdx.x, vecs = a.hidden >> 3;
    const E* x = static_cast<const E*>(a.x) + row * a.ld_x;
    const E* r = a.res ? static_cast<const E*>(a.res) + row * a.ld_res : nullptr;
    float v[NV][8], ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = i * blockDim.x + threadIdx.x;
        if (c < vecs) {
            load8(x + 8 * c, true, 8, v[i]);
            if (r) {
                float t[8];
                load8(r + 8 * c, true, 8, t);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] += t[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
    }
    ss = block_total(ss, red);
    const float rstd = rsqrtf(ss / (float)a.hidden + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
    const size_t base = (size_t)row * a.hidden;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = i * blockDim.x + threadIdx.x;
        const bool in = c < vecs;
        if (in && a.sum) store8(static_cast<E*>(a.sum) + base + 8 * c, true, 8, v[i]);
        float w[8], top = 0.f;
        if (in) load8(static_cast<const E*>(a.w) + 8 * c, true, 8, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[i][j] = in ? v[i][j] * rstd * w[j] : 0.f;
            top = max_nan(top, fabsf(v[i][j]));
        }
        if (in && a.y) store8(static_cast<E*>(a.y) + base + 8 * c, true, 8, v[i]);
        if (a.codes) {  // sixteen threads hold the 128 features of one scale
#pragma unroll
            for (int o = 8; o; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
            // an all-zero group keeps scale 1; the floor keeps 1 / scale finite
            float s = top / 448.f;
            if (top == 0.f) s = 1.f;
            else if (s < 1.17549435e-38f) s = 1.17549435e-38f;
            if (in) {
                const float inv = 1.f / s;
                uint32_t q[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[i][4 * h] * inv, v[i][4 * h + 1] * inv),
                                                                 __NV_SATFINITE, __NV_E4M3);
                    const uint32_t hi = __nv_cvt_float2_to_fp8x2(
                        make_float2(v[i][4 * h + 2] * inv, v[i][4 * h + 3] * inv), __NV_SATFINITE, __NV_E4M3);
                    q[h] = lo | (hi << 16);
                }
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.codes) + base + 8 * c) = make_uint2(q[0], q[1]);
                if ((threadIdx.x & 15) == 0)
                    a.scales[(size_t)row * ((a.hidden + kGroup - 1) / kGroup) + (8 * c) / kGroup] = s;
            }
        }
    }
}

// Block b takes rows b, b + gridDim, ...: dx of each, and the block's share
// of the weight's gradient in registers, written once to partial[b].
template <typename E, int NV>
__global__ void __launch_bounds__(1024) rms_norm_bwd_kernel(const NormBwdArgs a) {
    __shared__ float red[32];
    const int vecs = a.hidden >> 3;
    float dw[NV][8] = {};
    float w[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = i * blockDim.x + threadIdx.x;
        load8(static_cast<const E*>(a.w) + 8 * c, c < vecs, 0, w[i]);
    }
    for (int row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float rstd = a.rstd[row];
        float g[NV][8], xh[NV][8], dot = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * blockDim.x + threadIdx.x;
            const bool in = c < vecs;
            load8(static_cast<const E*>(a.sum) + row * a.ld_sum + 8 * c, in, 0, xh[i]);
            load8(static_cast<const E*>(a.dy) + row * a.ld_dy + 8 * c, in, 0, g[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                xh[i][j] *= rstd;
                dw[i][j] = fmaf(g[i][j], xh[i][j], dw[i][j]);
                g[i][j] *= w[i][j];
                dot = fmaf(g[i][j], xh[i][j], dot);
            }
        }
        dot = block_total(dot, red) / (float)a.hidden;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * blockDim.x + threadIdx.x;
            if (c >= vecs) continue;
            float o[8] = {};
            if (a.dsum) load8(static_cast<const E*>(a.dsum) + row * a.ld_dsum + 8 * c, true, 8, o);
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = fmaf(rstd, g[i][j] - xh[i][j] * dot, o[j]);
            store8(static_cast<E*>(a.dx) + (size_t)row * a.hidden + 8 * c, true, 8, o);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = i * blockDim.x + threadIdx.x;
        if (c < vecs) store8_f32(a.partial + (size_t)blockIdx.x * a.hidden + 8 * c, true, 8, dw[i]);
    }
}

// out[c] = sum over n rows of partial, in a fixed order: a block takes 32
// columns, its 32 warps every 32nd row each.
template <typename E>
__global__ void __launch_bounds__(1024) column_total_kernel(const float* partial, int n, int cols, E* out) {
    __shared__ float part[32][33];
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float t = 0.f;
    if (c < cols)
        for (int r = wp; r < n; r += 32) t += partial[(size_t)r * cols + c];
    part[wp][lane] = t;
    __syncthreads();
    t = warp_total(part[lane][wp]);  // warp wp adds up column wp of the block
    const int oc = blockIdx.x * 32 + wp;
    if (lane == 0 && oc < cols) out[oc] = Elem<E>::put(t);
}

constexpr int kActRows = 64;  // rows of one chunk of the activation's backward pass

// Block (x, y): rows x * 64 ..., columns y * 256 ...; warp w takes every 8th row.
template <typename E>
__global__ void __launch_bounds__(256) act_bwd_kernel(const ActBwdArgs a) {
    __shared__ float part[8][256];
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    const int c = blockIdx.y * 256 + lane * 8, n = a.cols - c;
    const int r0 = blockIdx.x * kActRows, r1 = min(a.rows, r0 + kActRows);
    const bool vec = (a.cols & 7) == 0;
    float t[8] = {};
    if (n > 0) {
        for (int r = r0 + wp; r < r1; r += 8) {
            float g[8];
            load8(static_cast<const E*>(a.dy) + r * a.ld_dy + c, vec, n, g);
            if (a.z) {
                float z[8];
                load8(static_cast<const E*>(a.z) + r * a.ld_z + c, vec, n, z);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float d;
                    act_both(a.act, z[j], d);
                    g[j] *= d;
                }
            }
            if (a.dz) store8(static_cast<E*>(a.dz) + r * a.ld_dz + c, vec, n, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) t[j] += g[j];
        }
    }
    if (!a.db) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) part[wp][lane * 8 + j] = t[j];
    __syncthreads();
    const int oc = blockIdx.y * 256 + threadIdx.x;
    if (oc < a.cols) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) s += part[w][threadIdx.x];
        a.partial[(size_t)blockIdx.x * a.cols + oc] = s;
    }
}

template <typename E>
cudaError_t column_total(const float* partial, int n, int cols, void* out, cudaStream_t st) {
    column_total_kernel<E><<<(cols + 31) / 32, 1024, 0, st>>>(partial, n, cols, static_cast<E*>(out));
    return cudaGetLastError();
}

// Threads of a row block with nv vectors of 8 per thread.
int row_threads(int hidden, int nv) { return (((hidden / 8 + nv - 1) / nv) + 31) / 32 * 32; }
int row_vectors(int hidden) {
    int nv = 1;
    while (row_threads(hidden, nv) > 1024) nv *= 2;
    return nv;
}

template <typename E>
cudaError_t norm(const NormArgs& a, cudaStream_t st) {
    const int nv = row_vectors(a.hidden), th = row_threads(a.hidden, nv);
    if (nv == 1) rms_norm_kernel<E, 1><<<a.rows, th, 0, st>>>(a);
    else if (nv == 2) rms_norm_kernel<E, 2><<<a.rows, th, 0, st>>>(a);
    else rms_norm_kernel<E, 4><<<a.rows, th, 0, st>>>(a);
    return cudaGetLastError();
}
template <typename E>
cudaError_t norm_bwd(const NormBwdArgs& a, cudaStream_t st) {
    const int nv = row_vectors(a.hidden), th = row_threads(a.hidden, nv), nb = norm_bwd_blocks(a.rows);
    if (nb) {
        if (nv == 1) rms_norm_bwd_kernel<E, 1><<<nb, th, 0, st>>>(a);
        else if (nv == 2) rms_norm_bwd_kernel<E, 2><<<nb, th, 0, st>>>(a);
        else rms_norm_bwd_kernel<E, 4><<<nb, th, 0, st>>>(a);
        if (cudaError_t e = cudaGetLastError()) return e;
    }
    return column_total<E>(a.partial, nb, a.hidden, a.dw, st);
}
template <typename E>
cudaError_t act_bwd(const ActBwdArgs& a, cudaStream_t st) {
    const int chunks = act_bwd_chunks(a.rows);
    if (chunks) {
        act_bwd_kernel<E><<<dim3(chunks, (a.cols + 255) / 256), 256, 0, st>>>(a);
        if (cudaError_t e = cudaGetLastError()) return e;
    }
    return a.db ? column_total<E>(a.partial, chunks, a.cols, a.db, st) : cudaSuccess;
}

}  // namespace

int norm_bwd_blocks(int rows) { return rows < 304 ? rows : 304; }
int act_bwd_chunks(int rows) { return (rows + kActRows - 1) / kActRows; }

cudaError_t launch_rms_norm(const NormArgs& a, int elem, cudaStream_t st) {
    return elem == PE_ELEM_BF16 ? norm<__nv_bfloat16>(a, st) : norm<__half>(a, st);
}
cudaError_t launch_rms_norm_bwd(const NormBwdArgs& a, int elem, cudaStream_t st) {
    return elem == PE_ELEM_BF16 ? norm_bwd<__nv_bfloat16>(a, st) : norm_bwd<__half>(a, st);
}
cudaError_t launch_act_bwd(const ActBwdArgs& a, int elem, cudaStream_t st) {
    return elem == PE_ELEM_BF16 ? act_bwd<__nv_bfloat16>(a, st) : act_bwd<__half>(a, st);
}

}  // namespace dense
}  // namespace pe
