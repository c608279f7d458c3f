// Matrix products of the dense operators: C[m, n] = sum_k A(m, k) B(n, k),
// then the epilogue.  A first, plain form: 64 x 64 tiles of C per block,
// 16-deep slices of both operands widened to fp32 in shared memory, 4 x 4
// accumulators per thread.
#include "dense.cuh"

namespace pe {
namespace dense {
namespace {

constexpr int TM = 64, TN = 64, TK = 16;

template <typename E>
__device__ __forceinline__ float fetch(const void* p, int64_t ld, int mn, int r, int k, const float* scale, int rows_per,
                                       int groups) {
    const size_t at = mn ? (size_t)k * ld + r : (size_t)r * ld + k;
    if (scale) {
        const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<const __nv_fp8_storage_t*>(p)[at], __NV_E4M3);
        return __half2float(__half(h)) * scale[(size_t)(r / rows_per) * groups + k / kGroup];
    }
    return Elem<E>::get(static_cast<const E*>(p)[at]);
}

template <typename E, int KIND>
__global__ void __launch_bounds__(256) product_kernel(const Product p) {
    __shared__ float sa[TK][TM + 1], sb[TK][TN + 1], su[TK][TN + 1];
    __shared__ float c[2][TM][TN + 4];
    const int m0 = blockIdx.x * TM, n0 = blockIdx.y * TN;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int groups = (p.K + kGroup - 1) / kGroup;
    const int N = KIND == EPI_GATED ? p.e.cols : p.N;
    float acc[4][4] = {}, acu[4][4] = {};
    for (int k0 = 0; k0 < p.K; k0 += TK) {
        for (int i = threadIdx.x; i < TM * TK; i += 256) {
            const int r = p.a_mn ? i % TM : i / TK, k = p.a_mn ? i / TM : i % TK;
            sa[k][r] = m0 + r < p.M && k0 + k < p.K ? fetch<E>(p.a, p.lda, p.a_mn, m0 + r, k0 + k, p.a_scale, 1, groups) : 0.f;
        }
        for (int i = threadIdx.x; i < TN * TK; i += 256) {
            const int r = p.b_mn ? i % TN : i / TK, k = p.b_mn ? i / TN : i % TK;
            const bool in = n0 + r < N && k0 + k < p.K;
            sb[k][r] = in ? fetch<E>(p.b, p.ldb, p.b_mn, n0 + r, k0 + k, p.b_scale, kGroup, groups) : 0.f;
            if (KIND == EPI_GATED) su[k][r] = in ? fetch<E>(p.b, p.ldb, 0, N + n0 + r, k0 + k, nullptr, 1, 1) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < TK; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[i][j] = fmaf(sa[k][ty * 4 + i], sb[k][tx * 4 + j], acc[i][j]);
                    if (KIND == EPI_GATED) acu[i][j] = fmaf(sa[k][ty * 4 + i], su[k][tx * 4 + j], acu[i][j]);
                }
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            c[0][ty * 4 + i][tx * 4 + j] = acc[i][j];
            c[1][ty * 4 + i][tx * 4 + j] = acu[i][j];
        }
    __syncthreads();
    for (int i = threadIdx.x; i < TM * TN / 8; i += 256) {
        const int r = i / (TN / 8), q = (i % (TN / 8)) * 8;
        float v[8], u[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = c[0][r][q + j];
            u[j] = c[1][r][q + j];
        }
        epilogue8<E, KIND>(p.e, m0 + r, n0 + q, v, u);
    }
}

template <typename E>
cudaError_t launch(const Product& p, EpiKind kind, cudaStream_t st) {
    const int N = kind == EPI_GATED ? p.e.cols : p.N;
    const dim3 grid((p.M + TM - 1) / TM, (N + TN - 1) / TN);
    if (kind == EPI_LINEAR) product_kernel<E, EPI_LINEAR><<<grid, 256, 0, st>>>(p);
    else if (kind == EPI_GATED) product_kernel<E, EPI_GATED><<<grid, 256, 0, st>>>(p);
    else product_kernel<E, EPI_GATED_BWD><<<grid, 256, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_product(const Product& p, EpiKind kind, int elem, uint32_t*, cudaStream_t st) {
    return elem == PE_ELEM_BF16 ? launch<__nv_bfloat16>(p, kind, st) : launch<__half>(p, kind, st);
}

}  // namespace dense
}  // namespace pe
