// Linear products with 4-bit weights: act(x W^T + bias) + residual, W from
// codes and scales as in an expert row (int4: q - 8 times an fp16 scale per
// 128 inputs; MXFP4: E2M1 times an E8M0 scale per 32; NVFP4: E2M1 times an
// E4M3 scale per 16 and the tensor's fp32 scale).
//
// Few rows (up to kW4Rows): codes are streamed once, 16 bytes a lane, from
// global memory into registers and become the operand there.  The tensor core
// is reached by mma.sync, whose A operand is registers: tcgen05 would want the
// decoded weights in shared or tensor memory, four times the codes' bytes
// written and read again, for products that HBM bounds.  A warp holds 16
// weight rows (the MMA's M) and all tokens (its N, 8 at a time) of every
// 128-input chunk that falls to it; lane (g, t) = (lane / 4, lane % 4) holds
// codes 32 t .. 32 t + 31 of rows g and g + 8, and since the order of the
// inputs within a product is free as long as both operands agree, no code
// changes lanes.  Warps of a block share 16 rows along K and add their sums in
// warp order through shared memory.
//
// Rounding: int4's q - 8 and E2M1 times its block scale are exact in 16 bits
// (a 2-bit times a 4-bit significand, or a power of two), int4's scales
// multiply fp32 sums of 128 inputs, and so does NVFP4's tensor scale in the
// end: weights are not rounded at all.
#include "experts.cuh"
#include "fp8_device.cuh"
#include "pe_device.cuh"

namespace pe {
namespace dense {
namespace {

constexpr int kWarps = 8, kChunk = 128;

// c += A B, A 16 x 16 and B 16 x 8 of E, fp32 sums.
template <typename E>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
#define PE_MMA(T)                                                                                                            \
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32." T "." T ".f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "     \
                 "{%0, %1, %2, %3};"                                                                                         \
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])                                                            \
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1))
    if (std::is_same<E, __half>::value) PE_MMA("f16");
    else PE_MMA("bf16");
#undef PE_MMA
}

template <typename E>
struct Pair;  // two E in a register
template <>
struct Pair<__nv_bfloat16> {
    using T = __nv_bfloat162;
    static __device__ __forceinline__ T both(float v) { return __float2bfloat162_rn(v); }
    // int4: 128, whose last mantissa bit is 1
    static constexpr uint32_t kInt = 0x43004300u;
    static constexpr float kIntBase = 128.f;
    // E2M1: 128 and the byte to add to it for a value
    static constexpr uint32_t kHigh = 0x43, kLow0 = 0x03020100u, kLow1 = 0x0C080604u;
    static constexpr float kBase = 128.f;
    static constexpr float kMostScale = 0x1p119f;
};
template <>
struct Pair<__half> {
    using T = __half2;
    static __device__ __forceinline__ T both(float v) { return __float2half2_rn(v); }
    static constexpr uint32_t kInt = 0x64006400u;  // 1024
    static constexpr float kIntBase = 1024.f;
    static constexpr uint32_t kHigh = 0x54, kLow0 = 0x30201000u, kLow1 = 0xC0806040u;  // 64, its last mantissa bit 1/16
    static constexpr float kBase = 64.f;
    static constexpr float kMostScale = 0x1p15f;
};
template <typename E>
__device__ __forceinline__ typename Pair<E>::T as_pair(uint32_t v) {
    return *reinterpret_cast<const typename Pair<E>::T*>(&v);
}
template <typename T>
__device__ __forceinline__ uint32_t bits_of(T v) {
    return *reinterpret_cast<const uint32_t*>(&v);
}

// int4: (q - 8) of codes (i, i + 4) of the eight in w, p[i], exactly.
template <typename E>
__device__ __forceinline__ void int4x8(uint32_t w, uint32_t (&p)[4]) {
    using P = Pair<E>;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        p[i] = bits_of(__hsub2(as_pair<E>(((w >> (4 * i)) & 0x000F000Fu) | P::kInt), P::both(P::kIntBase + 8.f)));
}

// E2M1: value times scale of codes (2i, 2i + 1) of the eight in w, p[i]; half:
// half the scale, twice.  2|v| is one of {0, 1, 2, 3, 4, 6, 8, 12}: its byte is
// looked up for four codes at once and makes kBase + 2|v|.  With bf16 that times
// half the scale less kBase times it is one exact multiply-add; with fp16, whose
// range is short, the subtraction comes first.
template <typename E>
__device__ __forceinline__ void e2m1x8(uint32_t w, typename Pair<E>::T half, typename Pair<E>::T less, uint32_t (&p)[4]) {
    using P = Pair<E>;
    const uint32_t mag = w & 0x77777777u;
    const uint32_t lo = __byte_perm(P::kLow0, P::kLow1, mag), hi = __byte_perm(P::kLow0, P::kLow1, mag >> 16);
    const uint32_t q[4] = {__byte_perm(lo, P::kHigh, 0x4140u), __byte_perm(lo, P::kHigh, 0x4342u),
                           __byte_perm(hi, P::kHigh, 0x4140u), __byte_perm(hi, P::kHigh, 0x4342u)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t b = w >> (8 * i);  // sign bits at 3 and 7
        const uint32_t m = std::is_same<E, __half>::value ? bits_of(__hmul2(__hsub2(as_pair<E>(q[i]), P::both(P::kBase)), half))
                                                          : bits_of(__hfma2(as_pair<E>(q[i]), half, less));
        p[i] = m ^ (((b << 12) & 0x8000u) | ((b << 24) & 0x80000000u));
    }
}

// Half a block scale, no larger than what leaves the arithmetic above finite
// (2^16 with fp16, whose values end below, 2^120 with bf16, for the scale).
template <typename E>
__device__ __forceinline__ float in_range(float s) {
    return s > Pair<E>::kMostScale ? Pair<E>::kMostScale : s;
}

// Half an E8M0 scale, 2^(e - 128); NaN for e = 255.
__device__ __forceinline__ float half_e8m0(uint32_t e) {
    if (e == 255u) return __uint_as_float(0x7FC00000u);
    return e >= 2u ? __uint_as_float((e - 1u) << 23) : __uint_as_float(0x00200000u << e);
}

// NT: eights of tokens.
template <typename E, int FMT, int NT>
__global__ void __launch_bounds__(kWarps * 32) w4_kernel(const __grid_constant__ W4Args a) {
    extern __shared__ float part[];  // [kWarps][NT * 8][16]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int n0 = blockIdx.x * 16;
    const int chunks = (a.K + kChunk - 1) / kChunk, groups = (a.K + w4_group(FMT) - 1) / w4_group(FMT);
    const int r0 = min(n0 + g, a.N - 1), r1 = min(n0 + g + 8, a.N - 1);
    const uint8_t* c0 = static_cast<const uint8_t*>(a.codes) + (size_t)r0 * (a.K / 2);
    const uint8_t* c1 = static_cast<const uint8_t*>(a.codes) + (size_t)r1 * (a.K / 2);
    float acc[NT][4] = {};
    pdl_wait();
    pdl_trigger();
    for (int c = warp; c < chunks; c += kWarps) {
        const int k = c * kChunk + 32 * t4;
        const bool there = k < a.K;  // K is a multiple of 32
        int4 w[2] = {};
        if (there) {
            w[0] = ld_stream(c0 + k / 2);
            w[1] = ld_stream(c1 + k / 2);
        }
        // scales: FMT int4 of the chunk's sums, else of this lane's two halves of 16 codes
        float s[2][2] = {};
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const size_t row = (size_t)(r ? r1 : r0) * groups;
            if (FMT == W4_INT4) {
                s[r][0] = __half2float(static_cast<const __half*>(a.scales)[row + c]);
            } else if (there && FMT == W4_MXFP4) {
                s[r][0] = s[r][1] = in_range<E>(half_e8m0(static_cast<const uint8_t*>(a.scales)[row + k / 32]));
            } else if (there) {
                // two E4M3 scales, at an even offset: groups is even where K is a multiple of 32
                const float2 f = e4m3x2(*reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(a.scales) + row + k / 16));
                s[r][0] = 0.5f * f.x, s[r][1] = 0.5f * f.y;
            }
        }
        float sum[NT][4] = {};
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // eight codes of each row
            uint32_t p[2][4];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint32_t word = q == 0 ? w[r].x : q == 1 ? w[r].y : q == 2 ? w[r].z : w[r].w;
                if (FMT == W4_INT4) int4x8<E>(word, p[r]);
                else e2m1x8<E>(word, Pair<E>::both(s[r][q / 2]), Pair<E>::both(-Pair<E>::kBase * s[r][q / 2]), p[r]);
            }
            const uint32_t a0[4] = {p[0][0], p[1][0], p[0][1], p[1][1]}, a1[4] = {p[0][2], p[1][2], p[0][3], p[1][3]};
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int t = 8 * j + g;
                int4 x = make_int4(0, 0, 0, 0);
                if (there && t < a.M) x = *reinterpret_cast<const int4*>(static_cast<const E*>(a.x) + t * a.ld_x + k + 8 * q);
                uint32_t b[4] = {(uint32_t)x.x, (uint32_t)x.y, (uint32_t)x.z, (uint32_t)x.w};
                if (FMT == W4_INT4) {  // inputs (i, i + 4)
                    const uint32_t o[4] = {__byte_perm(b[0], b[2], 0x5410), __byte_perm(b[0], b[2], 0x7632),
                                           __byte_perm(b[1], b[3], 0x5410), __byte_perm(b[1], b[3], 0x7632)};
                    mma16816<E>(sum[j], a0, o[0], o[1]);
                    mma16816<E>(sum[j], a1, o[2], o[3]);
                } else {
                    mma16816<E>(acc[j], a0, b[0], b[1]);
                    mma16816<E>(acc[j], a1, b[2], b[3]);
                }
            }
        }
        if (FMT == W4_INT4)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[j][i] = fmaf(s[i / 2][0], sum[j][i], acc[j][i]);
    }
    // part[warp][token][row]
    float* mine = part + warp * (NT * 8 * 16);
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) mine[(8 * j + 2 * t4 + (i & 1)) * 16 + g + 8 * (i / 2)] = acc[j][i];
    __syncthreads();
    const float ts = FMT == W4_NVFP4 ? a.tensor_scale[0] : 1.f;
    with_act(a.e.act, [&](auto act) {
        for (int u = threadIdx.x; u < 2 * a.M; u += kWarps * 32) {
            const int t = u / 2, col = n0 + 8 * (u & 1);
            float v[8] = {}, bias[8];
            epi_cols<E, EPI_LINEAR>(a.e, col, bias);
            const EpiIn in = epi_load<E, EPI_LINEAR>(a.e, t, col);
            for (int w = 0; w < kWarps; ++w)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] += part[w * (NT * 8 * 16) + t * 16 + 8 * (u & 1) + j];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= ts;
            epi_store<E, EPI_LINEAR, decltype(act)::value>(a.e, t, col, bias, in, v, v);
        }
    });
}

// Eight codes a thread.
template <typename E, int FMT>
__global__ void __launch_bounds__(256) w4_unpack_kernel(const __grid_constant__ W4Args a, E* out) {
    pdl_wait();
    pdl_trigger();
    const int groups = (a.K + w4_group(FMT) - 1) / w4_group(FMT), words = a.K / 8;
    const int64_t total = (int64_t)a.N * words;
    const float ts = FMT == W4_NVFP4 ? a.tensor_scale[0] : 1.f;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t n = i / words;
        const int k = (int)(i - n * words) * 8;
        const uint32_t w = static_cast<const uint32_t*>(a.codes)[i];
        const size_t at = (size_t)n * groups + k / w4_group(FMT);
        float s;
        if (FMT == W4_INT4) s = __half2float(static_cast<const __half*>(a.scales)[at]);
        else if (FMT == W4_MXFP4) s = in_range<E>(half_e8m0(static_cast<const uint8_t*>(a.scales)[at]));
        else s = 0.5f * ts * e4m3x2(static_cast<const uint8_t*>(a.scales)[at]).x;
        float v[8];
        if (FMT == W4_INT4) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = (float)((int)((w >> (4 * j)) & 15u) - 8) * s;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t q = w >> (4 * j);
                const float m = (float)((0xC8643210u >> (4 * (q & 7u))) & 15u);
                v[j] = (q & 8u) ? -m * s : m * s;
            }
        }
        store8(out + n * (int64_t)a.K + k, true, 8, v);
    }
}

template <typename E, int FMT, int NT>
cudaError_t launch(const W4Args& a, cudaStream_t st) {
    constexpr int bytes = kWarps * NT * 8 * 16 * 4;
    return launch_pdl(w4_kernel<E, FMT, NT>, dim3((a.N + 15) / 16), dim3(kWarps * 32), bytes, st, a);
}
template <typename E, int FMT>
cudaError_t by_rows(const W4Args& a, cudaStream_t st) {
    if (a.M <= 8) return launch<E, FMT, 1>(a, st);
    if (a.M <= 16) return launch<E, FMT, 2>(a, st);
    if (a.M <= 32) return launch<E, FMT, 4>(a, st);
    return launch<E, FMT, 8>(a, st);
}
template <typename E>
cudaError_t by_format(const W4Args& a, cudaStream_t st) {
    return a.fmt == W4_INT4 ? by_rows<E, W4_INT4>(a, st) : a.fmt == W4_MXFP4 ? by_rows<E, W4_MXFP4>(a, st) : by_rows<E, W4_NVFP4>(a, st);
}
template <typename E>
cudaError_t unpack(const W4Args& a, E* w, cudaStream_t st) {
    const int64_t blocks = ((int64_t)a.N * (a.K / 8) + 255) / 256;
    const dim3 grid((unsigned)(blocks < 152 * 32 ? blocks : 152 * 32));
    if (a.fmt == W4_INT4) return launch_pdl(w4_unpack_kernel<E, W4_INT4>, grid, dim3(256), 0, st, a, w);
    if (a.fmt == W4_MXFP4) return launch_pdl(w4_unpack_kernel<E, W4_MXFP4>, grid, dim3(256), 0, st, a, w);
    return launch_pdl(w4_unpack_kernel<E, W4_NVFP4>, grid, dim3(256), 0, st, a, w);
}

}  // namespace

cudaError_t launch_w4(const W4Args& a, int elem, cudaStream_t st) {
    return elem == PE_ELEM_BF16 ? by_format<__nv_bfloat16>(a, st) : by_format<__half>(a, st);
}
cudaError_t launch_w4_unpack(const W4Args& a, void* w, int elem, cudaStream_t st) {
    return elem == PE_ELEM_BF16 ? unpack(a, static_cast<__nv_bfloat16*>(w), st) : unpack(a, static_cast<__half*>(w), st);
}

}  // namespace dense
}  // namespace pe
