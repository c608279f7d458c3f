// Linear products with 4-bit weights: act(x W^T + bias) + residual, W from
// codes and scales as in an expert row (int4: q - 8 times an fp16 scale per
// 128 inputs; MXFP4: E2M1 times an E8M0 scale per 32; NVFP4: E2M1 times an
// E4M3 scale per 16 and the tensor's fp32 scale).
//
// Up to kW4Stream rows: codes are streamed once, 16 bytes a lane, from global
// memory into registers and become the operand there.  The tensor core is
// reached by mma.sync, whose A operand is registers: tcgen05 would want the
// decoded weights in shared memory, four times the codes' bytes written and read
// again (which pays from 17 rows on).  A warp holds 16 or 32 weight rows (the
// MMA's M) and all tokens (its N, 8 at a time) of every 128-input chunk that
// falls to it; lane (g, t) = (lane / 4, lane % 4) holds codes 32 t .. 32 t + 31
// of rows g and g + 8, and since the order of the inputs within a product is
// free as long as both operands agree, no code changes lanes.  The warps of a
// block share its rows along K, the next chunk on its way, and add their sums in
// warp order through shared memory.
//
// Bound by a block's latency (a launch, its first loads, three or four chunks, the
// sum over warps), and where weights are many by the rate of integer and logic
// instructions, which decoding is made of.  Weights in L2: 1 x 2048 to 2048 int4 2.6
// us, 1 x 4096 to 4096 5.0, 8 x 4096 to 4096 nvfp4 6.0, 1 x 8192 to 8192 int4 12.6
// (floor 5); from HBM the last three 5.7, 6.6 and 14.1.
//
// Rounding: int4's q - 8 and E2M1 times its block scale are exact in 16 bits
// (a 2-bit times a 4-bit significand, or a power of two), int4's scales
// multiply fp32 sums of 128 inputs, and so does NVFP4's tensor scale in the
// end.  MXFP4's scales reach past fp16 at both ends: with it they multiply sums
// of their 32 inputs, and a lane takes eight codes of each group instead of a
// group's 32.  So weights are not rounded at all.  Above kW4Rows they are unpacked
// to 16 bits for the dense products' kernels, which rounds int4's once, and
// MXFP4's where fp16 ends.
#include "experts.cuh"
#include "fp8_device.cuh"
#include "pe_device.cuh"
#include "w4_device.cuh"

namespace pe {
namespace dense {
namespace {

constexpr int kChunk = 128;  // inputs of a warp's step

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

// A warp's share of a 128-input chunk on its way: codes and raw scales of its
// rows g and g + 8 of RT tiles, and the tokens' inputs.  Where scales multiply
// sums of 32 inputs (kScaleSums) word i of a lane's codes, and its inputs i, are of
// group i: codes 32 i + 8 t .. 32 i + 8 t + 7 of the chunk.
template <int RT, int NT>
struct Chunk {
    int4 w[RT][2], x[4][NT];
    uint32_t s[RT][2];
};

__device__ __forceinline__ int& word_of(int4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Asks for chunk c.  k: the first input of this lane's 32.  K is a multiple of 32.
template <typename E, int FMT, int RT, int NT>
__device__ __forceinline__ void fetch(Chunk<RT, NT>& q, const uint8_t* const (&codes)[RT][2], const uint8_t* const (&scales)[RT][2],
                                      const E* const (&x)[NT], int K, int c, int k) {
    const bool whole = (c + 1) * kChunk <= K;
    if constexpr (kScaleSums<E, FMT>) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool there = whole || c * kChunk + 32 * i < K;
#pragma unroll
            for (int m = 0; m < RT; ++m)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    word_of(q.w[m][r], i) = there ? *reinterpret_cast<const uint32_t*>(codes[m][r] + c * (kChunk / 2) + 16 * i) : 0;
#pragma unroll
            for (int j = 0; j < NT; ++j)
                q.x[i][j] = there ? *reinterpret_cast<const int4*>(x[j] + c * kChunk + 32 * i) : make_int4(0, 0, 0, 0);
        }
        // a lane has one group's scale
#pragma unroll
        for (int m = 0; m < RT; ++m)
#pragma unroll
            for (int r = 0; r < 2; ++r) q.s[m][r] = whole || k < K ? scales[m][r][c * (kChunk / 32)] : 0;
        return;
    }
    if (whole || k < K) {  // else the lane has no inputs
#pragma unroll
        for (int m = 0; m < RT; ++m)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                q.w[m][r] = ld_stream(codes[m][r] + c * (kChunk / 2));
                // MXFP4: the scale of this lane's 32 codes; NVFP4: the two of them, at an even
                // offset, as a row of a multiple of 32 inputs has an even number of scales
                if (FMT == W4_MXFP4) q.s[m][r] = scales[m][r][c * (kChunk / 32)];
                if (FMT == W4_NVFP4) q.s[m][r] = *reinterpret_cast<const uint16_t*>(scales[m][r] + c * (kChunk / 16));
            }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) q.x[i][j] = *reinterpret_cast<const int4*>(x[j] + c * kChunk + 8 * i);
    } else {
        q = {};
    }
    // int4: the chunk's scale, for sums over all lanes' inputs
    if (FMT == W4_INT4)
#pragma unroll
        for (int m = 0; m < RT; ++m)
#pragma unroll
            for (int r = 0; r < 2; ++r) q.s[m][r] = *reinterpret_cast<const uint16_t*>(scales[m][r] + 2 * c);
}

// Adds chunk q's products.
template <typename E, int FMT, int RT, int NT>
__device__ __forceinline__ void multiply(const Chunk<RT, NT>& q, float (&acc)[RT][NT][4]) {
    float s[RT][2][2];
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            if (FMT == W4_INT4) {
                s[m][r][0] = __half2float(__ushort_as_half((unsigned short)q.s[m][r]));
            } else if (FMT == W4_MXFP4) {
                s[m][r][0] = s[m][r][1] = e8m0(q.s[m][r]);
            } else {
                const float2 f = e4m3x2(q.s[m][r]);
                s[m][r][0] = f.x, s[m][r][1] = f.y;
            }
        }
    float sum[RT][NT][4];
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[m][j][i] = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // eight codes of each row
        uint32_t b[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const uint32_t v[4] = {(uint32_t)q.x[i][j].x, (uint32_t)q.x[i][j].y, (uint32_t)q.x[i][j].z, (uint32_t)q.x[i][j].w};
            // inputs (h, h + 4), as the codes are decoded
            b[j][0] = __byte_perm(v[0], v[2], 0x5410), b[j][1] = __byte_perm(v[0], v[2], 0x7632);
            b[j][2] = __byte_perm(v[1], v[3], 0x5410), b[j][3] = __byte_perm(v[1], v[3], 0x7632);
        }
#pragma unroll
        for (int m = 0; m < RT; ++m) {
            uint32_t p[2][4];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                int4 w = q.w[m][r];
                const uint32_t word = word_of(w, i);
                if (FMT == W4_INT4) int4x8<E>(word, p[r]);
                else if (kScaleSums<E, FMT>) e2m1x8<E>(word, p[r]);
                else e2m1x8<E>(word, Pair<E>::both(s[m][r][i / 2]), p[r]);
            }
            const uint32_t a0[4] = {p[0][0], p[1][0], p[0][1], p[1][1]}, a1[4] = {p[0][2], p[1][2], p[0][3], p[1][3]};
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float(&d)[4] = FMT == W4_INT4 || kScaleSums<E, FMT> ? sum[m][j] : acc[m][j];
                mma16816<E>(d, a0, b[j][0], b[j][1]);
                mma16816<E>(d, a1, b[j][2], b[j][3]);
            }
            if constexpr (kScaleSums<E, FMT>) {  // the group's scale comes from the lane that has it
                float f[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) f[r] = __shfl_sync(0xffffffffu, s[m][r][0], i, 4);
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int h = 0; h < 4; ++h) acc[m][j][h] = fmaf(f[h / 2], sum[m][j][h], acc[m][j][h]), sum[m][j][h] = 0.f;
            }
        }
    }
    if (FMT == W4_INT4)
#pragma unroll
        for (int m = 0; m < RT; ++m)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][j][i] = fmaf(s[m][i / 2][0], sum[m][j][i], acc[m][j][i]);
}

// NT: eights of tokens; RT: tiles of 16 rows of a block; W: its warps.
template <typename E, int FMT, int NT, int RT, int W>
__global__ void __launch_bounds__(W * 32) w4_kernel(const __grid_constant__ W4Args a) {
    extern __shared__ float part[];  // [W][NT * 8][16 RT]
    constexpr int ROWS = 16 * RT;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int n0 = blockIdx.x * ROWS;
    const int chunks = (a.K + kChunk - 1) / kChunk, groups = (a.K + w4_group(FMT) - 1) / w4_group(FMT);
    const uint8_t *codes[RT][2], *scales[RT][2];
    const E* x[NT];
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const size_t row = min(n0 + 16 * m + 8 * r + g, a.N - 1);
            codes[m][r] = static_cast<const uint8_t*>(a.codes) + row * (a.K / 2) + (kScaleSums<E, FMT> ? 4 : 16) * t4;
            scales[m][r] = static_cast<const uint8_t*>(a.scales) +
                           (FMT == W4_INT4 ? 2 * row * groups : row * groups + t4 * (FMT == W4_MXFP4 ? 1 : 2));
        }
    // columns of B without a token take another token's, and nobody takes their sums
#pragma unroll
    for (int j = 0; j < NT; ++j) x[j] = static_cast<const E*>(a.x) + min(8 * j + g, a.M - 1) * a.ld_x + (kScaleSums<E, FMT> ? 8 : 32) * t4;
    float acc[RT][NT][4] = {};
    pdl_wait();
    pdl_trigger();
    Chunk<RT, NT> q[2];
    auto ask = [&](Chunk<RT, NT>& to, int c) {
        if (c < chunks) fetch<E, FMT, RT, NT>(to, codes, scales, x, a.K, c, c * kChunk + 32 * t4);
    };
    ask(q[0], warp);
    for (int c = warp; c < chunks; c += 2 * W) {  // one chunk ahead, two places in turn
        ask(q[1], c + W);
        multiply<E, FMT, RT, NT>(q[0], acc);
        ask(q[0], c + 2 * W);
        if (c + W < chunks) multiply<E, FMT, RT, NT>(q[1], acc);
    }
    float* mine = part + warp * (NT * 8 * ROWS);
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) mine[(8 * j + 2 * t4 + (i & 1)) * ROWS + 16 * m + g + 8 * (i / 2)] = acc[m][j][i];
    __syncthreads();
    const float ts = FMT == W4_NVFP4 ? a.tensor_scale[0] : 1.f;
    with_act(a.e.act, [&](auto act) {
        for (int u = threadIdx.x; u < 2 * RT * a.M; u += W * 32) {
            const int t = u / (2 * RT), at = 8 * (u % (2 * RT)), col = n0 + at;
            float v[8] = {}, bias[8];
            epi_cols<E, EPI_LINEAR>(a.e, col, bias);
            const EpiIn in = epi_load<E, EPI_LINEAR>(a.e, t, col);
#pragma unroll
            for (int w = 0; w < W; ++w)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] += part[w * (NT * 8 * ROWS) + t * ROWS + at + j];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= ts;
            epi_store<E, EPI_LINEAR, decltype(act)::value>(a.e, t, col, bias, in, v, v);
        }
    });
}

// NVFP4 without the tensor's scale, which multiplies the product's sums.  Eight
// codes a thread: 4096 x 4096 in 7 us, the rate of HBM though L2 holds it.
template <typename E, int FMT>
__global__ void __launch_bounds__(256) w4_unpack_kernel(const __grid_constant__ W4Args a, E* out) {
    pdl_wait();
    pdl_trigger();
    const int groups = (a.K + w4_group(FMT) - 1) / w4_group(FMT), words = a.K / 8;
    const int64_t total = (int64_t)a.N * words;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t n = i / words;
        const int k = (int)(i - n * words) * 8;
        const uint32_t w = static_cast<const uint32_t*>(a.codes)[i];
        const size_t at = (size_t)n * groups + k / w4_group(FMT);
        float s;
        if (FMT == W4_INT4) s = __half2float(static_cast<const __half*>(a.scales)[at]);
        else if (FMT == W4_MXFP4) s = 0.5f * e8m0(static_cast<const uint8_t*>(a.scales)[at]);
        else s = 0.5f * e4m3x2(static_cast<const uint8_t*>(a.scales)[at]).x;
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

template <typename E, int FMT, int NT, int RT>
cudaError_t launch(const W4Args& a, cudaStream_t st) {
    constexpr int W = 8, bytes = W * NT * 8 * 16 * RT * 4;
    return launch_pdl(w4_kernel<E, FMT, NT, RT, W>, dim3((a.N + 16 * RT - 1) / (16 * RT)), dim3(W * 32), bytes, st, a);
}
// 32 rows of a block share the tokens' inputs, 16 make twice as many blocks:
// the former where there are enough of them and a warp has four chunks or more
// (1 x 4096 to 4096 int4 5.0 us, with 16 6.3; 1 x 4096 to 2048 4.8 and 3.7; 1 x
// 2880 to 5120 5.6 and 5.3).
template <typename E, int FMT>
cudaError_t by_rows(const W4Args& a, cudaStream_t st) {
    const bool two = a.N >= 4096 && a.K >= 4096;
    if (a.M <= 8) return two ? launch<E, FMT, 1, 2>(a, st) : launch<E, FMT, 1, 1>(a, st);
    return two ? launch<E, FMT, 2, 2>(a, st) : launch<E, FMT, 2, 1>(a, st);
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
