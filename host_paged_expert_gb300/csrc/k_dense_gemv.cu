// Matrix products of one to four rows: C[t, n] = sum_k x(t, k) W(n, k), then
// the epilogue.
//
// With so few rows a weight is used a handful of times, and the tensor core's
// setup (barriers, TMEM, a cluster's meeting) costs more than the arithmetic.
// So: a warp holds two weight rows (EPI_GATED: gate and up of one feature),
// its lanes stream them in 16-byte pieces, four of each in flight, multiply
// with the tokens' pieces (which all warps share through L1) and add up in
// fp32; up to eight warps of a block share a row where rows are few.  The sum
// is a fixed tree: lanes, then warps in order.
//
// Bound by HBM, or by a launch's latency where the weights sit in L2: 1 x 8192
// to 8192 20.1 us (6680 GB/s), 1 x 4096 to 2048 2.9 us (3.2 with bias and
// residual), gated feed-forward 1 x 2048 x 768 4.5 us.  From two tokens on the multiply-adds count, and the
// tensor cores take over where weights are many.
//
// The second product of a feed-forward block asks for its first pieces of the
// weights while the first product still runs.
#include "dense.cuh"
#include "fp8_device.cuh"
#include "pe_device.cuh"

namespace pe {
namespace dense {
namespace {

constexpr int kWarps = 8, kAhead = 4;
// Weight bytes up to which the next launch may move in early: it hides the
// next one's start (gated feed-forward 1 x 2048 x 768, 9 MB: 4.6 instead of 4.7
// us; 1 x 4096 x 2048, 17 MB: no gain), but its waiting blocks slow a long
// stream (1 x 8192 x 8192, 134 MB: 22.0 us instead of 19.7).
constexpr size_t kLetGo = 32u << 20;

struct Plan {
    int share;    // warps per pair of rows
    int early;    // ask for weights before the previous kernel is done
};

template <typename E>
__device__ __forceinline__ float dot8(int4 w, int4 x, float acc);
template <>
__device__ __forceinline__ float dot8<__nv_bfloat16>(int4 w, int4 x, float acc) {
    return dot8_bf16(w, x, acc);
}
template <>
__device__ __forceinline__ float dot8<__half>(int4 w, int4 x, float acc) {
    float a[8], b[8];
    unpack8<__half>(w, a);
    unpack8<__half>(x, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc = fmaf(a[i], b[i], acc);
    return acc;
}

// sixteen E4M3 codes
__device__ __forceinline__ void unpack16(int4 r, float (&v)[16]) {
    const uint32_t w[4] = {(uint32_t)r.x, (uint32_t)r.y, (uint32_t)r.z, (uint32_t)r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 lo = e4m3x2(w[i]), hi = e4m3x2(w[i] >> 16);
        v[4 * i] = lo.x, v[4 * i + 1] = lo.y, v[4 * i + 2] = hi.x, v[4 * i + 3] = hi.y;
    }
}

template <typename E, int KIND, bool FP8, int NT>
__global__ void __launch_bounds__(kWarps * 32) gemv_kernel(const __grid_constant__ Product p, const Plan q) {
    constexpr int PIECE = FP8 ? 16 : 8;  // elements of 16 bytes
    constexpr int ES = FP8 ? 1 : 2;
    __shared__ float part[kWarps][NT * 2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int groups = kWarps / q.share, group = warp / q.share, mine = warp % q.share;
    const int col = (blockIdx.x * groups + group) * (KIND == EPI_GATED ? 1 : 2);
    const int n0 = min(col, p.N - 1), n1 = min(KIND == EPI_GATED ? p.e.cols + col : col + 1, p.N - 1);
    const uint8_t* w0 = static_cast<const uint8_t*>(p.b) + (size_t)n0 * p.ldb * ES;
    const uint8_t* w1 = static_cast<const uint8_t*>(p.b) + (size_t)n1 * p.ldb * ES;
    const uint8_t* x = static_cast<const uint8_t*>(p.a);
    const int pieces = p.K / PIECE, step = q.share * 32;
    float acc[NT][2] = {};
    int4 a[kAhead], b[kAhead];
    auto fetch = [&](int c) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = c + u * step;
            a[u] = b[u] = make_int4(0, 0, 0, 0);
            if (i < pieces) {
                a[u] = ld_stream(w0 + 16 * (size_t)i);
                b[u] = ld_stream(w1 + 16 * (size_t)i);
            }
        }
    };
    int c = mine * 32 + lane;
    if (!q.early) pdl_wait();
    fetch(c);
    if (q.early) pdl_wait();
    if ((size_t)p.N * p.K * ES <= kLetGo) pdl_trigger();
    while (c - lane < pieces) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = c + u * step;
            if (i < pieces) {
                if (FP8) {
                    const int groups_k = (p.K + kGroup - 1) / kGroup, g = i * PIECE / kGroup;
                    float wa[16], wb[16];
                    unpack16(a[u], wa);
                    unpack16(b[u], wb);
                    const float sa = p.b_scale[(size_t)(n0 / kGroup) * groups_k + g];
                    const float sb = p.b_scale[(size_t)(n1 / kGroup) * groups_k + g];
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        if (t < p.M) {
                            float xv[16], da = 0.f, db = 0.f;
                            unpack16(*reinterpret_cast<const int4*>(x + t * p.lda + 16 * (size_t)i), xv);
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                da = fmaf(wa[j], xv[j], da);
                                db = fmaf(wb[j], xv[j], db);
                            }
                            const float sx = p.a_scale[(size_t)t * groups_k + g];
                            acc[t][0] = fmaf(da, sa * sx, acc[t][0]);
                            acc[t][1] = fmaf(db, sb * sx, acc[t][1]);
                        }
                } else {
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        if (t < p.M) {
                            const int4 xv = *reinterpret_cast<const int4*>(x + t * p.lda * ES + 16 * (size_t)i);
                            acc[t][0] = dot8<E>(a[u], xv, acc[t][0]);
                            acc[t][1] = dot8<E>(b[u], xv, acc[t][1]);
                        }
                }
            }
        }
        c += kAhead * step;
        if (c - lane < pieces) fetch(c);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float s = warp_sum(acc[t][r]);
            if (lane == 0) part[warp][2 * t + r] = s;
        }
    __syncthreads();
    // lane 2t + r of the first warp of a group: token t, row r
    const int t = lane >> 1, r = lane & 1;
    if (mine == 0 && t < NT) {
        float s = 0.f, u = 0.f;
        for (int i = 0; i < q.share; ++i) {
            s += part[warp + i][2 * t + r];
            if (KIND == EPI_GATED) u += part[warp + i][2 * t + 1];
        }
        if (KIND == EPI_GATED) {
            if (r == 0) epi_store1<E, KIND>(p.e, t, col, s, u);
        } else {
            epi_store1<E, KIND>(p.e, t, col + r, s, 0.f);
        }
    }
}

template <typename E, int KIND, bool FP8>
cudaError_t launch(const Product& p, int chain, cudaStream_t st) {
    constexpr int PER = KIND == EPI_GATED ? 1 : 2;  // result columns of a group
    Plan q = {};
    q.early = chain == CHAIN_AFTER;
    const int pieces = p.K / (FP8 ? 16 : 8);
    auto blocks = [&](int share) { return (int)(((long long)p.e.cols + PER * (kWarps / share) - 1) / (PER * (kWarps / share))); };
    // warps share rows until there are two blocks per SM, as long as each lane
    // still has two pieces of a row
    q.share = 1;
    while (q.share < kWarps && blocks(q.share) < 304 && pieces >= 128 * q.share) q.share *= 2;
    const dim3 grid(blocks(q.share)), block(kWarps * 32);
    if (p.M == 1) return launch_pdl(gemv_kernel<E, KIND, FP8, 1>, grid, block, 0, st, p, q);
    if (p.M == 2) return launch_pdl(gemv_kernel<E, KIND, FP8, 2>, grid, block, 0, st, p, q);
    return launch_pdl(gemv_kernel<E, KIND, FP8, kGemvRows>, grid, block, 0, st, p, q);
}

template <typename E>
cudaError_t launch_kind(const Product& p, EpiKind kind, int chain, cudaStream_t st) {
    if (p.a_scale) return launch<E, EPI_LINEAR, true>(p, chain, st);
    return kind == EPI_LINEAR ? launch<E, EPI_LINEAR, false>(p, chain, st) : launch<E, EPI_GATED, false>(p, chain, st);
}

}  // namespace

cudaError_t launch_gemv(const Product& p, EpiKind kind, int elem, int chain, cudaStream_t st) {
    if (p.M > kGemvRows || p.a_mn || p.b_mn || kind > EPI_GATED) return cudaErrorInvalidValue;
    return elem == PE_ELEM_BF16 ? launch_kind<__nv_bfloat16>(p, kind, chain, st) : launch_kind<__half>(p, kind, chain, st);
}

}  // namespace dense
}  // namespace pe
