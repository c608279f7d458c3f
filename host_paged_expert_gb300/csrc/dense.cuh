// Device and host declarations shared by the dense operators (RMS norm,
// linear, gated feed-forward): element types, activations and the epilogue
// that every matrix-product kernel applies to eight consecutive columns of a
// result row.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <limits.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "pe.h"

namespace pe {
namespace dense {

constexpr int kGroup = 128;  // features sharing one scale of an 8-bit row; rows and columns of a weight block

// Rows are counted in int.  A loop over rows steps past the last one by its
// launch's stride, at most 4864 rows, and sizes are rounded up to a tile or a
// chunk, at most 4096 rows: PE_MAX_ROWS leaves 65535 below INT_MAX.
static_assert(INT_MAX - PE_MAX_ROWS == 65535, "room for a stride past the last row");

// What a matrix product does with its accumulators before they are stored.
enum EpiKind {
    EPI_LINEAR = 0,     // act(v + bias) + residual; optionally v + bias is kept
    EPI_GATED = 1,      // act(gate) * up of two accumulators; optionally both are kept
    EPI_GATED_BWD = 2,  // from dh and the kept gate and up: their gradients and h
};

struct Epi {
    int act;             // pe_act
    int rows, cols;      // valid rows and columns of the result (EPI_GATED*: columns of h)
    int out_f32;         // EPI_LINEAR: out holds fp32 instead of the element type
    int vec;             // every row pointer below is 16-byte aligned and cols % 8 = 0
    void* out;           // EPI_GATED_BWD: [rows, 2 cols], gradients of gate and up
    int64_t ld_out;
    const void* bias;    // [cols] or NULL
    const void* res;     // [rows, cols] or NULL
    int64_t ld_res;
    void* keep;          // EPI_LINEAR: [rows, cols] v + bias; EPI_GATED: [rows, 2 cols] gate, up; or NULL
    int64_t ld_keep;
    const void* gu;      // EPI_GATED_BWD: [rows, 2 cols] kept gate and up
    void* h;             // EPI_GATED_BWD: [rows, cols], or NULL
};

// One matrix product C[m, n] = sum_k A(m, k) B(n, k) with an epilogue.  A
// and B are row-major matrices in memory: [M, K] (mn = 0) or [K, M] (mn = 1),
// and likewise for B.  EPI_GATED: B is [2 cols, K], gate rows then up rows.
struct Product {
    const void* a;
    int64_t lda;
    int a_mn;
    const void* b;
    int64_t ldb;
    int b_mn;
    int M, N, K;
    const float* a_scale;  // E4M3 operands: [M, ceil(K/128)] and [ceil(N/128), ceil(K/128)]; else NULL
    const float* b_scale;
    Epi e;
};

// Every kernel of the dense operators is launched programmatically: it waits
// for the launch before it to be done (pdl_wait) before it touches global
// memory, and does not let the next one start before that (by pdl_trigger, or
// by its end), so whatever ran two launches back is done by the time a kernel
// runs.  CHAIN_AFTER: the
// launch before this product is one of the same call that does not write its
// B, so B may be read before the wait.
enum { CHAIN_NONE = 0, CHAIN_AFTER = 1 };

// elem: pe_elem of the 16-bit operands and of every 16-bit tensor of the epilogue.
cudaError_t launch_product(const Product& p, EpiKind kind, int elem, int chain, uint32_t* err, cudaStream_t st);

// Independent EPI_LINEAR products of 16-bit results, in any order or all at once.
cudaError_t launch_products(const Product* p, int count, int elem, uint32_t* err, cudaStream_t st);

// The kernels behind launch_product: tiles of 256 rows x tn (256 or 128)
// columns on CTA pairs, and tiles of 128 columns x nt rows whose K axis a
// cluster of `split` CTAs shares.
struct SplitShape {
    int nt, split;
};
// Polls after which a wait inside one of these kernels gives up.  A poll
// suspends the thread for up to a microsecond or so by itself, so this is
// seconds.
constexpr uint32_t kPolls = 1u << 22;
// Other limits, by the role that waits (the producer of copies, the issuer of
// MMAs, the warps that read the sums), for the self-test of the waits.  Its
// kernels are instances of their own: a limit that is no constant takes up to
// 0.4 us of a product (512 x 2048 to 2048 10.4 instead of 9.9 us).
struct WaitLimits {
    uint32_t copies, mma, sums;
};
// launch_pairs: up to kMostProducts EPI_LINEAR products of 16-bit operands in one launch, else one.
constexpr int kMostProducts = 3;
cudaError_t launch_pairs(const Product* p, int count, EpiKind kind, int elem, int tn, uint32_t* err, cudaStream_t st,
                         const WaitLimits* limits = nullptr);
cudaError_t launch_split(const Product& p, EpiKind kind, int elem, const SplitShape& s, int chain, uint32_t* err,
                         cudaStream_t st, const WaitLimits* limits = nullptr);
// Up to kGemvRows rows, forward products: weights streamed by warps, no tensor core.
constexpr int kGemvRows = 4;
cudaError_t launch_gemv(const Product& p, EpiKind kind, int elem, int chain, cudaStream_t st);
// K blocks of 64 that one accumulator takes where the result is fp32, of kb in all.
int split_blocks(const SplitShape& s, int kb);
// CTAs of this shape that the current device holds at once.
int split_resident(const SplitShape& s);

// Tensor map of an operand of `rows` rows and depth k: boxes of 128 bytes
// along K by box_rows rows, or (mn: stored [k, rows]) of 64 rows by 64 along
// K, swizzled over 128 bytes.
bool encode_operand(CUtensorMap* m, const void* base, int64_t ld, int rows, int k, bool mn, bool fp8, int box_rows);

struct NormArgs {
    const void *x, *res, *w;
    int64_t ld_x, ld_res;
    float eps;
    void *y, *sum, *codes;
    float *scales, *rstd;
    int rows, hidden;
};
cudaError_t launch_rms_norm(const NormArgs& a, int elem, cudaStream_t st);

struct NormBwdArgs {
    const void *dy, *dsum, *sum, *w;
    int64_t ld_dy, ld_dsum, ld_sum;
    const float* rstd;
    void *dx, *dw;
    float* partial;  // [norm_bwd_blocks(rows)][hidden]
    int rows, hidden;
};
int norm_bwd_blocks(int rows);
cudaError_t launch_rms_norm_bwd(const NormBwdArgs& a, int elem, cudaStream_t st);

// dz = dy * act'(z) (written with row pitch ld_dz when dz is not NULL) and
// its column sums (db, when not NULL).
struct ActBwdArgs {
    const void *dy, *z;
    int64_t ld_dy, ld_z;
    void* dz;
    int64_t ld_dz;
    void* db;
    float* partial;  // [act_bwd_chunks(rows, cols)][cols], when db is not NULL
    int act, rows, cols;
};
// Chunks are of kSumRows rows or more, so that one row of column sums for every
// kSumRows rows of dy is always enough room for `partial`, whatever the chunk.
constexpr int kSumRows = 32;
int act_bwd_chunks(int rows, int cols);
cudaError_t launch_act_bwd(const ActBwdArgs& a, int elem, cudaStream_t st);

#ifdef __CUDACC__

template <typename E>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
    static __device__ __forceinline__ float2 unpack(uint32_t v) {
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&p);
    }
    static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<__half> {
    static __device__ __forceinline__ float2 unpack(uint32_t v) {
        return __half22float2(*reinterpret_cast<const __half2*>(&v));
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __half2 p = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&p);
    }
    static __device__ __forceinline__ float get(__half v) { return __half2float(v); }
    static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
};

// 16 bytes that are read once.  Loads of these kernels are coherent ones: a
// block may be resident, waiting for the launch before it, while that launch
// still writes what the block will read, and the read-only path is only for
// memory that nothing writes as long as the kernel lives.
__device__ __forceinline__ int4 ld_stream(const void* p) {
    int4 v;
    asm volatile("ld.global.L1::no_allocate.v4.s32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Eight consecutive elements at p[0..7].  vec: p is 16-byte aligned and all
// eight exist; else the first n of them are touched one by one.
template <typename E>
__device__ __forceinline__ void load8(const E* p, bool vec, int n, float (&v)[8]) {
    if (vec) {
        const int4 r = *reinterpret_cast<const int4*>(p);
        const uint32_t w[4] = {(uint32_t)r.x, (uint32_t)r.y, (uint32_t)r.z, (uint32_t)r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = Elem<E>::unpack(w[i]);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? Elem<E>::get(p[i]) : 0.f;
    }
}
template <typename E>
__device__ __forceinline__ void store8(E* p, bool vec, int n, const float (&v)[8]) {
    if (vec) {
        int4 r;
        r.x = (int)Elem<E>::pack(v[0], v[1]);
        r.y = (int)Elem<E>::pack(v[2], v[3]);
        r.z = (int)Elem<E>::pack(v[4], v[5]);
        r.w = (int)Elem<E>::pack(v[6], v[7]);
        *reinterpret_cast<int4*>(p) = r;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = Elem<E>::put(v[i]);
    }
}
__device__ __forceinline__ void store8_f32(float* p, bool vec, int n, const float (&v)[8]) {
    if (vec) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = v[i];
    }
}

// e^x and 1/y by the special-function unit, about 2 ulp each, subnormals as
// zero (y is at least 1 here).  The rounding of x log2(e) adds 2^-23 |x| to
// e^x's relative error: 2e-6 at |x| = 17, 1e-5 at 80, far below the rounding
// to 16 bits; a result stored in fp32 shows it.
__device__ __forceinline__ float exp_f(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
    return r;
}
__device__ __forceinline__ float rcp_f(float y) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y));
    return r;
}
__device__ __forceinline__ float sigmoid_f(float x) { return rcp_f(1.f + exp_f(-x)); }

constexpr float kSqrt2OverPi = 0.7978845608028654f;
constexpr float kGeluCubic = 0.044715f;

// (1 + tanh u) / 2 = 1 / (1 + e^-2u) with u = sqrt(2/pi) (z + 0.044715 z^3): as
// the sigmoid it keeps its relative accuracy where it is small (1 + tanh(u)
// has none left from z = -5 on).
__device__ __forceinline__ float gelu_gate(float z) { return sigmoid_f(2.f * kSqrt2OverPi * (z + kGeluCubic * z * z * z)); }

// Phi(z), and e = e^(-z^2/2).  0.5 + 0.5 erf(z / sqrt 2) cancels at z < 0 (at z
// = -5 a tenth of it is lost), so the tail is computed as such: Phi(-y) = e t
// Q(t), t = 1 / (1 + 0.28 y), the form of Hastings' approximations (1955), with
// Q fitted here: degree 8, the relative error of t Q(t) against
// erfcx(y / sqrt 2) / 2 levelled over 0 < t <= 1 at 1.7e-7.  In fp32 within 5e-7,
// plus what e^x loses (1021 x 2880 to 1536 fp16 with GELU 14.0 us; by erff, with
// the cancellation, 14.5, by erfcf 16.2).
__device__ __forceinline__ float normal_cdf(float z, float& e) {
    const float t = rcp_f(fmaf(0.28f, fabsf(z), 1.f));
    e = exp_f(-0.5f * z * z);
    float q = 0.024719977751374245f;
    q = fmaf(q, t, -0.09359313547611237f);
    q = fmaf(q, t, 0.09242812544107437f);
    q = fmaf(q, t, -0.006449178792536259f);
    q = fmaf(q, t, 0.07277500629425049f);
    q = fmaf(q, t, 0.08363079279661179f);
    q = fmaf(q, t, 0.10308466106653214f);
    q = fmaf(q, t, 0.11169980466365814f);
    q = fmaf(q, t, 0.11170385777950287f);
    const float tail = t * q * e;
    return z > 0.f ? 1.f - tail : tail;
}

// act(z)
__device__ __forceinline__ float act_fwd(int act, float z) {
    switch (act) {
        case PE_ACT_SILU: return z * sigmoid_f(z);
        case PE_ACT_GELU: {
            float e;
            return z * normal_cdf(z, e);
        }
        case PE_ACT_GELU_TANH: return z * gelu_gate(z);
        case PE_ACT_RELU: return z > 0.f ? z : (z != z ? z : 0.f);
        default: return z;
    }
}
// act(z) and its slope d at z
__device__ __forceinline__ float act_both(int act, float z, float& d) {
    switch (act) {
        case PE_ACT_SILU: {
            const float s = sigmoid_f(z);
            d = s * (1.f + z * (1.f - s));
            return z * s;
        }
        case PE_ACT_GELU: {
            float e;
            const float c = normal_cdf(z, e);
            d = c + z * e * 0.3989422804014327f;
            return z * c;
        }
        case PE_ACT_GELU_TANH: {
            // s + z s' with s' = 2 u' s (1 - s), which is 0 long before z^2 overflows
            const float s = gelu_gate(z), p = s * (1.f - s);
            d = p > 0.f ? fmaf(z * p, 2.f * kSqrt2OverPi * (1.f + 3.f * kGeluCubic * z * z), s) : s;
            return z * s;
        }
        case PE_ACT_RELU: d = z > 0.f ? 1.f : 0.f; return z > 0.f ? z : (z != z ? z : 0.f);
        default: d = 1.f; return z;
    }
}

// f with the activation as a compile-time constant: callers put the choice
// outside of their loops, whose code then holds one activation only (a loop
// over all five costs more in fetched instructions than in arithmetic).
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
    switch (act) {
        case PE_ACT_SILU: f(std::integral_constant<int, PE_ACT_SILU>{}); break;
        case PE_ACT_GELU: f(std::integral_constant<int, PE_ACT_GELU>{}); break;
        case PE_ACT_GELU_TANH: f(std::integral_constant<int, PE_ACT_GELU_TANH>{}); break;
        case PE_ACT_RELU: f(std::integral_constant<int, PE_ACT_RELU>{}); break;
        default: f(std::integral_constant<int, PE_ACT_NONE>{}); break;
    }
}

template <typename E>
__device__ __forceinline__ void unpack8(int4 r, float (&v)[8]) {
    const uint32_t w[4] = {(uint32_t)r.x, (uint32_t)r.y, (uint32_t)r.z, (uint32_t)r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = Elem<E>::unpack(w[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

// The epilogue works on eight consecutive columns of a row: epi_cols loads
// what all rows of these columns share, epi_load what the epilogue reads of
// one row (ahead of its use, several rows at a time), epi_store finishes.
// Rows and columns past the result load zeros and store nothing.
struct EpiIn {
    int4 a, b;
};

// Whether the epilogue keeps nothing and stores 16-bit vectors.
template <int KIND>
__device__ __forceinline__ bool epi_light(const Epi& e) {
    return KIND == EPI_LINEAR && e.vec && !e.keep && !e.out_f32;
}

// bias of columns col..col+7
template <typename E, int KIND>
__device__ __forceinline__ void epi_cols(const Epi& e, int col, float (&bias)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) bias[i] = 0.f;
    if (KIND == EPI_LINEAR && e.bias && col < e.cols)
        load8(static_cast<const E*>(e.bias) + col, e.vec != 0, e.cols - col, bias);
}
template <typename E, int KIND>
__device__ __forceinline__ EpiIn epi_load(const Epi& e, int row, int col) {
    EpiIn in;
    in.a = in.b = make_int4(0, 0, 0, 0);
    if (row >= e.rows || col >= e.cols) return in;
    if (KIND == EPI_LINEAR) {
        if (e.res && e.vec) in.a = *reinterpret_cast<const int4*>(static_cast<const E*>(e.res) + row * e.ld_res + col);
    } else if (KIND == EPI_GATED_BWD) {
        const E* p = static_cast<const E*>(e.gu) + row * e.ld_keep + col;
        in.a = *reinterpret_cast<const int4*>(p);
        in.b = *reinterpret_cast<const int4*>(p + e.cols);
    }
    return in;
}
// v: the accumulators (of gate for EPI_GATED, where u holds up's; of dh for
// EPI_GATED_BWD).  The one rounding to 16 bits is at each store.
template <typename E, int KIND, int ACT>
__device__ __forceinline__ void epi_store(const Epi& e, int row, int col, const float (&bias)[8], const EpiIn& in,
                                          float (&v)[8], const float (&u)[8]) {
    const int n = e.cols - col;
    if (row >= e.rows || n <= 0) return;
    if (KIND == EPI_LINEAR) {
        const bool vec = e.vec != 0;  // cols % 8 = 0: all eight exist
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += bias[i];
        if (e.keep) store8(static_cast<E*>(e.keep) + row * e.ld_keep + col, vec, n, v);
        if (ACT != PE_ACT_NONE)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = act_fwd(ACT, v[i]);
        if (e.res) {
            float r[8];
            if (vec) unpack8<E>(in.a, r);
            else load8(static_cast<const E*>(e.res) + row * e.ld_res + col, false, n, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += r[i];
        }
        if (e.out_f32) store8_f32(static_cast<float*>(e.out) + row * e.ld_out + col, vec, n, v);
        else store8(static_cast<E*>(e.out) + row * e.ld_out + col, vec, n, v);
    } else if (KIND == EPI_GATED) {  // cols is a multiple of 8 from here on
        if (e.keep) {
            E* k = static_cast<E*>(e.keep) + row * e.ld_keep + col;
            store8(k, true, 8, v);
            store8(k + e.cols, true, 8, u);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = act_fwd(ACT, v[i]) * u[i];
        store8(static_cast<E*>(e.out) + row * e.ld_out + col, true, 8, v);
    } else {
        float a[8], d[8], w[8];
        unpack8<E>(in.a, a);
        unpack8<E>(in.b, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            a[i] = act_both(ACT, a[i], d[i]);
            d[i] *= v[i] * w[i];  // dg
            w[i] *= a[i];         // h
            a[i] *= v[i];         // du
        }
        E* o = static_cast<E*>(e.out) + row * e.ld_out + col;
        store8(o, true, 8, d);
        store8(o + e.cols, true, 8, a);
        if (e.h) store8(static_cast<E*>(e.h) + row * (int64_t)e.cols + col, true, 8, w);
    }
}

// epi_store where epi_light holds, with a third less code.
template <typename E, int ACT>
__device__ __forceinline__ void epi_store_light(const Epi& e, int row, int col, const float (&bias)[8], const EpiIn& in,
                                                float (&v)[8]) {
    if (e.bias)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += bias[i];
    if (ACT != PE_ACT_NONE)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = act_fwd(ACT, v[i]);
    if (e.res) {
        float r[8];
        unpack8<E>(in.a, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += r[i];
    }
    if (row < e.rows && col < e.cols) store8(static_cast<E*>(e.out) + row * e.ld_out + col, true, 8, v);
}

// The same for a single element (EPI_LINEAR, EPI_GATED).
template <typename E, int KIND>
__device__ __forceinline__ void epi_store1(const Epi& e, int row, int col, float v, float u) {
    if (row >= e.rows || col >= e.cols) return;
    E* keep = static_cast<E*>(e.keep) + row * e.ld_keep + col;
    if (KIND == EPI_LINEAR) {
        if (e.bias) v += Elem<E>::get(static_cast<const E*>(e.bias)[col]);
        if (e.keep) *keep = Elem<E>::put(v);
        v = act_fwd(e.act, v);
        if (e.res) v += Elem<E>::get(static_cast<const E*>(e.res)[row * e.ld_res + col]);
        if (e.out_f32) static_cast<float*>(e.out)[row * e.ld_out + col] = v;
        else static_cast<E*>(e.out)[row * e.ld_out + col] = Elem<E>::put(v);
    } else {
        if (e.keep) {
            keep[0] = Elem<E>::put(v);
            keep[e.cols] = Elem<E>::put(u);
        }
        static_cast<E*>(e.out)[row * e.ld_out + col] = Elem<E>::put(act_fwd(e.act, v) * u);
    }
}

#endif  // __CUDACC__

}  // namespace dense
}  // namespace pe
