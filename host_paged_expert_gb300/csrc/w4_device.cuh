// Decoding of 4-bit codes to pairs of 16-bit numbers, shared by the kernels of
// linear products with 4-bit weights.
//
// Integer and logic instructions, permutations and the multiply-adds of packed
// 16-bit numbers all run at half the rate of plain ones on this chip (measured:
// 2 a cycle and SM each), on two pipes.  So a pair's two codes stay at bits 0 and
// 16, and what can be a multiplication is one.
#pragma once

#include "experts.cuh"

namespace pe {
namespace dense {

template <typename E>
struct Pair;  // two E in a register
template <>
struct Pair<__nv_bfloat16> {
    using T = __nv_bfloat162;
    static __device__ __forceinline__ T both(float v) { return __float2bfloat162_rn(v); }
    static constexpr uint32_t kInt = 0x43004300u;  // 128, whose last mantissa bit is 1
    static constexpr float kIntBase = 128.f;
    static constexpr float kUnbias = 0x1p126f;  // E2M1's bias is 1, this type's 127
};
template <>
struct Pair<__half> {
    using T = __half2;
    static __device__ __forceinline__ T both(float v) { return __float2half2_rn(v); }
    static constexpr uint32_t kInt = 0x64006400u;  // 1024
    static constexpr float kIntBase = 1024.f;
    static constexpr float kUnbias = 0x1p14f;
};
template <typename E>
__device__ __forceinline__ typename Pair<E>::T as_pair(uint32_t v) {
    return *reinterpret_cast<const typename Pair<E>::T*>(&v);
}
template <typename T>
__device__ __forceinline__ uint32_t bits_of(T v) {
    return *reinterpret_cast<const uint32_t*>(&v);
}

// int4: (q - 8) of codes (i, i + 4) of the eight in w, p[i], exactly: q becomes
// the last bits of kIntBase + q, of which kIntBase + 8 is taken.
template <typename E>
__device__ __forceinline__ void int4x8(uint32_t w, uint32_t (&p)[4]) {
    using P = Pair<E>;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        p[i] = bits_of(__hsub2(as_pair<E>(((w >> (4 * i)) & 0x000F000Fu) | P::kInt), P::both(P::kIntBase + 8.f)));
}

// E2M1 of codes (i, i + 4) of the eight in w, p[i], exactly.  The code's sign
// and its exponent and mantissa become the element's, which is then right but
// for the difference of the biases (a subnormal code is a subnormal element).
template <typename E>
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t (&p)[4]) {
    using P = Pair<E>;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t n = (w >> (4 * i)) & 0x000F000Fu;
        uint32_t r;
        if (std::is_same<E, __half>::value) r = ((n * 0x200u) & 0x0E000E00u) | ((n * 0x1000u) & 0x80008000u);
        else r = (n * 0x1040u) & 0x81C081C0u;  // n << 12 | n << 6
        p[i] = bits_of(__hmul2(as_pair<E>(r), P::both(P::kUnbias)));
    }
}
// The same times a scale: a 2-bit times a 4-bit significand, or a power of two,
// exact wherever E holds the product.  E4M3's products fp16 and bf16 hold (2^-10
// to 2688), E8M0's bf16 as far as fp32 does.
template <typename E>
__device__ __forceinline__ void e2m1x8(uint32_t w, typename Pair<E>::T scale, uint32_t (&p)[4]) {
    e2m1x8<E>(w, p);
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = bits_of(__hmul2(as_pair<E>(p[i]), scale));
}

// fp16 holds E8M0's products from 2^-23 to 2^13 only, so with it these scales
// multiply the fp32 sums of their 32 inputs (8 x 4096 to 4096 7.2 us, 32 x 4096 to
// 32000 56; with the scales in fp16 and that range 6.1 and 49).
template <typename E, int FMT>
constexpr bool kScaleSums = FMT == W4_MXFP4 && std::is_same<E, __half>::value;

// 2^(e - 127); NaN for e = 255.
__device__ __forceinline__ float e8m0(uint32_t e) {
    return __uint_as_float(e == 255u ? 0x7FC00000u : e ? e << 23 : 0x00400000u);
}
}  // namespace dense
}  // namespace pe
