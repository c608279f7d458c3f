// Shared by the tensor-core kernels whose epilogue turns a warp's 32 x 32
// blocks through a patch of shared memory, and whose tiles are walked by
// persistent CTA pairs.
#pragma once

#include "dense.cuh"

namespace pe {
namespace dense {

constexpr int kRaster = 8;  // tile rows walked together, so that the other operand's tiles are shared in L2

// A patch holds a warp's block as rows of 128 bytes, whose 16-byte chunks are
// XOR-swizzled by the row.
// Eight columns 8 c8 .. of row r.
__device__ __forceinline__ void patch_get(const uint8_t* patch, int r, int c8, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(patch + r * 128 + (((2 * c8) ^ (r & 7)) << 4));
    const float4 b = *reinterpret_cast<const float4*>(patch + r * 128 + (((2 * c8 + 1) ^ (r & 7)) << 4));
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// What the epilogue of a warp's 32 x 32 block reads, asked for before the
// block's accumulators are there.
template <typename E, int KIND>
struct Ahead {
    float factor, bias[8];
    EpiIn in[4];
    __device__ __forceinline__ void load(const Epi& e, int lane, int row0, int col0) {
        const int col = col0 + 8 * (lane & 3);
        factor = KIND == EPI_SCALED ? e.factor[0] : 1.f;
        epi_cols<E, after_factor(KIND)>(e, col, bias);
#pragma unroll
        for (int it = 0; it < 4; ++it) in[it] = epi_load<E, after_factor(KIND)>(e, row0 + it * 8 + (lane >> 2), col);
    }
    // eight columns of a row of the patch
    __device__ __forceinline__ void get(const uint8_t* patch, int r, int c8, float (&v)[8]) const {
        patch_get(patch, r, c8, v);
        if (KIND == EPI_SCALED)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= factor;
    }
};

template <typename E, int KIND>
__device__ __forceinline__ void patch_out(const Epi& e, const uint8_t* patch, int lane, int row0, int col0,
                                          const Ahead<E, KIND>& x) {
    const int c8 = lane & 3, row = row0 + (lane >> 2), col = col0 + 8 * c8;
    with_act(e.act, [&](auto act) {
        constexpr int ACT = decltype(act)::value;
        if (epi_light<after_factor(KIND)>(e)) {
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                float v[8];
                x.get(patch, it * 8 + (lane >> 2), c8, v);
                epi_store_light<E, ACT>(e, row + it * 8, col, x.bias, x.in[it], v);
            }
        } else {
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                float v[8], u[8];
                x.get(patch, it * 8 + (lane >> 2), c8, v);
                if (KIND == EPI_GATED) patch_get(patch + 4096, it * 8 + (lane >> 2), c8, u);
                epi_store<E, after_factor(KIND), ACT>(e, row + it * 8, col, x.bias, x.in[it], v, u);
            }
        }
    });
}

// x / d and x % d without a division: the product with 2^32 / d, rounded down,
// is the quotient or one less.
struct Divide {
    uint32_t d, inv;
    static Divide by(uint32_t d) { return {d, d > 1 ? (uint32_t)((uint64_t(1) << 32) / d) : 0xffffffffu}; }
    __device__ __forceinline__ uint32_t operator()(uint32_t x, uint32_t& rest) const {
        uint32_t q = __umulhi(x, inv);
        rest = x - q * d;
        if (rest >= d) rest -= d, ++q;
        return q;
    }
};

}  // namespace dense
}  // namespace pe
