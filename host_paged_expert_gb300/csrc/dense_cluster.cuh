// Shared by the kernels that split K over a cluster: the cluster's sum of a
// tile over distributed shared memory.
#pragma once

#include "dense.cuh"
#include "dense_tc.cuh"

namespace pe {
namespace dense {

constexpr int kRows = 128;  // weight rows of a tile

// Adds up the cluster's partials of units of eight columns in a row, in rank
// order, and applies the epilogue.  Each thread asks for all the parts of
// several units before it adds the first: the round trip to another SM's
// shared memory is paid once.
// split: CTAs of the cluster, at most SPLIT.
template <typename E, int KIND, int SPLIT, int THREADS>
__device__ __forceinline__ void reduce(const Epi& e, const uint8_t* ring, int nt, int split, int rank, int t0, int f0) {
    constexpr int NF = KIND == EPI_GATED ? kRows / 2 : kRows, U = NF / 8, G = KIND == EPI_GATED ? 2 : 1;
    constexpr int BATCH = 4 / (SPLIT * G) > 1 ? 4 / (SPLIT * G) : 1;
    // each rank takes whole rows, as many as the others
    const int rows = min(nt, e.rows - t0), mine = (rows + split - 1) / split, r0 = rank * mine;
    const int total = min(mine, rows - r0) * U;
    uint32_t from[SPLIT];
#pragma unroll
    for (int r = 0; r < SPLIT; ++r) from[r] = tc::map_rank(tc::smem_u32(ring), r < split ? r : 0);
    // the stride between a thread's units is a multiple of U: its columns stay the same
    const int u0 = (int)threadIdx.x, col = f0 + (u0 % U) * 8;
    float bias[8];
    epi_cols<E, after_factor(KIND)>(e, col, bias);
    const float factor = KIND == EPI_SCALED ? e.factor[0] : 1.f;
    for (int ub = u0; ub < total; ub += THREADS * BATCH) {
        float v[BATCH][G][8];
        EpiIn in[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int u = ub + i * THREADS, t = r0 + u / U;
            const uint32_t at = (uint32_t)(t * kRows + (u0 % U) * 8) * 4;
            in[i] = epi_load<E, after_factor(KIND)>(e, u < total ? t0 + t : e.rows, col);
            if (u >= total) continue;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                float4 a[SPLIT][2];
#pragma unroll
                for (int r = 0; r < SPLIT; ++r)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (SPLIT <= 2 || r < split) a[r][h] = tc::ld_cluster_f4(from[r] + at + g * NF * 4 + h * 16);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][g][j] = 0.f;
#pragma unroll
                for (int r = 0; r < SPLIT; ++r)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (SPLIT > 2 && r >= split) continue;
                        float* d = v[i][g] + 4 * h;
                        d[0] += a[r][h].x, d[1] += a[r][h].y, d[2] += a[r][h].z, d[3] += a[r][h].w;
                    }
                if (KIND == EPI_SCALED)
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[i][g][j] *= factor;
            }
        }
        with_act(e.act, [&](auto act) {
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int u = ub + i * THREADS;
                if (u < total) {
                    if (epi_light<after_factor(KIND)>(e))
                        epi_store_light<E, decltype(act)::value>(e, t0 + r0 + u / U, col, bias, in[i], v[i][0]);
                    else
                        epi_store<E, after_factor(KIND), decltype(act)::value>(e, t0 + r0 + u / U, col, bias, in[i], v[i][0], v[i][G - 1]);
                }
            }
        });
    }
}

}  // namespace dense
}  // namespace pe
