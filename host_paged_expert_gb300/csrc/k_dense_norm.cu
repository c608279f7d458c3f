// RMS norm with the residual's addition and an 8-bit output, its backward
// pass, and the activation's backward pass with its column sums.  All of them
// are bound by HBM: each element is read and written once, in 16-byte
// vectors, and held in registers in between.  Measured (a plain copy
// moves 6786 GB/s): 16384 x 4096 with residual and 8-bit output
// 97 us (6270 GB/s), 16384 x 4096 backward 92 us (5800 GB/s); a single row
// 1.6 us, a launch's latency.
#include "dense.cuh"
#include "pe_device.cuh"

namespace pe {
namespace dense {
namespace {

// Threads of a row block: one vector of 8 each, more where a row has over 512
// vectors.  (16384 x 4096 with an 8-bit output: 97 us with up to 512 threads,
// 102 us with 256, 135 us with 128; 8192 x 8192 without: 85, 114, 114 us.)
// Rows of over 1024 vectors take up to 1024 threads: at 64 registers each a
// block fills the SM (4096 x 9000: 75 us, 99 us with 288 threads).
constexpr int kMostThreads = 512, kWideThreads = 1024;

__device__ __forceinline__ float warp_total(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over the block, the same on every thread (and in the same order on
// every run).  red: 32 floats of shared memory that no thread still reads; two
// of them, taken in turn, make one barrier per sum enough.
__device__ __forceinline__ float block_total(float v, float* red) {
    const int warps = blockDim.x >> 5;
    v = warp_total(v);
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.f;
    for (int i = 0; i < warps; ++i) t += red[i];
    return t;
}

// The larger of two magnitudes; NaN wins, so that a NaN reaches the scale.
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// A block takes rows b, b + gridDim, ...: NV vectors of 8 elements per thread,
// held in registers between the sum of squares and the output; the next row's
// loads are in flight meanwhile.  The norm is taken of the fp32 sum, before it
// is rounded for the residual stream.  RAW: rows of more than 8192 columns are
// held as they were read, and each vector of the next row is asked for as soon
// as this row's is used up (2048 x 32768: 99 us, 5400 GB/s; 107 us with the
// fp32 values in registers; 4096 x 16384 106 and 123 us).
template <typename E, int NV, bool RAW>
__global__ void __launch_bounds__(RAW ? kWideThreads : kMostThreads, RAW ? 1 : 2) rms_norm_kernel(const NormArgs a) {
    __shared__ float red[2][32];
    pdl_wait();
    const int vecs = a.hidden >> 3;
    constexpr int NW = RAW ? 1 : NV;  // weights stay in registers where there is room
    int4 xn[NV], rn[NV], w[NW];
    auto weight = [&](int i) {
        const int c = i * blockDim.x + threadIdx.x;
        return c < vecs ? *reinterpret_cast<const int4*>(static_cast<const E*>(a.w) + 8 * c) : make_int4(0, 0, 0, 0);
    };
    auto fetch1 = [&](int row, int i) {
        const int c = i * blockDim.x + threadIdx.x;
        if (c < vecs) {
            xn[i] = ld_stream(static_cast<const E*>(a.x) + row * a.ld_x + 8 * c);
            if (a.res) rn[i] = ld_stream(static_cast<const E*>(a.res) + row * a.ld_res + 8 * c);
        }
    };
    auto fetch = [&](int row) {
#pragma unroll
        for (int i = 0; i < NV; ++i) fetch1(row, i);
    };
    // the sum that is normed, of vector i
    auto value = [&](int i, float (&o)[8]) {
        if (i * blockDim.x + threadIdx.x < vecs) {
            unpack8<E>(xn[i], o);
            if (a.res) {
                float t[8];
                unpack8<E>(rn[i], t);
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] += t[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = 0.f;
        }
    };
    int row = blockIdx.x;
    fetch(row);
#pragma unroll
    for (int i = 0; i < NW; ++i)
        if (!RAW) w[i] = weight(i);
    for (int turn = 0; row < a.rows; row += gridDim.x, turn ^= 1) {
        float keep[RAW ? 1 : NV][8], ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float(&v)[8] = keep[RAW ? 0 : i];
            value(i, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
        }
        const bool more = gridDim.x < a.rows - row;
        if (!RAW && more) fetch(row + gridDim.x);
        ss = block_total(ss, red[turn]);
        const float rstd = rsqrtf(ss / (float)a.hidden + a.eps);
        if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
        const size_t base = (size_t)row * a.hidden;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * blockDim.x + threadIdx.x;
            const bool in = c < vecs;
            float(&v)[8] = keep[RAW ? 0 : i];
            if (RAW) {
                value(i, v);
                if (more) fetch1(row + gridDim.x, i);
            }
            if (in && a.sum) store8(static_cast<E*>(a.sum) + base + 8 * c, true, 8, v);
            float wf[8], top = 0.f;
            unpack8<E>(RAW ? weight(i) : w[RAW ? 0 : i], wf);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = in ? v[j] * rstd * wf[j] : 0.f;
                top = max_nan(top, fabsf(v[j]));
            }
            if (in && a.y) store8(static_cast<E*>(a.y) + base + 8 * c, true, 8, v);
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
                        const uint32_t lo = __nv_cvt_float2_to_fp8x2(
                            make_float2(v[4 * h] * inv, v[4 * h + 1] * inv), __NV_SATFINITE, __NV_E4M3);
                        const uint32_t hi = __nv_cvt_float2_to_fp8x2(
                            make_float2(v[4 * h + 2] * inv, v[4 * h + 3] * inv), __NV_SATFINITE, __NV_E4M3);
                        q[h] = lo | (hi << 16);
                    }
                    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.codes) + base + 8 * c) = make_uint2(q[0], q[1]);
                    if ((threadIdx.x & 15) == 0)
                        a.scales[(size_t)row * ((a.hidden + kGroup - 1) / kGroup) + (8 * c) / kGroup] = s;
                }
            }
        }
    }
}

// Short rows share a block: its `groups` groups of threads take a row each.
// Every group keeps its share of the weight's gradient in registers, the
// groups' shares are added in order through shared memory and written once
// to partial[block].  The next row's loads are in flight while a row is
// reduced.
template <typename E, int NV>
__global__ void __launch_bounds__(kMostThreads, NV == 1 ? 2 : 1) rms_norm_bwd_kernel(const NormBwdArgs a, int groups) {
    __shared__ float red[2][32];
    __shared__ float share[NV == 1 ? 8 * kMostThreads / 2 : 1];
    pdl_wait();
    const int vecs = a.hidden >> 3, th = blockDim.x / groups, group = threadIdx.x / th, tid = threadIdx.x - group * th;
    const int w0 = group * (th >> 5), warps = th >> 5;  // the group's first warp, and how many
    float dw[NV][8] = {};
    int4 sn[NV], yn[NV], dn[NV];
    float rn = 0.f;
    auto fetch = [&](int row) {
        rn = a.rstd[row];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * th + tid;
            sn[i] = yn[i] = dn[i] = make_int4(0, 0, 0, 0);
            if (c < vecs) {
                sn[i] = ld_stream(static_cast<const E*>(a.sum) + row * a.ld_sum + 8 * c);
                yn[i] = ld_stream(static_cast<const E*>(a.dy) + row * a.ld_dy + 8 * c);
                if (a.dsum) dn[i] = ld_stream(static_cast<const E*>(a.dsum) + row * a.ld_dsum + 8 * c);
            }
        }
    };
    auto weight = [&](int i) {
        const int c = i * th + tid;
        return c < vecs ? *reinterpret_cast<const int4*>(static_cast<const E*>(a.w) + 8 * c) : make_int4(0, 0, 0, 0);
    };
    int4 w[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) w[i] = weight(i);
    const int step = gridDim.x * groups;
    int row = blockIdx.x * groups + group;
    if (row < a.rows) fetch(row);
    for (int turn = 0; row < a.rows; row += step, turn ^= 1) {
        const float rstd = rn;
        float g[NV][8], xh[NV][8], dot = 0.f;
        int4 d[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float wf[8];
            unpack8<E>(sn[i], xh[i]);
            unpack8<E>(yn[i], g[i]);
            unpack8<E>(w[i], wf);
            d[i] = dn[i];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                xh[i][j] *= rstd;
                dw[i][j] = fmaf(g[i][j], xh[i][j], dw[i][j]);
                g[i][j] *= wf[j];
                dot = fmaf(g[i][j], xh[i][j], dot);
            }
        }
        if (step < a.rows - row) fetch(row + step);
        dot = warp_total(dot);
        if (warps > 1) {
            if ((threadIdx.x & 31) == 0) red[turn][threadIdx.x >> 5] = dot;
            asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(th) : "memory");
            dot = 0.f;
            for (int i = 0; i < warps; ++i) dot += red[turn][w0 + i];
        }
        dot /= (float)a.hidden;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * th + tid;
            if (c >= vecs) continue;
            float o[8];
            unpack8<E>(d[i], o);  // zeros without dsum
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = fmaf(rstd, g[i][j] - xh[i][j] * dot, o[j]);
            store8(static_cast<E*>(a.dx) + (size_t)row * a.hidden + 8 * c, true, 8, o);
        }
    }
    if (NV == 1 && groups > 1) {
        for (int g = 0; g < groups; ++g) {
            if (group == g && tid < vecs) {
                float* at = share + 8 * tid;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (g) dw[0][j] += at[j];
                    at[j] = dw[0][j];
                }
            }
            __syncthreads();
        }
        if (group != groups - 1) return;  // the last group holds the sum
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = i * th + tid;
        if (c < vecs) store8_f32(a.partial + (size_t)blockIdx.x * a.hidden + 8 * c, true, 8, dw[i]);
    }
}

// The same for rows of more than 8192 columns, whose fp32 values no longer
// fit: the row is held as it was read, the block's share of the weight's
// gradient lies in shared memory (each thread its own columns, so that no
// barrier is needed), and each vector of the next row is asked for as soon as
// this row's is used up.  2048 x 32768: 129 us, 4160 GB/s (402 us with the
// fp32 values in 128 registers of 512 threads, which spilled far more).  At
// four vectors a thread its 64 registers still spill 160 bytes (bf16; 124 in
// fp16).
template <typename E, int NV>
__global__ void __launch_bounds__(kWideThreads, 1) rms_norm_bwd_wide_kernel(const NormBwdArgs a) {
    extern __shared__ float4 dw[];  // the first halves of all vectors, then the second ones
    __shared__ float red[2][32];
    pdl_wait();
    const int vecs = a.hidden >> 3;
    int4 sn[NV], yn[NV], dn[NV];
    auto fetch1 = [&](int row, int i) {
        const int c = i * blockDim.x + threadIdx.x;
        if (c < vecs) {
            sn[i] = ld_stream(static_cast<const E*>(a.sum) + row * a.ld_sum + 8 * c);
            yn[i] = ld_stream(static_cast<const E*>(a.dy) + row * a.ld_dy + 8 * c);
            if (a.dsum) dn[i] = ld_stream(static_cast<const E*>(a.dsum) + row * a.ld_dsum + 8 * c);
        }
    };
    int row = blockIdx.x;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = i * blockDim.x + threadIdx.x;
        sn[i] = yn[i] = dn[i] = make_int4(0, 0, 0, 0);
        fetch1(row, i);
        if (c < vecs) dw[c] = dw[vecs + c] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int turn = 0; row < a.rows; row += gridDim.x, turn ^= 1) {
        const float rstd = a.rstd[row];
        // dy * w and sum * rstd of vector i; dyx: the weight's gradient of this row
        auto parts = [&](int i, int c, float (&g)[8], float (&xh)[8], float (&dyx)[8]) {
            float wf[8];
            unpack8<E>(sn[i], xh);
            unpack8<E>(yn[i], g);
            unpack8<E>(*reinterpret_cast<const int4*>(static_cast<const E*>(a.w) + 8 * c), wf);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                xh[j] *= rstd;
                dyx[j] = g[j] * xh[j];
                g[j] *= wf[j];
            }
        };
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * blockDim.x + threadIdx.x;
            if (c >= vecs) continue;
            float g[8], xh[8], dyx[8];
            parts(i, c, g, xh, dyx);
            float4 lo = dw[c], hi = dw[vecs + c];
            lo.x += dyx[0], lo.y += dyx[1], lo.z += dyx[2], lo.w += dyx[3];
            hi.x += dyx[4], hi.y += dyx[5], hi.z += dyx[6], hi.w += dyx[7];
            dw[c] = lo, dw[vecs + c] = hi;
#pragma unroll
            for (int j = 0; j < 8; ++j) dot = fmaf(g[j], xh[j], dot);
        }
        dot = block_total(dot, red[turn]) / (float)a.hidden;
        const bool more = gridDim.x < a.rows - row;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = i * blockDim.x + threadIdx.x;
            if (c >= vecs) continue;
            float g[8], xh[8], dyx[8], o[8];
            parts(i, c, g, xh, dyx);
            unpack8<E>(dn[i], o);  // zeros without dsum
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = fmaf(rstd, g[j] - xh[j] * dot, o[j]);
            if (more) fetch1(row + gridDim.x, i);
            store8(static_cast<E*>(a.dx) + (size_t)row * a.hidden + 8 * c, true, 8, o);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = i * blockDim.x + threadIdx.x;
        if (c >= vecs) continue;
        const float4 lo = dw[c], hi = dw[vecs + c];
        const float t[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        store8_f32(a.partial + (size_t)blockIdx.x * a.hidden + 8 * c, true, 8, t);
    }
}

// out[c] = sum over n rows of partial, in a fixed order: a block takes 32
// columns, its 32 warps every 32nd row each.
template <typename E>
__global__ void __launch_bounds__(1024) column_total_kernel(const float* partial, int n, int cols, E* out) {
    __shared__ float part[32][33];
    pdl_wait();
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

// The activation's backward pass: a block takes 8 * vx columns (vx threads, a
// power of two of at most a warp, so that narrow matrices fill the warps too)
// and a chunk of rows, four rows of a thread at a time, held as they were read.
// A chunk is one such batch, so that every SM has several blocks; four where
// there are more than 16 blocks per SM, so that the chunks' column sums (fp32)
// stay a small part of the traffic.
constexpr int kActThreads = 256, kActBatch = 4;
static_assert(kActThreads / 32 * kActBatch >= kSumRows, "a chunk has at least kSumRows rows");
int act_vx(int cols) {
    int vx = 1;
    while (vx < 32 && 8 * vx < cols) vx *= 2;
    return vx;
}
int act_rows(int rows, int cols) {
    const int vx = act_vx(cols), batch = kActThreads / vx * kActBatch;
    const long long blocks = (long long)((rows + batch - 1) / batch) * ((cols + 8 * vx - 1) / (8 * vx));
    return blocks > 16 * 152 ? 4 * batch : batch;
}

// Eight elements as they lie in memory; zeros past the n-th.
template <typename E>
__device__ __forceinline__ int4 raw8(const E* p, bool vec, int n) {
    if (vec) return ld_stream(p);
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (2 * i < n ? q[2 * i] : 0u) | (2 * i + 1 < n ? (uint32_t)q[2 * i + 1] << 16 : 0u);
    return make_int4(w[0], w[1], w[2], w[3]);
}

// gelu_tanh adds this to a projection's backward pass: 4098 x 2592 15 us, 7826
// x 88 12 us (24 and 24 us with 256 columns a block and chunks of 128 rows).
template <typename E>
__global__ void __launch_bounds__(kActThreads) act_bwd_kernel(const ActBwdArgs a, int vx, int chunk) {
    __shared__ alignas(16) float part[kActThreads * 8];  // [rows at a time][8 vx columns]
    pdl_wait();
    const int x = threadIdx.x & (vx - 1), y = threadIdx.x / vx, step = kActThreads / vx;
    const int across = (a.cols + 8 * vx - 1) / (8 * vx), by = blockIdx.x / across, bx = blockIdx.x - by * across;
    const int c = (bx * vx + x) * 8, n = a.cols - c;
    const int r0 = by * chunk, r1 = min(a.rows - r0, chunk) + r0;
    const bool vec = (a.cols & 7) == 0;
    float t[8] = {};
    if (n > 0) {
        with_act(a.act, [&](auto act) {
            constexpr int ACT = decltype(act)::value;
            for (int rb = r0 + y; rb < r1; rb += kActBatch * step) {
                int4 gr[kActBatch], zr[kActBatch];
#pragma unroll
                for (int i = 0; i < kActBatch; ++i) {
                    const int r = rb + i * step;
                    if (r >= r1) break;
                    gr[i] = raw8(static_cast<const E*>(a.dy) + r * a.ld_dy + c, vec, n);
                    if (ACT != PE_ACT_NONE) zr[i] = raw8(static_cast<const E*>(a.z) + r * a.ld_z + c, vec, n);
                }
#pragma unroll
                for (int i = 0; i < kActBatch; ++i) {
                    const int r = rb + i * step;
                    if (r >= r1) break;
                    float g[8];
                    unpack8<E>(gr[i], g);
                    if (ACT != PE_ACT_NONE) {
                        float z[8];
                        unpack8<E>(zr[i], z);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            float d;
                            act_both(ACT, z[j], d);
                            g[j] *= d;
                        }
                    }
                    if (a.dz) store8(static_cast<E*>(a.dz) + r * a.ld_dz + c, vec, n, g);
#pragma unroll
                    for (int j = 0; j < 8; ++j) t[j] += g[j];
                }
            }
        });
    }
    if (!a.db) return;
    const int width = 8 * vx;
    store8_f32(part + y * width + 8 * x, true, 8, t);
    __syncthreads();
    const int oc = bx * width + threadIdx.x;
    if (threadIdx.x < width && oc < a.cols) {
        float s = 0.f;
        for (int i = 0; i < step; ++i) s += part[i * width + threadIdx.x];
        a.partial[(size_t)by * a.cols + oc] = s;
    }
}

template <typename E>
cudaError_t column_total(const float* partial, int n, int cols, void* out, cudaStream_t st) {
    return launch_pdl(column_total_kernel<E>, dim3((cols + 31) / 32), dim3(1024), 0, st, partial, n, cols,
                      static_cast<E*>(out));
}

int row_threads(int hidden, int nv) { return (((hidden / 8 + nv - 1) / nv) + 31) / 32 * 32; }
bool wide_row(int hidden) { return hidden > 2 * 8 * kMostThreads; }
int row_vectors(int hidden) { return row_threads(hidden, 1) <= kMostThreads ? 1 : row_threads(hidden, 2) <= kWideThreads ? 2 : 4; }
constexpr int kSms = 152;
// Threads per SM that the forward pass's grid counts on: with the next row
// always on its way these keep HBM busy, and more only make the last rows
// uneven (16384 x 1032: 22.8 us, 26.2 with 1536, 23.6 with 2048).
constexpr int kResident = 1024;

template <typename E>
cudaError_t norm(const NormArgs& a, cudaStream_t st) {
    const int nv = row_vectors(a.hidden), th = row_threads(a.hidden, nv);
    // as many blocks as fit, and no more: a block's next row is then always on its way
    const int fit = kSms * (kResident / th > 0 ? kResident / th : 1), nb = a.rows < fit ? a.rows : fit;
    if (nv == 4) return launch_pdl(rms_norm_kernel<E, 4, true>, dim3(nb), dim3(th), 0, st, a);
    if (wide_row(a.hidden)) return launch_pdl(rms_norm_kernel<E, 2, true>, dim3(nb), dim3(th), 0, st, a);
    if (nv == 2) return launch_pdl(rms_norm_kernel<E, 2, false>, dim3(nb), dim3(th), 0, st, a);
    return launch_pdl(rms_norm_kernel<E, 1, false>, dim3(nb), dim3(th), 0, st, a);
}
template <typename E, int NV>
cudaError_t norm_bwd_wide(const NormBwdArgs& a, int th, int nb, cudaStream_t st) {
    const size_t smem = (size_t)a.hidden * sizeof(float);  // at most 128 KB: one block per SM
    if (cudaError_t e = cudaFuncSetAttribute(rms_norm_bwd_wide_kernel<E, NV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             8 * kWideThreads * NV * (int)sizeof(float)))
        return e;
    return launch_pdl(rms_norm_bwd_wide_kernel<E, NV>, dim3(nb), dim3(th), smem, st, a);
}
template <typename E>
cudaError_t norm_bwd(const NormBwdArgs& a, cudaStream_t st) {
    const int nv = row_vectors(a.hidden), th = row_threads(a.hidden, nv);
    // rows that share a block: as many as its threads allow, 15 barriers and
    // (half of the threads, so that their gradients fit) shared memory
    int groups = nv == 1 && th <= kMostThreads / 2 ? kMostThreads / th : 1;
    if (groups > 15) groups = 15;
    if (groups > a.rows) groups = a.rows > 0 ? a.rows : 1;
    const int most = wide_row(a.hidden) ? kSms : norm_bwd_blocks(a.rows), want = (a.rows + groups - 1) / groups;
    const int nb = want < most ? want : most;
    if (nb) {
        const dim3 grid(nb), block(th * groups);
        cudaError_t e;
        if (nv == 4) e = norm_bwd_wide<E, 4>(a, th, nb, st);
        else if (wide_row(a.hidden)) e = norm_bwd_wide<E, 2>(a, th, nb, st);
        else if (nv == 2) e = launch_pdl(rms_norm_bwd_kernel<E, 2>, grid, block, 0, st, a, groups);
        else e = launch_pdl(rms_norm_bwd_kernel<E, 1>, grid, block, 0, st, a, groups);
        if (e) return e;
    }
    return column_total<E>(a.partial, nb, a.hidden, a.dw, st);
}
template <typename E>
cudaError_t act_bwd(const ActBwdArgs& a, cudaStream_t st) {
    const int chunks = act_bwd_chunks(a.rows, a.cols), vx = act_vx(a.cols);
    if (chunks) {
        const dim3 grid(chunks * ((a.cols + 8 * vx - 1) / (8 * vx)));
        if (cudaError_t e = launch_pdl(act_bwd_kernel<E>, grid, dim3(kActThreads), 0, st, a, vx, act_rows(a.rows, a.cols))) return e;
    }
    return a.db ? column_total<E>(a.partial, chunks, a.cols, a.db, st) : cudaSuccess;
}

}  // namespace

int norm_bwd_blocks(int rows) { return rows < 2 * kSms ? rows : 2 * kSms; }
int act_bwd_chunks(int rows, int cols) {
    const int chunk = act_rows(rows, cols);
    return (rows + chunk - 1) / chunk;
}

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
