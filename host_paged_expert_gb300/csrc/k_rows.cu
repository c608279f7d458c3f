// Rows to their experts and back: out[place[t, i]] = x[t]; out[t] = the
// weighted sum of y[place[t, i]] over i, plus a residual; and the sum's
// gradients, dy[place[t, i]] = w[t, i] dout[t] and dw[t, i] = <dout[t],
// y[place[t, i]]>.
//
// All of them move rows and do little else, so they are bound by HBM: a
// thread holds 16 bytes of a token's row, asks for up to eight of its rows'
// pieces at once, and adds in fp32 in the order of i.  A block takes one
// token of wide rows, several of narrow ones.  8191 x 8 x 2048, bf16: to the
// experts 47 us, back with weights and a residual 55, its gradients 89 (6.1 to 6.5
// TB/s; the copy's rate is 6.8).
#include "experts.cuh"
#include "pe_device.cuh"

namespace pe {
namespace dense {
namespace {

constexpr int kThreads = 256, kBatch = 8;  // entries of a token in flight

__device__ __forceinline__ float weight_of(const RowsArgs& a, int64_t entry) { return a.weights ? a.weights[entry] : 1.f; }

// per: threads of a token (a power of two); a block holds kThreads / per tokens.
template <typename E, bool WEIGHTED>
__global__ void __launch_bounds__(kThreads) expand_kernel(const RowsArgs a, int per) {
    pdl_wait();
    pdl_trigger();
    const int64_t t = (int64_t)blockIdx.x * (kThreads / per) + threadIdx.x / per;
    if (t >= a.tokens) return;
    const int pieces = a.hidden / 8;
    for (int c = threadIdx.x % per; c < pieces; c += per) {
        const int4 v = ld_stream(static_cast<const E*>(a.x) + t * a.ld_x + c * 8);
        float f[8];
        if (WEIGHTED) unpack8<E>(v, f);
        for (int i0 = 0; i0 < a.k; i0 += kBatch) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int i = i0 + u;
                if (i >= a.k) break;
                const int row = a.place[t * a.k + i];
                if ((unsigned)row >= (unsigned)a.rows) continue;
                E* to = static_cast<E*>(a.out) + (int64_t)row * a.hidden + c * 8;
                if (WEIGHTED) {
                    const float w = a.weights[t * a.k + i];
                    float o[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = w * f[j];
                    store8(to, true, 8, o);
                } else {
                    *reinterpret_cast<int4*>(to) = v;
                }
            }
        }
    }
}

template <typename E>
__global__ void __launch_bounds__(kThreads) combine_kernel(const RowsArgs a, int per) {
    pdl_wait();
    pdl_trigger();
    const int64_t t = (int64_t)blockIdx.x * (kThreads / per) + threadIdx.x / per;
    if (t >= a.tokens) return;
    const int pieces = a.hidden / 8;
    for (int c = threadIdx.x % per; c < pieces; c += per) {
        float sum[8] = {};
        for (int i0 = 0; i0 < a.k; i0 += kBatch) {
            int4 v[kBatch];
            float w[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int i = i0 + u, row = i < a.k ? a.place[t * a.k + i] : -1;
                const bool there = (unsigned)row < (unsigned)a.rows;
                w[u] = there ? weight_of(a, t * a.k + i) : 0.f;
                v[u] = there ? ld_stream(static_cast<const E*>(a.y) + row * a.ld_y + c * 8) : make_int4(0, 0, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                float f[8];
                unpack8<E>(v[u], f);
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j] = fmaf(w[u], f[j], sum[j]);
            }
        }
        if (a.res) {
            float r[8];
            unpack8<E>(ld_stream(static_cast<const E*>(a.res) + t * a.ld_res + c * 8), r);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] += r[j];
        }
        store8(static_cast<E*>(a.out) + t * (int64_t)a.hidden + c * 8, true, 8, sum);
    }
}

// x: dout.  The dot products of a batch of entries are added up over the
// token's threads: lanes by a transposed butterfly, then warps in order.
// Three blocks of an SM: 89 us for 8191 x 8 x 2048 (6.4 TB/s); two 113, four 97.
template <typename E>
__global__ void __launch_bounds__(kThreads, 3) combine_bwd_kernel(const RowsArgs a, int per) {
    __shared__ float part[kThreads / 32][kBatch];
    pdl_wait();
    pdl_trigger();
    const int slot = threadIdx.x / per, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * (kThreads / per) + slot;
    const bool live = t < a.tokens;
    const int pieces = a.hidden / 8;
    for (int i0 = 0; i0 < a.k; i0 += kBatch) {
        float dot[kBatch] = {};
        int row[kBatch];
        float w[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int i = i0 + u;
            row[u] = live && i < a.k ? a.place[t * a.k + i] : -1;
            if ((unsigned)row[u] >= (unsigned)a.rows) row[u] = -1;
            w[u] = row[u] >= 0 ? weight_of(a, t * a.k + i) : 0.f;
        }
        for (int c = threadIdx.x % per; live && c < pieces; c += per) {
            const int4 dv = *reinterpret_cast<const int4*>(static_cast<const E*>(a.x) + t * a.ld_x + c * 8);
            int4 v[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                v[u] = row[u] >= 0 ? ld_stream(static_cast<const E*>(a.y) + row[u] * a.ld_y + c * 8) : make_int4(0, 0, 0, 0);
            float d[8];
            unpack8<E>(dv, d);
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                if (row[u] < 0) continue;
                float f[8], o[8];
                unpack8<E>(v[u], f);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    dot[u] = fmaf(d[j], f[j], dot[u]);
                    o[j] = w[u] * d[j];
                }
                store8(static_cast<E*>(a.out) + (int64_t)row[u] * a.hidden + c * 8, true, 8, o);
            }
        }
        // per >= 32: every lane of a warp has the same token
        const float s = warp_sum_rows<kBatch>(dot, lane);
        constexpr int LANES = 32 / kBatch;
        if (lane % LANES == 0) part[warp][lane / LANES] = s;
        __syncthreads();
        const int warps = per / 32, u = threadIdx.x % per;
        if (live && u < kBatch && i0 + u < a.k) {
            float sum = 0.f;
            for (int v = 0; v < warps; ++v) sum += part[slot * warps + v][u];
            a.dweights[t * a.k + i0 + u] = sum;
        }
        __syncthreads();
    }
}

// Threads of a token: enough for its row at one piece each, as far as a block goes.
int threads_per_token(int hidden, int least) {
    int per = least;
    while (per < kThreads && per < hidden / 8) per *= 2;
    return per;
}
dim3 grid_of(const RowsArgs& a, int per) {
    const int n = kThreads / per;
    return dim3((unsigned)((a.tokens + (int64_t)n - 1) / n));
}

template <typename E>
cudaError_t expand(const RowsArgs& a, cudaStream_t st) {
    const int per = threads_per_token(a.hidden, 1);
    return a.weights ? launch_pdl(expand_kernel<E, true>, grid_of(a, per), dim3(kThreads), 0, st, a, per)
                     : launch_pdl(expand_kernel<E, false>, grid_of(a, per), dim3(kThreads), 0, st, a, per);
}
template <typename E>
cudaError_t combine(const RowsArgs& a, cudaStream_t st) {
    const int per = threads_per_token(a.hidden, 1);
    return launch_pdl(combine_kernel<E>, grid_of(a, per), dim3(kThreads), 0, st, a, per);
}
template <typename E>
cudaError_t combine_bwd(const RowsArgs& a, cudaStream_t st) {
    // two pieces a thread: half as many sums over threads (one piece 94, two 89, four 90 us for 8191 x 8 x 2048)
    const int per = threads_per_token(a.hidden / 2, 32);
    return launch_pdl(combine_bwd_kernel<E>, grid_of(a, per), dim3(kThreads), 0, st, a, per);
}

}  // namespace

cudaError_t launch_expand(const RowsArgs& a, int elem, cudaStream_t st) {
    return elem == PE_ELEM_BF16 ? expand<__nv_bfloat16>(a, st) : expand<__half>(a, st);
}
cudaError_t launch_combine(const RowsArgs& a, int elem, cudaStream_t st) {
    return elem == PE_ELEM_BF16 ? combine<__nv_bfloat16>(a, st) : combine<__half>(a, st);
}
cudaError_t launch_combine_bwd(const RowsArgs& a, int elem, cudaStream_t st) {
    return elem == PE_ELEM_BF16 ? combine_bwd<__nv_bfloat16>(a, st) : combine_bwd<__half>(a, st);
}

}  // namespace dense
}  // namespace pe
