// The router's choice for every token, and each chosen entry's row in the
// order sorted by expert; the gradient of the logits.
//
// Top-k: a warp holds a token's logits as order-preserving keys, lane l the
// experts EPL l .. EPL l + EPL - 1, so that the lowest lane with the largest
// key holds the lowest such expert.  A pick is a warp maximum and a vote on who
// has it; that lane writes the expert down and takes its key away.
//
// Places: an expert is chosen at most once per token, so 32 tokens' choices of
// it are the bits of one word, and an entry's rank among its expert's is a
// popcount of the bits below its token's.  A block takes a chunk of tokens, kTokens
// at a time, and leaves ranks inside the chunk and the chunk's counts; a
// second launch adds up the counts of the chunks before each one and of all
// experts before.  Up to kAloneTokens one block does it all in one launch.
// Nothing depends on the order of atomics: the bits are OR-ed, the counts whole
// numbers.
//
// Bound by the picks' instructions, a warp maximum among them (439 a token with
// 8 of 128): 16384 tokens 15 us, of which the first launch 12; 8 tokens 2.9 us.
// That launch's 128 blocks of 128 tokens issue in 91 % of their SMs' cycles, for
// three quarters of its time; 24 SMs have none, as chunks are whole words.
#include "experts.cuh"
#include "pe_device.cuh"

namespace pe {
namespace dense {
namespace {

constexpr int kThreads = 1024;                  // a warp per token
constexpr int kWords = 4, kTokens = 32 * kWords;  // tokens of a batch
constexpr int kAloneTokens = 32;  // a chunk's least: 64 tokens of 128 experts 6.0 us in one launch, 5.2 in two
constexpr int kMostChunks = 152;

// Order-preserving key of a logit: NaN as -infinity, -0 as +0; never 0, the
// key of what was picked.
__device__ __forceinline__ uint32_t key_of(float v) {
    if (v != v) v = -INFINITY;
    const uint32_t u = __float_as_uint(v + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key) {
    return __uint_as_float((key & 0x80000000u) ? key & 0x7fffffffu : ~key);
}

// A token's logits on their way.  vec: rows of whole, aligned fours.
template <int EPL>
__device__ __forceinline__ void fetch(const float* row, int experts, bool vec, int lane, float (&v)[EPL]) {
    if (EPL % 4 == 0 && vec) {
#pragma unroll
        for (int q = 0; q < EPL; q += 4) {
            const int e = lane * EPL + q;
            const float4 f = e < experts ? *reinterpret_cast<const float4*>(row + e) : make_float4(0.f, 0.f, 0.f, 0.f);
            v[q] = f.x, v[(q + 1) % EPL] = f.y, v[(q + 2) % EPL] = f.z, v[(q + 3) % EPL] = f.w;
        }
    } else {
#pragma unroll
        for (int q = 0; q < EPL; ++q) v[q] = lane * EPL + q < experts ? row[lane * EPL + q] : 0.f;
    }
}

// SORTED: a lane's keys are put in order first (by neighbours, so that equal
// ones stay in the order of their experts), and a pick takes its head away;
// else a pick looks for the largest left.  Up to eight keys a lane: 16384 tokens
// of 256 experts 22.3 us sorted, 23.6 not.  `chosen`: the warp's, in shared memory.
template <int EPL>
__device__ __forceinline__ void pick(const float (&v0)[EPL], int experts, int k, int lane, uint16_t* chosen, float& w) {
    constexpr bool SORTED = EPL <= 8;
    uint32_t key[EPL], at = 0;  // SORTED: at, four bits each, the places of the keys
#pragma unroll
    for (int q = 0; q < EPL; ++q) key[q] = lane * EPL + q < experts ? key_of(v0[q]) : 0;
    if (SORTED) {
        uint32_t from[EPL];
#pragma unroll
        for (int q = 0; q < EPL; ++q) from[q] = q;
#pragma unroll
        for (int n = EPL - 1; n > 0; --n)
#pragma unroll
            for (int q = 0; q < n; ++q) {
                const bool swap = key[q] < key[q + 1];
                const uint32_t f = from[q], hi = max(key[q], key[q + 1]);
                key[q + 1] = min(key[q], key[q + 1]);
                key[q] = hi;
                from[q] = swap ? from[q + 1] : f;
                from[q + 1] = swap ? f : from[q + 1];
            }
#pragma unroll
        for (int q = 0; q < EPL; ++q) at |= from[q] << (4 * q);
    }
    uint32_t mine = 0;  // key of this lane's pick
    const uint32_t below = (1u << lane) - 1;
    for (int j = 0; j < k; ++j) {
        uint32_t best = key[0];
        if (!SORTED) {
            at = 0;
#pragma unroll
            for (int q = 1; q < EPL; ++q)
                if (key[q] > best) best = key[q], at = q;
        }
        const uint32_t top = __reduce_max_sync(0xffffffffu, best), have = __ballot_sync(0xffffffffu, best == top);
        if (best == top && !(have & below)) {
            chosen[j] = (uint16_t)(lane * EPL + (SORTED ? at & 15u : at));
            if (SORTED) {
#pragma unroll
                for (int q = 0; q + 1 < EPL; ++q) key[q] = key[q + 1];
                key[EPL - 1] = 0;
                at >>= 4;
            } else {
#pragma unroll
                for (int q = 0; q < EPL; ++q)
                    if (q == (int)at) key[q] = 0;
            }
        }
        if (lane == j) mine = top;
    }
    __syncwarp();
    // the softmax over the chosen; infinities that lead share the weight
    const float v = logit_of(mine), lead = __shfl_sync(0xffffffffu, v, 0);
    float p = lane < k ? (v == lead ? 1.f : expf(v - lead)) : 0.f, sum = p;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    w = __fdiv_rn(p, sum);
}

// Sum of v over the threads before this one; total over all.
__device__ __forceinline__ int scan_block(int v, int* part, int& total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = kThreads / 32;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += n;
    }
    if (lane == 31) part[warp] = s;
    __syncthreads();
    if (warp == 0) {
        int p = lane < warps ? part[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, p, o);
            if (lane >= o) p += n;
        }
        part[lane] = p;
    }
    __syncthreads();
    total = part[warps - 1];
    return s - v + (warp ? part[warp - 1] : 0);
}

// ALONE: the one block of its launch, which finishes the places and offsets.
template <int EPL, bool ALONE>
__global__ void __launch_bounds__(kThreads) choose_kernel(const RouteArgs a, int chunk_tokens, bool vec) {
    __shared__ uint32_t bits[kMaxGroups][kWords];  // bit t of word w: token 32 w + t of the batch chose this expert
    __shared__ int run[kMaxGroups], part[32];
    __shared__ uint16_t chosen[kTokens / 32][32][kMostTopK];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < a.experts; e += kThreads) {
        run[e] = 0;
#pragma unroll
        for (int w = 0; w < kWords; ++w) bits[e][w] = 0;
    }
    pdl_wait();
    pdl_trigger();
    __syncthreads();
    const int t0 = blockIdx.x * chunk_tokens, t1 = min(a.tokens - t0, chunk_tokens) + t0;
    constexpr bool AHEAD = EPL <= 16;  // registers for the next token's logits
    for (int tb = t0; tb < t1; tb += kTokens) {
        // a warp's tokens of the batch: one of each word
        float next[EPL];
        if (AHEAD && tb + warp < t1) fetch<EPL>(a.logits + (tb + warp) * a.ld, a.experts, vec, lane, next);
#pragma unroll 1
        for (int w = 0; w < kWords; ++w) {
            const int t = tb + 32 * w + warp;
            if (t >= t1) break;
            float v[EPL], weight;
            if (AHEAD) {
#pragma unroll
                for (int q = 0; q < EPL; ++q) v[q] = next[q];
                if (w + 1 < kWords && t1 - t > 32) fetch<EPL>(a.logits + (t + 32) * a.ld, a.experts, vec, lane, next);
            } else {
                fetch<EPL>(a.logits + t * a.ld, a.experts, vec, lane, v);
            }
            pick<EPL>(v, a.experts, a.k, lane, chosen[w][warp], weight);
            if (lane < a.k) {
                const int id = chosen[w][warp][lane];
                a.ids[(int64_t)t * a.k + lane] = id;
                a.weights[(int64_t)t * a.k + lane] = weight;
                atomicOr(&bits[id][w], 1u << warp);
            }
        }
        __syncthreads();
        // ranks: entries of the batch in turn, whole lines at a time
        const int entries = min(kTokens, t1 - tb) * a.k;
        for (int i = threadIdx.x; i < entries; i += kThreads) {
            const int t = i / a.k, id = chosen[t / 32][t % 32][i - t * a.k];
            int rank = run[id] + __popc(bits[id][t / 32] & ((1u << t % 32) - 1));
            for (int w = 0; w < t / 32; ++w) rank += __popc(bits[id][w]);
            a.place[(int64_t)tb * a.k + i] = rank;
        }
        __syncthreads();
        for (int e = threadIdx.x; e < a.experts; e += kThreads) {
            int n = run[e];
#pragma unroll
            for (int w = 0; w < kWords; ++w) n += __popc(bits[e][w]), bits[e][w] = 0;
            run[e] = n;
        }
        __syncthreads();
    }
    if (!ALONE) {
        for (int e = threadIdx.x; e < a.experts; e += kThreads) a.counts[(int64_t)blockIdx.x * a.experts + e] = run[e];
        return;
    }
    int total;
    const int n = threadIdx.x < a.experts ? run[threadIdx.x] : 0, before = scan_block(n, part, total);
    static_assert(kMaxGroups <= kThreads, "an expert per thread");
    if (threadIdx.x < a.experts) a.offsets[threadIdx.x] = run[threadIdx.x] = before;
    if (threadIdx.x == 0) a.offsets[a.experts] = total;
    __syncthreads();
    // written by this thread or, before a barrier, by another one of the block
    for (int i = threadIdx.x; i < a.tokens * a.k; i += kThreads) a.place[i] += run[a.ids[i]];
}

__global__ void __launch_bounds__(kThreads) place_kernel(const RouteArgs a, int chunk_tokens) {
    __shared__ int before[kMaxGroups], all[kMaxGroups], part[32];
    for (int e = threadIdx.x; e < a.experts; e += kThreads) before[e] = all[e] = 0;
    pdl_wait();
    pdl_trigger();
    const int t0 = blockIdx.x * chunk_tokens, t1 = min(a.tokens - t0, chunk_tokens) + t0;
    const int64_t first_entry = (int64_t)t0 * a.k + threadIdx.x, last_entry = (int64_t)t1 * a.k;
    int id0 = 0, place0 = 0;  // asked for ahead of the sums
    if (first_entry < last_entry) id0 = a.ids[first_entry], place0 = a.place[first_entry];
    __syncthreads();
    // a group of threads per expert's share of the chunks
    const int lanes = min(kThreads, (a.experts + 31) / 32 * 32), shares = kThreads / lanes;
    const int share = threadIdx.x / lanes, e0 = threadIdx.x % lanes;
    if (share < shares && e0 < a.experts) {
        int b = 0, s = 0;
        for (int c0 = share; c0 < (int)gridDim.x; c0 += 8 * shares) {
            int n[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) n[u] = c0 + u * shares < (int)gridDim.x ? a.counts[(int64_t)(c0 + u * shares) * a.experts + e0] : 0;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                s += n[u];
                if (c0 + u * shares < (int)blockIdx.x) b += n[u];
            }
        }
        atomicAdd(&before[e0], b);
        atomicAdd(&all[e0], s);
    }
    __syncthreads();
    int total;
    const int n = threadIdx.x < a.experts ? all[threadIdx.x] : 0, first = scan_block(n, part, total);
    if (threadIdx.x < a.experts) {
        before[threadIdx.x] += first;
        if (blockIdx.x == 0) a.offsets[threadIdx.x] = first;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[a.experts] = total;
    __syncthreads();
    if (first_entry < last_entry) a.place[first_entry] = place0 + before[id0];
    for (int64_t i = first_entry + kThreads; i < last_entry; i += kThreads) a.place[i] += before[a.ids[i]];
}

// dlogits[t, ids[i]] = w_i (dw_i - sum_j w_j dw_j), zero elsewhere; an expert
// named twice gets both.  A warp per token.
__global__ void __launch_bounds__(256) route_bwd_kernel(const RouteBwdArgs a) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (t >= a.tokens) return;
    float w = 0.f, d = 0.f;
    int id = -1;
    if (lane < a.k) {
        w = a.weights[t * a.k + lane];
        d = a.dweights[t * a.k + lane];
        id = a.ids[t * a.k + lane];
    }
    float dot = w * d;
#pragma unroll
    for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    const float g = w * (d - dot);
    float sum = 0.f;
    bool first = true;
    for (int j = 0; j < a.k; ++j) {
        const int other = __shfl_sync(0xffffffffu, id, j);
        const float v = __shfl_sync(0xffffffffu, g, j);
        if (other == id) {
            sum += v;
            if (j < lane) first = false;
        }
    }
    float* row = a.dlogits + t * a.experts;
    if (a.experts % 4 == 0) {
        for (int e = lane; e < a.experts / 4; e += 32) reinterpret_cast<float4*>(row)[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    } else {
        for (int e = lane; e < a.experts; e += 32) row[e] = 0.f;
    }
    __syncwarp();  // the zeros are there before the values
    if (lane < a.k && first && id >= 0 && id < a.experts) row[id] = sum;
}

// Tokens of a chunk: whole words of 32, in at most kMostChunks chunks.
int chunk_of(int tokens) {
    const int words = (tokens - 1) / 32 + 1;
    return ((words - 1) / kMostChunks + 1) * 32;
}

template <int EPL>
cudaError_t choose(const RouteArgs& a, cudaStream_t st) {
    const bool vec = a.experts % 4 == 0 && a.ld % 4 == 0 && reinterpret_cast<uintptr_t>(a.logits) % 16 == 0;
    if (a.tokens <= kAloneTokens) return launch_pdl(choose_kernel<EPL, true>, dim3(1), dim3(kThreads), 0, st, a, a.tokens, vec);
    const int chunks = route_chunks(a.tokens);
    if (cudaError_t e = launch_pdl(choose_kernel<EPL, false>, dim3(chunks), dim3(kThreads), 0, st, a, chunk_of(a.tokens), vec)) return e;
    return launch_pdl(place_kernel, dim3(chunks), dim3(kThreads), 0, st, a, chunk_of(a.tokens));
}

}  // namespace

int route_chunks(int tokens) { return (tokens - 1) / chunk_of(tokens) + 1; }

cudaError_t launch_route_tokens(const RouteArgs& a, cudaStream_t st) {
    const int epl = (a.experts + 31) / 32;
    return epl <= 1   ? choose<1>(a, st)
           : epl <= 2 ? choose<2>(a, st)
           : epl <= 4 ? choose<4>(a, st)
           : epl <= 8 ? choose<8>(a, st)
           : epl <= 16 ? choose<16>(a, st)
                      : choose<32>(a, st);
}

cudaError_t launch_route_bwd(const RouteBwdArgs& a, cudaStream_t st) {
    return launch_pdl(route_bwd_kernel, dim3((a.tokens + 7) / 8), dim3(256), 0, st, a);
}

}  // namespace dense
}  // namespace pe
