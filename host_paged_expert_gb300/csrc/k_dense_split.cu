// Matrix products of few rows or few tiles: C[m, n] = sum_k A(m, k) B(n, k),
// then the epilogue, with the K axis split over a cluster.
//
// A decode step's product reads each weight once and is bound by HBM, or by
// latency when the weights sit in L2; what counts is that every SM has many
// bytes in flight from the first moment on.  So the weights' rows lie along
// the MMA's M (128 per tile, all lanes of TMEM used) and the tokens along its
// N (16 to 128), the opposite of the large-tile kernel, and the K blocks of
// one tile are shared out among the CTAs of a cluster.  Each CTA streams its
// share through TMA (128 weight rows x 128 bytes a stage), accumulates in
// TMEM, and leaves its fp32 partial in shared memory; after a cluster
// barrier the CTAs add up the partials over distributed shared memory, each
// a part of the tile, in rank order, so the result does not depend on timing,
// needs no workspace and no second launch.
//
// What bounds it: a K block of 64 takes 0.24 us whatever the tokens (four
// MMAs of 128 rows), a launch 2 us and 0.026 us per token of the tile, and the
// partials cross the cluster at 1.7 TB/s: 8 x 2048 to 128 with fp32 results 3.8
// us, 64 x 2048 to 2048 5.9 us, 64 x 4096 to 4096 9.4 us (floor 4.9).
//
// The second product of a feed-forward block starts early: it loads its
// weights while the first one still runs (programmatic dependent launch) and
// waits only for the activations.
//
// E4M3: each 128-deep stage is one scale group and goes to a TMEM buffer of
// its own, added with its scales to fp32 registers.  fp32 results: the MMA
// truncates each addition to its accumulator (2.3e-6 relative after 2048
// terms), so no more than 512 terms go into one accumulator while TMEM has
// room, and those are added in registers.
#include "dense.cuh"
#include "dense_cluster.cuh"
#include "dense_tc.cuh"
#include "pe_device.cuh"

namespace pe {
namespace dense {

namespace {

constexpr int kThreads = 256;  // warp 0 TMA, 1 MMA, 2 TMEM, 4..7 epilogue; all of them add up
constexpr int kP = kRows * 128;  // bytes of their stage
constexpr int kMaxStages = 8;

struct Plan {
    int nt;       // tokens of a tile (MMA N), a multiple of 16
    int q_bytes;  // bytes of their stage
    int stages;
    int split;    // CTAs along K
    int ftiles;   // tiles of 128 weight rows
    int subs;     // accumulators per tile
    int sub_len;  // stages that one of them takes (16-bit operands)
    int cols;     // TMEM columns
    int early;    // load weights before the previous kernel is done
    WaitLimits limit;
};

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages], acc_full[8], acc_empty[8], drain;
    uint32_t tmem;
};

// LIMITED: the waits' limits are the launch's.
template <typename E, int KIND, bool FP8, bool LIMITED>
__global__ void __launch_bounds__(kThreads, 2)
    split_kernel(const __grid_constant__ CUtensorMap tp, const __grid_constant__ CUtensorMap tq,
                 const __grid_constant__ Product p, const __grid_constant__ Plan q, uint32_t* err) {
    constexpr int BK = FP8 ? 128 : 64;                            // elements of a 128-byte row
    constexpr int NF = KIND == EPI_GATED ? kRows / 2 : kRows;  // result columns of a tile
    auto polls = [](uint32_t limit) { return LIMITED ? limit : kPolls; };
    extern __shared__ uint8_t dyn[];
    __shared__ Shared S;
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // block = ((token tile) * feature tiles + feature tile) * split + rank
    const int rank = blockIdx.x % q.split, tile = blockIdx.x / q.split, ft = tile % q.ftiles;
    const int f0 = ft * NF, t0 = tile / q.ftiles * q.nt;
    const int kall = (p.K + BK - 1) / BK;
    const int kb0 = (int)((long long)kall * rank / q.split), nkb = (int)((long long)kall * (rank + 1) / q.split) - kb0;
    const int stage = kP + q.q_bytes;

    const int pre = min(q.stages, nkb);  // the ring's first round finds it empty
    auto load_p = [&](int i, int s) {
        uint8_t* a = ring + s * stage;
        const int k = (kb0 + i) * BK;
        if (p.b_mn) {
            tc::tma_load_2d(a, &tp, &S.full[s], f0, k);
            tc::tma_load_2d(a + kP / 2, &tp, &S.full[s], f0 + 64, k);
        } else {
            tc::tma_load_2d(a, &tp, &S.full[s], k, f0);
            tc::tma_load_2d(a + kP / 2, &tp, &S.full[s], k, f0 + (KIND == EPI_GATED ? p.e.cols : 64));
        }
    };
    auto load_q = [&](int i, int s) {
        uint8_t* b = ring + s * stage + kP;
        const int k = (kb0 + i) * BK;
        if (p.a_mn)
            for (int c = 0; c * 8192 < q.q_bytes; ++c) tc::tma_load_2d(b + c * 8192, &tq, &S.full[s], t0 + 64 * c, k);
        else tc::tma_load_2d(b, &tq, &S.full[s], k, t0);
    };
    // The producer does not wait for the block: its first loads go out while
    // TMEM is allocated, and it has no use for the address.
    if (warp == 0) {
        const bool lead = tc::elect_one();
        if (lead) {
            for (int i = 0; i < q.stages; ++i) {
                tc::mbar_init(&S.full[i], 1);
                tc::mbar_init(&S.empty[i], 1);
            }
            for (int i = 0; i < 8; ++i) {
                tc::mbar_init(&S.acc_full[i], 1);
                tc::mbar_init(&S.acc_empty[i], 4);
            }
            tc::mbar_init(&S.drain, 1);
            tc::fence_barrier_init();
            tc::tma_prefetch(&tp);
            tc::tma_prefetch(&tq);
        }
        __syncwarp();
        asm volatile("bar.arrive 2, %0;" ::"n"(kThreads) : "memory");
        if (!q.early) pdl_wait();
        if (lead)
            for (int i = 0; i < pre; ++i) {
                tc::mbar_arrive_expect_tx(&S.full[i], stage);
                load_p(i, i);
                if (!q.early) load_q(i, i);
            }
        __syncwarp();
    } else {
        if (warp == 2) tc::tmem_alloc(&S.tmem, q.cols);
        tc::fence_before_sync();
        asm volatile("bar.sync 2, %0;" ::"n"(kThreads) : "memory");
        tc::fence_after_sync();
    }
    const uint32_t tmem = warp == 0 ? 0 : *reinterpret_cast<volatile uint32_t*>(&S.tmem);
    if (warp == 3) {  // what ran before this kernel is done before the next one starts
        pdl_wait();
        pdl_trigger();
    }

    if (warp == 0) {
        // ---- producer
        const bool lead = tc::elect_one();
        if (q.early) {
            pdl_wait();
            if (lead)
                for (int i = 0; i < pre; ++i) load_q(i, i);
        }
        int i = pre, s = 0;
        uint32_t phase = 0;
        for (; i < nkb; ++i) {
            if (!tc::mbar_spin(&S.empty[s], phase, err, polls(q.limit.copies))) break;
            if (lead) {
                tc::mbar_arrive_expect_tx(&S.full[s], stage);
                load_p(i, s);
                load_q(i, s);
            }
            if (++s == q.stages) s = 0, phase ^= 1;
        }
        // the block does not end before its copies have landed (all of them were used, unless a wait gave up)
        bool landed = true;
        for (int j = max(0, i - q.stages); landed && j < i; ++j)
            landed = tc::mbar_wait(&S.full[j % q.stages], (j / q.stages) & 1, err, PE_DEVERR_TIMEOUT, tc::kLeavePolls);
        if (!landed) tc::settle();
    } else if (warp == 1) {
        // ---- MMA issuer
        const bool lead = tc::elect_one();
        constexpr int FMT = FP8 ? 0 : std::is_same<E, __nv_bfloat16>::value ? 1 : 0;
        const uint32_t id = tc::idesc(FMT, p.b_mn, p.a_mn, kRows, q.nt);
        const uint32_t pstep = (p.b_mn ? 2048 : 32) >> 4, qstep = (p.a_mn ? 2048 : 32) >> 4;
        const uint64_t a0 = tc::operand_desc(tc::smem_u32(ring), p.b_mn), b0 = tc::operand_desc(tc::smem_u32(ring) + kP, p.a_mn);
        int s = 0, buf = 0, in_buf = 0;
        uint32_t phase = 0, buf_phase = 1;
        pdl_wait();  // a wait's limit is for this kernel's own copies, not for the launch before it
        for (int i = 0; i < nkb; ++i) {
            // FP8: each stage has the next buffer to itself; else a buffer takes sub_len stages
            if (FP8 && !tc::mbar_spin(&S.acc_empty[buf], buf_phase, err, polls(q.limit.mma))) break;
            if (!tc::mbar_spin(&S.full[s], phase, err, polls(q.limit.mma))) break;
            tc::fence_after_sync();
            if (lead) {
                const uint64_t a = a0 + (uint32_t)(s * stage >> 4), b = b0 + (uint32_t)(s * stage >> 4);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    tc::mma<false, FP8>(tmem + buf * q.nt, a + k * pstep, b + k * qstep, id, (!FP8 && in_buf) || k);
                tc::mma_commit(&S.empty[s]);
                if (FP8) tc::mma_commit(&S.acc_full[buf]);
                else if (i == nkb - 1) tc::mma_commit(&S.acc_full[0]);
            }
            __syncwarp();
            if (++s == q.stages) s = 0, phase ^= 1;
            if (FP8 || ++in_buf == q.sub_len) {
                in_buf = 0;
                if (++buf == q.subs) buf = 0, buf_phase ^= 1;
            }
        }
        // nor before its MMAs, which read shared memory and write TMEM
        if (lead) tc::mma_commit(&S.drain);
        tc::mbar_wait(&S.drain, 0, err, PE_DEVERR_TIMEOUT, tc::kLeavePolls);
    } else if (warp >= 4) {
        // ---- accumulators to part[token][weight row]
        pdl_wait();
        const int quarter = warp & 3;
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        float* part = reinterpret_cast<float*>(ring) + quarter * 32 + lane;
        if (FP8) {  // nt <= 64: two chunks of 32 tokens
            float acc[2][32];
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int j = 0; j < 32; ++j) acc[c][j] = 0.f;
            const float* bs = p.b_scale + (size_t)ft * kall + kb0;
            int buf = 0;
            uint32_t phase = 0;
            for (int i = 0; i < nkb; ++i) {
                const float ws = bs[i];
                float xs[2];  // the scale of this lane's token of each chunk
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int t = t0 + c * 32 + lane;
                    xs[c] = t < p.M && c * 32 + lane < q.nt ? ws * p.a_scale[(size_t)t * kall + kb0 + i] : 0.f;
                }
                if (!tc::mbar_spin(&S.acc_full[buf], phase, err, polls(q.limit.sums))) break;
                tc::fence_after_sync();
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    if (c * 32 < q.nt) {
                        uint32_t r[32];
                        tc::tmem_ld32(lanes + buf * q.nt + c * 32, r);
                        tc::tmem_ld_wait(r);
#pragma unroll
                        for (int n = 0; n < 32; ++n)
                            acc[c][n] = fmaf(__uint_as_float(r[n]), __shfl_sync(0xffffffffu, xs[c], n), acc[c][n]);
                    }
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&S.acc_empty[buf]);
                if (++buf == q.subs) buf = 0, phase ^= 1;
            }
            // every warp is past its last buffer, so every MMA is done with the ring
            asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (c * 32 + j < q.nt) part[(c * 32 + j) * kRows] = acc[c][j];
        } else {
            if (tc::mbar_spin(&S.acc_full[0], 0, err, polls(q.limit.sums))) {
                tc::fence_after_sync();
                // the next chunk is on its way while this one is stored; two arrays in turn
                uint32_t r[2][32];
                const int last = (nkb - 1) / q.sub_len;  // accumulators 0..last hold parts
                tc::tmem_ld32(lanes, r[0]);
                for (int c0 = 0; c0 < q.nt; c0 += 64) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int c = c0 + 32 * h;
                        if (c >= q.nt) break;
                        tc::tmem_ld_wait(r[h]);
                        for (int b = 1; b <= last; ++b) {
                            tc::tmem_ld32(lanes + b * q.nt + c, r[h ^ 1]);
                            tc::tmem_ld_wait(r[h ^ 1]);
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                r[h][j] = __float_as_uint(__uint_as_float(r[h][j]) + __uint_as_float(r[h ^ 1][j]));
                        }
                        if (c + 32 < q.nt) tc::tmem_ld32(lanes + c + 32, r[h ^ 1]);
#pragma unroll
                        for (int j = 0; j < 16; ++j) part[(c + j) * kRows] = __uint_as_float(r[h][j]);
                        if (c + 16 < q.nt)
#pragma unroll
                            for (int j = 16; j < 32; ++j) part[(c + j) * kRows] = __uint_as_float(r[h][j]);
                    }
                }
            }
            tc::fence_before_sync();
        }
    }
    pdl_wait();
    __syncwarp();
    __syncthreads();
    if (q.split > 1) {
        tc::cluster_arrive();
        tc::cluster_wait();
    }

    // ---- the tile's sum over the cluster, and the epilogue
    if (q.split == 1) reduce<E, KIND, 1, kThreads>(p.e, ring, q.nt, 1, rank, t0, f0);
    else if (q.split == 2) reduce<E, KIND, 2, kThreads>(p.e, ring, q.nt, 2, rank, t0, f0);
    else if (q.split <= 4) reduce<E, KIND, 4, kThreads>(p.e, ring, q.nt, q.split, rank, t0, f0);
    else reduce<E, KIND, 8, kThreads>(p.e, ring, q.nt, q.split, rank, t0, f0);
    // no CTA leaves while another may read its partial
    if (q.split > 1) {
        tc::cluster_arrive_relaxed();
        tc::cluster_wait();
    }
    tc::fence_after_sync();
    if (warp == 2) tc::tmem_dealloc(tmem, q.cols);
}

constexpr int kMaxSmem = 226 * 1024;  // what a block may have, less the static part
// Up to kPairTokens tokens two blocks share an SM, so that one's epilogue
// hides under the other's stream and a dependent launch can move in early;
// above, one.  Their shared memory (between kTwo and kHalf, or at least kOne
// bytes) decides how many fit, and their TMEM has to fit as well: a block that
// waited for columns held by a block of its own cluster would wait forever.
constexpr int kPairTokens = 64, kTwo = 80 * 1024, kHalf = 110 * 1024, kOne = 116 * 1024;
int block_bytes(int nt) { return nt <= kPairTokens ? kHalf : kMaxSmem; }
int tmem_cols(int nt) { return nt <= kPairTokens ? 256 : 512; }

// Accumulators of a tile whose result is fp32: one for every 8 blocks of 64,
// as far as TMEM goes.
int sub_count(const SplitShape& s, int kb) {
    const int share = (kb + s.split - 1) / s.split, want = (share + 7) / 8, most = (tmem_cols(s.nt) - 32) / s.nt;
    return want < most ? want : most;
}

template <typename E, int KIND, bool FP8, bool LIMITED = false>
cudaError_t launch(const Product& p, const SplitShape& s, int chain, uint32_t* err, cudaStream_t st,
                   const WaitLimits& limits = {}) {
    static std::atomic<uint64_t> ready;  // devices whose attribute is set
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    auto kernel = split_kernel<E, KIND, FP8, LIMITED>;
    if (dev >= 64 || !(ready.load() >> dev & 1)) {
        if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem)) return e;
        if (dev < 64) ready.fetch_or(uint64_t(1) << dev);
    }
    Plan q = {};
    q.nt = s.nt;
    q.split = s.split;
    q.q_bytes = 128 * (p.a_mn && s.nt < 64 ? 64 : p.a_mn ? (s.nt + 63) / 64 * 64 : s.nt);
    const int kall = (p.K + (FP8 ? 127 : 63)) / (FP8 ? 128 : 64), share = (kall + s.split - 1) / s.split;
    const int block = kP + q.q_bytes, part = s.nt * kRows * 4;
    q.stages = (block_bytes(s.nt) - 1024) / block;
    if (q.stages > kMaxStages) q.stages = kMaxStages;
    if (q.stages > share) q.stages = share;
    int bytes = 1024 + (q.stages * block > part ? q.stages * block : part);
    // no fewer than what keeps the count of blocks per SM
    if (s.nt <= kPairTokens && bytes < kTwo) bytes = kTwo;
    if (s.nt > kPairTokens && bytes < kOne) bytes = kOne;
    q.subs = FP8 ? 4 : p.e.out_f32 ? sub_count(s, kall) : 1;
    q.sub_len = (share + q.subs - 1) / q.subs;
    q.cols = 32;
    while (q.cols < (q.nt + 31) / 32 * 32 + q.nt * (q.subs - 1)) q.cols *= 2;
    if (q.cols > tmem_cols(s.nt) || kall < s.split || s.split > 8 || s.nt > (FP8 ? 64 : 128)) return cudaErrorInvalidValue;
    constexpr int NF = KIND == EPI_GATED ? kRows / 2 : kRows;
    q.ftiles = (p.e.cols + NF - 1) / NF;
    const long long blocks = (long long)q.ftiles * ((p.M + s.nt - 1) / s.nt) * s.split;
    if (blocks > INT_MAX) return cudaErrorInvalidValue;
    q.early = chain == CHAIN_AFTER;
    q.limit = limits;
    CUtensorMap tp, tq;
    if (!encode_operand(&tp, p.b, p.ldb, p.N, p.K, p.b_mn, FP8, 64) || !encode_operand(&tq, p.a, p.lda, p.M, p.K, p.a_mn, FP8, s.nt))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)s.split, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, tp, tq, p, q, err);
}

template <typename E>
cudaError_t launch_kind(const Product& p, EpiKind kind, const SplitShape& s, int chain, uint32_t* err, cudaStream_t st) {
    if (p.a_scale) return launch<E, EPI_LINEAR, true>(p, s, chain, err, st);
    if (kind == EPI_LINEAR) return launch<E, EPI_LINEAR, false>(p, s, chain, err, st);
    if (kind == EPI_SCALED) return launch<E, EPI_SCALED, false>(p, s, chain, err, st);
    if (kind == EPI_GATED) return launch<E, EPI_GATED, false>(p, s, chain, err, st);
    return launch<E, EPI_GATED_BWD, false>(p, s, chain, err, st);
}

}  // namespace

int split_blocks(const SplitShape& s, int kb) {
    const int share = (kb + s.split - 1) / s.split, n = sub_count(s, kb);
    return (share + n - 1) / n;
}

int split_resident(const SplitShape& s) {
    static std::atomic<int> known[2][9];  // one or two blocks per SM; CTAs along K
    const int two = s.nt <= kPairTokens, at = s.split;
    int n = known[two][at].load();
    if (n) return n;
    n = 152;  // where the runtime does not say
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)s.split, 1, 1};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)s.split);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = block_bytes(s.nt);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto k = split_kernel<__nv_bfloat16, EPI_LINEAR, false, false>;
    int c = 0;
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&c, k, &cfg) == cudaSuccess && c > 0)
        n = c * s.split;
    // The runtime counts one block per SM for a kernel that allocates TMEM;
    // two do run where they fit (64 x 512 x 19456, 152 blocks: 5.2 us; 304
    // blocks: 6.5; 305: 10.5).
    n <<= two;
    known[two][at].store(n);
    return n;
}

cudaError_t launch_split(const Product& p, EpiKind kind, int elem, const SplitShape& s, int chain, uint32_t* err,
                         cudaStream_t st, const WaitLimits* limits) {
    if (limits)
        return p.a_scale ? launch<__nv_bfloat16, EPI_LINEAR, true, true>(p, s, chain, err, st, *limits)
                         : launch<__nv_bfloat16, EPI_LINEAR, false, true>(p, s, chain, err, st, *limits);
    return elem == PE_ELEM_BF16 ? launch_kind<__nv_bfloat16>(p, kind, s, chain, err, st)
                                : launch_kind<__half>(p, kind, s, chain, err, st);
}

}  // namespace dense
}  // namespace pe
