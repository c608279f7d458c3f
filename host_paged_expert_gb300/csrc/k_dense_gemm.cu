// Matrix products of the dense operators: C[m, n] = sum_k A(m, k) B(n, k),
// then the epilogue.
//
// pair_kernel: persistent CTA pairs (two SMs), 256 x 256 tiles of C (or 256 x
// 128, below).  Each CTA's TMA producer streams its half of A and of B (128
// rows x 128 bytes each, 128-byte swizzle) into a ring of stages; one thread
// of the pair's leader issues the 256 x 256 tcgen05.mma, which reads both
// CTAs' shared memory, so a byte of B feeds 256 rows instead of 128.
// Accumulators live in TMEM, two buffers of 256 columns, so that the epilogue
// warps drain one tile while the next is multiplied.  Each epilogue warp turns
// its 32 x 32 blocks through a swizzled shared-memory patch, after which eight
// lanes hold eight rows' 64 contiguous bytes and every load and store of the
// epilogue is coalesced.
//
// Operands may be row-major along K or along M / N (the backward products
// read the same tensors transposed): both have a swizzled layout that the
// MMA's descriptors name, so nothing is transposed in memory.
//
// A launch may hold several products (dx and the weights' gradients of a
// backward pass): their tiles are dealt out as one sequence.
//
// Bound by the tensor cores: bf16 8192^3 566 us (1940 TFLOP/s), 4096^3 79 us
// with the tensor pipe active 90 % of the cycles; 256 tiles fill 76 pairs'
// four waves to 84 %.  Where K is short the epilogue shows, its instructions
// and its waits for TMEM and the patch (issue slots 37 % busy): with eight
// warps a 256 x 256 tile takes 2.9 us at K = 128, its K blocks 0.53.  So tiles
// of 256 x 128 columns, the choice for short K and heavy epilogues, have
// sixteen epilogue warps (8192 x 256 to 8192 40 us, 53 with eight; with
// gelu_tanh 57, with bias, residual and kept values too 97); in tiles of 256
// columns their patches cost a stage (4096^3 2 % slower), gate and up would
// need twice the patches.
//
// E4M3 operands: a stage is 128 deep, one scale group.  Each stage's product
// goes to its own TMEM buffer and the epilogue warps add it, times the row's
// and the block's scale, to fp32 accumulators in registers, while the next
// stage is multiplied.  What bounds that is the epilogue warps' wait for TMEM
// (0.45 us a stage, the MMA 0.27), and each tile's own epilogue is exposed:
// 4864 x 8192 x 4096 132 us (2480 TFLOP/s), 8192 x 2048 x 6144 124 us (1660).
// Narrower accumulators (128 columns, four of them) were slower: the MMA then
// reads shared memory faster than it can (0.54 us a stage); sixteen epilogue
// warps have too few registers.
#include "dense.cuh"
#include "dense_tc.cuh"
#include "dense_tile.cuh"
#include "pe_device.cuh"

namespace pe {
namespace dense {

namespace {

// Epilogue warps (warps 4 and on; warp 0 TMA, 1 MMA, 2 TMEM).
constexpr int epi_warps(int kind, bool fp8, int tn) { return fp8 || kind == EPI_GATED || tn == 256 ? 8 : 16; }
constexpr int threads(int kind, bool fp8, int tn) { return 128 + 32 * epi_warps(kind, fp8, tn); }
constexpr int kTile = 256;             // rows of C per CTA pair
constexpr int kHalf = 128;             // of which each CTA has these
constexpr int kOperand = kHalf * 128;  // bytes of A's stage in one CTA
constexpr int kMaxStages = 8;

// TN: columns of C per pair (of gate and up together), 256 or 128.
constexpr int patch_bytes(int kind) { return kind == EPI_GATED ? 8192 : 4096; }
constexpr int stage_bytes(int tn) { return kOperand + tn / 2 * 128; }
constexpr int stages(int kind, bool fp8, int tn) {
    const int n = (225 * 1024 - epi_warps(kind, fp8, tn) * patch_bytes(kind)) / stage_bytes(tn);
    return n < kMaxStages ? n : kMaxStages;
}
constexpr int smem_bytes(int kind, bool fp8, int tn) {
    return 1024 + stages(kind, fp8, tn) * stage_bytes(tn) + epi_warps(kind, fp8, tn) * patch_bytes(kind);
}

// Registers: 128 x (72 + 2 x 216) = 384 x 168, what the block is launched with.
constexpr int kRegsFew = 72, kRegsMany = 216;

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drain;
    uint32_t tmem;
};

// One warp's 32 x 32 fp32 block, lane = row: to the patch, rows of 128 bytes
// whose 16-byte chunks are XOR-swizzled by the row.
__device__ __forceinline__ void patch_put(uint8_t* patch, int lane, const uint32_t (&r)[32]) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
        *reinterpret_cast<uint4*>(patch + lane * 128 + ((j ^ (lane & 7)) << 4)) =
            make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
}

// Products that one launch computes: their tiles are dealt out to the pairs
// as one sequence, so that a product's last wave is filled by the next one's
// tiles.
template <int N>
struct Work {
    CUtensorMap a[N], b[N];
    Product p[N];
    int tiles[N];
    Divide across[N];  // by a product's tiles along its columns
    int count;
    WaitLimits limit;
};

// A pair's way through them: tiles pair, pair + pairs, ...
struct Walk {
    int t, i = 0, base = 0;
    template <int N>
    __device__ __forceinline__ bool find(const Work<N>& w) {
        if (N == 1) return t < w.tiles[0];
        while (i < w.count && t - base >= w.tiles[i]) base += w.tiles[i++];
        return i < w.count;
    }
    // row and column of the tile in its product: kRaster tile rows at a time,
    // down each column of them
    __device__ __forceinline__ void at(const Product& p, const Divide& across, int& m, int& n) const {
        const int tm = (p.M + kTile - 1) / kTile, x = t - base;
        uint32_t r;
        const int first = (int)across((uint32_t)x / kRaster, r) * kRaster, rows = min(kRaster, tm - first);
        const uint32_t in = r * kRaster + x % kRaster;  // of the tile among the group's
        n = (int)(rows == kRaster ? in / kRaster : in / rows);
        m = first + (int)(in - n * rows);
    }
};

// LIMITED: the waits' limits are the launch's.
// NP: products that the launch may hold.  With one, its fields are constants
// of the instructions; found by index they cost 5 % of a large product's time.
template <typename E, int KIND, bool FP8, int TN, int NP, bool LIMITED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(threads(KIND, FP8, TN), 1)
    pair_kernel(const __grid_constant__ Work<NP> work, uint32_t* err) {
    constexpr int STAGES = stages(KIND, FP8, TN), kStage = stage_bytes(TN);
    constexpr int BK = FP8 ? 128 : 64;                      // elements of a 128-byte row
    constexpr int NT = KIND == EPI_GATED ? TN / 2 : TN;  // result columns of a tile
    auto polls = [](uint32_t limit) { return LIMITED ? limit : kPolls; };
    extern __shared__ uint8_t dyn[];
    __shared__ Shared S;
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = tc::cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    Walk walk{pair};

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            tc::mbar_init(&S.full[i], 1);
            tc::mbar_init(&S.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&S.acc_full[i], 1);
            tc::mbar_init(&S.acc_empty[i], 2 * epi_warps(KIND, FP8, TN));  // of both CTAs
        }
        tc::mbar_init(&S.drain, 1);
        tc::fence_barrier_init();
        tc::tma_prefetch(&work.a[0]);
        tc::tma_prefetch(&work.b[0]);
    }
    if (warp == 2) tc::tmem_alloc_pair(&S.tmem, 2 * TN);
    tc::fence_before_sync();
    __syncthreads();
    tc::cluster_arrive_relaxed();
    tc::cluster_wait();
    tc::fence_after_sync();
    const uint32_t tmem = S.tmem;
    pdl_wait();
    if (warp == 3) pdl_trigger();

    if (warp < 4) {
        if (FP8) tc::reg_dec<kRegsFew>();
        if (warp == 0) {
            // ---- producer
            const bool lead = tc::elect_one();
            const uint32_t bar0 = tc::map_rank(tc::smem_u32(&S.full[0]), 0);  // the leader's
            uint32_t s = 0, phase = 1, issued = 0;
            bool ok = true;
            for (; ok && walk.find(work); walk.t += pairs) {
                const Product& p = work.p[NP == 1 ? 0 : walk.i];
                const CUtensorMap &ta = work.a[NP == 1 ? 0 : walk.i], &tb = work.b[NP == 1 ? 0 : walk.i];
                const int kblocks = (p.K + BK - 1) / BK;
                int mt, nt;
                walk.at(p, work.across[NP == 1 ? 0 : walk.i], mt, nt);
                const int m0 = mt * kTile + (int)rank * kHalf;
                const int n0 = KIND == EPI_GATED ? (int)rank * p.e.cols + nt * NT : nt * NT + (int)rank * (TN / 2);
                for (int kb = 0; kb < kblocks; ++kb) {
                    if (!(ok = tc::mbar_spin(&S.empty[s], phase, err, polls(work.limit.copies)))) break;
                    if (lead) {
                        if (rank == 0) tc::mbar_arrive_expect_tx(&S.full[s], 2 * kStage);
                        const uint32_t bar = bar0 + 8 * s;
                        uint8_t* a = ring + s * kStage;
                        uint8_t* b = a + kOperand;
                        if (p.a_mn) {
                            tc::tma_load_2d_pair(a, &ta, bar, m0, kb * BK);
                            tc::tma_load_2d_pair(a + 8192, &ta, bar, m0 + 64, kb * BK);
                        } else {
                            tc::tma_load_2d_pair(a, &ta, bar, kb * BK, m0);
                        }
                        if (p.b_mn) {
                            tc::tma_load_2d_pair(b, &tb, bar, n0, kb * BK);
                            if (TN == 256) tc::tma_load_2d_pair(b + 8192, &tb, bar, n0 + 64, kb * BK);
                        } else {
                            tc::tma_load_2d_pair(b, &tb, bar, kb * BK, n0);
                        }
                    }
                    __syncwarp();
                    ++issued;
                    if (++s == STAGES) s = 0, phase ^= 1;
                }
            }
            // The leader's MMAs arrive on this CTA's barriers: stay until the last of
            // them have (a stage never used passes at once).
            for (int i = 0; ok && i < STAGES; ++i) {
                ok = tc::mbar_spin(&S.empty[s], phase, err, polls(work.limit.copies));
                if (++s == STAGES) s = 0, phase ^= 1;
            }
            // After a wait gave up: let the copies land before the block ends.  The
            // leader's barriers tell of both CTAs' where both asked for a stage.
            if (!ok) {
                bool landed = rank == 0;
                for (uint32_t i = issued > STAGES ? issued - STAGES : 0; landed && i < issued; ++i)
                    landed = tc::mbar_wait(&S.full[i % STAGES], (i / STAGES) & 1, err, PE_DEVERR_TIMEOUT, tc::kLeavePolls);
                if (!landed) tc::settle();
            }
        } else if (warp == 1 && rank == 0) {
            // ---- MMA issuer
            const bool lead = tc::elect_one();
            constexpr int FMT = FP8 ? 0 : std::is_same<E, __nv_bfloat16>::value ? 1 : 0;
            uint32_t s = 0, phase = 0, buf = 0, buf_phase = 1;
            bool ok = true;
            for (; ok && walk.find(work); walk.t += pairs) {
                const Product& p = work.p[NP == 1 ? 0 : walk.i];
                const int kblocks = (p.K + BK - 1) / BK;
                const uint32_t id = tc::idesc(FMT, p.a_mn, p.b_mn, kTile, TN);
                const uint32_t astep = (p.a_mn ? 2048 : 32) >> 4, bstep = (p.b_mn ? 2048 : 32) >> 4;
                const uint64_t a0 = tc::operand_desc(tc::smem_u32(ring), p.a_mn);
                const uint64_t b0 = tc::operand_desc(tc::smem_u32(ring) + kOperand, p.b_mn);
                for (int kb = 0; kb < kblocks; ++kb) {
                    if ((FP8 || kb == 0) && !(ok = tc::mbar_spin(&S.acc_empty[buf], buf_phase, err, polls(work.limit.mma)))) break;
                    if (!(ok = tc::mbar_spin(&S.full[s], phase, err, polls(work.limit.mma)))) break;
                    tc::fence_after_sync();
                    const bool last = FP8 || kb == kblocks - 1;
                    if (lead) {
                        const uint64_t a = a0 + s * (kStage >> 4), b = b0 + s * (kStage >> 4);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            tc::mma<true, FP8>(tmem + buf * TN, a + k * astep, b + k * bstep, id, (!FP8 && kb) || k);
                        tc::mma_commit_pair(&S.empty[s]);
                        if (last) tc::mma_commit_pair(&S.acc_full[buf]);
                    }
                    __syncwarp();
                    if (++s == STAGES) s = 0, phase ^= 1;
                    if (last) {
                        buf ^= 1;
                        if (buf == 0) buf_phase ^= 1;
                    }
                }
            }
            // the other CTA's epilogue warps arrive here too: stay until the last of them have
            for (int i = 0; ok && i < 2; ++i) {
                ok = tc::mbar_spin(&S.acc_empty[buf], buf_phase, err, polls(work.limit.mma));
                buf ^= 1;
                if (buf == 0) buf_phase ^= 1;
            }
            if (!ok) {  // the MMAs already issued read shared memory and write TMEM
                if (lead) tc::mma_commit_pair_here(&S.drain);
                tc::mbar_wait(&S.drain, 0, err, PE_DEVERR_TIMEOUT, tc::kLeavePolls);
            }
        }
    } else {
        // ---- epilogue
        if (FP8) tc::reg_inc<kRegsMany>();
        const int ew = warp - 4, quarter = warp & 3, half = ew >> 2;
        uint8_t* patch = ring + STAGES * kStage + ew * patch_bytes(KIND);
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t release = tc::map_rank(tc::smem_u32(&S.acc_empty[0]), 0);  // of the pair's leader
        uint32_t use_acc = 0;
        bool ok = true;
        for (; ok && walk.find(work); walk.t += pairs) {
            const Product& p = work.p[NP == 1 ? 0 : walk.i];
            const int kblocks = (p.K + BK - 1) / BK;
            int mt, nt;
            walk.at(p, work.across[NP == 1 ? 0 : walk.i], mt, nt);
            const int row0 = mt * kTile + (int)rank * kHalf + quarter * 32;
            if (FP8) {
                uint64_t acc[4][16];  // pairs of fp32
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[c][i] = 0;
                const int row = row0 + lane, nb = (nt * NT + half * 128) / kGroup;
                const bool live = row < p.M && nt * NT + half * 128 < p.N;
                const float* as = p.a_scale + (size_t)(live ? row : 0) * kblocks;
                const float* bs = p.b_scale + (size_t)(live ? nb : 0) * kblocks;
                float next = live ? as[0] * bs[0] : 0.f;
                if (p.e.res && p.e.vec && live) {  // the residual's 256 bytes on their way to L2
                    const uint8_t* rp = static_cast<const uint8_t*>(p.e.res) + 2 * (row * p.e.ld_res + nt * NT + half * 128);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (nt * NT + half * 128 + 64 * i < p.N) asm volatile("prefetch.global.L2 [%0];" ::"l"(rp + 128 * i));
                }
                for (int kb = 0; kb < kblocks && ok; ++kb) {
                    const uint64_t sc = tc::pack2(__float_as_uint(next), __float_as_uint(next));
                    if (kb + 1 < kblocks && live) next = as[kb + 1] * bs[kb + 1];
                    const uint32_t buf = use_acc & 1, at = lanes + buf * TN + half * 128;
                    if (!(ok = tc::mbar_spin(&S.acc_full[buf], (use_acc >> 1) & 1, err, polls(work.limit.sums)))) break;
                    tc::fence_after_sync();
                    ++use_acc;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        // 64 columns at once; the other warp of this scheduler adds while this one reads
                        uint32_t r[2][32];
                        tc::tmem_ld32(at + h * 64, r[0]);
                        tc::tmem_ld32(at + h * 64 + 32, r[1]);
                        tc::tmem_ld_wait(r[0], r[1]);
                        if (h == 1) {
                            tc::fence_before_sync();
                            if (lane == 0) tc::mbar_arrive_cluster(release + 8 * buf);
                        }
#pragma unroll
                        for (int c = 0; c < 2; ++c)
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                acc[2 * h + c][i] = tc::fma2(tc::pack2(r[c][2 * i], r[c][2 * i + 1]), sc, acc[2 * h + c][i]);
                    }
                }
                if (!ok) break;
                const int col0 = nt * NT + half * 128;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    Ahead<E, KIND> x;
                    x.load(p.e, lane, row0, col0 + c * 32);
                    uint32_t o[32];
#pragma unroll
                    for (int i = 0; i < 16; ++i) tc::unpack2(acc[c][i], o[2 * i], o[2 * i + 1]);
                    __syncwarp();
                    patch_put(patch, lane, o);
                    __syncwarp();
                    patch_out<E, KIND>(p.e, patch, lane, row0, col0 + c * 32, x);
                }
            } else {
                const uint32_t buf = use_acc & 1;
                constexpr int SHARE = epi_warps(KIND, FP8, TN) / 4;  // warps that share a tile's columns
                Ahead<E, KIND> x;
                x.load(p.e, lane, row0, nt * NT + half * (NT / SHARE));
                if (!(ok = tc::mbar_spin(&S.acc_full[buf], (use_acc >> 1) & 1, err, polls(work.limit.sums)))) break;
                ++use_acc;
                tc::fence_after_sync();
                constexpr int CH = NT / SHARE / 32;  // 32-column chunks of this warp's share
                const int c0 = half * (NT / SHARE);
                const uint32_t at = lanes + buf * TN + c0;
#pragma unroll 1
                for (int c = 0; c < CH; ++c) {
                    uint32_t r[32];
                    tc::tmem_ld32(at + c * 32, r);
                    tc::tmem_ld_wait(r);
                    __syncwarp();  // the patch's last readers are done
                    patch_put(patch, lane, r);
                    if (KIND == EPI_GATED) {
                        tc::tmem_ld32(at + TN / 2 + c * 32, r);
                        tc::tmem_ld_wait(r);
                        patch_put(patch + 4096, lane, r);
                    }
                    if (c == CH - 1) {
                        tc::fence_before_sync();
                        if (lane == 0) tc::mbar_arrive_cluster(release + 8 * buf);
                    }
                    __syncwarp();
                    patch_out<E, KIND>(p.e, patch, lane, row0, nt * NT + c0 + c * 32, x);
                    if (c + 1 < CH) x.load(p.e, lane, row0, nt * NT + c0 + (c + 1) * 32);
                }
            }
        }
    }
    // neither CTA leaves, and no TMEM is freed, while the other may still use it
    // (what each sends to the other's barriers was waited for above, so that
    // the meeting has nothing to order)
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::cluster_arrive_relaxed();
    tc::cluster_wait();
    tc::fence_after_sync();
    if (warp == 2) tc::tmem_dealloc_pair(tmem, 2 * TN);
}

// Pairs that the device holds at once, looked up once per kernel.
template <typename E, int KIND, bool FP8, int TN, int NP, bool LIMITED>
cudaError_t resident_pairs(int* out) {
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    int n = dev < 64 ? known[dev].load() : 0;
    if (!n) {
        auto k = pair_kernel<E, KIND, FP8, TN, NP, LIMITED>;
        if (cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(KIND, FP8, TN))) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(threads(KIND, FP8, TN));
        cfg.dynamicSmemBytes = smem_bytes(KIND, FP8, TN);
        if (cudaError_t e = cudaOccupancyMaxActiveClusters(&n, k, &cfg)) return e;
        if (n < 1) return cudaErrorLaunchOutOfResources;
        if (dev < 64) known[dev].store(n);
    }
    *out = n;
    return cudaSuccess;
}

template <typename E, int KIND, bool FP8, int TN, int NP = 1, bool LIMITED = false>
cudaError_t launch(const Product* p, int count, uint32_t* err, cudaStream_t st, const WaitLimits& limits = {}) {
    if (count < 1 || count > NP) return cudaErrorInvalidValue;
    Work<NP> w;
    w.count = count;
    w.limit = limits;
    long long tiles = 0;
    for (int i = 0; i < count; ++i) {
        if (!encode_operand(&w.a[i], p[i].a, p[i].lda, p[i].M, p[i].K, p[i].a_mn, FP8, kHalf) ||
            !encode_operand(&w.b[i], p[i].b, p[i].ldb, p[i].N, p[i].K, p[i].b_mn, FP8, TN / 2))
            return cudaErrorInvalidValue;
        w.p[i] = p[i];
        constexpr int NT = KIND == EPI_GATED ? TN / 2 : TN;
        const long long n = (long long)((p[i].M + kTile - 1) / kTile) * ((p[i].e.cols + NT - 1) / NT);
        if ((tiles += n) > INT_MAX / 2) return cudaErrorInvalidValue;
        w.tiles[i] = (int)n;
        w.across[i] = Divide::by((p[i].e.cols + NT - 1) / NT);
    }
    int pairs = 0;
    if (cudaError_t e = resident_pairs<E, KIND, FP8, TN, NP, LIMITED>(&pairs)) return e;
    if (tiles < pairs) pairs = (int)tiles;
    return launch_pdl(pair_kernel<E, KIND, FP8, TN, NP, LIMITED>, dim3(2 * pairs), dim3(threads(KIND, FP8, TN)), smem_bytes(KIND, FP8, TN), st, w, err);
}

template <typename E>
cudaError_t launch_kind(const Product* p, int count, EpiKind kind, int tn, uint32_t* err, cudaStream_t st) {
    if (p->a_scale) return launch<E, EPI_LINEAR, true, 256>(p, count, err, st);
    if (count > 1 && kind == EPI_LINEAR)
        return tn == 256 ? launch<E, EPI_LINEAR, false, 256, kMostProducts>(p, count, err, st)
                         : launch<E, EPI_LINEAR, false, 128, kMostProducts>(p, count, err, st);
    if (kind == EPI_LINEAR)
        return tn == 256 ? launch<E, EPI_LINEAR, false, 256>(p, count, err, st)
                         : launch<E, EPI_LINEAR, false, 128>(p, count, err, st);
    if (kind == EPI_SCALED)
        return tn == 256 ? launch<E, EPI_SCALED, false, 256>(p, count, err, st)
                         : launch<E, EPI_SCALED, false, 128>(p, count, err, st);
    if (kind == EPI_GATED)
        return tn == 256 ? launch<E, EPI_GATED, false, 256>(p, count, err, st)
                         : launch<E, EPI_GATED, false, 128>(p, count, err, st);
    return tn == 256 ? launch<E, EPI_GATED_BWD, false, 256>(p, count, err, st)
                     : launch<E, EPI_GATED_BWD, false, 128>(p, count, err, st);
}

}  // namespace

namespace {
using PFN_encode = PFN_cuTensorMapEncodeTiled_v12000;
PFN_encode encode_fn() {
    static PFN_encode fn = [] {
        void* q = nullptr;
        cudaDriverEntryPointQueryResult r;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &q, 12000, cudaEnableDefault, &r);
        return e == cudaSuccess && r == cudaDriverEntryPointSuccess ? reinterpret_cast<PFN_encode>(q) : nullptr;
    }();
    return fn;
}
}  // namespace

bool encode_boxes(CUtensorMap* m, const void* base, int rank, const uint64_t* dims, const uint64_t* strides, const uint32_t* box,
                  bool fp8) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint32_t step[3] = {1, 1, 1};
    // the type only sizes the elements: nothing is converted on the way
    return fn(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, rank, const_cast<void*>(base), dims,
              strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_operand(CUtensorMap* m, const void* base, int64_t ld, int rows, int k, bool mn, bool fp8, int box_rows) {
    const uint64_t dims[2] = {(uint64_t)(mn ? rows : k), (uint64_t)(mn ? k : rows)}, strides[1] = {(uint64_t)ld * (fp8 ? 1 : 2)};
    const uint32_t box[2] = {fp8 ? 128u : 64u, mn ? 64u : (uint32_t)box_rows};
    return encode_boxes(m, base, 2, dims, strides, box, fp8);
}

cudaError_t launch_pairs(const Product* p, int count, EpiKind kind, int elem, int tn, uint32_t* err, cudaStream_t st,
                         const WaitLimits* limits) {
    if (limits)
        return p->a_scale ? launch<__nv_bfloat16, EPI_LINEAR, true, 256, 1, true>(p, count, err, st, *limits)
                          : launch<__nv_bfloat16, EPI_LINEAR, false, 256, 1, true>(p, count, err, st, *limits);
    return elem == PE_ELEM_BF16 ? launch_kind<__nv_bfloat16>(p, count, kind, tn, err, st)
                                : launch_kind<__half>(p, count, kind, tn, err, st);
}

}  // namespace dense
}  // namespace pe
