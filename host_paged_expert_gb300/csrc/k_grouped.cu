// Matrix products grouped by expert: rows offsets[g] .. offsets[g + 1] - 1
// meet the weights of expert g, ragged groups and empty ones among them.
//
// Features lie along the MMA's M and rows along its N, which goes in steps of
// 32: experts of a layer have some tens or hundreds of rows each, of which
// tiles of 256 rows along M would leave half unused.  Persistent CTA pairs take
// tiles of 256 features (128 of gate and 128 of up) x up to 256 rows of one
// group; a group's rows are shared out evenly over the fewest tiles.  Each CTA
// streams its half of both operands (TMA, 128-byte swizzle) into a ring of
// stages; one thread of the pair's leader issues the MMAs; accumulators live
// in TMEM, two buffers of 256 columns, so that the epilogue of a tile runs
// under the next one's products.  An epilogue warp holds 32 features x 32 rows
// with a feature per lane and turns them through a patch of shared memory, as
// the dense products' kernel does, with the block transposed on its way in.
//
// Offsets are on the device: every CTA makes a table of the groups' tiles for
// itself and walks it, 32 groups a look.  They are clamped to [0, rows] and
// never decrease, whatever they hold, so no access leaves the operands.
//
// Weights' gradients (GROUP_WEIGHTS) sum over a group's rows, which lie along
// K.  The last block of 64 rows runs into the next group, whose rows may hold
// anything: a warp of each CTA zeroes what is not the group's, in both operands,
// before the leader may multiply.  The result of an empty group is zeros.
//
// Bound by HBM where experts have few rows: 128 experts of 2048 x 768, 2048 x 8
// rows, gate, up and down 218 us (1.21 GB of weights; 91 % of the copy's rate
// with the rows), 4 x 8 rows through 2048 to 1536 28 us (183 MB).  With 4096 x 8
// rows: gate and up 178 us, kept in fp32 too 208; down 102; dg, du and h 137; dx
// 178; dW13 228 and dW2 122 (tensor pipe active 39 % of the time: tiles of many
// rows are bound by their MMAs, of few by their stores; 175 us for dW13 with 256
// rows each).  A block of 64 of a full tile takes 540 cycles, in which each SM
// takes in 32 KB, about what it can.
#include "experts.cuh"
#include "dense_tc.cuh"
#include "dense_tile.cuh"
#include "pe_device.cuh"

namespace pe {
namespace dense {
namespace {

constexpr int kEpiWarps = 8, kThreads = 128 + 32 * kEpiWarps;  // warp 0 TMA, 1 MMA, 2 TMEM, 3 clears tails, 4..11 epilogue
constexpr int kTile = 256, kHalf = 128;  // features (and rows, at most) of a pair's tile, of a CTA's share
constexpr int kOperand = kHalf * 128, kStage = 2 * kOperand;
constexpr int kMaxStages = 6;
constexpr int kBox = 32;  // rows of a copy of the rows' operand
constexpr int kSmem = 227 * 1024;

constexpr int patch_bytes(int kind) { return kind == GROUP_GATED ? 8192 : 4096; }  // of a warp

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages], raw[kMaxStages], acc_full[2], acc_empty[2], drain;
    uint32_t tmem;
};

struct Work {
    CUtensorMap w, x;
    CUtensorMap w_tail, x_tail, out;  // GROUP_WEIGHTS: boxes of 16 rows, the result
    const int32_t* offsets;
    int groups, rows, features, depth, w_mn;
    int ftiles;        // tiles along the features
    int ntiles;        // GROUP_WEIGHTS: along the other side
    Divide across;     // by ftiles (GROUP_WEIGHTS: by a group's tiles)
    Divide down;       // GROUP_WEIGHTS: by ftiles
    int stages;
    WaitLimits limit;
    Epi e;
};

// One tile: group, feature tile, first row (GROUP_WEIGHTS: first column of the
// other side), the group's end, and the MMA's N.
struct Tile {
    int g, f, n0, end, nt;
    int k0, kn;  // first row along K (GROUP_WEIGHTS; else 0) and the depth
};

// Rows of a group's tiles: shared out evenly over the fewest of them.
__device__ __forceinline__ int tile_rows(int rows) {
    const int tiles = (rows + kTile - 1) / kTile;
    return tiles <= 1 ? (rows + 31) / 32 * 32 : ((rows + tiles - 1) / tiles + 31) / 32 * 32;
}

struct Table {
    int32_t *off, *end;  // rows ahead of each group; tiles up to each group's end
};

// A pair's way through the tiles: every `pairs`-th, group by group.  (Dealt out
// evenly by size, from large to small or large and small in turn, they took as
// long or longer: it is the mixture of tiles bound by the tensor cores with
// tiles bound by their stores that counts.)
template <int KIND>
struct Walk {
    Table tab;
    int t, pairs, i = 0;
    __device__ __forceinline__ void next() { t += pairs; }
    __device__ __forceinline__ bool find(const Work& w, int lane) {
        if constexpr (KIND == GROUP_WEIGHTS) {
            return t < w.groups * (w.ftiles * w.ntiles);
        } else {
            for (; i < w.groups; i += 32) {
                const uint32_t past = __ballot_sync(0xffffffffu, i + lane < w.groups && tab.end[i + lane] > t);
                if (past) {
                    i += __ffs(past) - 1;
                    return true;
                }
            }
            return false;
        }
    }
    __device__ __forceinline__ Tile at(const Work& w) const {
        Tile r;
        uint32_t rest;
        if (KIND == GROUP_WEIGHTS) {
            r.g = (int)w.across((uint32_t)t, rest);
            uint32_t f;
            r.n0 = (int)w.down(rest, f) * kTile;
            r.f = (int)f;
            r.k0 = tab.off[r.g], r.kn = tab.off[r.g + 1] - r.k0;
            r.end = w.depth;
            r.nt = min(kTile, (w.depth - r.n0 + 31) / 32 * 32);
            return r;
        }
        r.g = i;
        const int r0 = tab.off[i], r1 = tab.off[i + 1], rows = r1 - r0, tiles = (rows + kTile - 1) / kTile;
        const int x = t - (i ? tab.end[i - 1] : 0);
        // kRaster row tiles at a time, across all features
        const int first = (int)w.across((uint32_t)x / kRaster, rest) * kRaster, n = min(kRaster, tiles - first);
        const uint32_t in = rest * kRaster + x % kRaster;
        r.f = (int)(n == kRaster ? in / kRaster : in / n);
        r.nt = tile_rows(rows);
        r.n0 = r0 + (first + (int)(in - r.f * n)) * r.nt;
        r.end = r1;
        r.k0 = 0, r.kn = w.depth;
        return r;
    }
};

// A tail's block is copied kEarly blocks ahead of its turn, so that it is clear
// by then: the place among a tile's copies of its last block.
constexpr int kEarly = 3;
template <bool WEIGHTS>
__device__ __forceinline__ int early_at(int depth) {
    const int last = (depth + 63) / 64 - 1;
    return WEIGHTS && depth % 64 ? max(0, last - kEarly) : last;
}

// A warp's 32 features x 32 rows, lane = feature: to the patch, a row of the
// result per 128 bytes (the layout of patch_get).
__device__ __forceinline__ void patch_put_t(uint8_t* patch, int lane, const uint32_t (&r)[32]) {
    const uint32_t in = (lane & 3) * 4, chunk = lane >> 2;
#pragma unroll
    for (int j = 0; j < 32; ++j) *reinterpret_cast<uint32_t*>(patch + j * 128 + ((chunk ^ (j & 7)) << 4) + in) = r[j];
}

// By one warp: offsets, clamped and never decreasing, and tiles up to each
// group's end.
__device__ __forceinline__ void make_table(const Work& w, const Table& tab, int lane) {
    int high = min(max(w.offsets[0], 0), w.rows), tiles = 0;
    if (lane == 0) tab.off[0] = high;
    for (int b = 0; b < w.groups; b += 32) {
        const int i = b + lane;
        int v = i < w.groups ? min(w.offsets[i + 1], w.rows) : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v = max(v, n);
        }
        v = max(v, high);
        int before = __shfl_up_sync(0xffffffffu, v, 1);
        if (lane == 0) before = high;
        int n = i < w.groups ? (v - before + kTile - 1) / kTile * w.ftiles : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int m = __shfl_up_sync(0xffffffffu, n, o);
            if (lane >= o) n += m;
        }
        n += tiles;
        if (i < w.groups) tab.off[i + 1] = v, tab.end[i] = n;
        high = __shfl_sync(0xffffffffu, v, 31);
        tiles = __shfl_sync(0xffffffffu, n, 31);
    }
}

// Named barrier of two warps that exchange gate and up; true if `ok` of both.
__device__ __forceinline__ bool couple_and(int id, bool ok) {
    int r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %2, 0;\n\t"
        "barrier.cta.red.and.pred.aligned q, %1, 64, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"((int)ok)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void couple_sync(int id) { asm volatile("barrier.cta.sync.aligned %0, 64;" ::"r"(id) : "memory"); }

// What the epilogue of a warp's 32 x 32 block reads, asked for before the
// block's accumulators are there, and what it does with them: nothing but
// rounding, or (GROUP_GATED_BWD) the gradients of gate and up and h from dh and
// the fp32 gate and up that the forward call kept.
template <typename E, int KIND>
struct Before {
    __device__ __forceinline__ void load(const Epi&, int, int, int) {}
    __device__ __forceinline__ void out(const Epi& e, const uint8_t* patch, int lane, int row0, int col0) const {
        const int c8 = lane & 3, col = col0 + 8 * c8;
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            const int rr = it * 8 + (lane >> 2), row = row0 + rr;
            float v[8];
            patch_get(patch, rr, c8, v);
            if (row < e.rows && col < e.cols) store8(static_cast<E*>(e.out) + row * e.ld_out + col, true, 8, v);
        }
    }
};
template <typename E>
struct Before<E, GROUP_GATED_BWD> {
    float4 g[4][2], u[4][2];
    __device__ __forceinline__ void load(const Epi& e, int lane, int row0, int col0) {
        const int col = col0 + 8 * (lane & 3);
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            const int row = row0 + it * 8 + (lane >> 2);
            if (row >= e.rows || col >= e.cols) continue;
            const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(e.gu) + row * e.ld_keep + col);
            const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(e.gu) + row * e.ld_keep + e.cols + col);
            g[it][0] = p[0], g[it][1] = p[1], u[it][0] = q[0], u[it][1] = q[1];
        }
    }
    __device__ __forceinline__ void out(const Epi& e, const uint8_t* patch, int lane, int row0, int col0) const {
        const int c8 = lane & 3, col = col0 + 8 * c8;
        with_act(e.act, [&](auto act) {
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const int rr = it * 8 + (lane >> 2), row = row0 + rr;
                if (row >= e.rows || col >= e.cols) continue;
                float v[8];
                patch_get(patch, rr, c8, v);
                float a[8] = {g[it][0].x, g[it][0].y, g[it][0].z, g[it][0].w, g[it][1].x, g[it][1].y, g[it][1].z, g[it][1].w};
                float b[8] = {u[it][0].x, u[it][0].y, u[it][0].z, u[it][0].w, u[it][1].x, u[it][1].y, u[it][1].z, u[it][1].w};
                float d[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    a[i] = act_both(decltype(act)::value, a[i], d[i]);
                    d[i] *= v[i] * b[i];  // dg
                    b[i] *= a[i];         // h
                    a[i] *= v[i];         // du
                }
                E* o = static_cast<E*>(e.out) + row * e.ld_out + col;
                store8(o, true, 8, d);
                store8(o + e.cols, true, 8, a);
                if (e.h) store8(static_cast<E*>(e.h) + row * (int64_t)e.cols + col, true, 8, b);
            }
        });
    }
};

// LIMITED: the waits' limits are the launch's.
template <typename E, int KIND, bool LIMITED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) grouped_kernel(const __grid_constant__ Work w, uint32_t* err) {
    constexpr bool WEIGHTS = KIND == GROUP_WEIGHTS, GATED = KIND == GROUP_GATED;
    constexpr int BK = 64;
    auto polls = [](uint32_t limit) { return LIMITED ? limit : kPolls; };
    extern __shared__ uint8_t dyn[];
    __shared__ Shared S;
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~(uintptr_t)1023);
    uint8_t* patches = ring + w.stages * kStage;
    int32_t* off = reinterpret_cast<int32_t*>(patches + kEpiWarps * patch_bytes(KIND));
    const Table tab = {off, off + w.groups + 1};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = tc::cluster_rank();
    Walk<KIND> walk{tab, (int)(blockIdx.x >> 1), (int)(gridDim.x >> 1)};

    if (threadIdx.x == 0) {
        for (int i = 0; i < w.stages; ++i) {
            tc::mbar_init(&S.full[i], WEIGHTS ? 2 : 1);
            tc::mbar_init(&S.empty[i], 1);
            tc::mbar_init(&S.raw[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&S.acc_full[i], 1);
            tc::mbar_init(&S.acc_empty[i], 2 * kEpiWarps);
        }
        tc::mbar_init(&S.drain, 1);
        tc::fence_barrier_init();
        tc::tma_prefetch(&w.w);
        tc::tma_prefetch(&w.x);
    }
    if (warp == 2) tc::tmem_alloc_pair(&S.tmem, 512);
    pdl_wait();
    if (warp == 3) {
        make_table(w, tab, lane);
        pdl_trigger();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::cluster_arrive_relaxed();
    tc::cluster_wait();
    tc::fence_after_sync();
    const uint32_t tmem = S.tmem;

    if (warp == 0) {
        // ---- producer
        const bool lead = tc::elect_one();
        const uint32_t bar0 = tc::map_rank(tc::smem_u32(&S.full[0]), 0);  // the leader's
        uint32_t s = 0, phase = 1;
        bool ok = true;
        for (; ok && walk.find(w, lane); walk.next()) {
            const Tile tl = walk.at(w);
            const int f0 = GATED ? tl.f * kHalf + (int)rank * 64 : tl.f * kTile + (int)rank * kHalf;
            const int f1 = GATED ? w.features + f0 : f0 + 64;
            const int n0 = tl.n0 + (int)rank * (tl.nt / 2), boxes = (tl.nt / 2 + kBox - 1) / kBox;
            const int blocks = (tl.kn + BK - 1) / BK, early = early_at<WEIGHTS>(tl.kn);
            for (int j = 0; j < blocks; ++j) {
                const int k = (!WEIGHTS || j < early ? j : j == early ? blocks - 1 : j - 1) * BK;
                if (!(ok = tc::mbar_spin(&S.empty[s], phase, err, polls(w.limit.copies)))) break;
                if (lead) {
                    uint8_t* a = ring + s * kStage;
                    uint8_t* b = a + kOperand;
                    const uint32_t bar = bar0 + 8 * s;
                    if (WEIGHTS) {
                        const int kk = tl.k0 + k;
                        if (tl.kn - k >= BK) {
                            if (rank == 0) tc::mbar_arrive_expect_tx(&S.full[s], 2 * kStage);
                            else tc::mbar_arrive_cluster(bar);
                            tc::tma_load_2d_pair(a, &w.w, bar, f0, kk);
                            tc::tma_load_2d_pair(a + 8192, &w.w, bar, f0 + 64, kk);
                            tc::tma_load_2d_pair(b, &w.x, bar, n0, kk);
                            tc::tma_load_2d_pair(b + 8192, &w.x, bar, n0 + 64, kk);
                        } else {  // for the warp that clears the tail: as many rows as the MMAs will read
                            const int steps = (tl.kn - k + 15) / 16;
                            tc::mbar_arrive_expect_tx(&S.raw[s], steps * 4 * 2048);
                            for (int i = 0; i < steps; ++i) {
                                tc::tma_load_2d(a + i * 2048, &w.w_tail, &S.raw[s], f0, kk + 16 * i);
                                tc::tma_load_2d(a + i * 2048 + 8192, &w.w_tail, &S.raw[s], f0 + 64, kk + 16 * i);
                                tc::tma_load_2d(b + i * 2048, &w.x_tail, &S.raw[s], n0, kk + 16 * i);
                                tc::tma_load_2d(b + i * 2048 + 8192, &w.x_tail, &S.raw[s], n0 + 64, kk + 16 * i);
                            }
                        }
                    } else {
                        if (rank == 0) tc::mbar_arrive_expect_tx(&S.full[s], 2 * (kOperand + boxes * kBox * 128));
                        if (w.w_mn) {
                            tc::tma_load_3d_pair(a, &w.w, bar, f0, k, tl.g);
                            tc::tma_load_3d_pair(a + 8192, &w.w, bar, f1, k, tl.g);
                        } else {
                            tc::tma_load_3d_pair(a, &w.w, bar, k, f0, tl.g);
                            tc::tma_load_3d_pair(a + 8192, &w.w, bar, k, f1, tl.g);
                        }
                        for (int i = 0; i < boxes; ++i) tc::tma_load_2d_pair(b + i * kBox * 128, &w.x, bar, k, n0 + i * kBox);
                    }
                }
                __syncwarp();
                if (++s == (uint32_t)w.stages) s = 0, phase ^= 1;
            }
        }
        // The leader's MMAs arrive on this CTA's barriers: stay until the last of
        // them have (a stage never used passes at once).
        for (int i = 0; ok && i < w.stages; ++i) {
            ok = tc::mbar_spin(&S.empty[s], phase, err, polls(w.limit.copies));
            if (++s == (uint32_t)w.stages) s = 0, phase ^= 1;
        }
        if (!ok) tc::settle();  // copies may be on their way
    } else if (warp == 1 && rank == 0) {
        // ---- MMA issuer
        const bool lead = tc::elect_one();
        constexpr int FMT = std::is_same<E, __nv_bfloat16>::value ? 1 : 0;
        const int a_mn = WEIGHTS || w.w_mn, b_mn = WEIGHTS;
        const uint32_t astep = (a_mn ? 2048 : 32) >> 4, bstep = (b_mn ? 2048 : 32) >> 4;
        const uint64_t a0 = tc::operand_desc(tc::smem_u32(ring), a_mn), b0 = tc::operand_desc(tc::smem_u32(ring) + kOperand, b_mn);
        uint32_t s = 0, phase = 0, buf = 0, buf_phase = 1;
        bool ok = true;
        for (; ok && walk.find(w, lane); walk.next()) {
            const Tile tl = walk.at(w);
            if (tl.kn <= 0) continue;  // zeros
            const uint32_t id = tc::idesc(FMT, a_mn, b_mn, kTile, tl.nt);
            if (!(ok = tc::mbar_spin(&S.acc_empty[buf], buf_phase, err, polls(w.limit.mma)))) break;
            const int blocks = (tl.kn + BK - 1) / BK, early = early_at<WEIGHTS>(tl.kn);
            uint32_t s_tail = 0, phase_tail = 0;
            for (int j = 0; j < blocks; ++j) {
                if (WEIGHTS && j == early && j < blocks - 1) {  // the tail's stage: at the end
                    s_tail = s, phase_tail = phase;
                    if (++s == (uint32_t)w.stages) s = 0, phase ^= 1;
                }
                const bool last = j == blocks - 1, late = WEIGHTS && last && early < blocks - 1;
                const uint32_t at = late ? s_tail : s, ph = late ? phase_tail : phase;
                const uint32_t limit = polls(w.limit.mma);
                if (!(ok = WEIGHTS ? tc::mbar_spin_cluster(&S.full[at], ph, err, limit) : tc::mbar_spin(&S.full[at], ph, err, limit))) break;
                tc::fence_after_sync();
                if (lead) {
                    const uint64_t a = a0 + at * (kStage >> 4), b = b0 + at * (kStage >> 4);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (!WEIGHTS || !last || j * BK + 16 * i < tl.kn)
                            tc::mma<true, false>(tmem + buf * kTile, a + i * astep, b + i * bstep, id, j || i);
                    tc::mma_commit_pair(&S.empty[at]);
                    if (last) tc::mma_commit_pair(&S.acc_full[buf]);
                }
                __syncwarp();
                if (!late && ++s == (uint32_t)w.stages) s = 0, phase ^= 1;
            }
            buf ^= 1;
            if (buf == 0) buf_phase ^= 1;
        }
        // the other CTA's epilogue warps arrive here too: stay until the last of them have
        for (int i = 0; ok && i < 2; ++i) {
            ok = tc::mbar_spin(&S.acc_empty[buf], buf_phase, err, polls(w.limit.mma));
            buf ^= 1;
            if (buf == 0) buf_phase ^= 1;
        }
        if (!ok) {  // the MMAs already issued read shared memory and write TMEM
            if (lead) tc::mma_commit_pair_here(&S.drain);
            tc::mbar_wait(&S.drain, 0, err, PE_DEVERR_TIMEOUT, tc::kLeavePolls);
        }
    } else if (WEIGHTS && warp == 3) {
        // ---- tails: rows of the next group, up to the MMA's step of 16, become zeros
        const uint32_t bar0 = tc::map_rank(tc::smem_u32(&S.full[0]), 0);
        uint32_t s = 0, phases = 0;
        bool ok = true;
        for (; ok && walk.find(w, lane); walk.next()) {
            const Tile tl = walk.at(w);
            const int blocks = (tl.kn + BK - 1) / BK, rem = tl.kn % BK;
            if (rem) {
                const uint32_t at = (s + early_at<true>(tl.kn)) % w.stages;
                if (!(ok = tc::mbar_spin(&S.raw[at], phases >> at & 1, err, polls(w.limit.copies)))) break;
                phases ^= 1u << at;
                // a row along K is 128 bytes of each of four boxes
                uint8_t* to = ring + at * kStage + (lane >> 3) * 8192 + (lane & 7) * 16;
                for (int r = rem; r < (rem + 15) / 16 * 16; ++r) *reinterpret_cast<uint4*>(to + r * 128) = make_uint4(0, 0, 0, 0);
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive_cluster_release(bar0 + 8 * at);
            }
            s = (s + blocks) % w.stages;
        }
    } else if (warp >= 4) {
        // ---- epilogue
        const int ew = warp - 4, quarter = warp & 3, half = ew >> 2;
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t release = tc::map_rank(tc::smem_u32(&S.acc_empty[0]), 0);  // of the pair's leader
        uint32_t use_acc = 0;
        bool ok = true;
        for (; walk.find(w, lane); walk.next()) {
            const Tile tl = walk.at(w);
            const uint32_t buf = use_acc & 1, at = lanes + buf * kTile;
            auto let_go = [&] {
                tc::fence_before_sync();
                if (lane == 0) tc::mbar_arrive_cluster(release + 8 * buf);
            };
            if constexpr (WEIGHTS) {
                // boxes of 32 rows (lane = row) x 64 columns, swizzled as the map has
                // it, stored by TMA, which leaves out what is past the result
                const int m = tl.f * kTile + (int)rank * kHalf + quarter * 32;
                if (tl.kn > 0) {
                    if (!(ok = tc::mbar_spin(&S.acc_full[buf], (use_acc >> 1) & 1, err, polls(w.limit.sums)))) break;
                    ++use_acc;
                    tc::fence_after_sync();
                }
#pragma unroll 1
                for (int c = 0; c < kHalf; c += 64) {
                    uint32_t r[64];
                    if (tl.kn > 0) {
                        uint32_t q[2][32];
                        tc::tmem_ld32(at + half * kHalf + c, q[0]);
                        tc::tmem_ld32(at + half * kHalf + c + 32, q[1]);
                        tc::tmem_ld_wait(q[0], q[1]);
                        if (c + 64 == kHalf) let_go();
#pragma unroll
                        for (int j = 0; j < 64; ++j) r[j] = q[j / 32][j % 32];
                    } else {
#pragma unroll
                        for (int j = 0; j < 64; ++j) r[j] = 0;
                    }
                    const int col = tl.n0 + half * kHalf + c;
                    if (m >= w.features || col >= w.depth) continue;
                    uint8_t* patch = patches + ew * patch_bytes(KIND);
                    if (lane == 0) tc::tma_store_read<0>();
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        uint4 v;
                        v.x = Elem<E>::pack(__uint_as_float(r[8 * j]), __uint_as_float(r[8 * j + 1]));
                        v.y = Elem<E>::pack(__uint_as_float(r[8 * j + 2]), __uint_as_float(r[8 * j + 3]));
                        v.z = Elem<E>::pack(__uint_as_float(r[8 * j + 4]), __uint_as_float(r[8 * j + 5]));
                        v.w = Elem<E>::pack(__uint_as_float(r[8 * j + 6]), __uint_as_float(r[8 * j + 7]));
                        *reinterpret_cast<uint4*>(patch + lane * 128 + ((j ^ (lane & 7)) << 4)) = v;
                    }
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) tc::tma_store_3d(&w.out, patch, col, m, tl.g);
                }
            } else {
                Epi e = w.e;
                e.rows = tl.end;
                const int live = min(tl.nt, tl.end - tl.n0);  // rows of this tile
                ok = tc::mbar_spin(&S.acc_full[buf], (use_acc >> 1) & 1, err, polls(w.limit.sums));
                const int couple = 1 + half * 2 + (quarter & 1);
                if (GATED) ok = couple_and(couple, ok);
                if (!ok) break;
                ++use_acc;
                tc::fence_after_sync();
                if (half * 32 >= live) let_go();
                if constexpr (GATED) {
                    const int f = tl.f * kHalf + (int)rank * 64 + (quarter & 1) * 32, part = quarter >> 1;
                    uint8_t* mine = patches + (couple - 1) * (2 * patch_bytes(KIND));
                    uint32_t turn = 0;
#pragma unroll 1
                    for (int c = half * 32; c < live; c += 64, turn ^= 8192) {
                        uint32_t r[32];
                        tc::tmem_ld32(at + c, r);
                        tc::tmem_ld_wait(r);
                        if (c + 64 >= live) let_go();
                        patch_put_t(mine + turn + part * 4096, lane, r);
                        couple_sync(couple);  // two patches in turn: the partner may still read the other one
                        const int c8 = lane & 3, col = f + 8 * c8;
                        with_act(e.act, [&](auto act) {
#pragma unroll
                            for (int it = 0; it < 2; ++it) {
                                const int rr = (2 * part + it) * 8 + (lane >> 2);
                                float v[8], u[8];
                                patch_get(mine + turn, rr, c8, v);
                                patch_get(mine + turn + 4096, rr, c8, u);
                                const int row = tl.n0 + c + rr;
                                if (row >= e.rows || col >= e.cols) continue;
                                if (e.keep) {
                                    float* k = static_cast<float*>(e.keep) + row * e.ld_keep + col;
                                    store8_f32(k, true, 8, v);
                                    store8_f32(k + e.cols, true, 8, u);
                                }
#pragma unroll
                                for (int j = 0; j < 8; ++j) v[j] = act_fwd(decltype(act)::value, v[j]) * u[j];
                                store8(static_cast<E*>(e.out) + row * e.ld_out + col, true, 8, v);
                            }
                        });
                    }
                    couple_sync(couple);  // nor may the next tile's first patch meet its readers
                } else {
                    const int f = tl.f * kTile + (int)rank * kHalf + quarter * 32;
                    uint8_t* patch = patches + ew * patch_bytes(KIND);
#pragma unroll 1
                    for (int c = half * 32; c < live; c += 64) {
                        Before<E, KIND> x;
                        x.load(e, lane, tl.n0 + c, f);
                        uint32_t r[32];
                        tc::tmem_ld32(at + c, r);
                        tc::tmem_ld_wait(r);
                        if (c + 64 >= live) let_go();
                        __syncwarp();  // the patch's last readers are done
                        patch_put_t(patch, lane, r);
                        __syncwarp();
                        x.out(e, patch, lane, tl.n0 + c, f);
                    }
                }
            }
        }
    }
    if (WEIGHTS && warp >= 4 && lane == 0) tc::tma_store_done();
    // neither CTA leaves, and no TMEM is freed, while the other may still use it
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::cluster_arrive_relaxed();
    tc::cluster_wait();
    tc::fence_after_sync();
    if (warp == 2) tc::tmem_dealloc_pair(tmem, 512);
}

int table_bytes(int groups) { return 4 * (2 * groups + 1); }
// Stages of the ring that fit next to the patches and the table.
int stages_of(GroupKind kind, int groups) {
    const int room = kSmem - 1024 - (int)sizeof(Shared) - kEpiWarps * patch_bytes(kind) - table_bytes(groups);
    return room / kStage < kMaxStages ? room / kStage : kMaxStages;
}

// Pairs that the device holds at once, looked up once per kernel.
template <typename E, int KIND, bool LIMITED>
cudaError_t resident_pairs(int* out) {
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    int n = dev < 64 ? known[dev].load() : 0;
    if (!n) {
        auto k = grouped_kernel<E, KIND, LIMITED>;
        const int bytes = kSmem - (int)sizeof(Shared);
        if (cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = bytes;
        if (cudaError_t e = cudaOccupancyMaxActiveClusters(&n, k, &cfg)) return e;
        if (n < 1) return cudaErrorLaunchOutOfResources;
        if (dev < 64) known[dev].store(n);
    }
    *out = n;
    return cudaSuccess;
}

template <typename E, int KIND, bool LIMITED = false>
cudaError_t launch(const Grouped& p, uint32_t* err, cudaStream_t st, const WaitLimits& limits = {}) {
    constexpr bool WEIGHTS = KIND == GROUP_WEIGHTS;
    constexpr int NF = KIND == GROUP_GATED ? kHalf : kTile;
    Work w = {};
    if (WEIGHTS) {
        const uint64_t wd[2] = {(uint64_t)p.features, (uint64_t)p.rows}, ws[1] = {2 * (uint64_t)p.ld_w};
        const uint64_t xd[2] = {(uint64_t)p.depth, (uint64_t)p.rows}, xs[1] = {2 * (uint64_t)p.ld_x};
        const uint64_t od[3] = {(uint64_t)p.depth, (uint64_t)p.features, (uint64_t)p.groups}, os[2] = {2 * od[0], 2 * od[0] * od[1]};
        const uint32_t whole[2] = {64, 64}, tail[2] = {64, 16}, out[3] = {64, 32, 1};
        if (!encode_boxes(&w.w, p.w, 2, wd, ws, whole, false) || !encode_boxes(&w.x, p.x, 2, xd, xs, whole, false) ||
            !encode_boxes(&w.w_tail, p.w, 2, wd, ws, tail, false) || !encode_boxes(&w.x_tail, p.x, 2, xd, xs, tail, false) ||
            !encode_boxes(&w.out, p.e.out, 3, od, os, out, false))
            return cudaErrorInvalidValue;
    } else {
        const uint64_t lines = (uint64_t)p.features * (KIND == GROUP_GATED ? 2 : 1), k = p.depth;
        const uint64_t dims[3] = {p.w_mn ? lines : k, p.w_mn ? k : lines, (uint64_t)p.groups};
        const uint64_t strides[2] = {2 * dims[0], 2 * dims[0] * dims[1]};
        const uint32_t box[3] = {64, 64, 1};
        if (!encode_boxes(&w.w, p.w, 3, dims, strides, box, false) ||
            !encode_operand(&w.x, p.x, p.ld_x, p.rows, p.depth, false, false, kBox))
            return cudaErrorInvalidValue;
    }
    w.offsets = p.offsets;
    w.groups = p.groups;
    w.rows = p.rows;
    w.features = p.features;
    w.depth = p.depth;
    w.w_mn = p.w_mn;
    w.ftiles = (p.features + NF - 1) / NF;
    w.ntiles = (p.depth + kTile - 1) / kTile;
    w.across = Divide::by(WEIGHTS ? w.ftiles * w.ntiles : w.ftiles);
    w.down = Divide::by(w.ftiles);
    w.stages = stages_of((GroupKind)KIND, p.groups);
    w.limit = limits;
    w.e = p.e;
    w.e.cols = p.features;
    w.e.vec = 1;
    // no more tiles than these, wherever the offsets lie
    const long long most = WEIGHTS ? (long long)p.groups * w.ftiles * w.ntiles
                                   : ((long long)p.rows / kTile + (p.groups < p.rows ? p.groups : p.rows)) * w.ftiles;
    if (most > INT_MAX / 2 || w.stages < 2) return cudaErrorInvalidValue;
    int pairs = 0;
    if (cudaError_t e = resident_pairs<E, KIND, LIMITED>(&pairs)) return e;
    if (most < pairs) pairs = (int)most;
    const int bytes = 1024 + w.stages * kStage + kEpiWarps * patch_bytes(KIND) + table_bytes(p.groups);
    return launch_pdl(grouped_kernel<E, KIND, LIMITED>, dim3(2 * pairs), dim3(kThreads), bytes, st, w, err);
}

template <typename E>
cudaError_t launch_kind(const Grouped& p, GroupKind kind, uint32_t* err, cudaStream_t st) {
    switch (kind) {
        case GROUP_ROWS: return launch<E, GROUP_ROWS>(p, err, st);
        case GROUP_GATED: return launch<E, GROUP_GATED>(p, err, st);
        case GROUP_GATED_BWD: return launch<E, GROUP_GATED_BWD>(p, err, st);
        default: return launch<E, GROUP_WEIGHTS>(p, err, st);
    }
}

}  // namespace

cudaError_t launch_grouped(const Grouped& p, GroupKind kind, int elem, uint32_t* err, cudaStream_t st, const WaitLimits* limits) {
    if (limits)
        return kind == GROUP_WEIGHTS ? launch<__nv_bfloat16, GROUP_WEIGHTS, true>(p, err, st, *limits)
               : kind == GROUP_GATED ? launch<__nv_bfloat16, GROUP_GATED, true>(p, err, st, *limits)
                                     : launch<__nv_bfloat16, GROUP_ROWS, true>(p, err, st, *limits);
    return elem == PE_ELEM_BF16 ? launch_kind<__nv_bfloat16>(p, kind, err, st) : launch_kind<__half>(p, kind, err, st);
}

}  // namespace dense
}  // namespace pe
