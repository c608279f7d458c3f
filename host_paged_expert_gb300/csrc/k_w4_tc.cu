// Linear products with 4-bit weights of some tens of rows: the weights are
// decoded to 16 bits on their way into shared memory and multiplied on tcgen05.
//
// As in the 16-bit kernel of this size the weights' rows lie along the MMA's M
// (128 per tile), the tokens along its N (16 to 64), and the K blocks of a tile
// are shared out among the CTAs of a cluster, which add their fp32 partials in
// rank order over distributed shared memory.  Sixteen warps read codes (64 bytes
// of a row by two lanes, the next ones on their way), decode them and write the
// operand in the swizzle that the MMA's descriptor names, eight of them a pair of
// 64-deep blocks, the others the next pair; TMA brings the tokens.
//
// Each pair, 128 inputs, has a TMEM buffer of its own.  Eight more warps add it
// to fp32 registers, where a lane has a weight row: int4's group scale multiplies
// it there, so int4's weights are not rounded, and E2M1 times its block scale is
// exact in 16 bits.  But MXFP4's scales reach past fp16: with it a pair has four
// buffers, one for each 32 inputs, and their scales multiply them too.
//
// Bound by the decoding warps, their instructions and the latency of their
// loads.  NVFP4, 32 x 8192 to 19456 (152 tiles, one a CTA; 64 pairs of blocks):
// 44.5 us.  With two of a pair's eight MMAs 43.2, without the sums 43.8, without
// writing what is decoded 45.8; without the arithmetic of decoding 34.1, with the
// first codes loaded only 35.7.  (A chain of MMAs alone takes 72 cycles for 128
// rows, 16 inputs and up to 32 tokens, 77 for 64, 85 for 128 and 129 for 256: 0.28
// us of a pair's 0.69.)  Weights in L2, 32 x 4096 to 4096 10 to 11 us, to 32000 40
// to 48; from HBM 10.4 (int4) and 46 to 49.
#include "experts.cuh"
#include "dense_cluster.cuh"
#include "dense_tc.cuh"
#include "fp8_device.cuh"
#include "pe_device.cuh"
#include "w4_device.cuh"

#include <algorithm>

namespace pe {
namespace dense {
namespace {

constexpr int kDecoders = 8;  // warps that decode a pair of blocks, of which two sets take every other one
constexpr int kThreads = 384 + 64 * kDecoders;  // warp 0 TMA, 1 MMA, 2 TMEM, 4..11 sums, 12..27 decoding; all of them add up
constexpr int kP = kRows * 128;  // bytes of a block of weights: 128 rows of 64 inputs
constexpr int kStages = 4;       // of a pair of blocks each
constexpr int kAhead = 2;        // pairs of blocks whose codes are on their way to a thread
constexpr int kMostTokens = 64;
// Sums of a pair of blocks that have scales of their own (kScaleSums: of each 32
// inputs), and places for such sums in TMEM.
template <typename E, int FMT>
constexpr int kSums = kScaleSums<E, FMT> ? 4 : 1;
template <typename E, int FMT>
constexpr int kPlaces = kScaleSums<E, FMT> ? 2 : kStages;

struct Plan {
    int nt, q_bytes;  // tokens of a tile, a multiple of 16; bytes of their block
    int split, ftiles;
    WaitLimits limit;
};
struct Shared {
    uint64_t full[kStages], done[kStages], acc_empty[kStages], drain;
    uint32_t tmem;
};

// Codes of one pair of blocks on their way to a thread: 32 of its row in each
// block, and their raw scales.
template <int FMT>
struct Codes {
    int4 w[2];
    uint32_t s[2];
};

// LIMITED: the waits' limits are the launch's.
template <typename E, int FMT, bool LIMITED>
__global__ void __launch_bounds__(kThreads, 1)
    w4_tc_kernel(const __grid_constant__ CUtensorMap tx, const __grid_constant__ W4Args a, const __grid_constant__ Plan q, uint32_t* err) {
    auto polls = [](uint32_t limit) { return LIMITED ? limit : kPolls; };
    constexpr int SUMS = kSums<E, FMT>, PLACES = kPlaces<E, FMT>, COLUMNS = PLACES * SUMS * kMostTokens;  // of TMEM
    extern __shared__ uint8_t dyn[];
    __shared__ Shared S;
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blockIdx.x % q.split, tile = blockIdx.x / q.split;
    const int f0 = tile % q.ftiles * kRows, t0 = tile / q.ftiles * q.nt;
    const int pairs_all = (a.K + 127) / 128;
    const int p0 = (int)((long long)pairs_all * rank / q.split), np = (int)((long long)pairs_all * (rank + 1) / q.split) - p0;
    const int stage = 2 * (kP + q.q_bytes);  // weights of both blocks, then tokens
    const int groups = (a.K + w4_group(FMT) - 1) / w4_group(FMT);

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(&S.full[i], 1 + kDecoders);  // the copy of the tokens, the decoding warps
            tc::mbar_init(&S.done[i], 1);
            tc::mbar_init(&S.acc_empty[i], 8);
        }
        tc::mbar_init(&S.drain, 1);
        tc::fence_barrier_init();
        tc::tma_prefetch(&tx);
    }
    if (warp == 2) tc::tmem_alloc(&S.tmem, COLUMNS);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = S.tmem;
    pdl_wait();
    if (warp == 3) pdl_trigger();

    if (warp == 0) {
        // ---- the tokens' copies
        const bool lead = tc::elect_one();
        bool ok = true;
        int p = 0;
        for (; p < np; ++p) {
            const int s = p % kStages;
            if (!(ok = tc::mbar_spin(&S.done[s], (p / kStages & 1) ^ 1, err, polls(q.limit.copies)))) break;
            if (lead) {
                uint8_t* to = ring + s * stage + 2 * kP;
                tc::mbar_arrive_expect_tx(&S.full[s], 2 * q.q_bytes);
                tc::tma_load_2d(to, &tx, &S.full[s], (p0 + p) * 128, t0);
                tc::tma_load_2d(to + q.q_bytes, &tx, &S.full[s], (p0 + p) * 128 + 64, t0);
            }
            __syncwarp();
        }
        // the block does not end before its copies have landed
        for (int j = max(0, p - kStages); ok && j < p; ++j)
            ok = tc::mbar_wait(&S.full[j % kStages], (j / kStages) & 1, err, PE_DEVERR_TIMEOUT, tc::kLeavePolls);
        if (!ok) tc::settle();
    } else if (warp == 1) {
        // ---- MMA issuer
        const bool lead = tc::elect_one();
        constexpr int FMT16 = std::is_same<E, __nv_bfloat16>::value ? 1 : 0;
        const uint32_t id = tc::idesc(FMT16, 0, 0, kRows, q.nt);
        const uint64_t a0 = tc::operand_desc(tc::smem_u32(ring), false), b0 = tc::operand_desc(tc::smem_u32(ring) + 2 * kP, false);
        for (int p = 0; p < np; ++p) {
            const int s = p % kStages, place = p % PLACES;
            if (!tc::mbar_spin(&S.acc_empty[place], (p / PLACES & 1) ^ 1, err, polls(q.limit.mma))) break;
            if (!tc::mbar_spin(&S.full[s], p / kStages & 1, err, polls(q.limit.mma))) break;
            tc::fence_after_sync();
            if (lead) {
                const uint64_t da = a0 + (uint32_t)(s * stage >> 4), db = b0 + (uint32_t)(s * stage >> 4);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    tc::mma<false, false>(tmem + (place * SUMS + k * SUMS / 8) * kMostTokens, da + (k / 4 * kP >> 4) + k % 4 * 2,
                                          db + (k / 4 * q.q_bytes >> 4) + k % 4 * 2, id, k % (8 / SUMS));
                tc::mma_commit(&S.done[s]);
            }
            __syncwarp();
        }
        // the block does not end before its MMAs, which read shared memory and write TMEM
        if (lead) tc::mma_commit(&S.drain);
        tc::mbar_wait(&S.drain, 0, err, PE_DEVERR_TIMEOUT, tc::kLeavePolls);
    } else if (warp >= 4 && warp < 12) {
        // ---- sums: a lane has a weight row, a warp half of the tokens, 16 or 32
        const int quarter = warp & 3, share = q.nt > 32 ? 32 : 16, c0 = (warp - 4) / 4 * share, row = min(f0 + quarter * 32 + lane, a.N - 1);
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16) + c0;
        float acc[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) acc[j] = 0.f;
        // The raw scales of a pair's sums (past K, of nothing), two pairs ahead; what
        // is loaded rests until its turn (fp16 with MXFP4, 32 x 4096 to 32000: 56 us;
        // one pair ahead 77).
        uint32_t raw[2][2] = {};
        auto scales = [&](int p, uint32_t(&to)[2]) {
            to[0] = to[1] = 0;
            const int at = SUMS * (p0 + p);
            if (p >= np) return;
            if constexpr (FMT == W4_INT4) {
                to[0] = static_cast<const uint16_t*>(a.scales)[(size_t)row * groups + at];
            } else if constexpr (SUMS > 1) {
                const uint8_t* from = static_cast<const uint8_t*>(a.scales) + (size_t)row * groups + at;
                if (groups % 2 == 0) {
                    to[0] = *reinterpret_cast<const uint16_t*>(from);
                    if (at + 2 < groups) to[1] = *reinterpret_cast<const uint16_t*>(from + 2);
                } else {
#pragma unroll
                    for (int i = 0; i < SUMS; ++i)
                        if (at + i < groups) to[i / 2] |= (uint32_t)from[i] << (8 * (i & 1));
                }
            }
        };
        scales(0, raw[0]);
        scales(1, raw[1]);
        bool ok = true;
        for (int p = 0; p < np; ++p) {
            const uint32_t bits = raw[0][0] | raw[0][1] << 16;
            raw[0][0] = raw[1][0], raw[0][1] = raw[1][1];
            scales(p + 2, raw[1]);
            if (!(ok = tc::mbar_spin(&S.done[p % kStages], p / kStages & 1, err, polls(q.limit.sums)))) break;
            tc::fence_after_sync();
            const int place = p % PLACES;
            if (c0 < q.nt) {
#pragma unroll
                for (int i = 0; i < SUMS; ++i) {
                    const float f = FMT == W4_INT4 ? __half2float(__ushort_as_half((unsigned short)bits))
                                    : SUMS > 1   ? e8m0(bits >> (8 * i) & 255u)
                                                 : 1.f;
#pragma unroll
                    for (int h = 0; h < 32; h += 16) {
                        if (h >= share) continue;
                        uint32_t r[16];
                        tc::tmem_ld16(lanes + (place * SUMS + i) * kMostTokens + h, r);
                        tc::tmem_ld_wait(r);
#pragma unroll
                        for (int j = 0; j < 16; ++j) acc[h + j] = fmaf(f, __uint_as_float(r[j]), acc[h + j]);
                    }
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&S.acc_empty[place]);
        }
        const float ts = FMT == W4_NVFP4 ? a.tensor_scale[0] : 1.f;
        // every warp is past its last buffer, so every MMA is done with the ring
        asm volatile("bar.sync 1, 256;" ::: "memory");
        float* part = reinterpret_cast<float*>(ring) + c0 * kRows + quarter * 32 + lane;
        if (ok)
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (j < share && c0 + j < q.nt) part[j * kRows] = acc[j] * ts;
    } else if (warp >= 12) {
        // ---- decoding: lanes 2 i and 2 i + 1 have 64 inputs of a row, 16 rows a warp
        const int half = lane & 1, r0 = (warp - 12) % kDecoders * 16 + (lane >> 1), set = (warp - 12) / kDecoders;
        const size_t row = min(f0 + r0, a.N - 1);
        const uint8_t* codes = static_cast<const uint8_t*>(a.codes) + row * (a.K / 2) + 16 * half;
        const uint8_t* scales = static_cast<const uint8_t*>(a.scales) + row * groups;
        auto fetch = [&](int p, Codes<FMT>& to) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int k = (p0 + p) * 128 + 64 * b + 32 * half;
                to.w[b] = make_int4(0, 0, 0, 0);
                to.s[b] = 0;
                if (p < np && k < a.K) {  // K is a multiple of 32; the tokens' copy has zeros past it
                    to.w[b] = *reinterpret_cast<const int4*>(codes + (p0 + p) * 64 + 32 * b);
                    if (FMT == W4_MXFP4 && SUMS == 1) to.s[b] = scales[k / 32];
                    if (FMT == W4_NVFP4) to.s[b] = *reinterpret_cast<const uint16_t*>(scales + k / 16);
                }
            }
        };
        Codes<FMT> c[kAhead];
#pragma unroll
        for (int h = 0; h < kAhead; ++h) fetch(set + 2 * h, c[h]);
        uint8_t* to[4];  // of eight codes' places in a stage
#pragma unroll
        for (int j = 0; j < 4; ++j) to[j] = ring + r0 * 128 + (((4 * half + j) ^ (r0 & 7)) << 4);
        bool ok = true;
        uint32_t s = set, phase = 1;
        for (int pb = set; ok && pb < np; pb += 2 * kAhead) {
#pragma unroll
            for (int h = 0; h < kAhead; ++h) {
                const int p = pb + 2 * h;
                if (!ok || p >= np) continue;
                ok = tc::mbar_spin(&S.done[s], phase, err, polls(q.limit.copies));
                if (!ok) continue;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    float f[2];
                    if (FMT == W4_MXFP4 && SUMS == 1) {
                        f[0] = f[1] = e8m0(c[h].s[b]);
                    } else if (FMT == W4_NVFP4) {
                        const float2 v = e4m3x2(c[h].s[b]);
                        f[0] = v.x, f[1] = v.y;
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int4 w = c[h].w[b];
                        const uint32_t word = j == 0 ? w.x : j == 1 ? w.y : j == 2 ? w.z : w.w;
                        uint32_t v[4];
                        if (FMT == W4_INT4) int4x8<E>(word, v);
                        else if (SUMS > 1) e2m1x8<E>(word, v);
                        else e2m1x8<E>(word, Pair<E>::both(f[j / 2]), v);
                        // (0, 4) (1, 5) (2, 6) (3, 7) to the inputs' order
                        uint4 o;
                        o.x = __byte_perm(v[0], v[1], 0x5410), o.y = __byte_perm(v[2], v[3], 0x5410);
                        o.z = __byte_perm(v[0], v[1], 0x7632), o.w = __byte_perm(v[2], v[3], 0x7632);
                        *reinterpret_cast<uint4*>(to[j] + s * stage + b * kP) = o;
                    }
                }
                fetch(p + 2 * kAhead, c[h]);
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&S.full[s]);
                if ((s += 2) >= kStages) s -= kStages, phase ^= 1;
            }
        }
    }
    __syncwarp();
    __syncthreads();
    if (q.split > 1) {
        tc::cluster_arrive();
        tc::cluster_wait();
    }
    if (q.split == 1) reduce<E, EPI_LINEAR, 1, kThreads>(a.e, ring, q.nt, 1, rank, t0, f0);
    else if (q.split == 2) reduce<E, EPI_LINEAR, 2, kThreads>(a.e, ring, q.nt, 2, rank, t0, f0);
    else reduce<E, EPI_LINEAR, 4, kThreads>(a.e, ring, q.nt, q.split, rank, t0, f0);
    // no CTA leaves while another may read its partial
    if (q.split > 1) {
        tc::cluster_arrive_relaxed();
        tc::cluster_wait();
    }
    tc::fence_after_sync();
    if (warp == 2) tc::tmem_dealloc(tmem, COLUMNS);
}

// CTAs along K: as many as fill the SMs in one wave, four at most (32 rows,
// nvfp4, with 1, 2, 3 and 4 of them: 4096 x 4096, 32 tiles, 22, 14, 12 and 11 us;
// 2880 x 5120, 40 tiles, 16, 12, 11 and 18; 8192 x 8192, 64 tiles, 38, 23, 35 and
// 30; 4096 x 32000, 250 tiles, 44, 57, 71 and 75).
int split_of(int tiles, int pairs) {
    int n = 4;
    while (n > 1 && (tiles * n > 152 || n > pairs)) --n;
    return n;
}

template <typename E, int FMT, bool LIMITED = false>
cudaError_t launch(const W4Args& a, uint32_t* err, cudaStream_t st, const WaitLimits& limits = {}) {
    static std::atomic<uint64_t> ready;  // devices whose attribute is set
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    auto kernel = w4_tc_kernel<E, FMT, LIMITED>;
    constexpr int most = 1024 + kStages * 2 * (kP + kMostTokens * 128);
    if (dev >= 64 || !(ready.load() >> dev & 1)) {
        if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most)) return e;
        if (dev < 64) ready.fetch_or(uint64_t(1) << dev);
    }
    Plan q = {};
    q.limit = limits;
    const int ttiles = (a.M + kMostTokens - 1) / kMostTokens;
    if ((long long)((a.N + kRows - 1) / kRows) * ttiles > INT_MAX / 4) return cudaErrorInvalidValue;
    q.nt = ((a.M + ttiles - 1) / ttiles + 15) / 16 * 16;
    q.q_bytes = q.nt * 128;
    q.ftiles = (a.N + kRows - 1) / kRows;
    q.split = split_of(q.ftiles * ttiles, (a.K + 127) / 128);
    const long long blocks = (long long)q.ftiles * ttiles * q.split;
    if (blocks > INT_MAX) return cudaErrorInvalidValue;
    CUtensorMap tx;
    if (!encode_operand(&tx, a.x, a.ld_x, a.M, a.K, false, false, q.nt)) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = most;  // a block per SM
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)q.split, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, tx, a, q, err);
}
template <typename E>
cudaError_t by_format(const W4Args& a, uint32_t* err, cudaStream_t st) {
    return a.fmt == W4_INT4 ? launch<E, W4_INT4>(a, err, st) : a.fmt == W4_MXFP4 ? launch<E, W4_MXFP4>(a, err, st) : launch<E, W4_NVFP4>(a, err, st);
}

}  // namespace

cudaError_t launch_w4_tc(const W4Args& a, int elem, uint32_t* err, cudaStream_t st, const WaitLimits* limits) {
    if (limits) return launch<__nv_bfloat16, W4_INT4, true>(a, err, st, *limits);
    return elem == PE_ELEM_BF16 ? by_format<__nv_bfloat16>(a, err, st) : by_format<__half>(a, err, st);
}

}  // namespace dense
}  // namespace pe
