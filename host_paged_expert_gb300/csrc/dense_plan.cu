// Which kernel and which tiles a matrix product takes: the least of the
// times that these models give.  They were fitted to GB300 measurements of
// both kernels (94 plain bf16 products of 8 to 2048 rows and 60 of 512 to 8192
// on CTA pairs, operands in L2, in microseconds), agree with them to 8 % and 3
// % and choose a shape 1 to 2 % slower than the best one on average:
//
//   rows x K x cols   CTA pairs, 256 / 128 columns   cluster split (tokens, CTAs along K)
//   8 x 2048 x 2048        13.3 / 9.8                 9.8 (16, 1)   6.8 (16, 2)   5.0 (16, 4)   4.5 (16, 8)
//   64 x 4096 x 4096       22.1 / 16.5               18.8 (64, 1)  12.4 (64, 2)   9.5 (64, 4)  11.9 (64, 8)
//   256 x 2048 x 2048      13.8 / 9.9                11.1 (64, 1)   8.7 (64, 2)  10.2 (64, 4)  20.4 (64, 8)
//   400 x 8192 x 1024      39.4 / 29.5               34.8 (64, 1)  20.7 (64, 2)  17.8 (64, 4)  15.9 (128, 4)
//   1024 x 2048 x 2048     14.2 / 11.1               14.1 (64, 1)  21.2 (64, 2)  37.0 (64, 4)  13.2 (128, 1)
//   2048 x 4096 x 4096     41.0 / 57.4               87.5 (64, 1)
//   8192 x 256 x 4096      24.4 / 22.0
//   4096 x 512 x 4096      18.1 / 18.3
//   4096 x 1024 x 4096     23.9 / 29.2
//   16 x 2048 x 12288                                7.8 (16, 2)   7.65 (16, 3) 11.5 (16, 4)
//   300 x 6144 x 2048                               21.5 (64, 2)  17.2 (64, 3)  24.1 (64, 4)
//
//   rows x K x cols   warps streaming weights        best cluster split
//   1 x 4096 x 2048         2.9                       5.8
//   1 x 8192 x 8192        20.1                      25.1
//   2 x 4096 x 4096         6.6                       7.0
//   4 x 2048 x 2048         4.2                       4.6
//   4 x 4096 x 4096        10.1                       7.0
//   4 x 8192 x 8192        42.2                      24.6
#include <algorithm>
#include <cmath>

#include "dense.cuh"

namespace pe {
namespace dense {
namespace {

constexpr double kPairs = 76;

int up(long long a, long long b) { return (int)((a + b - 1) / b); }

// Of a launch of CTA pairs: starting it, filling the pipeline and the last
// tile's epilogue (`full` of it for tiles with all their rows); a K block of
// a tile; what each further tile costs beyond its K blocks; and how often one
// can follow another where K is short, a plain epilogue and some of its K
// blocks.  `heavier`: what `epi_extra` takes, against tiles of 128 columns.
struct PairCost {
    double fixed, full, block, gap, epi, slope, heavier;
};
constexpr PairCost kWide = {5.2, 0.1, 0.265, 0.5, 2.65, 0.11, 2.7}, kNarrow = {3.15, 0.45, 0.205, 0.42, 1.25, 0.03, 1.0};

// What a linear epilogue does besides converting and storing (8192 x 256 to
// 8192, 27 tiles of 128 columns a pair: plain 40 us, gelu_tanh 57, bias and
// residual 69, gelu_tanh with its input kept 68, all of it 97); narrow tiles
// of gate and up have half the epilogue warps; an fp32 store costs what the
// read of a residual does (4096 x 512 to 32000, 53 tiles a pair: 128 us).
// EPI_GATED_BWD, which reads and stores the most, is not measured and counts
// as a plain one.
double epi_extra(const Product& p, EpiKind kind, int tn) {
    if (kind == EPI_GATED) return tn == 128 ? 0.7 : 0.0;
    if (kind != EPI_LINEAR) return 0;
    return (p.e.act != PE_ACT_NONE ? 0.8 : 0.0) + (p.e.bias ? 0.2 : 0.0) + (p.e.res ? 0.9 : 0.0) + (p.e.keep ? 0.5 : 0.0) +
           (p.e.out_f32 ? 0.9 : 0.0);
}

double tile_time(const PairCost& c, int kb, double extra) {
    return std::max(kb * c.block + c.gap, c.epi + kb * c.slope + c.heavier * extra);
}

// 8-bit operands: every tile's epilogue is exposed (its warps add up the K
// blocks), 3.3 us.
double pair_time(const Product& p, EpiKind kind, int tn) {
    const bool fp8 = p.a_scale != nullptr;
    const int kb = up(p.K, fp8 ? 128 : 64), cols = kind == EPI_GATED ? tn / 2 : tn;
    const double waves = std::max(1.0, std::ceil((double)up(p.M, 256) * up(p.e.cols, cols) / kPairs));
    if (fp8) return 3.0 + waves * (kb * 0.45 + 3.3);
    const PairCost& c = tn == 256 ? kWide : kNarrow;
    const double extra = epi_extra(p, kind, tn);
    return c.fixed + (c.full + c.heavier * extra) * std::min(1.0, p.M / 256.0) + kb * c.block +
           (waves - 1) * tile_time(c, kb, extra);
}

// The same with the K blocks of one CTA, or all weights from HBM (L2 where
// they may stay there); two CTAs on an SM, which some SMs have as soon as
// there are more than one each, take half as long again; partial sums cross
// the cluster.
double split_time(const Product& p, EpiKind kind, const SplitShape& s) {
    const bool fp8 = p.a_scale != nullptr;
    const int kb = up(p.K, fp8 ? 128 : 64), share = up(kb, s.split);
    const double base = (double)up(p.e.cols, kind == EPI_GATED ? 64 : 128) * up(p.M, s.nt), ctas = base * s.split;
    const double block = fp8 ? 0.28 + 0.0035 * s.nt : s.nt <= 64 ? 0.24 : 0.26;
    const double slots = split_resident(s);  // fewer than the SMs hold: a cluster stays within a GPC
    const double fixed = 1.83 + 0.0265 * s.nt + (s.split > 1 ? 0.4 : 0.0), waves = std::max(1.0, std::ceil(ctas / slots));
    const double shared = s.nt <= 64 && ctas / waves > slots / 2 ? 1.47 : 1.0;
    const double bytes = (double)p.N * p.K * (fp8 ? 1 : 2), stream = bytes / (bytes > 64e6 ? 6.2e6 : 11e6);
    return fixed * waves + std::max(stream, share * block * shared * waves) + base * s.nt * 512.0 * (s.split - 1) / 1.7e6 +
           0.055 * (s.split - 1);
}

// Weights at what HBM and L2 gave, less with each further row; or the
// multiply-adds with operands from L1.
double gemv_time(const Product& p) {
    const bool fp8 = p.a_scale != nullptr;
    const double weights = (double)p.N * p.K;
    return 1.7 + std::max(weights * (fp8 ? 1 : 2) / 7.2e6 * (1 + 0.3 * (p.M - 1)), p.M * weights / (fp8 ? 5.0e6 : 6.3e6));
}

// The best kernel for one product and its time.
struct Choice {
    double us = 1e30;
    int tn = 0;            // CTA pairs with tiles of so many columns
    bool gemv = false;
    SplitShape shape = {};  // else a cluster split
};

Choice choose(const Product& p, EpiKind kind) {
    const bool fp8 = p.a_scale != nullptr, f32 = p.e.out_f32 != 0;
    const int kb = up(p.K, fp8 ? 128 : 64);
    Choice c;
    bool bounded = !f32 || fp8;  // whether the best kernel keeps its accumulators to 8 blocks, where that matters
    // fp32 results of more than 8 blocks stay with the kernel that bounds the terms of one accumulator, and
    // so do those of ragged columns, stored one by one (cluster split / CTA pairs: 700 x 512 x 777 8.6 / 12.6
    // us, 6508 x 344 x 310 15.8 / 17.0; with whole vectors 6508 x 344 x 304 11.1 / 8.5, 8192 x 512 x 512 14.1 /
    // 9.9, 4096 x 512 x 32000 328 / 128)
    if (!f32 || fp8 || (kb <= 8 && p.e.vec))
        for (int t = 256; t >= (fp8 ? 256 : 128); t /= 2) {
            const double us = pair_time(p, kind, t);
            if (us < c.us) c.us = us, c.tn = t, bounded = true;
        }
    for (int most = 32; most <= (fp8 ? 64 : 128); most *= 2) {
        // rows shared out evenly over the fewest tiles of at most `most`
        SplitShape s;
        const int tiles = up(p.M, most);
        s.nt = up(up(p.M, tiles), 16) * 16;
        for (s.split = 1; s.split <= 8 && s.split <= kb; ++s.split) {
            const double us = split_time(p, kind, s);
            const bool fits = !f32 || fp8 || split_blocks(s, kb) <= 8;
            if (fits > bounded || (fits == bounded && us < c.us)) c.us = us, c.tn = 0, c.shape = s, bounded = fits;
        }
    }
    if (p.M <= kGemvRows && !p.a_mn && !p.b_mn && kind != EPI_GATED_BWD) {
        const double us = gemv_time(p);
        if (us < c.us) c.us = us, c.gemv = true;
    }
    return c;
}

cudaError_t launch_choice(const Choice& c, const Product& p, EpiKind kind, int elem, int chain, uint32_t* err,
                          cudaStream_t st) {
    if (c.gemv) return launch_gemv(p, kind, elem, chain, st);
    if (c.tn) return launch_pairs(&p, 1, kind, elem, c.tn, err, st);
    return launch_split(p, kind, elem, c.shape, chain, err, st);
}

// Products of 16-bit operands in one launch: the busiest pair, whose tiles
// take their K blocks or their epilogue, whichever is longer.
double group_time(const Product* p, int count, int tn) {
    const PairCost& c = tn == 256 ? kWide : kNarrow;
    double load[(int)kPairs] = {};
    long long t = 0;
    for (int i = 0; i < count; ++i) {
        const long long n = (long long)up(p[i].M, 256) * up(p[i].e.cols, tn);
        const double tile = tile_time(c, up(p[i].K, 64), 0), whole = (double)(n / (int)kPairs) * tile;
        for (int j = 0; j < (int)kPairs; ++j)
            load[j] += whole + (((j - t) % (int)kPairs + (int)kPairs) % (int)kPairs < n % (int)kPairs ? tile : 0);
        t += n;
    }
    const double most = *std::max_element(load, load + (int)kPairs);
    return c.fixed + c.full + most;
}

}  // namespace

cudaError_t launch_product(const Product& p, EpiKind kind, int elem, int chain, uint32_t* err, cudaStream_t st) {
    return launch_choice(choose(p, kind), p, kind, elem, chain, err, st);
}

cudaError_t launch_products(const Product* p, int count, int elem, uint32_t* err, cudaStream_t st) {
    if (count > kMostProducts) return cudaErrorInvalidValue;
    Choice c[kMostProducts];
    Product by_k[kMostProducts];  // the longest tiles first
    double apart = 0;
    for (int i = 0; i < count; ++i) {
        c[i] = choose(p[i], EPI_LINEAR);
        apart += c[i].us;
        by_k[i] = p[i];
    }
    std::sort(by_k, by_k + count, [](const Product& a, const Product& b) { return a.K > b.K; });
    if (count > 1)
        for (int tn = 256; tn >= 128; tn /= 2)
            if (group_time(by_k, count, tn) < apart && group_time(by_k, count, tn) <= group_time(by_k, count, 384 - tn))
                return launch_pairs(by_k, count, EPI_LINEAR, elem, tn, err, st);
    for (int i = 0; i < count; ++i)
        if (cudaError_t e = launch_choice(c[i], p[i], EPI_LINEAR, elem, CHAIN_NONE, err, st)) return e;
    return cudaSuccess;
}

}  // namespace dense
}  // namespace pe
