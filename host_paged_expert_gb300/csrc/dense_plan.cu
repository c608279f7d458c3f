// Which kernel and which tiles a matrix product takes: the least of the
// times that these models give.  They were fitted to GB300 measurements of
// both kernels (plain bf16 products, operands in L2, in microseconds) and
// agree with them to about 10 % from one row to 2048:
//
//   rows x K x cols   CTA pairs, 256 / 128 columns   cluster split (tokens, CTAs along K)
//   1 x 2048 x 2048        13.9 / -                  11.5 (16, 1)   7.8 (16, 2)   5.5 (16, 8)
//   64 x 4096 x 4096       25.4 / -                  21.2 (64, 1)  13.7 (64, 2)  10.5 (64, 4)
//   256 x 2048 x 2048      17.1 / 12.7               13.4 (64, 1)  10.0 (64, 2)  11.3 (64, 4)
//   512 x 8192 x 1024      42.3 / 31.4               37.0 (64, 1)  21.9 (64, 2)  17.9 (128, 4)
//   1024 x 2048 x 2048     17.1 / 13.1               17.1 (64, 1)  21.9 (64, 2)  16.3 (128, 1)
//   1024 x 4096 x 4096     26.6 / 32.8               49.3 (64, 1)
//
//   rows x K x cols   warps streaming weights        best cluster split
//   1 x 4096 x 2048         2.7                       6.8
//   1 x 8192 x 8192        18.6                      24.2
//   2 x 4096 x 4096         6.2                       8.2
//   4 x 2048 x 2048         4.0                       5.7
//   4 x 8192 x 8192        40.4                      24.4
//   8 x 2048 x 2048         8.1                       6.1
#include <algorithm>
#include <cmath>

#include "dense.cuh"

namespace pe {
namespace dense {
namespace {

constexpr double kSms = 152, kPairs = 76;

int up(long long a, long long b) { return (int)((a + b - 1) / b); }

// Launch, filling the pipeline and the last tile's epilogue; then the K
// blocks of each wave of tiles, under which the other epilogues hide unless K
// is short.  8-bit operands: every tile's epilogue is exposed (its warps add
// up the K blocks), 3.3 us.
double pair_time(const Product& p, EpiKind kind, int tn) {
    const bool fp8 = p.a_scale != nullptr;
    const int kb = up(p.K, fp8 ? 128 : 64), cols = kind == EPI_GATED ? tn / 2 : tn;
    const double waves = std::max(1.0, std::ceil((double)up(p.M, 256) * up(p.e.cols, cols) / kPairs));
    if (fp8) return 5.5 + waves * (kb * 0.46 + 3.3);
    const double block = tn == 256 ? 0.265 : 0.195, epi = tn == 256 ? 3.5 : 1.8;
    const double full = tn == 256 ? 3.1 : 1.6, fixed = tn == 256 ? 5.5 : 4.7;
    return fixed + full * std::min(1.0, p.M / 256.0) + waves * kb * block + (waves - 1) * std::max(0.0, epi - kb * block);
}

// The same with the K blocks of one CTA (or all weights from HBM); blocks on one SM share its tensor
// core; partial sums cross the cluster at about 1.6 TB/s.
double split_time(const Product& p, EpiKind kind, const SplitShape& s) {
    const bool fp8 = p.a_scale != nullptr;
    const int kb = up(p.K, fp8 ? 128 : 64), share = up(kb, s.split);
    const double base = (double)up(p.e.cols, kind == EPI_GATED ? 64 : 128) * up(p.M, s.nt), ctas = base * s.split;
    const double block = fp8 ? 0.26 + 0.0045 * s.nt : s.nt <= 64 ? 0.245 : 0.275;
    const double slots = s.nt <= 64 ? 2 * kSms : kSms;
    const double fixed = 3.6 + 0.0245 * s.nt, waves = std::max(1.0, std::ceil(ctas / slots));
    const double stream = (double)p.N * p.K * (fp8 ? 1 : 2) / 6.2e6;  // the weights at HBM's rate
    return fixed * waves + std::max(stream, share * block * std::max(1.0, ctas / kSms)) +
           base * s.nt * 512.0 * (s.split - 1) / 1.6e6 + 0.1 * (s.split - 1);
}

// Weights at what HBM and L2 gave, or the multiply-adds with operands from L1.
double gemv_time(const Product& p) {
    const bool fp8 = p.a_scale != nullptr;
    const double weights = (double)p.N * p.K;
    return 1.7 + std::max(weights * (fp8 ? 1 : 2) / 7.2e6, p.M * weights / (fp8 ? 5.0e6 : 6.3e6));
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
    // fp32 results stay with the kernel that bounds the terms of one accumulator
    if (!f32 || fp8)
        for (int t = 256; t >= (fp8 ? 256 : 128); t /= 2) {
            const double us = pair_time(p, kind, t);
            if (us < c.us) c.us = us, c.tn = t;
        }
    bool bounded = !f32 || fp8;  // whether the best shape keeps its accumulators to 8 blocks, where that matters
    for (int most = 32; most <= (fp8 ? 64 : 128); most *= 2) {
        // rows shared out evenly over the fewest tiles of at most `most`
        SplitShape s;
        const int tiles = up(p.M, most);
        s.nt = up(up(p.M, tiles), 16) * 16;
        for (s.split = 1; s.split <= 8 && s.split <= kb; s.split *= 2) {
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

// Products of 16-bit operands in one launch: the pair with the most K blocks.
double group_time(const Product* p, int count, int tn) {
    double load[(int)kPairs] = {};
    long long t = 0;
    for (int i = 0; i < count; ++i) {
        const long long n = (long long)up(p[i].M, 256) * up(p[i].e.cols, tn);
        const double kb = up(p[i].K, 64), whole = (double)(n / (int)kPairs) * kb;
        for (int j = 0; j < (int)kPairs; ++j)
            load[j] += whole + (((j - t) % (int)kPairs + (int)kPairs) % (int)kPairs < n % (int)kPairs ? kb : 0);
        t += n;
    }
    const double most = *std::max_element(load, load + (int)kPairs);
    return (tn == 256 ? 8.6 : 6.3) + most * (tn == 256 ? 0.265 : 0.195);
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
