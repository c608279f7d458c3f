"""Which kernel a product takes, on the CPU: csrc/dense_plan.cu is host code,
compiled here with stand-ins for the launches that print what was chosen."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "host_paged_expert_gb300", "csrc")

MAIN = r"""
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include "dense_plan.cu"
namespace pe { namespace dense {
cudaError_t launch_pairs(const Product*, int count, EpiKind, int, int tn, uint32_t*, cudaStream_t, const WaitLimits*) {
    printf("pairs %d %d\n", tn, count);
    return cudaSuccess;
}
cudaError_t launch_split(const Product&, EpiKind, int, const SplitShape& s, int, uint32_t*, cudaStream_t, const WaitLimits*) {
    printf("split %d %d\n", s.nt, s.split);
    return cudaSuccess;
}
cudaError_t launch_gemv(const Product&, EpiKind, int, int, cudaStream_t) { puts("gemv"); return cudaSuccess; }
// as k_dense_split.cu has them on a GB300
int split_blocks(const SplitShape& s, int kb) {
    const int share = (kb + s.split - 1) / s.split, most = ((s.nt <= 64 ? 256 : 512) - 32) / s.nt;
    const int want = (share + 7) / 8, n = want < most ? want : most;
    return (share + n - 1) / n;
}
int split_resident(const SplitShape& s) { return (s.nt <= 64 ? 2 : 1) * (152 / s.split * s.split); }
} }
int main(int argc, char** argv) {  // M K N kind f32 fp8, for each product of the call
    using namespace pe::dense;
    Product p[kMostProducts] = {};
    static const float scale = 1;
    int n = 0;
    for (int i = 1; i + 5 < argc; i += 6, ++n) {
        p[n].M = atoi(argv[i]), p[n].K = atoi(argv[i + 1]), p[n].N = p[n].e.cols = atoi(argv[i + 2]);
        p[n].e.rows = p[n].M, p[n].e.out_f32 = atoi(argv[i + 4]), p[n].e.vec = p[n].N % 8 == 0;
        if (atoi(argv[i + 5])) p[n].a_scale = p[n].b_scale = &scale;
        if (atoi(argv[i + 3]) == EPI_GATED) p[n].N *= 2;
    }
    return n == 1 ? launch_product(p[0], (EpiKind)atoi(argv[4]), 0, CHAIN_NONE, nullptr, nullptr) : launch_products(p, n, 0, nullptr, nullptr);
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    from host_paged_expert_gb300 import build

    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("plan")
    src, exe = d / "plan.cpp", d / "plan"
    src.write_text(MAIN)
    inc = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "include")
    subprocess.run([cxx, "-O1", "-std=c++17", f"-I{CSRC}", f"-I{os.path.join(ROOT, 'include')}", f"-I{inc}", str(src), "-o", str(exe)], check=True)

    def choose(*products):
        out = subprocess.run([str(exe), *[str(v) for p in products for v in p]], check=True, capture_output=True, text=True).stdout
        return [line.split()[0] for line in out.splitlines()]

    return choose


@pytest.mark.parametrize("m,k,n", [(6508, 344, 304), (8192, 512, 512), (16384, 512, 4096), (4096, 512, 32000), (20000, 8, 16)])
def test_large_fp32_results_of_short_k_take_pairs(plan, m, k, n):
    """Up to 512 terms one accumulator holds them all, on either kernel."""
    assert plan((m, k, n, 0, 1, 0)) == plan((m, k, n, 0, 0, 0)) == ["pairs"]


@pytest.mark.parametrize("m,k,n", [(2048, 4096, 4096), (8192, 520, 512), (300, 2048, 128)])
def test_fp32_results_of_long_k_bound_their_accumulators(plan, m, k, n):
    assert plan((m, k, n, 0, 1, 0)) == ["split"]


@pytest.mark.parametrize("m,k,n", [(6508, 344, 310), (700, 512, 777), (20000, 64, 127)])
def test_fp32_results_of_ragged_columns(plan, m, k, n):
    """Stored one by one, for which the kernel of pairs has the slower epilogue."""
    assert plan((m, k, n, 0, 1, 0)) == ["split"]


def test_other_choices(plan):
    assert plan((1, 4096, 2048, 0, 0, 0)) == ["gemv"]
    assert plan((8, 2048, 128, 0, 1, 0)) == ["split"]
    assert plan((64, 2048, 2048, 0, 0, 0)) == ["split"]
    assert plan((4096, 4096, 4096, 0, 0, 0)) == ["pairs"]
    assert plan((4096, 4096, 4096, 0, 1, 1)) == ["pairs"]
    assert plan((2048, 2048, 6144, 1, 0, 0)) == ["pairs"]
    # a backward pass: dx and dw in one launch
    assert plan((1021, 1536, 2880, 0, 0, 0), (1536, 1021, 2880, 0, 0, 0)) == ["pairs"]
