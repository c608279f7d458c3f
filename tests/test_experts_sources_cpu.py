"""Rules of the sources of the resident experts' and 4-bit products' kernels
that no run shows (as test_dense_sources_cpu, which see)."""

import re

import pytest

from test_dense_sources_cpu import code, early_reads


@pytest.mark.parametrize("name,loads", [("k_grouped.cu", 4), ("k_w4_tc.cu", 1)])
def test_tensor_memory_is_read_after_its_wait(name, loads):
    text = code(name).replace("tmem_ld16(", "tmem_ld32(")
    assert text.count("tmem_ld32(") >= loads
    assert not early_reads(text), early_reads(text)


@pytest.mark.parametrize("name", ["k_grouped.cu", "k_route.cu", "k_rows.cu", "k_w4.cu", "k_w4_tc.cu", "experts.cuh", "w4_device.cuh", "dense_tile.cuh",
                                  "dense_cluster.cuh"])
def test_loads_are_coherent(name):
    assert not re.findall(r"__ldg|\bldg16|\bld_nc_na|\.nc\b", code(name))


def test_grouped_kernel_stays_until_the_last_arrivals():
    """MMAs of a pair arrive on the other CTA's `empty` barriers, its epilogue
    warps on the leader's `acc_empty`, and stores leave from shared memory: each
    is waited for before the block ends."""
    text = code("k_grouped.cu")
    text = text[text.index("grouped_kernel(") :]
    producer, rest = text[text.index("if (warp == 0) {") :].split("} else if (warp == 1 && rank == 0) {", 1)
    issuer = rest[: rest.index("} else if (WEIGHTS && warp == 3) {")]
    assert producer.rindex("mbar_spin(&S.empty[s]") > producer.rindex("tma_load_2d_pair(")
    assert issuer.rindex("mbar_spin(&S.acc_empty[buf]") > issuer.rindex("mma_commit_pair(&S.acc_full[buf])")
    assert text.index("tma_store_done()") > text.index("tma_store_3d(")
    assert text.index("tma_store_done()") < text.rindex("cluster_arrive_relaxed()")


def test_cleared_tails_are_handed_over():
    """Rows that a warp clears reach the tensor core of the pair's leader: a proxy
    fence by every lane, then a release that the leader's wait acquires."""
    text = code("k_grouped.cu")
    clear = text[text.index("S.raw[at], phases") :]
    order = [clear.index(w) for w in ("make_uint4(0, 0, 0, 0)", "fence_proxy_async_smem()", "__syncwarp()", "mbar_arrive_cluster_release(")]
    assert order == sorted(order)
    assert "WEIGHTS ? tc::mbar_spin_cluster(&S.full[at]" in text


@pytest.mark.parametrize("name", ["k_grouped.cu", "k_w4_tc.cu"])
def test_every_wait_of_a_role_has_the_launchs_limit(name):
    """So that the self-test can make each of them run out."""
    text = code(name)
    assert text.count("mbar_spin") >= 5 and text.count("polls(") >= 5
    assert not re.findall(r"err,\s*kPolls", text)


def test_split_weights_wait_for_the_launch_before():
    """The kernel of 17 to 128 rows counts its polls once the launch before is done."""
    text = code("k_w4_tc.cu")
    assert text.index("pdl_wait();") < text.index("mbar_spin(")
