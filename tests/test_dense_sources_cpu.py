"""Rules of the dense kernels' sources that no run shows: what the compiler
happens to do today may hide a breach of them."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "host_paged_expert_gb300", "csrc")
KERNELS = ["k_dense_gemm.cu", "k_dense_split.cu", "k_dense_gemv.cu", "k_dense_norm.cu"]


def code(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def early_reads(text):
    """Uses of a tensor-memory load's registers before the wait that names
    them: PTX leaves their content undefined until tcgen05.wait::ld, and only a
    wait that takes the registers keeps the compiler from moving their use
    ahead of it."""
    found, pending = [], set()
    for line in text.splitlines():
        flat = line.replace(" ", "")
        load, wait = re.search(r"tmem_ld32\(.*,\s*([^,;]+)\);", line), re.search(r"tmem_ld_wait\(([^;]*)\);", line)
        if "__global__" in line:
            pending = set()
        elif load:
            pending.add(load.group(1).replace(" ", ""))
        elif wait:
            for reg in wait.group(1).replace(" ", "").split(","):
                # a wait for r[h] is one for r[0], the first of the turns
                turns = reg.split("[")[0] + "[" if re.search(r"\[[a-z]\]$", reg) else None
                pending = {p for p in pending if p != reg and not (turns and re.fullmatch(re.escape(turns) + r"\d\]", p))}
        else:
            for reg in pending:
                # r[0] may be reached as r[i]; of arrays taken in turn, r[h ^ 1] is not r[h]
                name = reg.split("[")[0] if re.search(r"\[\d+\]$", reg) else reg
                if re.search(r"(?<![\w.])" + re.escape(name) + r"(?!\w)", flat if "[" in name else line):
                    found.append(line.strip())
    return found


@pytest.mark.parametrize("name", ["k_dense_gemm.cu", "k_dense_split.cu"])
def test_tensor_memory_is_read_after_its_wait(name):
    text = code(name)
    assert text.count("tmem_ld32(") >= 3
    assert not early_reads(text), early_reads(text)


def test_the_rule_finds_an_early_read():
    at = "tc::tmem_ld32(a, n);\n"
    assert early_reads(at + "r[j] = n[j];\ntc::tmem_ld_wait(n);\n")
    assert early_reads(at + "tc::tmem_ld_wait();\nr[j] = n[j];\n")
    assert early_reads("tc::tmem_ld32(a, r[h ^ 1]);\nx = r[h ^ 1][j];\n")
    assert early_reads("tc::tmem_ld32(a, r[1]);\nx = r[c][j];\n")
    assert not early_reads(at + "r[j] = 0;\ntc::tmem_ld_wait(n);\nr[j] = n[j];\n")
    assert not early_reads("tc::tmem_ld32(a, r[h ^ 1]);\nx = r[h][j];\ntc::tmem_ld_wait(r[h ^ 1]);\n")


@pytest.mark.parametrize("name", KERNELS + ["dense.cuh", "dense_tc.cuh"])
def test_loads_are_coherent(name):
    """A block may be resident, waiting for the launch before it, while that
    launch writes the block's inputs: the read-only path (which holds for
    memory that nothing writes while the kernel lives) is not for them."""
    assert not re.findall(r"__ldg|\bldg16|\bld_nc_na|\.nc\b", code(name))


def test_pair_kernel_stays_until_the_last_arrivals():
    """The MMAs of a pair arrive on the other CTA's `empty` barriers and its
    epilogue warps on the leader's `acc_empty`: the meeting at the kernel's end
    is a relaxed one, so each CTA has to have waited for what is sent to it."""
    text = code("k_dense_gemm.cu")
    producer, rest = text[text.index("if (warp == 0) {") :].split("} else if (warp == 1 && rank == 0) {", 1)
    issuer = rest[: rest.index("} else {\n")]
    assert producer.rindex("mbar_spin(&S.empty[s]") > producer.rindex("tma_load_2d_pair(")
    assert issuer.rindex("mbar_spin(&S.acc_empty[buf]") > issuer.rindex("mma_commit_pair(&S.acc_full[buf])")


def test_split_kernel_waits_for_its_own_copies_only():
    """A wait that counts its polls starts once the launch before is done:
    however long that one takes, it uses up no limit."""
    text = code("k_dense_split.cu")
    issuer, rest = text[text.index("} else if (warp == 1) {") :].split("} else if (warp >= 4) {", 1)
    for part in (issuer, rest[: rest.index("__syncthreads();")]):
        assert "pdl_wait();" in part and part.index("pdl_wait();") < part.index("mbar_spin(")


def test_binding_holds_the_lock_again_before_an_exception_goes_on():
    """What a call lets go it takes back by a destructor: the macros' block
    would leave a C++ exception (of torch's stream lookup) without the lock that
    its translation into a Python one needs."""
    text = code("py_dense.cpp")
    assert "Py_BEGIN_ALLOW_THREADS" not in text
    assert re.search(r"~\w+\(\)\s*\{\s*PyEval_RestoreThread\(", text)
