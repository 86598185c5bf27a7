"""Rules that the kernels' sources keep, checked on the text (comments left out)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "swiglu_gated_mlp_gb300", "csrc")


def code(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


OVERLAPPING = sorted(os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cu")) if "pdl_wait(" in code(p))


def test_the_fused_kernels_are_covered():
    assert {"backward_pair.cu", "fused_large_m_pair.cu", "fused_small_m.cu", "lora_shrink.cu"} <= set(OVERLAPPING)


@pytest.mark.parametrize("name", OVERLAPPING + ["ptx.cuh", "lora_lb.cuh"])
def test_no_read_only_loads_where_grids_overlap(name):
    # A read-only load asks for memory that nothing writes while the kernel is resident, and
    # may be moved ahead of the grid-dependency wait. A kernel that starts while the one
    # before it still writes its inputs may not use one, nor promise it by __restrict__.
    text = code(os.path.join(CSRC, name))
    for word in ("__ldg", "ld.global.nc", "__restrict__"):
        assert word not in text, word


REMOTE = sorted(os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cu")) if "ld_shared_cluster_v4(" in code(p))


@pytest.mark.parametrize("name", REMOTE)
def test_reads_of_a_peers_memory_come_before_its_end(name):
    # The barrier that holds a CTA until its peers have read its shared memory releases, or (relaxed,
    # which orders no reads) comes behind stores of all that was read: no part that is left out of
    # the sums is loaded.
    text = code(os.path.join(CSRC, name))
    after = text[text.rindex("ld_shared_cluster_v4("):]
    first = re.search(r"cluster_(sync|arrive_release|arrive)\(", after).group(1)
    if first == "arrive":
        assert re.search(r"if \(k < splits\)\s+a\[k\] = ld_shared_cluster_v4\(mapa_shared\(local, static_cast<uint32_t>\(k\)\)", text)
        assert text.count("ld_shared_cluster_v4(") == 1


PAIRED = sorted(os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cu")) if "tmem_alloc_pair(" in code(p))


def test_the_pair_kernels_are_covered():
    assert PAIRED == ["backward_pair.cu", "fused_large_m_pair.cu", "fused_resident_pair.cu", "int8_gemm.cu"]


@pytest.mark.parametrize("name", PAIRED)
def test_pairs_allocate_tensor_memory_in_step(name):
    # Nothing bounds the wait of a CTA pair's allocation, so both CTAs run by then, all grids before
    # have completed, the right to allocate goes behind a barrier, and neither CTA leaves before both
    # have given the memory back.
    text = re.sub(r"\s+", " ", code(os.path.join(CSRC, name)))
    assert text.count("tmem_alloc_pair(") == 1
    before, rest = text.split("if (warp == 1) tmem_alloc_pair(")
    assert re.search(r"cluster_arrive\(\); cluster_wait\(\); [^;]*pdl_wait\(\); $", before), before[-120:]
    wait = before.rsplit(";", 2)[1]  # what is waited on: always, or with any condition by the warp that allocates
    assert wait.strip() == "pdl_wait()" or re.search(r"\|\| warp == 1\) pdl_wait\(\)$", wait), wait
    assert re.search(r"^[^;]*; tc_fence_before\(\); cluster_arrive\(\); if \(warp != 0\) cluster_wait\(\); "
                     r"tc_fence_after\(\); if \(warp == 1\) tmem_relinquish_pair\(\);", rest), rest[:200]
    assert "cluster_arrive(); cluster_wait();" in rest.split("tmem_dealloc_pair(")[1]
