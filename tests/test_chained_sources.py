"""Kernels launched beside the one before them (programmatic dependent launch)
read what that kernel may have written only behind griddep_wait.  Loads through
the read-only path (__ldg) need not stay behind it: the compiler may move one
whose address it knows.  So these kernels use none, or make the address unknown
until the wait is over."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "blackwell_tile_gemm_gb300", "csrc")


def code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


@pytest.mark.parametrize("name", ["group_rows.cu", "grouped_kernel.cuh"])
def test_no_read_only_loads_by_intrinsic(name):
    text = code(name)
    assert "griddep_wait()" in text
    assert "__ldg(" not in text and "__restrict__" not in text


def test_the_rank_value_kernel_reads_its_rows_behind_the_wait():
    text = code("gemm_lora.cu")
    assert text.count("__ldg(") == 1                # load8, for rows of A and of `down`
    body = text[text.index("lora_down_kernel(const DownArgs p)"):text.index("constexpr int kLongRun")]
    wait = body.index("griddep_wait()")
    opaque = body.index('asm volatile("" : "+l"(A))')
    assert wait < opaque < body.index("load8(A +")
    assert "load8(p.A" not in body
    # `down` by an id, the ids by plain loads behind the wait.
    assert wait < body.index("p.ids[row0 + lane]") < body.index("p.down + id * p.stride_down")


def test_the_chained_row_copy_reads_its_index_behind_the_wait():
    """Its rows may go through the read-only path: their addresses come from it."""
    text = code("gemm_gather.cu")
    body = text[text.index("void gather_rows_kernel"):text.index("size_t gather_workspace_bytes")]
    assert "kChained ? __ldcg(idx + i)" in body
    assert body.index("griddep_wait()") < body.index("__ldcg(idx + i)") < body.index("__ldg(av + k)")


def test_epilogue_warps_that_meet_later_agree_on_every_wait():
    """A wait that runs out in one warp and completes in the next must not send
    the one home and the other to a barrier of both: where a plan has split
    tiles, whose warps all meet, one thread decides every wait of the epilogue,
    also those of the whole tiles before (whose own S is 1)."""
    text = code("grouped_kernel.cuh")
    body = text[text.index("auto acc_ready = "):text.index("auto hand_back = ")]
    assert "C::kTail && plan.S > 1" in body
    assert not re.search(r"(?<!plan\.)\bS > 1", body)
    # Every wait for an accumulator goes through it.
    assert text.count("mbar_wait(&accf_bar") == body.count("mbar_wait(&accf_bar") == 2
