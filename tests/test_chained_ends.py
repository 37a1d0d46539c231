"""The loss, token rows and balance kernels are launched beside the one before them:
what that may have written they read behind griddep_wait, and not through loads that
the compiler may move before it (read-only intrinsics, restricted pointers)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "blackwell_tile_gemm_gb300", "csrc")


def code(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


@pytest.mark.parametrize("name", ["xent_kernel.cuh", "gemm_xent.cu", "embed_rows.cu",
                                  "balance_loss.cu", "grouped_sliced.cu"])
def test_no_read_only_loads(name):
    text = code(name)
    assert "__ldg(" not in text and "__restrict__" not in text and "ld_global_nc" not in text


@pytest.mark.parametrize("name,unchained", [("gemm_xent.cu", ["xent_zero_kernel"]),
                                            ("embed_rows.cu", []), ("balance_loss.cu", []),
                                            ("xent_kernel.cuh", [])])
def test_every_chained_kernel_waits(name, unchained):
    """Each kernel has its own wait, before it reads anything that a pointer leads to."""
    text = code(name)
    parts = re.split(r"__global__", text)[1:]
    assert parts
    for part in parts:
        kernel = re.search(r"(\w+_kernel)\(", part).group(1)
        body = part[part.index("{"):]
        if kernel in unchained:
            assert "griddep_wait" not in body.split("__global__")[0][:2000].split("\n}\n")[0]
            continue
        assert "griddep_wait();" in body, kernel
        before = body[:body.index("griddep_wait();")]
        for read in (r"\[row\]", "__ldc", r"p\.(ids|targets|sorted|order|lse|grad)\["):
            assert not re.search(read, before), (kernel, read)
