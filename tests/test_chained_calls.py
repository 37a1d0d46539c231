"""Before its griddep_wait a chained kernel of the loss, token rows and balance only sets up
what is on chip: it calls nothing but what is named here, so that no read of memory can hide
in a helper."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "blackwell_tile_gemm_gb300", "csrc")

ON_CHIP = {"for", "if", "while", "sizeof", "min", "static_cast", "reinterpret_cast", "constexpr",
           "smem_addr", "cluster_ctarank", "map_to_cta", "mbar_init", "fence_barrier_init",
           "prefetch_tensormap", "tmem_alloc", "tmem_relinquish", "tc_fence_before_sync",
           "tc_fence_after_sync", "__syncthreads", "cluster_sync", "__align__",
           "griddep_wait"}


def kernels(name):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    for part in re.split(r"__global__", text)[1:]:
        kernel = re.search(r"(\w+_kernel)\(", part).group(1)
        body = part[part.index("{"):]
        body = body[:body.index("\n}\n")]
        if "griddep_wait();" in body:
            yield kernel, body


@pytest.mark.parametrize("name,count", [("xent_kernel.cuh", 1), ("gemm_xent.cu", 2),
                                        ("embed_rows.cu", 7), ("balance_loss.cu", 3)])
def test_nothing_else_is_called_before_the_wait(name, count):
    found = list(kernels(name))
    assert len(found) == count, [k for k, _ in found]
    for kernel, body in found:
        before = body[:body.index("griddep_wait();")]
        called = set(re.findall(r"(\w+)\s*(?:<[^<>();]*>)?\s*\(", before))
        assert called <= ON_CHIP, (kernel, called - ON_CHIP)
        # No pointer of the arguments is followed either.
        assert not re.search(r"p\.\w+\s*\[|\*\s*p\.\w+\s*[;,)]|->", before), kernel


def test_a_read_in_a_helper_is_seen():
    body = "{\n  const int a = helper(p);\n  griddep_wait();\n"
    called = set(re.findall(r"(\w+)\s*(?:<[^<>();]*>)?\s*\(", body[:body.index("griddep_wait();")]))
    assert called - ON_CHIP == {"helper"}
