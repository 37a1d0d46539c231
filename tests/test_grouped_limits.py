"""Extents of the grouped and adapter calls close to 2^31 are refused before any
CUDA call: the kernels count rows, columns and terms in 32 bits and go past an
extent by up to a tile, so 2^31 - 1 rows of one group wrapped to none."""
import pytest

import blackwell_tile_gemm_gb300 as tg
from blackwell_tile_gemm_gb300 import build as tgbuild

A16 = 0x10000           # a 16-byte aligned fake device address (never dereferenced)
TOO_MANY = [2 ** 31 - 1, 2 ** 31 - 255, 2 ** 31 - 4095]


@pytest.fixture(scope="module")
def L():
    tgbuild.build()
    return tg.lib()


def sizes(axis, n):
    s = dict(M=8, N=64, K=64)
    s[axis] = n
    return s["M"], s["N"], s["K"]


def up8(n):
    return (n + 7) // 8 * 8


@pytest.mark.parametrize("n", TOO_MANY)
@pytest.mark.parametrize("axis", ["M", "N", "K"])
def test_grouped_calls_refuse(L, axis, n):
    M, N, K = sizes(axis, n)
    assert L.gemm_bf16_grouped(A16, up8(K), M, None, A16, 1, M, A16, up8(K), 0, A16, up8(N), N, K, 0,
                               None, 0, None) == tg.TG_ERR_UNSUPPORTED
    assert L.gemm_bf16_grouped_dgrad(A16, up8(N), A16, 1, M, A16, up8(K), 0, A16, up8(K), N, K, 0, 0,
                                     None) == tg.TG_ERR_UNSUPPORTED
    assert L.gemm_bf16_grouped_wgrad(A16, up8(N), A16, up8(K), M, None, A16, 1, M, A16, up8(K), 0, N,
                                     K, 0, 0, None) == tg.TG_ERR_UNSUPPORTED


@pytest.mark.parametrize("n", TOO_MANY)
@pytest.mark.parametrize("axis", ["M", "N", "K"])
def test_lora_refuses(L, axis, n):
    M, N, K = sizes(axis, n)
    assert L.gemm_bf16_lora(A16, up8(K), A16, up8(K), A16, A16, up8(K), 0, A16, 8, 0, None, 1, 8, A16,
                            up8(N), M, N, K, 0, None, 0, None) == tg.TG_ERR_UNSUPPORTED
