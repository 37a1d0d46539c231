"""Calls of the loss, token rows and balance that the binding or the library has to
refuse, without a GPU."""
import pytest
import torch

import blackwell_tile_gemm_gb300 as tg
from blackwell_tile_gemm_gb300 import build as tgbuild

A16 = 0x10000           # a 16-byte aligned fake device address (never dereferenced)
BAD, ALIGN, UNSUP = tg.TG_ERR_INVALID_ARG, tg.TG_ERR_MISALIGNED, tg.TG_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    tgbuild.build()
    return tg.lib()


@pytest.fixture
def no_library(monkeypatch):
    class Refuse:
        def __getattr__(self, name):
            raise AssertionError("the binding called the library")
    monkeypatch.setattr(tg, "_lib", Refuse())


@pytest.mark.parametrize("loss", [None, A16])
@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), BAD), (dict(scale=0.0), BAD), (dict(lse=None), BAD), (dict(t=None), BAD),
    (dict(d=2), BAD), (dict(ldda=60), BAD), (dict(ldda=66), ALIGN), (dict(M=2 ** 30), UNSUP),
    (dict(flags=1), UNSUP), (dict(dA=None, dB=None), 0), (dict(K=0), 0)])
def test_gradient_with_the_loss_rejects_before_launch(L, kw, code, loss):
    a = dict(t=A16, lse=A16, scale=1.0, dA=A16, ldda=64, dB=A16, M=100, N=500, K=64, d=0, flags=0)
    a.update(kw)
    assert L.gemm_bf16_xent_grad_ex(A16, 64, A16, 64, a["t"], a["lse"], loss, None, a["scale"],
                                    a["dA"], a["ldda"], a["dB"], 64, a["M"], a["N"], a["K"], a["d"],
                                    a["flags"], None) == code


@pytest.mark.parametrize("loss", [torch.zeros(7), torch.zeros(8, 1), torch.zeros(8).double(),
                                  torch.zeros(16)[::2]])
def test_a_loss_of_another_form_is_refused(no_library, loss):
    A, B = torch.zeros(8, 16, dtype=torch.bfloat16), torch.zeros(9, 16, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        tg.gemm_bf16_xent_grad(A, B, torch.zeros(8, dtype=torch.int32), torch.zeros(8), loss=loss)


@pytest.mark.parametrize("rows", [2, 5])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_of_a_router_that_share_memory_are_refused(no_library, rows, dtype):
    """One row for all tokens, or rows that overlap: reading them a row's width apart would
    leave the tensor."""
    ids = torch.zeros(rows, 2, dtype=torch.int32)
    fine = torch.zeros(rows, 8, dtype=dtype)
    for shared in (torch.zeros(8, dtype=dtype).expand(rows, 8),
                   torch.zeros(64, dtype=dtype).as_strided((rows, 8), (4, 1))):
        for call in (lambda: tg.balance_loss(shared, ids),
                     lambda: tg.balance_loss_grad(shared, ids, torch.zeros(8)),
                     lambda: tg.balance_loss_grad(fine, ids, torch.zeros(8), D=shared)):
            with pytest.raises(ValueError, match="overlap"):
                call()


XENT, GRAD, TABLE, BALANCE = (tg.TG_CALL_GEMM_BF16_XENT, tg.TG_CALL_GEMM_BF16_XENT_GRAD,
                              tg.TG_CALL_EMBED_ROWS_GRAD, tg.TG_CALL_BALANCE_LOSS)
MOST = 2 ** 31 - 1


@pytest.mark.parametrize("call,sizes,d,code", [
    (XENT, (MOST, 1, 1), 0, UNSUP), (XENT, (2 ** 31 - 4096, 2 ** 31 - 4096, 1), 0, UNSUP),
    (GRAD, (MOST, 1, MOST), 1, UNSUP), (GRAD, (1, MOST, MOST), 1, UNSUP),
    (GRAD, (MOST, MOST, MOST), 0, UNSUP), (GRAD, (2 ** 30, 1000, 64), 0, UNSUP),
    (GRAD, (100, 1000, 64), 2, BAD), (TABLE, (2 ** 30 + 1, 1, 1), 0, BAD),
    (TABLE, (1, 1, 256 * 65535 + 1), 0, UNSUP), (BALANCE, (9, tg.TG_MAX_GROUPS + 1, 1), 0, BAD)])
def test_no_workspace_is_named_for_sizes_that_are_refused(L, call, sizes, d, code):
    """(Some of them have no 64-bit number of bytes at all.)"""
    with pytest.raises(tg.TgError) as e:
        tg.workspace_bytes(call, *sizes, d_dtype=d)
    assert e.value.code == code


@pytest.mark.parametrize("call,sizes,d", [
    (XENT, (2 ** 31 - 4096, 16000, 64), 0), (XENT, (1, 2 ** 31 - 4096, 64), 0),
    (GRAD, (2 ** 31 - 4096, 1000, 64), 1), (GRAD, (2 ** 30 - 2048, 1000, 64), 0),
    (GRAD, (1000, 2 ** 31 - 4096, 64), 0), (GRAD, (64, 1000, 2 ** 31 - 4096), 0),
    (TABLE, (2 ** 30, MOST, 256 * 65535), 0), (BALANCE, (9, tg.TG_MAX_GROUPS, 1), 0)])
def test_the_largest_sizes_have_a_workspace(L, call, sizes, d):
    assert 0 < tg.workspace_bytes(call, *sizes, d_dtype=d) < 2 ** 50


def test_the_gradient_with_the_loss_as_packed_words(L):
    import struct

    def call(words):
        return L.tg_call_packed(tg.TG_FN_GEMM_BF16_XENT_GRAD_EX,
                                struct.pack("=%dq" % len(words), *words), len(words))
    one = struct.unpack("=I", struct.pack("=f", 1.0))[0]
    # A, lda, B, ldb, targets, lse, loss, grad, scale, dA, ldda, dB, lddb, M, N, K, type, flags, stream
    words = [A16, 64, A16, 64, A16, A16, A16, 0, one, 0, 64, 0, 64, 100, 500, 64, 0, 0, 0]
    assert call(words) == 0                                   # neither gradient is wanted
    assert call(words[:-1]) == BAD
    assert call(words[:8] + [-1] + words[9:]) == BAD          # no float
    assert call(words[:9] + [A16, 60] + words[11:]) == BAD
