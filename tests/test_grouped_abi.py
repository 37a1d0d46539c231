"""Refusals of the grouped calls, tg_group_rows and gemm_bf16_lora without a
GPU: the library's before any CUDA call, and the binding's before the library."""
import ctypes

import pytest
import torch

import blackwell_tile_gemm_gb300 as tg
from blackwell_tile_gemm_gb300 import build as tgbuild

A16 = 0x10000           # a 16-byte aligned fake device address (never dereferenced)


@pytest.fixture(scope="module")
def L():
    tgbuild.build()
    return tg.lib()


BAD, ALIGN, UNSUP = tg.TG_ERR_INVALID_ARG, tg.TG_ERR_MISALIGNED, tg.TG_ERR_UNSUPPORTED


def forward(L, **kw):
    a = dict(A=A16, lda=64, a_rows=100, idx=None, off=A16, groups=4, M=100, B=A16, ldb=64,
             gsb=64 * 64, D=A16, ldd=64, N=64, K=64, d=0, epi=None, flags=0)
    a.update(kw)
    return L.gemm_bf16_grouped(a["A"], a["lda"], a["a_rows"], a["idx"], a["off"], a["groups"], a["M"],
                               a["B"], a["ldb"], a["gsb"], a["D"], a["ldd"], a["N"], a["K"], a["d"],
                               a["epi"], a["flags"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), BAD), (dict(N=-1), BAD), (dict(K=-1), BAD), (dict(a_rows=-1), BAD),
    (dict(M=2 ** 31), BAD), (dict(groups=0), BAD), (dict(groups=tg.TG_MAX_GROUPS + 1), BAD),
    (dict(d=2), BAD), (dict(flags=1), UNSUP), (dict(off=None), BAD),
    (dict(A=None), BAD), (dict(B=None), BAD), (dict(D=None), BAD),
    (dict(lda=56), BAD), (dict(ldb=56), BAD), (dict(ldd=56), BAD),
    (dict(lda=68), ALIGN), (dict(ldb=68), ALIGN), (dict(ldd=66), ALIGN),
    (dict(A=A16 + 2), ALIGN), (dict(B=A16 + 8), ALIGN), (dict(D=A16 + 4), ALIGN),
    (dict(gsb=64 * 64 - 8), BAD), (dict(gsb=64 * 64 + 4), ALIGN),
    (dict(a_rows=99), BAD),                       # fewer rows of A than the product has
    (dict(a_rows=0, idx=A16), BAD),
    (dict(M=2 ** 31 - 1, N=2 ** 31 - 8, ldd=2 ** 31 - 8, gsb=2 ** 40), UNSUP),   # tiles
])
def test_forward_rejects_before_launch(L, kw, code):
    assert forward(L, **kw) == code


def test_forward_epilogue_and_empty_problems(L):
    bad = tg.tg_epilogue(9, 0.0, 0.0, None)
    assert forward(L, epi=ctypes.byref(bad)) == BAD
    assert forward(L, epi=ctypes.byref(tg.tg_epilogue(tg.TG_EPI_BIAS_COL, 0, 0, None))) == BAD
    assert forward(L, M=0, A=None, D=None, off=None) == tg.TG_OK
    assert forward(L, N=0, B=None, D=None) == tg.TG_OK


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), BAD), (dict(groups=0), BAD), (dict(d=5), BAD), (dict(flags=2), UNSUP),
    (dict(off=None), BAD), (dict(G=None), BAD), (dict(B=None), BAD), (dict(D=None), BAD),
    (dict(ldg=60), BAD), (dict(ldg=68), ALIGN), (dict(ldb=60), BAD), (dict(ldd=60), BAD),
    (dict(D=A16 + 8), ALIGN), (dict(gsb=8), BAD), (dict(M=0), 0), (dict(K=0), 0),
])
def test_dgrad_rejects_before_launch(L, kw, code):
    a = dict(G=A16, ldg=64, off=A16, groups=4, M=100, B=A16, ldb=64, gsb=64 * 64, D=A16, ldd=64,
             N=64, K=64, d=0, flags=0)
    a.update(kw)
    assert L.gemm_bf16_grouped_dgrad(a["G"], a["ldg"], a["off"], a["groups"], a["M"], a["B"],
                                     a["ldb"], a["gsb"], a["D"], a["ldd"], a["N"], a["K"], a["d"],
                                     a["flags"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), BAD), (dict(groups=0), BAD), (dict(d=5), BAD), (dict(flags=2), UNSUP),
    (dict(off=None), BAD), (dict(G=None), BAD), (dict(A=None), BAD), (dict(D=None), BAD),
    (dict(ldg=60), BAD), (dict(ldg=68), ALIGN), (dict(lda=60), BAD), (dict(ldd=60), BAD),
    (dict(D=A16 + 8), ALIGN), (dict(gsd=8), BAD), (dict(gsd=64 * 64 + 2), ALIGN),
    (dict(a_rows=99), BAD), (dict(a_rows=-1), BAD), (dict(N=0), 0), (dict(K=0), 0),
])
def test_wgrad_rejects_before_launch(L, kw, code):
    a = dict(G=A16, ldg=64, A=A16, lda=64, a_rows=100, idx=None, off=A16, groups=4, M=100, D=A16,
             ldd=64, gsd=64 * 64, N=64, K=64, d=0, flags=0)
    a.update(kw)
    assert L.gemm_bf16_grouped_wgrad(a["G"], a["ldg"], a["A"], a["lda"], a["a_rows"], a["idx"],
                                     a["off"], a["groups"], a["M"], a["D"], a["ldd"], a["gsd"],
                                     a["N"], a["K"], a["d"], a["flags"], None) == code


@pytest.mark.parametrize("n,groups,ids,off,order,code", [
    (-1, 4, A16, A16, A16, BAD), (2 ** 30 + 1, 4, A16, A16, A16, BAD), (8, 0, A16, A16, A16, BAD),
    (8, tg.TG_MAX_GROUPS + 1, A16, A16, A16, BAD), (8, 4, None, A16, A16, BAD),
    (8, 4, A16, None, A16, BAD), (8, 4, A16, A16, None, BAD),
])
def test_group_rows_rejects_before_launch(L, n, groups, ids, off, order, code):
    assert L.tg_group_rows(ids, n, groups, off, order, None, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), BAD), (dict(adapters=-1), BAD), (dict(rank=0), BAD), (dict(d=3), BAD),
    (dict(rank=12), UNSUP), (dict(rank=tg.TG_MAX_RANK + 8), UNSUP), (dict(flags=1), UNSUP),
    (dict(A=None), BAD), (dict(B=None), BAD), (dict(ids=None), BAD), (dict(down=None), BAD),
    (dict(up=None), BAD), (dict(D=None), BAD), (dict(lda=56), BAD), (dict(lda=68), ALIGN),
    (dict(ld_down=56), BAD), (dict(ld_up=8), BAD), (dict(ld_up=20, step_up=2048), ALIGN),
    (dict(down=A16 + 2), ALIGN), (dict(up=A16 + 8), ALIGN), (dict(step_down=64), BAD),
    (dict(step_up=64), BAD), (dict(step_down=16 * 64 + 4), ALIGN), (dict(ldd=60), BAD),
    (dict(D=A16 + 4), ALIGN), (dict(M=0), 0), (dict(N=0), 0),
])
def test_lora_rejects_before_launch(L, kw, code):
    a = dict(A=A16, lda=64, B=A16, ldb=64, ids=A16, down=A16, ld_down=64, step_down=16 * 64, up=A16,
             ld_up=16, step_up=16 * 64, scales=None, adapters=4, rank=16, D=A16, ldd=64, M=8, N=64,
             K=64, d=0, epi=None, flags=0)
    a.update(kw)
    assert L.gemm_bf16_lora(a["A"], a["lda"], a["B"], a["ldb"], a["ids"], a["down"], a["ld_down"],
                            a["step_down"], a["up"], a["ld_up"], a["step_up"], a["scales"],
                            a["adapters"], a["rank"], a["D"], a["ldd"], a["M"], a["N"], a["K"],
                            a["d"], a["epi"], a["flags"], None) == code


@pytest.mark.parametrize("call,shape,want", [
    (tg.TG_CALL_GROUP_ROWS, (2048, 64, 1), 0),                    # one CTA
    (tg.TG_CALL_GROUP_ROWS, (2049, 64, 1), 2 * 65 * 4),           # CTAs of 2048 rows
    (tg.TG_CALL_GROUP_ROWS, (1 << 22, 256, 1), 256 * 257 * 4),    # at most 256 of them
    (tg.TG_CALL_GEMM_BF16_LORA, (64, 16, 1), 64 * 16 * 6),
    (tg.TG_CALL_GEMM_BF16_LORA, (1000, 24, 1), 144128 + 1000 * 4 + (2 * (1000 // 192) + 2) * 4),
])
def test_workspace_bytes(L, call, shape, want):
    assert tg.workspace_bytes(call, *shape) == want


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


@pytest.mark.parametrize("call,exc", [
    (lambda: tg.group_rows(torch.zeros(4, dtype=torch.int64), 4), TypeError),
    (lambda: tg.group_rows(i32(4, 2), 4), TypeError),
    (lambda: tg.group_rows(i32(8)[::2], 4), TypeError),
    (lambda: tg.gemm_bf16_grouped(bf16(8, 16), bf16(2, 4, 32), i32(3)), ValueError),      # K
    (lambda: tg.gemm_bf16_grouped(bf16(8, 16), bf16(4, 16), i32(3)), ValueError),         # B 2-D
    (lambda: tg.gemm_bf16_grouped(torch.zeros(8, 16), bf16(2, 4, 16), i32(3)), TypeError),
    (lambda: tg.gemm_bf16_grouped(bf16(8, 16), bf16(2, 4, 16), i32(2)), ValueError),      # offsets
    (lambda: tg.gemm_bf16_grouped(bf16(8, 16), bf16(2, 4, 16), i32(3).long()), TypeError),
    (lambda: tg.gemm_bf16_grouped(bf16(16, 8).T, bf16(2, 4, 16), i32(3)), ValueError),    # stride
    (lambda: tg.gemm_bf16_grouped(bf16(8, 16), bf16(2, 4, 16), i32(3), torch.zeros(8, 5)),
     ValueError),
    (lambda: tg.gemm_bf16_grouped(bf16(8, 16), bf16(2, 4, 16), i32(3), bias=torch.zeros(4)),
     ValueError),                                                                # not one a group
    (lambda: tg.gemm_bf16_grouped(bf16(8, 16), bf16(2, 4, 16), i32(3), bias=torch.zeros(2, 4),
                                  affine=(1.0, 0.0)), ValueError),
    (lambda: tg.gemm_bf16_grouped(bf16(8, 16), bf16(2, 4, 16), i32(3), out_dtype=torch.float16),
     ValueError),
    (lambda: tg.gemm_bf16_grouped_dgrad(bf16(8, 5), bf16(2, 4, 16), i32(3)), ValueError),
    (lambda: tg.gemm_bf16_grouped_wgrad(bf16(8, 5), bf16(7, 16), i32(3)), ValueError),
    (lambda: tg.gemm_bf16_grouped_wgrad(bf16(8, 5), bf16(7, 16), i32(3), row_idx=i32(7)),
     ValueError),
    (lambda: tg.gemm_bf16_grouped_wgrad(bf16(8, 5), bf16(8, 16), i32(1)), ValueError),
    (lambda: tg.gemm_bf16_lora(bf16(8, 16), bf16(4, 16), i32(7), bf16(2, 8, 16), bf16(2, 4, 8)),
     ValueError),                                                                # ids
    (lambda: tg.gemm_bf16_lora(bf16(8, 16), bf16(4, 16), i32(8), bf16(2, 8, 16), bf16(2, 5, 8)),
     ValueError),                                                                # up
    (lambda: tg.gemm_bf16_lora(bf16(8, 16), bf16(4, 16), i32(8), bf16(2, 8, 16), bf16(2, 4, 8),
                               scales=torch.zeros(3)), TypeError),
    (lambda: tg.gemm_bf16_lora(bf16(8, 16), bf16(4, 16), i32(8), bf16(3, 8, 16), bf16(2, 4, 8)),
     ValueError),
])
def test_binding_rejects_before_calling_the_library(monkeypatch, call, exc):
    class Refuse:
        def __getattr__(self, name):
            raise AssertionError("the binding called the library")
    monkeypatch.setattr(tg, "_lib", Refuse())
    with pytest.raises(exc):
        call()


def test_packed_calls(L):
    """tg_call_packed checks what it unpacks and returns what the call does."""
    import struct
    rows = [A16, 0, 4, A16, A16, A16, 0]
    lora = [A16, 64, A16, 64, A16, A16, 64, 1024, A16, 16, 1024, 0, 4, 16, A16, 64, 0, 64, 64, 0, 0,
            0, 0]

    def call(fn, words, count=None):
        return L.tg_call_packed(fn, struct.pack("=%dq" % len(words), *words),
                                len(words) if count is None else count)
    assert call(tg.TG_FN_GEMM_BF16_LORA, lora) == 0                       # M = 0: nothing to do
    assert call(tg.TG_FN_GEMM_BF16_LORA, lora[:1] + [60] + lora[2:]) == 0
    assert call(tg.TG_FN_GEMM_BF16_LORA, lora[:13] + [12] + lora[14:]) == UNSUP   # rank 12
    assert call(tg.TG_FN_GEMM_BF16_LORA, lora[:16] + [-1] + lora[17:]) == BAD
    assert call(tg.TG_FN_GEMM_BF16_LORA, lora, 22) == BAD
    assert call(tg.TG_FN_GEMM_BF16_LORA, lora[:19] + [1 << 32] + lora[20:]) == BAD   # not an int
    assert call(tg.TG_FN_GROUP_ROWS, [A16, -1, 4, A16, A16, A16, 0]) == BAD
    assert call(5, rows) == BAD
    assert call(-1, rows) == BAD
    assert L.tg_call_packed(tg.TG_FN_GROUP_ROWS, None, 7) == BAD
