"""Refusals of the vocabulary loss, the token rows and the balance loss without a GPU:
the library's before any CUDA call, and the binding's before the library."""
import math
import struct

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


SIZES = [(dict(M=-1), BAD), (dict(N=-1), BAD), (dict(K=-1), BAD), (dict(M=2 ** 31), BAD),
         (dict(N=2 ** 31 - 4095, ldb=2 ** 31), UNSUP), (dict(M=2 ** 31 - 1), UNSUP),
         (dict(M=2 ** 31 - 4096, N=2 ** 31 - 4096), UNSUP),          # tiles
         (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD), (dict(scale=math.nan), BAD),
         (dict(scale=math.inf), BAD), (dict(scale=2e38), BAD), (dict(flags=1), UNSUP), (dict(t=None), BAD),
         (dict(A=None), BAD), (dict(B=None), BAD), (dict(lda=56), BAD), (dict(ldb=56), BAD),
         (dict(lda=68), ALIGN), (dict(ldb=68), ALIGN), (dict(A=A16 + 2), ALIGN),
         (dict(B=A16 + 8), ALIGN), (dict(lse=None), BAD)]


@pytest.mark.parametrize("kw,code", SIZES + [(dict(loss=None), BAD), (dict(M=0, A=None), 0)])
def test_xent_rejects_before_launch(L, kw, code):
    a = dict(A=A16, lda=64, B=A16, ldb=64, t=A16, scale=1.0, loss=A16, lse=A16, M=100, N=500, K=64,
             flags=0)
    a.update(kw)
    assert L.gemm_bf16_xent(a["A"], a["lda"], a["B"], a["ldb"], a["t"], a["scale"], a["loss"],
                            a["lse"], a["M"], a["N"], a["K"], a["flags"], None) == code


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(d=2), BAD), (dict(ldda=60), BAD), (dict(lddb=60), BAD), (dict(ldda=66), ALIGN),
    (dict(dA=A16 + 8), ALIGN), (dict(dB=A16 + 4), ALIGN), (dict(M=2 ** 30), UNSUP),
    (dict(dA=None, dB=None), 0), (dict(K=0), 0)])
def test_xent_grad_rejects_before_launch(L, kw, code):
    a = dict(A=A16, lda=64, B=A16, ldb=64, t=A16, lse=A16, grad=None, scale=1.0, dA=A16, ldda=64,
             dB=A16, lddb=64, M=100, N=500, K=64, d=0, flags=0)
    a.update(kw)
    assert L.gemm_bf16_xent_grad(a["A"], a["lda"], a["B"], a["ldb"], a["t"], a["lse"], a["grad"],
                                 a["scale"], a["dA"], a["ldda"], a["dB"], a["lddb"], a["M"], a["N"],
                                 a["K"], a["d"], a["flags"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), BAD), (dict(n=2 ** 30 + 1), BAD), (dict(rows=-1), BAD), (dict(rows=2 ** 31), BAD),
    (dict(K=-1), BAD), (dict(d=3), BAD), (dict(ids=None), BAD), (dict(W=None), BAD),
    (dict(D=None), BAD), (dict(ldw=56), BAD), (dict(ldw=68), ALIGN), (dict(ldd=56), BAD),
    (dict(ldd=66), ALIGN), (dict(W=A16 + 2), ALIGN), (dict(D=A16 + 4), ALIGN),
    (dict(K=256 * 65535 + 1), UNSUP), (dict(n=0, ids=None, D=None), 0), (dict(K=0), 0)])
def test_embed_rejects_before_launch(L, kw, code):
    a = dict(W=A16, ldw=64, rows=100, ids=A16, n=10, K=64, scale=1.0, D=A16, ldd=64, d=0)
    a.update(kw)
    assert L.embed_rows(a["W"], a["ldw"], a["rows"], a["ids"], a["n"], a["K"], a["scale"], a["D"],
                        a["ldd"], a["d"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), BAD), (dict(n=2 ** 30 + 1), BAD), (dict(rows=-1), BAD), (dict(rows=2 ** 31), BAD),
    (dict(K=-1), BAD), (dict(d=3), BAD), (dict(g=2), BAD), (dict(ids=None), BAD),
    (dict(G=None), BAD), (dict(D=None), BAD), (dict(ldg=56), BAD), (dict(ldg=66), ALIGN),
    (dict(ldd=56), BAD), (dict(ldd=66), ALIGN), (dict(G=A16 + 2), ALIGN), (dict(D=A16 + 4), ALIGN),
    (dict(add=2), BAD), (dict(K=256 * 65535 + 1), UNSUP), (dict(rows=0, D=None), 0),
    (dict(K=0), 0), (dict(n=0, add=1, G=None, ids=None), 0)])
def test_embed_grad_rejects_before_launch(L, kw, code):
    a = dict(G=A16, ldg=64, g=0, ids=A16, n=10, rows=100, K=64, scale=1.0, D=A16, ldd=64, d=0, add=0)
    a.update(kw)
    assert L.embed_rows_grad(a["G"], a["ldg"], a["g"], a["ids"], a["n"], a["rows"], a["K"],
                             a["scale"], a["D"], a["ldd"], a["d"], a["add"], None) == code


ROUTER = [(dict(M=-1), BAD), (dict(M=2 ** 31), BAD), (dict(E=0), BAD),
          (dict(E=tg.TG_MAX_GROUPS + 1), BAD), (dict(k=0), BAD), (dict(k=1025), BAD),
          (dict(M=2 ** 22, k=512), UNSUP), (dict(dtype=2), BAD), (dict(z=None), BAD),
          (dict(ids=None), BAD), (dict(ld=15), BAD), (dict(shares=None), BAD)]


@pytest.mark.parametrize("kw,code", ROUTER + [(dict(loss=None), BAD), (dict(counts=None), BAD)])
def test_balance_rejects_before_launch(L, kw, code):
    a = dict(z=A16, ld=16, dtype=0, ids=A16, k=2, M=10, E=16, loss=A16, counts=A16, shares=A16)
    a.update(kw)
    assert L.tg_balance_loss(a["z"], a["ld"], a["dtype"], a["ids"], a["k"], a["M"], a["E"], a["loss"],
                             a["counts"], a["shares"], None) == code


@pytest.mark.parametrize("kw,code", ROUTER + [(dict(D=None), BAD), (dict(ldd=15), BAD),
                                              (dict(d=3), BAD), (dict(M=0, z=None), 0)])
def test_balance_grad_rejects_before_launch(L, kw, code):
    a = dict(z=A16, ld=16, dtype=0, ids=A16, k=2, M=10, E=16, shares=A16, grad=None, D=A16, ldd=16,
             d=0)
    a.update(kw)
    assert L.tg_balance_loss_grad(a["z"], a["ld"], a["dtype"], a["ids"], a["k"], a["M"], a["E"],
                                  a["shares"], a["grad"], a["D"], a["ldd"], a["d"], None) == code


def test_packed_calls_take_floats_as_their_bits(L):
    def bits(x):
        return struct.unpack("=I", struct.pack("=f", x))[0]

    def call(fn, words):
        return L.tg_call_packed(fn, struct.pack("=%dq" % len(words), *words), len(words))
    xent = [A16, 64, A16, 64, A16, bits(1.0), A16, A16, 0, 500, 64, 0, 0]
    assert call(tg.TG_FN_GEMM_BF16_XENT, xent) == 0
    assert call(tg.TG_FN_GEMM_BF16_XENT, xent[:5] + [bits(-1.0)] + xent[6:]) == BAD
    assert call(tg.TG_FN_GEMM_BF16_XENT, xent[:5] + [-1] + xent[6:]) == BAD          # not 32 bits
    assert call(tg.TG_FN_GEMM_BF16_XENT, xent[:5] + [1 << 32] + xent[6:]) == BAD
    assert call(tg.TG_FN_GEMM_BF16_XENT, xent[:-1]) == BAD
    assert call(tg.TG_FN_EMBED_ROWS, [A16, 64, 9, A16, 0, 64, bits(2.0), A16, 64, 0, 0]) == 0
    assert call(tg.TG_FN_EMBED_ROWS, [A16, 64, 9, A16, -1, 64, bits(2.0), A16, 64, 0, 0]) == BAD
    assert call(tg.TG_FN_BALANCE_LOSS_GRAD, [A16, 8, 0, A16, 2, 0, 8, A16, 0, A16, 8, 0, 0]) == 0
    assert call(11, [0] * 7) == BAD


@pytest.mark.parametrize("call,shape,kw", [
    (tg.TG_CALL_GEMM_BF16_XENT, (1, 1, 1), {}),
    (tg.TG_CALL_GEMM_BF16_XENT, (8192, 128000, 4096), {}),
    (tg.TG_CALL_GEMM_BF16_XENT_GRAD, (100, 1000, 64), dict(d_dtype=tg.TG_D_BF16)),
    (tg.TG_CALL_GEMM_BF16_XENT_GRAD, (100000, 128000, 4096), dict(d_dtype=tg.TG_D_F32)),
    (tg.TG_CALL_EMBED_ROWS_GRAD, (1, 1, 1), {}),
    (tg.TG_CALL_EMBED_ROWS_GRAD, (1 << 20, 256000, 8192), {}),
    (tg.TG_CALL_BALANCE_LOSS, (1000, 64, 1), {})])
def test_workspace_bytes_are_known_without_a_device(L, call, shape, kw):
    n = tg.workspace_bytes(call, *shape, **kw)
    assert 0 < n < 8 << 30
    # What the largest call of a stream needs serves the smaller ones.
    smaller = tuple(max(1, x // 2) for x in shape)
    assert call == tg.TG_CALL_GEMM_BF16_XENT or tg.workspace_bytes(call, *smaller, **kw) <= n


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def f32(*shape):
    return torch.zeros(shape)


@pytest.mark.parametrize("call,exc", [
    (lambda: tg.gemm_bf16_xent(f32(8, 16), bf16(9, 16), i32(8)), TypeError),
    (lambda: tg.gemm_bf16_xent(bf16(8, 16), bf16(9, 24), i32(8)), ValueError),
    (lambda: tg.gemm_bf16_xent(bf16(8, 16), bf16(9, 16), i32(7)), ValueError),
    (lambda: tg.gemm_bf16_xent(bf16(8, 16), bf16(9, 16), i32(8).long()), TypeError),
    (lambda: tg.gemm_bf16_xent(bf16(16, 8).T, bf16(9, 16), i32(8)), ValueError),
    (lambda: tg.gemm_bf16_xent_grad(bf16(8, 16), bf16(9, 16), i32(8), f32(7)), TypeError),
    (lambda: tg.gemm_bf16_xent_grad(bf16(8, 16), bf16(9, 16), i32(8), None), TypeError),
    (lambda: tg.gemm_bf16_xent_grad(bf16(8, 16), bf16(9, 16), i32(8), f32(8), f32(8, 1)), TypeError),
    (lambda: tg.gemm_bf16_xent_grad(bf16(8, 16), bf16(9, 16), i32(8), f32(8), None, f32(8, 16),
                                    bf16(9, 16)), ValueError),
    (lambda: tg.gemm_bf16_xent_grad(bf16(8, 16), bf16(9, 16), i32(8), f32(8), None, bf16(9, 16)),
     ValueError),
    (lambda: tg.gemm_bf16_xent_grad(bf16(8, 16), bf16(9, 16), i32(8), f32(8), None, bf16(8, 16),
                                    rows=False), ValueError),
    (lambda: tg.gemm_bf16_xent_grad(bf16(8, 16), bf16(9, 16), i32(8), f32(8),
                                    out_dtype=torch.float16), ValueError),
    (lambda: tg.embed_rows(f32(8, 16), i32(3)), TypeError),
    (lambda: tg.embed_rows(bf16(8, 16), i32(3, 1)), TypeError),
    (lambda: tg.embed_rows(bf16(8, 16), i32(3), bf16(4, 16)), ValueError),
    (lambda: tg.embed_rows_grad(f32(3, 16).half(), i32(3), 8), TypeError),
    (lambda: tg.embed_rows_grad(f32(3, 16), i32(4), 8), ValueError),
    (lambda: tg.embed_rows_grad(f32(3, 16), i32(3), 8, accumulate=True), ValueError),
    (lambda: tg.embed_rows_grad(f32(3, 16), i32(3), -1), ValueError),
    (lambda: tg.embed_rows_grad(f32(3, 16), i32(3), 8, f32(9, 16)), ValueError),
    (lambda: tg.balance_loss(f32(4, 8).double(), i32(4, 2)), TypeError),
    (lambda: tg.balance_loss(f32(4, 8), i32(8)), TypeError),
    (lambda: tg.balance_loss(f32(4, 8), i32(5, 2)), ValueError),
    (lambda: tg.balance_loss(f32(8, 4).T, i32(4, 2)), ValueError),
    (lambda: tg.balance_loss_grad(f32(4, 8), i32(4, 2), f32(4)), TypeError),
    (lambda: tg.balance_loss_grad(f32(4, 8), i32(4, 2), f32(8), f32(2)), TypeError),
    (lambda: tg.balance_loss_grad(f32(4, 8), i32(4, 2), f32(8), D=f32(4, 9)), ValueError),
    # Right in everything, but on the host: an address would reach the device.
    (lambda: tg.gemm_bf16_xent(bf16(8, 16), bf16(9, 16), i32(8)), ValueError),
    (lambda: tg.gemm_bf16_xent_grad(bf16(8, 16), bf16(9, 16), i32(8), f32(8)), ValueError),
    (lambda: tg.embed_rows(bf16(8, 16), i32(3)), ValueError),
    (lambda: tg.embed_rows_grad(f32(3, 16), i32(3), 8), ValueError),
    (lambda: tg.balance_loss(f32(4, 8), i32(4, 2)), ValueError),
    (lambda: tg.balance_loss_grad(f32(4, 8), i32(4, 2), f32(8)), ValueError),
])
def test_binding_rejects_before_calling_the_library(monkeypatch, call, exc):
    class Refuse:
        def __getattr__(self, name):
            raise AssertionError("the binding called the library")
    monkeypatch.setattr(tg, "_lib", Refuse())
    with pytest.raises(exc):
        call()
