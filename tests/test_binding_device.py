"""The grouped and adapter calls refuse host tensors: their addresses would reach
a kernel as device addresses.  Right in everything else, all arguments or each in
turn on the host; tensors that only say they are on a GPU stand in for the
others, so nothing is launched."""
import pytest
import torch

import blackwell_tile_gemm_gb300 as tg


@pytest.fixture(autouse=True)
def no_library(monkeypatch):
    class Refuse:
        def __getattr__(self, name):
            raise AssertionError("the binding called the library")
    monkeypatch.setattr(tg, "_lib", Refuse())


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


CALLS = {
    "group_rows": (lambda a: tg.group_rows(a["ids"], 4), dict(ids=i32(8))),
    "grouped": (lambda a: tg.gemm_bf16_grouped(a["A"], a["B"], a["off"], a["D"], row_idx=a["idx"],
                                               bias=a["bias"]),
                dict(A=bf16(8, 16), B=bf16(2, 8, 16), off=i32(3), D=torch.zeros(8, 8), idx=i32(8),
                     bias=torch.zeros(2, 8))),
    "dgrad": (lambda a: tg.gemm_bf16_grouped_dgrad(a["G"], a["B"], a["off"], a["D"]),
              dict(G=bf16(8, 8), B=bf16(2, 8, 16), off=i32(3), D=torch.zeros(8, 16))),
    "wgrad": (lambda a: tg.gemm_bf16_grouped_wgrad(a["G"], a["A"], a["off"], a["D"],
                                                   row_idx=a["idx"]),
              dict(G=bf16(8, 8), A=bf16(8, 16), off=i32(3), D=torch.zeros(2, 8, 16), idx=i32(8))),
    "lora": (lambda a: tg.gemm_bf16_lora(a["A"], a["B"], a["ids"], a["down"], a["up"], a["D"],
                                         scales=a["s"], bias=a["bias"]),
             dict(A=bf16(8, 16), B=bf16(8, 16), ids=i32(8), down=bf16(2, 8, 16), up=bf16(2, 8, 8),
                  D=torch.zeros(8, 8), s=torch.zeros(2), bias=torch.zeros(8))),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_host_tensors_are_refused(name):
    call, args = CALLS[name]
    with pytest.raises(ValueError, match="device"):
        call(args)


class Elsewhere(torch.Tensor):
    """A host tensor that says it lives on the first GPU."""
    def get_device(self):
        return 0


@pytest.mark.parametrize("name,host", [(n, a) for n in sorted(CALLS) for a in CALLS[n][1]])
def test_one_host_tensor_among_others_is_refused(name, host, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    call, args = CALLS[name]
    mixed = {k: t if k == host else t.as_subclass(Elsewhere) for k, t in args.items()}
    with pytest.raises(ValueError, match="device"):
        call(mixed)
