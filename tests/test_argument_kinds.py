"""Arguments that are no tensors raise MoeError with MOE_ERR_INVALID_ARG, as wrong shapes do.

No GPU is needed: the checks are those behind the one for a CUDA device, which is stood in for, and every call is
refused before anything is enqueued."""
import pytest
import torch

import moe_expert_layer_top16_gb300 as moe
from moe_expert_layer_top16_gb300 import block, router

BAD = moe.MOE_ERR_INVALID_ARG


@pytest.fixture(autouse=True)
def host_device(monkeypatch):
    """CPU tensors pass for those of the current device, whose index is then -1; no entry point is reached."""
    def device(t, what):
        if not isinstance(t, torch.Tensor):
            block._bad(what + ": CUDA tensors are needed")
        return t.get_device()

    def reached():
        raise AssertionError("the call was not refused")
    for m in (block, router):
        monkeypatch.setattr(m, "_device", device)
        monkeypatch.setattr(m, "_current", lambda: -1)
        monkeypatch.setattr(m, "lib", reached)


def refused(f, *args, **kw):
    with pytest.raises(moe.MoeError) as e:
        f(*args, **kw)
    assert e.value.code == BAD


NO_TENSORS = [[1, 0], 3, "x", 2.5]


@pytest.mark.parametrize("no", NO_TENSORS, ids=str)
def test_router(no):
    x, i, f = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    refused(moe.select_experts, no, 2)
    refused(moe.select_experts, x, 2, mask=no)
    refused(moe.select_experts, x, 2, bias=no)
    refused(moe.select_experts, x, 2, score=no)
    refused(moe.balance_loss, no, i)
    refused(moe.balance_loss, x, no)
    refused(moe.balance_loss, x, i, sequences=no)
    refused(moe.router_backward, x, no, d_gates=f)
    refused(moe.router_backward, x, i, d_gates=no)
    refused(moe.router_backward, x, i, d_loss=no)
    refused(moe.router_backward, x, i, d_loss=torch.zeros(1), counts=no, tokens=no)


@pytest.mark.parametrize("no", NO_TENSORS, ids=str)
def test_products(no):
    c, s = torch.zeros(5, 4, 128, dtype=torch.uint8), torch.zeros(5, 4, 8, dtype=torch.uint8)
    x, i, w = torch.zeros(2, 256), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3)
    refused(moe.w4_matvec, no, c, s, idx=i)
    refused(moe.w4_matvec, x, no, s, idx=i)
    refused(moe.w4_matvec, x, c, no, idx=i)
    refused(moe.w4_matvec, x, c, s, idx=no)
    refused(moe.w4_matvec, x, c, s, idx=i, weights=no)
    refused(moe.w4_matvec, x, c, s, idx=i, up=no)
    refused(moe.w4_matvec, x, c, s, idx=i, up=(c, no))
    refused(moe.w4_matvec, x, c, s, idx=i, status=no)
    refused(moe.w4_matvec, x, c, s, idx=i, out=no)
    refused(moe.w4_matvec, x, c, s, idx=i, out=no, out_dtype=torch.float32)
    refused(moe.w4_matvec, x, c, s, idx=i, out_dtype=no)


@pytest.mark.parametrize("no", NO_TENSORS, ids=str)
def test_weights_of_slots(no):
    rows, pos = torch.zeros(6, 16), torch.zeros(2, 3, dtype=torch.int32)
    refused(moe.unpermute, rows, pos, no)
    refused(moe.unpermute_backward, torch.zeros(2, 16), rows, pos, no)
