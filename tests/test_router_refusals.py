"""What the router's operators refuse, on the host and before anything is
enqueued (no GPU is needed: the pointers are never followed)."""
import ctypes as C

import pytest
import torch

import moe_expert_layer_top16_gb300 as moe
from moe_expert_layer_top16_gb300 import build as mbuild
from moe_expert_layer_top16_gb300 import router

BAD, OK = moe.MOE_ERR_INVALID_ARG, moe.MOE_OK
P = 4096


@pytest.fixture(scope="module")
def L():
    mbuild.build()
    return moe.lib()


def made(kind, good, **kw):
    a = kind()
    for n, v in {**good, **kw}.items():
        setattr(a, n, v)
    return a


SELECT = dict(logits=P, ld_logits=64, bias=P, mask=P, idx=P, gates=P, T=4, E=64, k=4, dtype=1, score_fn=0, normalize=1, scale=1.0)
LOSS = dict(logits=P, ld_logits=64, idx=P, sequences=P, loss=P, counts=P, tokens=P, workspace=P, workspace_bytes=1 << 20, T=4, E=64, k=4, S=3, dtype=0, score_fn=1)
BACK = dict(logits=P, ld_logits=64, idx=P, d_gates=P, d_loss=P, counts=P, tokens=P, sequences=P, d_logits=P, ld_d_logits=64, T=4, E=64, k=4, S=3, dtype=0,
            score_fn=1, normalize=1, scale=1.0)
SHAPES = [dict(T=-1), dict(E=0), dict(E=1025, ld_logits=2000), dict(k=0), dict(k=33), dict(E=3), dict(dtype=3), dict(dtype=-1), dict(score_fn=2), dict(score_fn=-1),
          dict(logits=None), dict(logits=P + 1), dict(ld_logits=63), dict(idx=None), dict(idx=P + 2)]


@pytest.mark.parametrize("bad", SHAPES + [dict(score_fn=1), dict(bias=P + 1), dict(gates=None), dict(gates=P + 1)])
def test_select(L, bad):
    assert L.moe_select(made(router._SelectArgs, SELECT, **bad), None) == BAD


@pytest.mark.parametrize("bad", SHAPES + [dict(S=0), dict(S=(1 << 20) + 1), dict(sequences=None), dict(sequences=P + 1), dict(loss=None), dict(loss=P + 1), dict(counts=None),
                                          dict(counts=P + 1), dict(tokens=None), dict(tokens=P + 2), dict(workspace=None), dict(workspace=P + 8), dict(workspace_bytes=100)])
def test_balance_loss(L, bad):
    assert L.moe_balance_loss(made(router._BalanceLossArgs, LOSS, **bad), None) == BAD


@pytest.mark.parametrize("bad", SHAPES + [dict(d_gates=None, d_loss=None), dict(d_gates=P + 1), dict(d_loss=P + 1), dict(counts=None), dict(counts=P + 1), dict(tokens=None),
                                          dict(tokens=P + 1), dict(sequences=None), dict(sequences=P + 2), dict(S=0), dict(S=(1 << 20) + 1), dict(d_logits=None),
                                          dict(d_logits=P + 1), dict(ld_d_logits=63)])
def test_router_backward(L, bad):
    assert L.moe_router_backward(made(router._RouterBackwardArgs, BACK, **bad), None) == BAD


def test_null_and_empty(L):
    for f in (L.moe_select, L.moe_balance_loss, L.moe_router_backward):
        assert f(None, None) == BAD
    assert L.moe_select(made(router._SelectArgs, SELECT, T=0, logits=None, idx=None, gates=None), None) == OK
    assert L.moe_router_backward(made(router._RouterBackwardArgs, BACK, T=0, logits=None, idx=None, d_logits=None), None) == OK


def test_workspace(L):
    f = L.moe_balance_loss_workspace_bytes
    assert f(64, 32, 1) > 0 and f(64, 32, 9) > f(64, 32, 1) and f(0, 32, 1) == 0
    assert f(-1, 32, 1) == f(64, 0, 1) == f(64, 1025, 1) == f(64, 32, 0) == f(64, 32, (1 << 20) + 1) == 0


def test_binding():
    """CPU tensors and wrong shapes raise MoeError with MOE_ERR_INVALID_ARG."""
    x, i, f = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    w = "x"
    for call in (lambda: moe.select_experts(x, 2), lambda: moe.balance_loss(x, i), lambda: moe.router_backward(x, i, d_gates=f),
                 lambda: router._score("relu", w), lambda: router._logits(x[0], w), lambda: router._logits(torch.zeros(2, 1025), w), lambda: router._logits(x.int(), w),
                 lambda: router._logits(torch.zeros(2, 0), w), lambda: router._slots_of(i.long(), 4, 8, -1, w), lambda: router._slots_of(i, 5, 8, -1, w),
                 lambda: router._slots_of(i, 4, 1, -1, w), lambda: router._slots_of(None, 4, 8, -1, w), lambda: router._slots_of(i, 4, 8, 0, w),
                 lambda: router._slots_of(torch.zeros(4, 33, dtype=torch.int32), 4, 64, -1, w), lambda: router._sequences(i, -1, w),
                 lambda: router._sequences(i[0, :1], -1, w), lambda: router._sequences(i[0].long(), -1, w), lambda: router._sequences([0, 4], -1, w),
                 lambda: router._floats(f, (2, 4), -1, "f", w), lambda: router._floats(f.double(), (4, 2), -1, "f", w), lambda: router._floats(None, (4, 2), -1, "f", w),
                 lambda: router._ints(f, (4, 2), -1, "i", w), lambda: router._ints(i, (4,), -1, "i", w)):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.code == BAD
    assert router._sequences(None, -1, w) == (None, 1)
