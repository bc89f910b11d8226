"""What the products of a few rows with four-bit weights refuse, on the host and
before anything is enqueued (no GPU is needed: the pointers are never followed)."""
import pytest
import torch

import moe_expert_layer_top16_gb300 as moe
from moe_expert_layer_top16_gb300 import block
from moe_expert_layer_top16_gb300 import build as mbuild

BAD, OK = moe.MOE_ERR_INVALID_ARG, moe.MOE_OK
P = 4096


@pytest.fixture(scope="module")
def L():
    mbuild.build()
    return moe.lib()


GOOD = dict(codes=P, scales=P, up_codes=None, up_scales=None, x=P, ld_x=256, idx=P, weights=P, out=P, ld_out=64, T=2, k=4, G=8, M=64, K=256, group=32, x_per_slot=0,
            format=0, scale_dtype=0, x_dtype=1, out_dtype=1)
INTS = dict(format=1, group=64, scale_dtype=0)


def call(L, **kw):
    a = block._W4MatvecArgs()
    for n, v in {**GOOD, **kw}.items():
        setattr(a, n, v)
    return L.moe_w4_matvec(a, None)


@pytest.mark.parametrize("bad", [dict(codes=None), dict(codes=P + 8), dict(scales=None), dict(x=None), dict(x=P + 1), dict(ld_x=255), dict(out=None), dict(out=P + 1),
                                 dict(ld_out=63), dict(idx=P + 1), dict(weights=P + 2), dict(dev_status=P + 2), dict(T=-1), dict(k=0), dict(k=33), dict(T=2 ** 30), dict(G=0), dict(M=0),
                                 dict(G=2 ** 16, M=2 ** 15), dict(K=0), dict(K=48, ld_x=48), dict(K=2 ** 24 + 32, ld_x=2 ** 25), dict(group=64), dict(group=16), dict(format=2),
                                 dict(format=-1), dict(x_dtype=3), dict(out_dtype=-1), dict(idx=None), dict(idx=None, G=1), dict(up_codes=P, up_scales=P),
                                 dict(weights=None, up_codes=P), dict(weights=None, up_scales=P), dict(weights=None, up_codes=P + 8, up_scales=P),
                                 dict(INTS, group=48), dict(INTS, group=256), dict(INTS, scale_dtype=3), dict(INTS, scales=P + 2), dict(INTS, K=288, ld_x=288),
                                 dict(INTS, weights=None, up_codes=P, up_scales=P + 2)])
def test_entry_point(L, bad):
    assert call(L, **bad) == BAD


def test_null_and_empty(L):
    assert L.moe_w4_matvec(None, None) == BAD
    assert call(L, T=0, x=None, out=None, codes=None) == OK


def test_binding():
    """CPU tensors and wrong shapes raise MoeError with MOE_ERR_INVALID_ARG."""
    c, s, f = torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 8, dtype=torch.uint8), torch.zeros(4, 4)
    for bad in (lambda: moe.w4_matvec(torch.zeros(2, 256), c, s), lambda: moe.w4_matvec(None, c, s), lambda: block._w4(c, s[:, :4], 2, -1, "x"),
                lambda: block._w4(c, s.int(), 2, -1, "x"), lambda: block._w4(c, s, 3, -1, "x"), lambda: block._w4(c, s, 2, 0, "x"), lambda: block._w4(c.int(), s, 2, -1, "x"),
                lambda: block._w4(c, s[:3], 2, -1, "x"), lambda: block._w4(c, f[:, :1], 2, -1, "x"), lambda: block._w4(c, None, 2, -1, "x"),
                lambda: block._w4(c[:0], s[:0], 2, -1, "x")):
        with pytest.raises(moe.MoeError) as e:
            bad()
        assert e.value.code == BAD
    assert block._w4(c, s, 2, -1, "x")[2] == 32 and block._w4(c, f, 2, -1, "x")[2] == 64 and block._w4(c, f[:, :2], 2, -1, "x")[2] == 128
