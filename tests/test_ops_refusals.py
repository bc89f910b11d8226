"""What the operators round the layer refuse, on the host and before anything
is enqueued (no GPU is needed: the pointers are never followed)."""
import ctypes as C

import pytest
import torch

import moe_expert_layer_top16_gb300 as moe
from moe_expert_layer_top16_gb300 import block
from moe_expert_layer_top16_gb300 import build as mbuild

BAD, OK = moe.MOE_ERR_INVALID_ARG, moe.MOE_OK
P, ODD = C.c_void_p(4096), C.c_void_p(4097)


@pytest.fixture(scope="module")
def L():
    mbuild.build()
    return moe.lib()


def refuse(f, good, changes):
    for i, v in changes:
        args = list(good)
        args[i] = v
        assert f(*args) == BAD, (f.__name__, i, v)


def test_sort(L):
    refuse(L.moe_sort, [P, 4, 2, 8, P, P, P, None, 0, None],
           [(0, None), (1, -1), (2, 0), (2, 33), (3, 0), (3, 1025), (4, None), (5, None), (6, None), (0, ODD), (4, ODD),
            (1, 2 ** 30), (7, ODD)])
    need = L.moe_sort_workspace_bytes(9000, 16, 896)
    assert need > 0 and L.moe_sort_workspace_bytes(64, 16, 896) == 0 and L.moe_sort_workspace_bytes(-1, 16, 896) == 0
    refuse(L.moe_sort, [P, 9000, 16, 896, P, P, P, P, need, None], [(7, None), (8, need - 1)])


def test_permute(L):
    good = [P, 64, 64, 4, 2, P, 8, P, 64, None]
    refuse(L.moe_permute, good, [(0, None), (1, 63), (2, 0), (3, -1), (4, 0), (4, 33), (5, None), (5, ODD), (6, -1), (7, None), (8, 32)])
    for i, v in ((3, 0), (6, 0)):
        args = list(good)
        args[i] = v
        assert L.moe_permute(*args) == OK           # nothing to do


def test_unpermute(L):
    good = [P, 16, 0, 8, P, P, 4, 2, 16, P, 16, 0, None]
    refuse(L.moe_unpermute, good, [(0, None), (0, ODD), (1, 15), (2, 3), (2, -1), (3, -1), (4, None), (5, ODD), (6, -1), (7, 0),
                                   (7, 33), (8, 0), (9, None), (9, ODD), (10, 15), (11, 3)])
    good[6] = 0
    assert L.moe_unpermute(*good) == OK


def test_unpermute_backward(L):
    good = [P, 16, 0, P, 16, 0, 8, P, P, 4, 2, 16, P, 16, P, None]
    refuse(L.moe_unpermute_backward, good,
           [(0, None), (0, ODD), (1, 15), (2, 5), (3, None), (4, 15), (5, 3), (6, -1), (7, None), (8, ODD), (9, -1), (10, 0),
            (10, 33), (11, 0), (12, ODD), (13, 15), (14, ODD)])
    for change in ({9: 0}, {12: None, 14: None}):
        assert L.moe_unpermute_backward(*[change.get(i, v) if i in change else v for i, v in enumerate(good)]) == OK


def norm_args(**kw):
    a = block._BlockNormArgs()
    base = dict(x=4096, ld_x=64, y=4096, ld_y=64, w_post=4096, w_pre=4096, gate=4096, h=4096, ld_h=64, u=4096, ld_u=64, T=4, D=64,
                gate_kind=1, res_scale=1.0, eps=1e-6)
    base.update(kw)
    for k, v in base.items():
        setattr(a, k, v)
    return C.byref(a)


def test_block_norm(L):
    assert L.moe_block_norm(None, None) == BAD
    for bad in (dict(x=None), dict(x=4097), dict(ld_x=63), dict(ld_y=63), dict(ld_h=1), dict(ld_u=63), dict(T=-1), dict(D=0),
                dict(D=16385), dict(x_dtype=3), dict(y_dtype=-1), dict(u_dtype=3), dict(w_dtype=9), dict(gate_kind=3),
                dict(gate=None), dict(h=None), dict(y=None, u=None), dict(eps=-1.0), dict(eps=float("nan")), dict(w_post=4098),
                dict(gate=4097), dict(y=4098), dict(u=4097)):
        assert L.moe_block_norm(norm_args(**bad), None) == BAD, bad
    assert L.moe_block_norm(norm_args(T=0), None) == OK


def back_args(**kw):
    a = block._BlockNormBackwardArgs()
    base = dict(dh=4096, ld_dh=64, du=4096, ld_du=64, h=4096, ld_h=64, y=4096, ld_y=64, w_post=4096, w_pre=4096, gate=4096,
                dx=4096, ld_dx=64, dy=4096, ld_dy=64, dw_post=4096, dw_pre=4096, d_gate=4096, workspace=4096,
                workspace_bytes=1 << 20, T=4, D=64, gate_kind=1, res_scale=1.0, eps=1e-6)
    base.update(kw)
    for k, v in base.items():
        setattr(a, k, v)
    return C.byref(a)


def test_block_norm_backward(L):
    assert L.moe_block_norm_backward(None, None) == BAD
    for bad in (dict(dh=None, du=None), dict(h=None), dict(gate=None), dict(gate_kind=4), dict(gate_kind=0), dict(y=None),
                dict(workspace=None), dict(workspace=4100), dict(workspace_bytes=4 * 2 * 64 * 4 - 1), dict(ld_dx=63),
                dict(ld_dy=63), dict(ld_dh=63), dict(ld_du=63), dict(ld_h=63), dict(ld_y=63), dict(T=-1), dict(D=0), dict(D=16385),
                dict(x_dtype=3), dict(y_dtype=3), dict(u_dtype=3), dict(w_dtype=3), dict(dw_pre=4097), dict(d_gate=4098),
                dict(dx=4097), dict(du=None), dict(eps=-1e-9)):
        assert L.moe_block_norm_backward(back_args(**bad), None) == BAD, bad
    assert L.moe_block_norm_workspace_bytes(4, 64) == 4 * 2 * 64 * 4
    assert L.moe_block_norm_workspace_bytes(-1, 64) == 0 and L.moe_block_norm_workspace_bytes(4, 0) == 0
    none = dict(dw_post=None, dw_pre=None, d_gate=None)
    assert L.moe_block_norm_backward(back_args(T=0, **none), None) == OK


def test_four_bits(L):
    for f, good in ((L.moe_mxfp4_quantize, [P, 64, 0, 4, 64, P, P, None]),):
        refuse(f, good, [(0, None), (0, ODD), (1, 63), (2, 3), (3, -1), (4, 48), (4, 0), (5, None), (5, ODD), (6, None)])
        good[3] = 0
        assert f(*good) == OK
    good = [P, P, 4, 64, P, 64, 0, None]
    refuse(L.moe_mxfp4_decode, good, [(0, None), (0, ODD), (1, None), (2, -1), (3, 48), (4, None), (4, ODD), (5, 63), (6, 3)])
    good = [P, P, 2, 128, P, P, 16, 256, P, P, 128, 0, None, None]
    refuse(L.moe_mx4_gemm, good,
           [(0, None), (0, C.c_void_p(4104)), (1, None), (1, C.c_void_p(4098)), (2, 0), (2, 1025), (3, 0), (3, 2 ** 30 + 1), (4, None),
            (4, C.c_void_p(4104)), (5, None), (6, -1), (7, 64), (7, 192), (8, None), (8, ODD), (9, None), (9, ODD), (10, 127),
            (11, 3), (12, ODD)])
    good[6] = 0
    assert L.moe_mx4_gemm(*good) == OK


def test_forward_block(L):
    a = block._BlockArgs()
    assert L.moe_forward_block(None, C.byref(a), 1, None) == BAD
    assert L.moe_forward_block(None, None, 1, None) == BAD


def test_binding_refuses_what_it_can_see():
    """CPU tensors and wrong shapes raise MoeError with MOE_ERR_INVALID_ARG."""
    x = torch.zeros(4, 64)
    i = torch.zeros(4, 2, dtype=torch.int32)
    c, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    for f in (lambda: moe.sort_by_expert(i, 4), lambda: moe.permute(x, i), lambda: moe.unpermute(x, i),
              lambda: moe.permute_backward(x, i), lambda: moe.unpermute_backward(x, x, i), lambda: moe.block_norm(x, x),
              lambda: moe.block_norm_backward(x, None, x), lambda: moe.block_norm_backward(None, None, x),
              lambda: moe.mxfp4_quantize(x), lambda: moe.mxfp4_decode(c, s), lambda: moe.mx4_gemm(c, s, c, s)):
        with pytest.raises(moe.MoeError) as e:
            f()
        assert e.value.code == BAD
    d = -1                                  # the device index of CPU tensors
    for gate, per, T, D in ((torch.zeros(4), None, 4, 4), (torch.zeros(5), None, 4, 6), (torch.zeros(4), "row", 4, 6),
                            (torch.zeros(4), "channel", 4, 6), (None, "token", 4, 6)):
        with pytest.raises(moe.MoeError):
            block._gate(gate, per, T, D, d, "x")
    with pytest.raises(moe.MoeError):
        block._norm_weights("x", d, 6, torch.zeros(6), torch.zeros(6).bfloat16(), None)
    with pytest.raises(moe.MoeError):
        block._norm_weights("x", d, 6, torch.zeros(5), None, None)
    with pytest.raises(moe.MoeError):
        block._mx4(c, s[:, :1], "x")
    with pytest.raises(moe.MoeError):
        block._out_rows(torch.zeros(1, 8).expand(4, 8), 4, 8, torch.float32, d, "x")


def test_sizes_behind_the_last(L):
    """Sizes whose index arithmetic would leave its integers."""
    P16 = C.c_void_p(4096)
    assert L.moe_unpermute(P, 2 ** 31, 0, 8, P, P, 4, 2, 2 ** 30 + 1, P, 2 ** 31, 0, None) == BAD
    assert L.moe_unpermute_backward(P, 2 ** 31, 0, P, 2 ** 31, 0, 8, P, P, 4, 2, 2 ** 30 + 1, P, 2 ** 31, P, None) == BAD
    for rows, K in ((2 ** 44, 32), (2 ** 62, 64), (2 ** 20, 2 ** 60)):
        assert L.moe_mxfp4_quantize(P, K, 0, rows, K, P, P, None) == BAD
        assert L.moe_mxfp4_decode(P, P, rows, K, P, K, 0, None) == BAD
    assert L.moe_mx4_gemm(P16, P16, 1, 2 ** 31 - 255, P16, P16, 16, 128, None, P16, 2 ** 31, 0, None, None) == BAD


def test_stream_of_another_kind():
    x = torch.zeros(4, 64)
    for stream in (0, "s", None.__class__):
        with pytest.raises(moe.MoeError) as e:
            block._on(0, stream, moe.block_norm, x)
        assert e.value.code == BAD
    for n in (2 ** 31, 2 ** 40):
        with pytest.raises(moe.MoeError):
            block._int32(n, "x")
    block._int32(2 ** 31 - 1, "x")


def test_four_bit_product_behind_its_last_sizes(L):
    """K and N whose tile counts would leave 32 bits: 2^31 - 128 gave a negative number of stages, and with it an
    output that no product had been written to."""
    good = [P, P, 1, 1, P, P, 1, 128, None, P, 1, 0, None, None]
    for i, v in ((7, 2 ** 31 - 128), (7, 2 ** 24 + 128), (6, 2 ** 31 - 1), (6, 2 ** 31 - 255)):
        args = list(good)
        args[i] = v
        assert L.moe_mx4_gemm(*args) == BAD, (i, v)
