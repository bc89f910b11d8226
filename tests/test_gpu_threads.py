"""Entry points that encode TMA descriptors, as the first CUDA call of a host
thread: the thread has no context of its own yet."""
import threading

import pytest
import torch

import test_gpu_mx4 as base
import moe_expert_layer_top16_gb300 as moe

pytestmark = pytest.mark.gpu

DEV = base.DEV


def in_a_thread(call):
    got = []
    t = threading.Thread(target=lambda: got.append(call()))
    t.start()
    t.join()
    return got[0]


def sizes(M, N, K):
    ops = base.operands(M + N, 1, M, N, K)
    return [t.contiguous() for t in (ops[0][0], ops[1][0], ops[2], ops[3])]


@pytest.mark.parametrize("M,N,K", [(256, 40, 512), (512, 1024, 512), (130, 17, 640)])
def test_four_bit_product(M, N, K):
    a, sa, b, sb = sizes(M, N, K)
    want = moe.mx4_gemm(a, sa, b, sb)
    out = torch.empty_like(want)
    L, s, p = moe.lib(), torch.cuda.current_stream().cuda_stream, [t.data_ptr() for t in (a, sa, b, sb, out)]
    torch.cuda.synchronize()
    for _ in range(2):
        assert in_a_thread(lambda: L.moe_mx4_gemm(p[0], p[1], 1, M, p[2], p[3], N, K, None, p[4], M, 0, None, s)) == moe.MOE_OK
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        out.zero_()


@pytest.mark.parametrize("noalloc", [False, True])
@pytest.mark.parametrize("M,N,K", [(256, 40, 512), (512, 1024, 512)])
def test_eight_bit_product(M, N, K, noalloc):
    g = torch.Generator(device=DEV).manual_seed(1)
    a, sa, _, _ = sizes(M, N, K)
    b = torch.randint(0, 120, (N, K), generator=g, device=DEV, dtype=torch.int32).to(torch.uint8)
    sb = torch.full((N, K // 32), 127, dtype=torch.uint8, device=DEV)
    L, s = moe.lib(), torch.cuda.current_stream().cuda_stream
    f = L.moe_mx_gemm_noalloc if noalloc else L.moe_mx_gemm
    out = [torch.empty(N, M, device=DEV) for _ in range(2)]
    call = lambda o: f(a.data_ptr(), sa.data_ptr(), M, b.data_ptr(), sb.data_ptr(), N, K, o.data_ptr(), None, s)  # noqa: E731
    assert call(out[0]) == moe.MOE_OK
    torch.cuda.synchronize()
    assert in_a_thread(lambda: call(out[1])) == moe.MOE_OK
    torch.cuda.synchronize()
    assert torch.equal(*out)


def test_the_other_operators():
    """Which launch and encode nothing."""
    x = torch.randn(64, 256, device=DEV)
    idx = torch.randint(0, 9, (64, 4), device=DEV, dtype=torch.int32)
    calls = (lambda: moe.block_norm(x, x)[1], lambda: moe.sort_by_expert(idx, 9)[2], lambda: moe.mxfp4_quantize(x)[0],
             lambda: moe.block_norm_backward(x, x, x, x)["dy"])
    for call in calls:
        want = call()
        torch.cuda.synchronize()
        got = in_a_thread(call)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
