"""Launches that overlap the one before them, on data that change with every
call: the counts of the sort's first launch in a workspace that the calls
share, and scales that the quantiser has only just written."""
import pytest
import torch

import moe_expert_layer_top16_gb300 as moe

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.mark.parametrize("T,k,E", [(1000, 16, 896), (8192, 16, 896), (3001, 7, 61)])
def test_sorts_in_one_workspace(T, k, E):
    """Back to back, other experts each time, in the same workspace and outputs: a count left from the call before
    would show in the offsets."""
    g = torch.Generator(device=DEV).manual_seed(T)
    idx = [torch.randint(0, 1 + E // (1 + i % 5), (T, k), generator=g, device=DEV, dtype=torch.int32) for i in range(12)]
    L = moe.lib()
    size = L.moe_sort_workspace_bytes(T, k, E)
    assert size > 0
    work = torch.empty(size, dtype=torch.uint8, device=DEV)
    offsets, order, pos = (torch.empty(n, dtype=torch.int32, device=DEV) for n in (E + 1, T * k, T * k))
    kept = []
    torch.cuda.synchronize()
    for i in idx:
        assert L.moe_sort(i.data_ptr(), T, k, E, offsets.data_ptr(), order.data_ptr(), pos.data_ptr(), work.data_ptr(), size,
                          torch.cuda.current_stream().cuda_stream) == moe.MOE_OK
        kept.append((offsets.clone(), order.clone(), pos.clone()))
    for i, (o, s, p) in zip(idx, kept):
        flat = torch.where((i < 0) | (i >= E), E, i).reshape(-1).long()
        want = torch.sort(flat, stable=True)
        n = int((flat < E).sum())
        assert torch.equal(o.long(), torch.searchsorted(want.values, torch.arange(E + 1, device=DEV)))
        assert torch.equal(s[:n].long(), want.indices[:n]) and (s[n:] == -1).all()
        place = torch.full_like(flat, -1)
        place[want.indices[:n]] = torch.arange(n, device=DEV)
        assert torch.equal(p.long(), place)


@pytest.mark.parametrize("N,M,K", [(73, 256, 896), (600, 512, 640), (600, 512, 1024)])
def test_products_of_reused_operands(N, M, K):
    """Codes and scales rewritten in place before each product, without a wait: gathered scales (K not a multiple of
    512) and copied ones, single CTAs and pairs."""
    g = torch.Generator(device=DEV).manual_seed(K)
    L, s = moe.lib(), torch.cuda.current_stream().cuda_stream
    xs = [torch.randn(N, K, generator=g, device=DEV) * 2.0 ** (i % 7) for i in range(10)]
    w = moe.mxfp4_quantize(torch.randn(M, K, generator=g, device=DEV))
    codes = torch.empty(N, K // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(N, K // 32, dtype=torch.uint8, device=DEV)
    out = [torch.empty(N, M, device=DEV) for _ in xs]
    torch.cuda.synchronize()
    for x, o in zip(xs, out):
        assert L.moe_mxfp4_quantize(x.data_ptr(), K, 0, N, K, codes.data_ptr(), scales.data_ptr(), s) == moe.MOE_OK
        moe.mx4_gemm(*w, codes, scales, out=o)
    torch.cuda.synchronize()
    for x, o in zip(xs, out):
        q = moe.mxfp4_quantize(x)
        torch.cuda.synchronize()
        assert torch.equal(o, moe.mx4_gemm(*w, *q))
