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


CASES = ["alone", "kernel before the wait", "copy after the wait", "memset after the wait", "kernel after the wait"]


def prepared(kind):
    """An operator's call, its inputs and what it gives for them."""
    g = torch.Generator(device=DEV).manual_seed(len(kind))
    x, w = torch.randn(600, 1024, generator=g, device=DEV), torch.randn(512, 1024, generator=g, device=DEV)
    a, idx = moe.mxfp4_quantize(w), torch.randint(0, 61, (3000, 7), generator=g, device=DEV, dtype=torch.int32)
    call = {"product": lambda c, s, i, v: [moe.mx4_gemm(*a, c, s)], "sort": lambda c, s, i, v: moe.sort_by_expert(i, 61),
            "quantise": lambda c, s, i, v: moe.mxfp4_quantize(v),
            "gradients": lambda c, s, i, v: [moe.block_norm_backward(v, v, v, v, w_post=v[0], w_pre=v[1])["dw_post"]]}[kind]
    inputs = (*moe.mxfp4_quantize(x), idx, x)
    return call, inputs, [t.clone() for t in call(*inputs)]


def behind(call, inputs, late, other, case, cycles):
    """The call on `late`, which another stream fills from `inputs` after so many cycles, behind a wait for that stream."""
    main, side = torch.cuda.current_stream(), torch.cuda.Stream()
    side.wait_stream(main)
    with torch.cuda.stream(side):
        torch.cuda._sleep(cycles)
        for t, v in zip(late, inputs):
            t.copy_(v)
    if case == "kernel before the wait":
        moe.mxfp4_quantize(other)                 # which lets its successor start early
    main.wait_stream(side)
    if case == "copy after the wait":
        other.copy_(other * 2)
    if case == "memset after the wait":
        other.zero_()
    if case == "kernel after the wait":
        moe.mxfp4_quantize(other)
    return call(*late)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("kind", ["product", "sort", "quantise", "gradients"])
@pytest.mark.parametrize("case", CASES)
def test_behind_another_streams_work(kind, case, captured):
    """Eager, and as nodes of a graph whose launch depends on two others."""
    call, inputs, want = prepared(kind)
    late, other = [torch.full_like(t, 3) for t in inputs], torch.randn(64, 1024, device=DEV)
    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = behind(call, inputs, late, other, case, 2_000_000)
    for _ in range(2):
        for t in late:
            t.fill_(3)
        if captured:
            graph.replay()
        else:
            got = behind(call, inputs, late, other, case, 20_000_000)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
