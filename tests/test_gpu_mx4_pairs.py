"""Grouped four-bit products on CTA pairs (512 rows of B a group and more, on
average): items of few rows beside full ones, empty groups between others,
groups whose rows of A end inside a pair's 256.  The bound is test_gpu_mx4's:
(K + 8) 2^-22 of the sum of magnitudes plus half a step of the output's type.
fp16 ends at 65,504: an exact value of 65,520 (half a step further) and more
rounds to an infinity of its sign, which the random scales reach here and
there among the millions of values of a case."""
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import test_gpu_mx4 as base
import moe_expert_layer_top16_gb300 as moe

pytestmark = pytest.mark.gpu

DEV = base.DEV
F32, BF16, F16 = base.F32, base.BF16, base.F16


def check(ops, bounds, out, dtype, K):
    """base.check, group by group, where an exact value may lie outside fp16."""
    ac, as_, bc, bs = ops
    for g in range(ac.shape[0]):
        lo, hi = bounds[g], bounds[g + 1]
        if lo == hi:
            continue
        a, b = base.values(ac[g], as_[g]).to(DEV), base.values(bc[lo:hi], bs[lo:hi]).to(DEV)
        exact, mag = b @ a.T, b.abs() @ a.abs().T
        tol = mag * ((K + 8) * 2.0 ** -22)
        got = out[lo:hi].double()
        near = (got - exact).abs() <= tol + (exact.abs() + tol) * base.HALF[dtype]
        if dtype == F16:
            out_of_range = (exact.abs() + tol >= 65520) & (got == torch.sign(exact) * float("inf"))
            near = torch.where(exact.abs() - tol >= 65520, out_of_range, near | out_of_range)
        assert near.all(), f"group {g}"


@pytest.mark.parametrize("counts,M", [
    ([1500, 3], 130), ([0, 1600, 17], 384), ([600, 500, 1, 1000], 256), ([1, 1200], 200), ([192 * 4 + 1, 192 * 3 + 31], 257),
    ([0, 0, 2100, 0], 512), ([513, 511, 512, 600, 450], 129)])
@pytest.mark.parametrize("K", [128, 512, 640, 1536])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("lead", [0, 5])
def test_grouped_pairs(counts, M, K, dtype, lead):
    G = len(counts)
    N = lead + sum(counts) + 3
    assert N >= 512 * G and M > 128                        # the product's rule for pairs
    ops = base.operands(G + K, G, M, N, K)
    bounds = (lead + np.concatenate([[0], np.cumsum(counts)])).tolist()
    offsets = torch.tensor(bounds, dtype=torch.int32, device=DEV)
    keep = torch.full((N, M + 4), 7.0, device=DEV).to(dtype)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = moe.mx4_gemm(*ops, offsets=offsets, out=keep[:, :M], status=status)
    assert status.item() == 0
    check(ops, bounds, out, dtype, K)
    assert (keep[:bounds[0]] == 7).all() and (keep[bounds[-1]:] == 7).all() and (keep[:, M:] == 7).all()


@pytest.mark.parametrize("K", [384, 1024])
def test_not_a_number_stays_in_its_row(K):
    """Of pairs: the scales of a group's rows behind an item's last, and of the next group's rows of A, reach no column
    that is stored."""
    counts, M = [700, 9, 1000], 200
    bounds = np.concatenate([[0], np.cumsum(counts)]).tolist()
    ops = base.operands(3, 3, M, bounds[-1], K)
    offsets = torch.tensor(bounds, dtype=torch.int32, device=DEV)
    ref = moe.mx4_gemm(*ops, offsets=offsets)
    ops[3][700, 3] = 255                                   # first row of the second group
    ops[1][2, 5, 2] = 255                                  # a row of A of the third
    out = moe.mx4_gemm(*ops, offsets=offsets)
    bad = torch.zeros_like(ref, dtype=torch.bool)
    bad[700] = True
    bad[709:, 5] = True
    assert out[bad].isnan().all() and torch.equal(out[~bad], ref[~bad])


def threads_first_products():
    """Several host threads' first products, at once: all paired, each on a stream of its own."""
    n, M, N, K = 8, 512, 1024, 512
    ops = [base.operands(i, 1, M, N, K) for i in range(n)]
    out = [torch.empty(N, M, device=DEV) for _ in range(n)]
    torch.cuda.synchronize()
    go, bad = threading.Barrier(n), []

    def one(i):
        try:
            side = torch.cuda.Stream()
            go.wait()
            for _ in range(3):
                moe.mx4_gemm(ops[i][0][0], ops[i][1][0], ops[i][2], ops[i][3], out=out[i], stream=side)
            side.synchronize()
        except Exception as e:      # noqa: BLE001
            bad.append(e)
            go.abort()

    threads = [threading.Thread(target=one, args=(i,)) for i in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad
    for o, got in zip(ops, out):
        assert torch.equal(got, moe.mx4_gemm(o[0][0], o[1][0], o[2], o[3]))
        check(o, [0, N], got, F32, K)


def test_first_products_of_several_threads():
    """In a process of their own: nothing that they share has been asked for yet."""
    r = subprocess.run([sys.executable, "-c", "import sys; sys.path[:0] = %r; import test_gpu_mx4_pairs as t; t.threads_first_products()"
                        % (sys.path,)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_longest_k():
    """K = 2^24, the largest: sums of ones, which fp32 adds exactly, and of the last element alone."""
    K, M, N = 2 ** 24, 3, 2
    one = torch.full((M, K // 2), 0x22, dtype=torch.uint8, device=DEV)
    b = torch.full((N, K // 2), 0x22, dtype=torch.uint8, device=DEV)
    b[1] = 0
    b[1, -1] = 0x70                                        # 6 in the last place
    scales = torch.full((M, K // 32), 127, dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = moe.mx4_gemm(one, scales, b, scales[:N], status=status)
    assert status.item() == 0 and out.tolist() == [[2.0 ** 24] * M, [6.0] * M]
