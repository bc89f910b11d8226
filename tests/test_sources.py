"""What the CUDA sources have to keep and no run can show: values that the
whole process shares are published whole, and what a kernel launched before its
predecessor has ended reads of that predecessor goes through plain loads."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "moe_expert_layer_top16_gb300", "csrc")
UNITS = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h")))


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", UNITS)
def test_statics_are_safe_to_share(name):
    """A mutable static inside a function is written by whichever host thread comes first, while others read it."""
    plain = [m.group(0).strip() for m in re.finditer(r"^[ \t]+static (?!const |constexpr |__device__)[^;(]*;", code(name), re.M)
             if not re.match(r"\s+static (std::atomic<|std::mutex|std::once_flag|PerDevice )", m.group(0))]
    assert not plain


def kernels(text):
    """(name, parameters, body) of the kernels of a unit."""
    for m in re.finditer(r"__global__ void\s+(?:__launch_bounds__\([^)]*(?:\([^)]*\))?[^)]*\)\s+)?(\w+)\(", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[i], 0)
            i += 1
        end = text.index("\n}\n", i)
        yield m.group(1), text[m.end():i - 1], text[i:end]


def test_loads_behind_the_wait_are_plain():
    """sort_kernel and the four-bit product start while the kernel that writes their inputs still runs.  The
    non-coherent path (`__ldg`, or a `const __restrict__` parameter) is for memory that nobody writes while the kernel
    lives, and such loads may be moved over the wait."""
    found = {n: (p, b) for f in ("route.cu", "mx4.cu", "norm_back.cu") for n, p, b in kernels(code(f)) if "pdl_wait()" in b}
    assert set(found) == {"sort_kernel", "mx4_gemm_kernel", "norm_columns_kernel"}
    params, _ = found["sort_kernel"]
    # idx was there before the count began; the counts are what is waited for
    assert re.findall(r"const int32_t\* __restrict__ (\w+)", params) == ["idx"]
    for name in ("mx4_gemm_kernel", "norm_columns_kernel"):
        assert "__restrict__" not in found[name][0]
    assert "__ldg" not in code("mx4.cu")
    assert "__ldg" not in found["norm_columns_kernel"][1] and "__ldg" not in found["sort_kernel"][1]
