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


@pytest.mark.parametrize("name", ["gemm.cu", "mx4.cu"])
def test_statics_are_safe_to_share(name):
    """A mutable static inside a function is written by whichever host thread comes first, while others read it."""
    plain = [m.group(0).strip() for m in re.finditer(r"^[ \t]+static (?!const |constexpr |__device__)[^;(]*;", code(name), re.M)
             if not re.match(r"\s+static (std::atomic<|std::mutex|std::once_flag|PerDevice )", m.group(0))]
    assert not plain
