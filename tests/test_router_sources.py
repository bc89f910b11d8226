"""Source checks of the router's kernels that overlap the launch before them."""
from test_sources import code, kernels


def test_loads_behind_the_wait_are_plain():
    """balance_sum_kernel starts while the parts that it adds are still written: no load of it may take the
    non-coherent path, and nothing is read before the wait."""
    found = {n: (p, b) for f in ("select.cu", "matvec.cu") for n, p, b in kernels(code(f)) if "pdl_wait()" in b}
    assert set(found) == {"balance_sum_kernel"}
    params, body = found["balance_sum_kernel"]
    assert "__restrict__" not in params and "__ldg" not in body and "ld.global.nc" not in body
    assert "a.part" not in body[:body.index("pdl_wait()")]


def test_every_wait_is_bounded():
    """The products wait for their copies with a limit, and drain them with one."""
    text = code("matvec.cu")
    assert "mbar_wait(" in text and "while (!mbar_try_wait(bar, parity))" in text and "kWaitLimitNs" in text
    assert text.count("mbar_try_wait(") == 1
