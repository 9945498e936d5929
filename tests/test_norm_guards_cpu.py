"""What the norm refuses, beside test_mx_cpu.py."""
import pytest

from test_mx_cpu import INV, _norm, _op, lib  # noqa: F401 (fixture)


@pytest.mark.parametrize("eps", [float("inf"), 1e39])
def test_an_infinite_eps(lib, eps):  # noqa: F811
    """The norm would be zero, and its root has no digits to make that of: no answer rather than NaN."""
    assert _norm(lib, _op(eps=eps)) == INV
