"""Calls too large for a launch of one of their kernels are refused before any HIP call (no GPU)."""
import pytest

from test_mx_experts_host import UNSUPPORTED, forward, shape, size

OK, TOO_SMALL = 0, 3


@pytest.mark.parametrize("kw", [
    dict(T=1 << 28, H=64, E=8, k=2, I=1 << 14, N=1),    # gate_up: 2^22 row tiles by 64 column tiles
    dict(T=1 << 28, H=1 << 14, E=8, k=2, I=64, N=1),    # down: by 32
    dict(T=(1 << 28) + 1, H=64, E=8, k=2, I=1 << 14, N=2),
    dict(T=1, H=64, E=8, k=32, I=1 << 27, N=1),         # few assignments of experts too large for their form
    dict(T=16, H=1 << 27, E=64, k=2, I=64, N=1),
    dict(T=64, H=64, E=1024, k=8, I=1 << 29, N=1),      # few rows an expert
])
def test_refused(kw):
    assert forward(shape(**kw)) == size(shape(**kw)) == UNSUPPORTED


@pytest.mark.parametrize("kw", [
    dict(T=1 << 28, H=64, E=8, k=2, I=64, N=1),
    dict(T=1 << 28, H=64, E=8, k=2, I=1 << 14, N=256),  # the same in chunks
    dict(T=1, H=64, E=8, k=32, I=1 << 16, N=1),
    dict(T=1, H=64, E=8, k=32, I=1 << 24, N=1),
    dict(T=16, H=1 << 24, E=64, k=2, I=64, N=1),
])
def test_taken(kw):
    assert size(shape(**kw)) == OK
    assert forward(shape(**kw), n=256) == TOO_SMALL
