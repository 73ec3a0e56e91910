"""Argument checks of the 4-bit experts' entry points (no GPU: every call returns before any HIP call)."""
import ctypes

import pytest
import torch

import combine_top_route_expert_amd as moe

lib = moe.load_library()
INVALID, UNSUPPORTED, TOO_SMALL = 1, 2, 3
P = 0x10000000  # never dereferenced


def shape(T=8, H=256, E=4, k=2, I=128, N=2, dtype="bf16"):  # noqa: E741
    return moe.make_shape(T, H, E, k, I, 1, N, dtype)


def forward(s, **kw):
    a = dict(x=P, idx=P, tw=P, wgu=P, wgus=P, wd=P, wds=P, out=P, err=None, ws=P, n=1 << 40)
    a.update(kw)
    return lib.moe_mx_forward(ctypes.byref(s), *a.values(), None)


def size(s):
    b = ctypes.c_size_t()
    return lib.moe_mx_workspace_size(ctypes.byref(s), ctypes.byref(b))


@pytest.mark.parametrize("name,off", [(n, o) for n in ("x", "wgu", "wgus", "wd", "wds", "out", "ws") for o in (None, 8)] +
                         [(n, o) for n in ("idx", "tw") for o in (None, 2)] + [("err", 2)])
def test_forward_refuses(name, off):
    assert forward(shape(), **{name: None if off is None else P + off}) == INVALID


def test_workspace():
    s = shape(T=1000, H=2048, E=64, k=4, I=1024, N=2)
    need = moe.moe_mx_workspace_size(s)
    rows = 2 * 500 * 4
    blocks = rows // 32 + 64
    assert 0 < need - blocks * 50 * (2048 + 1024) - rows * (2 * 2048 + 2048 // 64) < 1 << 20
    assert forward(s, n=need - 1) == TOO_SMALL
    one, four = (moe.moe_mx_workspace_size(shape(T=16384, H=2048, E=128, k=8, I=768, N=n)) for n in (1, 4))
    assert abs(four / one - 0.5) < 0.02


@pytest.mark.parametrize("kw", [dict(dtype="f32"), dict(H=96), dict(I=32), dict(k=65), dict(E=2000)])
def test_limits(kw):
    s = shape(**kw)
    assert forward(s) == size(s) == UNSUPPORTED


def test_binding_refuses():
    s = shape(T=1, H=64, E=1, k=1, I=64, N=1)
    z = torch.zeros(1 << 14, dtype=torch.uint8)
    with pytest.raises(ValueError):                 # host tensors
        moe.moe_mx_forward(s, z, z, z, z, z, z, z, z, z)
