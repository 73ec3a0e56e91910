"""Argument checks of the 8-bit integer experts' entry points (no GPU: every call returns before any HIP call)."""
import ctypes

import pytest
import torch

import combine_top_route_expert_amd as moe

lib = moe.load_library()
OK, INVALID, UNSUPPORTED, TOO_SMALL = 0, 1, 2, 3
P = 0x10000000  # never dereferenced


def shape(T=8, H=256, E=4, k=2, I=128, N=2, dtype="bf16"):  # noqa: E741
    return moe.make_shape(T, H, E, k, I, 1, N, dtype)


def gate_up(s, chunk=0, **kw):
    a = dict(q=P, sc=P, src=P, off=P, w=P, ws=P, act=P)
    a.update(kw)
    return lib.moe_quant_gate_up_gather_pair(ctypes.byref(s), chunk, *a.values(), None)


def act(s, chunk=0, **kw):
    a = dict(act=P, off=P, q=P, sc=P)
    a.update(kw)
    return lib.moe_quant_act_pair(ctypes.byref(s), chunk, *a.values(), None)


def down(s, chunk=0, **kw):
    a = dict(q=P, sc=P, off=P, w=P, ws=P, y0=P, y1=P)
    a.update(kw)
    return lib.moe_quant_down_pair(ctypes.byref(s), chunk, *a.values(), None)


def forward(s, **kw):
    a = dict(q=P, sc=P, idx=P, w=P, wgu=P, wgus=P, wd=P, wds=P, out=P, err=None, ws=P, n=1 << 40)
    a.update(kw)
    return lib.moe_quant_forward(ctypes.byref(s), *a.values(), None)


@pytest.mark.parametrize("name,off", [(n, o) for n in ("q", "w", "act") for o in (None, 8)] +
                         [(n, o) for n in ("sc", "ws", "src", "off") for o in (None, 2)])
def test_gate_up_refuses(name, off):
    assert gate_up(shape(), **{name: None if off is None else P + off}) == INVALID


@pytest.mark.parametrize("name,off", [(n, o) for n in ("act", "q") for o in (None, 8)] +
                         [(n, o) for n in ("sc", "off") for o in (None, 2)])
def test_act_refuses(name, off):
    assert act(shape(), **{name: None if off is None else P + off}) == INVALID


@pytest.mark.parametrize("name,off", [(n, o) for n in ("q", "w", "y0", "y1") for o in (None, 8)] +
                         [(n, o) for n in ("sc", "ws", "off") for o in (None, 2)])
def test_down_refuses(name, off):
    assert down(shape(), **{name: None if off is None else P + off}) == INVALID


@pytest.mark.parametrize("name,off", [(n, o) for n in ("q", "wgu", "wd", "out", "ws") for o in (None, 8)] +
                         [(n, o) for n in ("sc", "idx", "w", "wgus", "wds") for o in (None, 2)] + [("err", 2)])
def test_forward_refuses(name, off):
    assert forward(shape(), **{name: None if off is None else P + off}) == INVALID


def test_workspace():
    s = shape(T=1000, H=2048, E=64, k=4, I=1024, N=2)
    need = moe.moe_quant_workspace_size(s)
    rows = 2 * 500 * 4
    assert 0 < need - rows * (2 * 2048 + 2 * 1024 + 1024 + 4) < 1 << 20
    assert forward(s, n=need - 1) == TOO_SMALL
    # two chunks resident at a time: four chunks take half of what one takes
    one, four = (moe.moe_quant_workspace_size(shape(T=16384, H=2048, E=128, k=8, I=768, N=n)) for n in (1, 4))
    assert abs(four / one - 0.5) < 0.02


@pytest.mark.parametrize("kw", [dict(H=131072), dict(I=131072), dict(H=36, dtype="f32"), dict(I=20, dtype="f32"),
                                dict(H=96), dict(I=32), dict(k=65), dict(E=2000)])
def test_limits(kw):
    s = shape(**kw)
    assert forward(s) == gate_up(s) == act(s) == down(s) == UNSUPPORTED
    b = ctypes.c_size_t()
    assert lib.moe_quant_workspace_size(ctypes.byref(s), ctypes.byref(b)) == UNSUPPORTED


def test_chunks():
    s = shape(T=3, N=4)
    for fn in (gate_up, act, down):
        assert fn(s, 4) == INVALID and fn(s, -1) == INVALID
    # chunk 3 of three tokens in four chunks is empty: nothing to do, nothing needed
    none = dict.fromkeys(("q", "sc", "off"))
    assert gate_up(s, 3, src=None, w=None, ws=None, act=None, **none) == OK
    assert act(s, 3, act=None, **none) == OK
    assert down(s, 3, w=None, ws=None, y0=None, y1=None, **none) == OK


def test_binding_refuses():
    s = shape(T=1, H=64, E=1, k=1, I=64, N=1)
    z = torch.zeros(1 << 14, dtype=torch.int8)
    with pytest.raises(ValueError):                 # host tensors
        moe.moe_quant_forward(s, z, z, z, z, z, z, z, z, z, z)


def test_binding_rows_of_a_pair_are_the_librarys():
    for T in (0, 1, 2, 3, 10, 97):
        for N in (1, 2, 3, 4, 7, 50):
            s = shape(T=T, N=N, k=3)
            for c in range(N):
                assert moe._rows_of_pair(s, c) == moe._pair_rows(s, c), (T, N, c)
            for bad in (-1, N):
                with pytest.raises(moe.MoeError):
                    moe._rows_of_pair(s, bad)
