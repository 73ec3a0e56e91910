"""Argument checks of the router, of dropout and of the 4-bit matrices' entry points (no GPU: every call returns before any
HIP call), and the references of their tests: gradients against differences, the generator against published outputs."""
import ctypes

import numpy as np
import pytest
import torch

import block_oracle as bo
import combine_top_route_expert_amd as moe

lib = moe.load_library()
OK, INVALID, UNSUPPORTED = 0, 1, 2
P = 0x10000000  # never dereferenced
NAN, INF = float("nan"), float("inf")


def shape(T=8, H=256, E=8, k=2, G=4, dtype="bf16"):
    return moe.make_shape(T, H, E, k, 128, G, 1, dtype)


def route(s, **kw):
    a = dict(dt=0, x=P, bias=P, score=0, limit=2, renorm=1, factor=1.0, idx=P, w=P)
    a.update(kw)
    return lib.moe_router_top_k(ctypes.byref(s), *a.values(), None)


def route_grad(s, **kw):
    a = dict(dt=0, x=P, idx=P, gw=P, score=0, renorm=1, factor=1.0, grad=P + 16)
    a.update(kw)
    return lib.moe_router_top_k_backward(ctypes.byref(s), *a.values(), None)


def dropout(s, **kw):
    a = dict(x=P, res=P, p=0.5, so=P, out=P)
    a.update(kw)
    return lib.moe_dropout_add(ctypes.byref(s), *a.values(), None)


@pytest.mark.parametrize("kw", [dict(dt=2), dict(dt=-1), dict(x=None), dict(x=P + 8), dict(bias=P + 2), dict(score=2),
                                dict(score=-1), dict(limit=-1), dict(limit=5), dict(factor=NAN), dict(factor=INF),
                                dict(factor=-INF), dict(idx=None), dict(idx=P + 2), dict(w=None), dict(w=P + 1)])
def test_route_refuses(kw):
    assert route(shape(), **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(dt=2), dict(x=None), dict(x=P + 8), dict(score=7), dict(factor=NAN), dict(idx=None),
                                dict(idx=P + 1), dict(gw=None), dict(gw=P + 2), dict(grad=None), dict(grad=P + 24),
                                dict(grad=P)])
def test_route_grad_refuses(kw):
    assert route_grad(shape(), **kw) == INVALID


def test_route_limits():
    assert route(shape(E=128, G=128), limit=3) == UNSUPPORTED
    assert route(shape(E=2000, G=1), limit=0) == UNSUPPORTED and route(shape(k=65)) == UNSUPPORTED
    assert route(shape(E=9, G=4)) == INVALID and route_grad(shape(E=9, G=4)) == INVALID
    none = dict(x=None, idx=None, w=None)
    assert route(shape(T=0), **none) == OK and route_grad(shape(T=0), x=None, idx=None, gw=None, grad=None) == OK


@pytest.mark.parametrize("kw", [dict(x=None), dict(x=P + 8), dict(res=P + 4), dict(p=-0.1), dict(p=1.0), dict(p=NAN),
                                dict(so=None), dict(so=P + 4), dict(out=None), dict(out=P + 2)])
def test_dropout_refuses(kw):
    assert dropout(shape(), **kw) == INVALID


def test_dropout_limits():
    assert dropout(shape(T=0), x=None, res=None, so=None, out=None) == OK
    assert dropout(shape(T=0), p=2.0) == INVALID
    assert dropout(shape(H=96)) == UNSUPPORTED


def matrices(rows, cols, **kw):
    """Status of all four calls on a matrix."""
    a = dict(dt=1, x=P, q=P, s=P)
    a.update(kw)
    b = ctypes.c_size_t()
    return (lib.moe_quantize_mx(rows, cols, a["dt"], a["x"], a["q"], a["s"], None),
            lib.moe_dequantize_mx(rows, cols, a["dt"], a["q"], a["s"], a["x"], None),
            lib.moe_pack_mx(rows, cols, a["x"], a["x"], a["q"], a["s"], None),
            lib.moe_mx_scale_size(rows, cols, ctypes.byref(b)))


@pytest.mark.parametrize("name,off", [(n, o) for n in ("x", "q", "s") for o in (None, 2)])
def test_matrices_refuse(name, off):
    ptr = None if off is None else P + off
    assert matrices(32, 64, **{name: ptr})[:3] == (INVALID,) * 3


def test_matrix_limits():
    assert matrices(-32, 64) == matrices(32, 0) == matrices(32, -64) == (INVALID,) * 4
    for rows, cols in ((31, 64), (48, 64), (32, 32), (32, 96), (32 << 31, 64), (32 << 20, 256 << 12)):
        assert matrices(rows, cols) == (UNSUPPORTED,) * 4, (rows, cols)
    assert matrices(0, 64, x=None, q=None, s=None) == (OK,) * 4
    assert matrices(32, 64, dt=2)[:2] == (INVALID,) * 2
    assert lib.moe_mx_scale_size(32, 64, None) == INVALID
    for rows, cols in ((32, 64), (64, 256), (96, 320), (4096, 7168)):
        assert moe.moe_mx_scale_size(rows, cols) == rows * 8 * -(-cols // 256)


def test_matrix_limit_of_a_launch():
    """32 rows by 256 columns are 256 threads of a launch, which holds less than 2^32."""
    for rows, cols in ((32 << 24, 64), (32 << 12, 256 << 12), (32 << 12, (256 << 12) - 192)):
        assert matrices(rows, cols) == (UNSUPPORTED,) * 4, (rows, cols)
    for rows, cols in (((32 << 24) - 32, 64), (32 << 12, (256 << 12) - 256)):
        assert moe.moe_mx_scale_size(rows, cols) == rows * 8 * -(-cols // 256)


def test_binding_refuses():
    s, z = shape(), torch.zeros(1 << 12)
    for call in (lambda: moe.moe_router_top_k(s, z, None, "softmax", 0, True, 1.0, z.int(), z),
                 lambda: moe.moe_router_top_k_backward(s, z, z.int(), z, "softmax", True, 1.0, z),
                 lambda: moe.moe_dropout_add(s, z.bfloat16(), None, 0.1, z.long(), z.bfloat16()),
                 lambda: moe.moe_quantize_mx(32, 64, "f32", z, z.byte(), z.byte()),
                 lambda: moe.moe_pack_mx(32, 64, z.byte(), z.byte(), z.byte(), z.byte()),
                 lambda: moe.moe_dequantize_mx(32, 64, "f32", z.byte(), z.byte(), z),
                 lambda: moe.moe_router_top_k(s, z, None, "relu", 0, True, 1.0, z.int(), z),
                 lambda: moe.moe_quantize_mx(32, 64, "f16", z, z.byte(), z.byte())):
        with pytest.raises(ValueError):  # host tensors, an unknown score, an unknown type
            call()


# ------------------------------------------------------------------ the references themselves
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_router_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(7)
    for E, k in ((5, 2), (12, 12), (30, 4)):
        row, g = rng.normal(size=E), rng.normal(size=k)
        ids = bo.route_row(row, None, score, 1, 0, k)
        ids[-1] = ids[0] if k == 4 else ids[-1]  # one expert twice
        grad, _ = bo.route_grad_row(row, ids, g, score, renorm, 2.5)
        h = 1e-5
        for e in range(E):
            up, down = row.copy(), row.copy()
            up[e] += h
            down[e] -= h
            d = sum(gj * (a - b) for gj, a, b in zip(g, bo.weights_row(up, ids, score, renorm, 2.5),
                                                     bo.weights_row(down, ids, score, renorm, 2.5))) / (2 * h)
            # the difference is off by h^2 / 6 times third derivatives (below 2.5 * 13 |g| k) and 2^-53 / h roundings
            assert abs(d - grad[e]) < 1e-7, (E, k, e)


def test_philox_against_published_outputs():
    """Known answers of Philox 4x32-10 from its authors' test vectors."""
    low = 0xFFFFFFFF
    assert bo.philox((0, 0, 0, 0), (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert bo.philox((low,) * 4, (low,) * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert bo.philox((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)) == \
        [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_quantizer_reference():
    x = np.zeros((1, 64))
    x[0, :9] = [6.0, 5.0, 2.5, 0.25, 0.75, -1.75, 3.5, -0.2, 1.25]
    codes, b = bo.quantize_row_major(x)
    assert b.tolist() == [[127, 0]] and codes[0, :9].tolist() == [7, 6, 4, 0, 2, 12, 6, 8, 2]
    x[0, 0] = 6.001
    assert bo.quantize_row_major(x)[1].tolist() == [[128, 0]]
    back = bo.values(*bo.quantize_row_major(np.random.default_rng(1).normal(size=(4, 64))))
    assert np.isfinite(back).all() and np.abs(back).max() > 0.5
