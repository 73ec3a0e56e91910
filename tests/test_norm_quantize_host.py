"""The layer norm's and the row quantiser's argument checks (no GPU: every call returns before any HIP call), and the
gradient formula of the tests' oracle against central differences."""
import ctypes

import numpy as np
import pytest
import torch

import combine_top_route_expert_amd as moe
import norm_oracle as no

lib = moe.load_library()
OK, INVALID, UNSUPPORTED, TOO_SMALL = 0, 1, 2, 3
P = 0x10000000  # never dereferenced
EPS = 1e-5


def shape(T=8, H=256, dtype="bf16"):
    return moe.make_shape(T, H, 4, 2, 64, 1, 1, dtype)


def norm(s, x=P, res=None, w=P, b=P, eps=EPS, sm=None, y=P, mean=P, rstd=P):
    return lib.moe_layer_norm(ctypes.byref(s), x, res, w, b, eps, sm, y, mean, rstd, None)


def norm_q(s, x=P, res=None, eps=EPS, sm=None, y=P, q=P, scale=P):
    return lib.moe_layer_norm_quantize(ctypes.byref(s), x, res, P, P, eps, sm, y, q, scale, None)


def grad(s, gy=P, x=P, w=P, mean=P, rstd=P, gs=None, gx=P, gw=P, gb=P, ws=P, n=None):
    n = moe.moe_layer_norm_backward_workspace_size(s) if n is None else n
    return lib.moe_layer_norm_backward(ctypes.byref(s), gy, x, w, mean, rstd, gs, gx, gw, gb, ws, n, None)


@pytest.mark.parametrize("kw", [dict(x=None), dict(y=None), dict(x=P + 2), dict(y=P + 8), dict(w=P + 2),
                                dict(b=P + 1), dict(mean=P + 2), dict(rstd=P + 3), dict(res=P), dict(sm=P),
                                dict(res=P + 4, sm=P), dict(res=P, sm=P + 4), dict(res=2 * P, sm=P, y=P), dict(eps=0.0), dict(eps=-1.0),
                                dict(eps=float("nan")), dict(eps=float("inf"))])
def test_norm_refuses(kw):
    assert norm(shape(), **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(x=None), dict(q=None), dict(scale=None), dict(q=P + 4), dict(scale=P + 2),
                                dict(y=P + 2), dict(res=P), dict(eps=0.0)])
def test_norm_quantize_refuses(kw):
    assert norm_q(shape(), **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(gy=None), dict(x=None), dict(mean=None), dict(rstd=None), dict(gx=None),
                                dict(ws=None), dict(ws=P + 16), dict(gy=P + 2), dict(gs=P + 8), dict(gx=P + 4),
                                dict(gw=P + 4), dict(gb=P + 8), dict(w=P + 2)])
def test_norm_backward_refuses(kw):
    assert grad(shape(), **kw) == INVALID


def test_norm_backward_workspace():
    s = shape()
    need = moe.moe_layer_norm_backward_workspace_size(s)
    assert need >= 2 * s.H * 4
    assert grad(s, n=2 * s.H * 4 - 1) == TOO_SMALL
    # never more than 256 groups of rows, whatever T
    assert moe.moe_layer_norm_backward_workspace_size(shape(T=1 << 20, H=16384)) == 256 * 2 * 16384 * 4


def test_norm_shape_limits():
    assert norm(shape(H=16384 + 64)) == UNSUPPORTED
    assert norm_q(shape(H=16384 + 64)) == UNSUPPORTED
    with pytest.raises(moe.MoeError):
        moe.moe_layer_norm_backward_workspace_size(shape(H=16384 + 64))
    assert norm(shape(H=96)) == UNSUPPORTED         # bf16 rows come in 64s
    assert norm(shape(H=6, dtype="f32")) == UNSUPPORTED
    bad = shape()
    bad.dtype = 9
    assert norm(bad) == INVALID


def test_no_tokens_is_a_noop():
    s = shape(T=0)
    assert norm(s, x=None, w=None, b=None, y=None, mean=None, rstd=None) == OK
    assert norm_q(s, x=None, y=None, q=None, scale=None) == OK
    assert grad(s, gy=None, x=None, mean=None, rstd=None, gx=None, gw=None, gb=None, ws=None, n=0) == OK


@pytest.mark.parametrize("args,code", [
    ((-1, 64, 1, P, P, P), INVALID), ((4, 0, 1, P, P, P), INVALID), ((4, 64, 2, P, P, P), INVALID),
    ((4, 64, 1, None, P, P), INVALID), ((4, 64, 1, P, None, P), INVALID), ((4, 64, 1, P, P, None), INVALID),
    ((4, 64, 1, P + 8, P, P), INVALID), ((4, 64, 1, P, P + 8, P), INVALID), ((4, 64, 1, P, P, P + 2), INVALID),
    ((4, 60, 1, P, P, P), UNSUPPORTED), ((4, 62, 0, P, P, P), UNSUPPORTED), ((0, 64, 1, None, None, None), OK)])
def test_quantize_rows_refuses(args, code):
    assert lib.moe_quantize_rows(*args, None) == code


def test_binding_refuses():
    s = shape(T=2, H=64)
    z = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):                 # host tensors
        moe.moe_layer_norm(s, z, None, None, None, EPS, None, z)
    with pytest.raises(ValueError):
        moe.moe_quantize_rows(2, 64, "fp16", z, z, z)


def test_gradient_formula_against_differences():
    rng = np.random.default_rng(1)
    s, w, b = rng.normal(size=(3, 12)) + 0.5, rng.normal(size=12), rng.normal(size=12)
    gy = rng.normal(size=(3, 12))
    _, mean, rstd = no.norm(s, w, b, EPS)
    dx, dw, db = no.norm_grad(gy, s, w, mean, rstd, None)
    loss = lambda s_, w_, b_: float((gy * no.norm(s_, w_, b_, EPS)[0]).sum())  # noqa: E731
    h = 1e-6
    for which, got in ((0, dx), (1, dw), (2, db)):
        args = [s, w, b]
        for i in np.ndindex(args[which].shape):
            up, dn = [a.copy() for a in args], [a.copy() for a in args]
            up[which][i] += h
            dn[which][i] -= h
            # central differences: h^2 times a third derivative of order 10, and 1e-16 |loss| / h
            assert abs((loss(*up) - loss(*dn)) / (2 * h) - got[i]) < 1e-7


def test_quantizer_oracle_by_hand():
    x = np.array([[127.0, 0.5, 1.5, -2.5, -127.0], [0, 0, 0, 0, 0], [2.0, 1.0, -1.0, 0.0, 0.01],
                  [np.inf, 1, 2, 3, 4], [1, np.nan, 2, 3, 4]])
    q, scale = no.quantize(x)
    assert q.tolist() == [[127, 0, 2, -2, -127], [0] * 5, [127, 64, -64, 0, 1], [0] * 5, [0] * 5]
    assert scale[0] == 1.0 and scale[1] == 0.0 and np.isnan(scale[3:]).all()


@pytest.mark.parametrize("H,offset,spread", no.OFFSETS)
def test_bound_about_the_mean_sees_mistakes(H, offset, spread):
    """float32 models of the norm: a float64 mean in two parts is within the bound; a row of zeros, flipped signs, a
    variance from the sum of squares, and a mean from one float32 sum or rounded to one float32 are not."""
    x = no.offset_rows(3, H, offset, spread)
    ref = no.norm(x.astype(np.float64), 1.0, 0.0, EPS)[0]
    bound = no.norm_bound_about_mean(x.astype(np.float64), np.ones(H), np.zeros(H), EPS, "f32")[0]
    f = np.float32

    def y_of(d, var=None):
        var = (d * d).sum(1, dtype=f) / f(H) if var is None else var
        return d * (f(1) / np.sqrt(var + f(EPS)))[:, None]

    within = lambda y: bool((np.abs(y.astype(np.float64) - ref) <= bound).all())  # noqa: E731
    mean = x.astype(np.float64).mean(1, keepdims=True)
    high = mean.astype(f)
    good = y_of((x - high) - (mean - high).astype(f))
    assert good.dtype == f and within(good)
    assert not within(np.zeros_like(x)) and not within(-good)
    one_pass = np.maximum((x * x).sum(1, dtype=f) / f(H) - high[:, 0] * high[:, 0], f(0))
    assert not within(y_of(x - high, one_pass))
    assert not within(y_of(x - high))
    single = x.reshape(3, -1, 4).cumsum(1, dtype=f)[:, -1].sum(1, dtype=f, keepdims=True) / f(H)
    assert not within(y_of(x - single))
