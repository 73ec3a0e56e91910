"""Layer norm (forward, backward, quantising form) and the row quantiser on the GPU against the float64 oracle.

Floating outputs are held element by element to bounds counted in roundings (norm_oracle); quantised values, scales and
the residual sum have to be equal."""
import numpy as np
import pytest
import torch

import combine_top_route_expert_amd as moe
import norm_oracle as no
from gpu_layer import say

pytestmark = pytest.mark.gpu
EPS = 1e-5
f64 = no.f64

# widths on both sides of every change of kernel (1024, 2048, 4096, 8192, 16384 values to a row)
WIDTHS = [("bf16", h) for h in (64, 320, 1024, 1088, 2048, 2112, 4096, 4160, 7168, 8192, 8256, 16384)] + \
         [("f32", h) for h in (4, 36, 324, 1028, 2052, 4100, 8196, 16384)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.load_library()


def shape(T, H, dtype):
    return moe.make_shape(T, H, 4, 2, 64, 1, 1, dtype)


def rows(T, H, dtype, seed, offset=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, H, generator=g, device="cuda") + offset
    x[:, :: max(1, H // 3)] *= 8.0
    return x.to(no.TORCH[dtype])


def params(H, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return 1 + 0.2 * torch.randn(H, generator=g, device="cuda"), 0.3 * torch.randn(H, generator=g, device="cuda")


def within(got, ref, bound, what):
    off = np.abs(f64(got) - ref) - bound
    at = np.unravel_index(np.argmax(off), off.shape)
    assert off[at] <= 0, f"{what}{at}: {f64(got)[at]!r} against {ref[at]!r}, bound {bound[at]:.3g}"


def guarded(n, tail, dtype, value):
    """A buffer of n elements with `tail` more behind it that nothing may write."""
    t = torch.full((n + tail,), value, dtype=dtype, device="cuda")
    return t, t[:n]


def quantizes(x, q, scale):
    rq, rs = no.quantize(f64(x))
    assert np.array_equal(q.cpu().numpy(), rq)
    assert np.array_equal(scale.cpu().numpy(), rs.astype(np.float32), equal_nan=True)


@pytest.mark.parametrize("dtype,H", WIDTHS)
@pytest.mark.parametrize("T,residual,affine", [(1, True, True), (5, False, True), (67, True, False)])
def test_norm(dtype, H, T, residual, affine):
    say(f"norm {dtype} T={T} H={H} residual={residual} affine={affine}")
    dt = no.TORCH[dtype]
    x = rows(T, H, dtype, 1, 2.0)
    r = rows(T, H, dtype, 2) if residual else None
    w, b = params(H, 3) if affine else (None, None)
    whole, y = guarded(T * H, 64, dt, 7.0)
    sm = torch.full((T, H), 7.0, dtype=dt, device="cuda") if residual else None
    mean, rstd = torch.full((T + 1,), 7.0, device="cuda"), torch.full((T + 1,), 7.0, device="cuda")
    moe.moe_layer_norm(shape(T, H, dtype), x, r, w, b, EPS, sm, y, mean, rstd)
    torch.cuda.synchronize()
    s = x
    if residual:
        s = (x.float() + r.float()).to(dt)
        assert torch.equal(sm, s)
    s64 = f64(s)
    w64, b64 = (f64(w), f64(b)) if affine else (np.ones(H), np.zeros(H))
    ref, m64, r64 = no.norm(s64, w64, b64, EPS)
    within(y.view(T, H), ref, no.norm_bound(s64, w64, b64, EPS, dtype), "y")
    within(mean[:T], m64, 57 * no.U32 * (np.abs(s64).mean(1) + np.abs(m64)), "mean")
    off = 2 * 56 * no.U32 * np.abs(s64).mean(1) * r64
    within(rstd[:T], r64, r64 * (33 * no.U32 + off), "rstd")
    assert bool((whole[T * H:] == 7.0).all()) and float(mean[T]) == 7.0 and float(rstd[T]) == 7.0
    # without the statistics: the same rows
    y2 = torch.empty_like(y)
    moe.moe_layer_norm(shape(T, H, dtype), x, r, w, b, EPS, sm, y2)
    assert torch.equal(y, y2)


@pytest.mark.parametrize("dtype,H", WIDTHS)
@pytest.mark.parametrize("T,residual", [(1, True), (66, False)])
def test_norm_quantize_is_the_two_calls(dtype, H, T, residual):
    say(f"norm_quantize {dtype} T={T} H={H}")
    dt, s = no.TORCH[dtype], shape(T, H, dtype)
    x, r, (w, b) = rows(T, H, dtype, 4), rows(T, H, dtype, 5) if residual else None, params(H, 6)
    sm = torch.empty(T, H, dtype=dt, device="cuda") if residual else None
    y, y2 = torch.empty(T, H, dtype=dt, device="cuda"), torch.empty(T, H, dtype=dt, device="cuda")
    q, q2, q3 = (torch.full((T, H), 99, dtype=torch.int8, device="cuda") for _ in range(3))
    sc, sc2, sc3 = (torch.full((T,), -1.0, device="cuda") for _ in range(3))
    moe.moe_layer_norm(s, x, r, w, b, EPS, sm, y)
    moe.moe_quantize_rows(T, H, dtype, y, q, sc)
    sm2 = torch.empty(T, H, dtype=dt, device="cuda") if residual else None
    moe.moe_layer_norm_quantize(s, x, r, w, b, EPS, sm2, y2, q2, sc2)
    moe.moe_layer_norm_quantize(s, x, r, w, b, EPS, sm2, None, q3, sc3)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(q, q2) and torch.equal(sc, sc2)
    assert torch.equal(q, q3) and torch.equal(sc, sc3)
    if residual:
        assert torch.equal(sm, sm2)
    quantizes(y, q, sc)


@pytest.mark.parametrize("dtype,H", WIDTHS)
@pytest.mark.parametrize("T,residual", [(1, False), (3, True), (5, True), (33, False), (1531, True)])
def test_norm_backward(dtype, H, T, residual):
    if T * H > 1531 * 4200:
        T = 700                                     # more rows than the 256 groups, all the same
    say(f"norm_backward {dtype} T={T} H={H}")
    s, dt = shape(T, H, dtype), no.TORCH[dtype]
    x, (w, b) = rows(T, H, dtype, 7, 1.0), params(H, 8)
    gy, gs = rows(T, H, dtype, 9), rows(T, H, dtype, 10) if residual else None
    y, mean, rstd = torch.empty_like(x), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    moe.moe_layer_norm(s, x, None, w, b, EPS, None, y, mean, rstd)
    gx = torch.full((T, H), 7.0, dtype=dt, device="cuda")
    wholew, gw = guarded(H, 4, torch.float32, 7.0)
    wholeb, gb = guarded(H, 4, torch.float32, 7.0)
    ws = torch.full((moe.moe_layer_norm_backward_workspace_size(s) + 256,), 0xff, dtype=torch.uint8, device="cuda")
    moe.moe_layer_norm_backward(s, gy, x, w, mean, rstd, gs, gx, gw, gb, ws[:-256])
    torch.cuda.synchronize()
    args = (f64(gy), f64(x), f64(w), f64(mean), f64(rstd), f64(gs) if residual else None)
    for got, ref, bound, what in zip((gx, gw, gb), no.norm_grad(*args), no.norm_grad_bounds(*args, dtype),
                                     ("grad_x", "grad_weight", "grad_bias")):
        within(got, ref, bound, what)
    assert bool((wholew[H:] == 7.0).all()) and bool((wholeb[H:] == 7.0).all()) and bool((ws[-256:] == 0xff).all())
    # each gradient alone, without parameters, and in place: the same bits
    gx2, gw2, gb2 = torch.empty_like(gx), torch.empty_like(gw), torch.empty_like(gb)
    moe.moe_layer_norm_backward(s, gy, x, w, mean, rstd, gs, gx2, gw2, None, ws)
    assert torch.equal(gx, gx2) and torch.equal(gw, gw2)
    moe.moe_layer_norm_backward(s, gy, x, w, mean, rstd, gs, gx2, None, gb2, ws)
    assert torch.equal(gx, gx2) and torch.equal(gb, gb2)
    for alias in ("gy", "x") + (("gs",) if residual else ()):
        t = dict(gy=gy.clone(), x=x.clone(), gs=gs.clone() if residual else None)
        moe.moe_layer_norm_backward(s, t["gy"], t["x"], w, mean, rstd, t["gs"], t[alias])
        assert torch.equal(gx, t[alias]), alias


def test_norm_backward_without_weight_and_rows():
    T, H = 9, 320
    s, x, gy = shape(T, H, "f32"), rows(T, H, "f32", 11), rows(T, H, "f32", 12)
    mean, rstd = x.mean(1), 1 / (x.var(1, unbiased=False) + EPS).sqrt()
    ws = torch.empty(moe.moe_layer_norm_backward_workspace_size(s), dtype=torch.uint8, device="cuda")
    a, b = torch.empty_like(x), torch.empty_like(x)
    gw, gw1 = torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    moe.moe_layer_norm_backward(s, gy, x, None, mean, rstd, None, a, gw, None, ws)
    moe.moe_layer_norm_backward(s, gy, x, torch.ones(H, device="cuda"), mean, rstd, None, b, gw1, None, ws)
    assert torch.equal(a, b) and torch.equal(gw, gw1)
    # no rows: parameter gradients of zero
    none = torch.empty(0, H, device="cuda")
    moe.moe_layer_norm_backward(shape(0, H, "f32"), none, none, None, mean[:0], rstd[:0], None, none, gw, gw1, ws)
    torch.cuda.synchronize()
    assert not gw.any() and not gw1.any()


def test_gradient_against_differences_of_the_forward():
    """Directional differences of the float32 forward kernel itself."""
    T, H = 6, 324
    s, x, (w, b), gy = shape(T, H, "f32"), rows(T, H, "f32", 13), params(H, 14), rows(T, H, "f32", 15)

    def loss(x_, w_, b_):
        y = torch.empty_like(x_)
        moe.moe_layer_norm(s, x_.contiguous(), None, w_, b_, EPS, None, y)
        return float((y.double() * gy.double()).sum())

    mean, rstd, y = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty_like(x)
    moe.moe_layer_norm(s, x, None, w, b, EPS, None, y, mean, rstd)
    gx, gw, gb = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    ws = torch.empty(moe.moe_layer_norm_backward_workspace_size(s), dtype=torch.uint8, device="cuda")
    moe.moe_layer_norm_backward(s, gy, x, w, mean, rstd, None, gx, gw, gb, ws)
    step = 2.0 ** -7
    g = torch.Generator(device="cuda").manual_seed(16)
    for which, got in ((0, gx), (1, gw), (2, gb)):
        v = torch.randn(got.shape, generator=g, device="cuda")
        up, dn = [x, w, b], [x, w, b]
        up[which], dn[which] = up[which] + step * v, dn[which] - step * v
        num = (loss(*up) - loss(*dn)) / (2 * step)
        want = float((got.double() * v.double()).sum())
        # the third-derivative term, step^2 / 6 of a sum of the size of `size`, and float32 noise of y over step
        size = float((got.double().abs() * v.double().abs()).sum())
        noise = 64 * no.U32 * float((y.double().abs() * gy.double().abs()).sum()) / step
        assert abs(num - want) <= 4 * step ** 2 * size + noise, (which, num, want)


def test_norm_in_place_and_bad_rows():
    T, H = 33, 2112
    s, (w, b) = shape(T, H, "bf16"), params(H, 17)
    x, r = rows(T, H, "bf16", 18), rows(T, H, "bf16", 19)
    sm, y = torch.empty_like(x), torch.empty_like(x)
    moe.moe_layer_norm(s, x, r, w, b, EPS, sm, y)
    for a, c in (("x", "r"), ("r", "x")):
        t = dict(x=x.clone(), r=r.clone())
        moe.moe_layer_norm(s, t["x"], t["r"], w, b, EPS, t[a], t[c])
        assert torch.equal(t[a], sm) and torch.equal(t[c], y)
    # a NaN, an infinity, a row of zeros and a row of the type's largest values: their rows only
    bad = x.clone()
    bad[3, 5], bad[9, 2111], bad[12], bad[20] = float("nan"), float("-inf"), 0.0, 3.3e38
    y2, q, sc = torch.empty_like(x), torch.empty(T, H, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    moe.moe_layer_norm_quantize(s, bad, None, w, None, EPS, None, y2, q, sc)
    y3 = torch.empty_like(x)
    moe.moe_layer_norm(s, x, None, w, None, EPS, None, y3)
    torch.cuda.synchronize()
    for row in range(T):
        if row in (3, 9, 20):                       # 20: the sum of the row leaves fp32's range
            assert bool(y2[row].isnan().all()) and bool(sc[row].isnan()) and not q[row].any(), row
        elif row == 12:
            assert not y2[row].any() and float(sc[row]) == 0.0 and not q[row].any()
        else:
            assert torch.equal(y2[row], y3[row]), row


def test_parameters_at_any_float():
    """weight, bias, mean, rstd and scale need only their own four bytes' alignment."""
    for dtype, H in (("bf16", 2112), ("f32", 1028)):
        T, s = 7, shape(7, H, dtype)
        x, (w, b) = rows(T, H, dtype, 30), params(H + 1, 31)
        y, y2, q, q2 = torch.empty_like(x), torch.empty_like(x), *(torch.empty(T, H, dtype=torch.int8, device="cuda")
                                                                   for _ in range(2))
        st, st2 = torch.empty(4, T + 1, device="cuda"), torch.empty(4, T, device="cuda")
        moe.moe_layer_norm(s, x, None, w[1:], b[1:], EPS, None, y, st[0, 1:], st[1, 1:])
        moe.moe_layer_norm(s, x, None, w[1:].clone(), b[1:].clone(), EPS, None, y2, st2[0], st2[1])
        moe.moe_layer_norm_quantize(s, x, None, w[1:], b[1:], EPS, None, None, q, st[2, 1:])
        moe.moe_quantize_rows(T, H, dtype, y2, q2, st2[2])
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(q, q2) and torch.equal(st[:3, 1:], st2[:3])
        gx, gx2, gw = torch.empty_like(x), torch.empty_like(x), torch.empty(H, device="cuda")
        ws = torch.empty(moe.moe_layer_norm_backward_workspace_size(s), dtype=torch.uint8, device="cuda")
        moe.moe_layer_norm_backward(s, x, x, w[1:], st[0, 1:], st[1, 1:], None, gx, gw, None, ws)
        moe.moe_layer_norm_backward(s, x, x, w[1:].clone(), st2[0], st2[1], None, gx2, gw.clone(), None, ws)
        assert torch.equal(gx, gx2)


def test_constant_rows_keep_their_precision():
    """A large common offset: the variance is that of the distances from the mean."""
    T, H = 4, 4096
    s = shape(T, H, "f32")
    x = 1000.0 + torch.arange(H, device="cuda").remainder(2).float().repeat(T, 1) / 64
    x[1] = 1000.0
    y = torch.empty_like(x)
    moe.moe_layer_norm(s, x, None, None, None, EPS, None, y)
    ref = no.norm(f64(x), 1.0, 0.0, EPS)[0]
    within(y, ref, no.norm_bound(f64(x), np.ones(H), np.zeros(H), EPS, "f32"), "y")
    assert not y[1].any()


@pytest.mark.parametrize("dtype,cols", [("bf16", 8), ("bf16", 768), ("bf16", 1032), ("bf16", 2048), ("bf16", 4088),
                                        ("bf16", 7168), ("bf16", 16384), ("bf16", 16392), ("bf16", 40000),
                                        ("f32", 4), ("f32", 1028), ("f32", 2052), ("f32", 4100), ("f32", 8196),
                                        ("f32", 16388)])
def test_quantize_rows(dtype, cols):
    for n in (1, 3, 130):
        say(f"quantize {dtype} rows={n} cols={cols}")
        x = rows(n, cols, dtype, 20)
        x = (x.float() * torch.logspace(-30, 30, n, device="cuda")[:, None]).to(no.TORCH[dtype])
        if n > 20:
            x[7], x[11, 0], x[13, cols - 1], x[17] = 0.0, float("nan"), float("inf"), -3.0e38
            x[19] = x[19] * 0 + 1e-40               # subnormal
        wq, q = guarded(n * cols, 16, torch.int8, 99)
        ws, sc = guarded(n, 4, torch.float32, 99.0)
        moe.moe_quantize_rows(n, cols, dtype, x, q, sc)
        torch.cuda.synchronize()
        quantizes(x, q.view(n, cols), sc)
        assert bool((wq[n * cols:] == 99).all()) and bool((ws[n:] == 99.0).all())


def test_quantize_ties_go_to_even():
    """Rows made of exact ties: 254 x / max is an odd number."""
    odd = torch.arange(-253, 254, 2, device="cuda").float()                  # 254 of them
    for dtype, p in (("bf16", 2.0), ("bf16", 2.0 ** -100), ("bf16", 2.0 ** 100), ("f32", 2.0),
                     ("f32", 77777.0), ("f32", 2.0 ** -20 * 12345), ("f32", 2.0 ** -126 * 2)):
        a = 127.0 * p
        x = torch.cat([odd * (p / 2), torch.tensor([a, -a], device="cuda")]).reshape(1, 256)
        x = x.to(no.TORCH[dtype])
        # 253 * 77777 has 25 bits: half of that row's values round to just beside a tie
        assert torch.equal(x[0, :254].double() * 2, odd.double() * p) or p == 77777.0
        q, sc = torch.empty(1, 256, dtype=torch.int8, device="cuda"), torch.empty(1, device="cuda")
        moe.moe_quantize_rows(1, 256, dtype, x, q, sc)
        quantizes(x, q, sc)
    # every row: half the largest value is a tie
    x = torch.randn(512, 64, device="cuda").to(torch.bfloat16)
    x[:, 0] = x.abs().amax(1)
    x[:, 1], x[:, 2] = x[:, 0] / 2, -x[:, 0] / 2
    q, sc = torch.empty(512, 64, dtype=torch.int8, device="cuda"), torch.empty(512, device="cuda")
    moe.moe_quantize_rows(512, 64, "bf16", x, q, sc)
    quantizes(x, q, sc)
    assert bool((q[:, 1] == 64).all()) and bool((q[:, 2] == -64).all())


def test_more_rows_than_one_launch_takes():
    n = (1 << 21) + 77
    say(f"quantize rows={n}")
    x = torch.randn(n, 8, device="cuda").to(torch.bfloat16)
    q, sc = torch.empty(n, 8, dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda")
    moe.moe_quantize_rows(n, 8, "bf16", x, q, sc)
    s = moe.make_shape(n, 64, 1, 1, 64, 1, 1, "bf16")
    xn = torch.randn(n, 64, device="cuda").to(torch.bfloat16)
    y = torch.full_like(xn, 7.0)
    moe.moe_layer_norm(s, xn, None, None, None, EPS, None, y)
    torch.cuda.synchronize()
    for part in (slice(0, 99), slice((1 << 21) - 50, (1 << 21) + 50), slice(n - 50, n)):
        quantizes(x[part], q[part], sc[part])
        within(y[part], no.norm(f64(xn[part]), 1.0, 0.0, EPS)[0],
               no.norm_bound(f64(xn[part]), np.ones(64), np.zeros(64), EPS, "bf16"), "y")


def test_streams_and_graph_replays():
    """On a side stream, and captured with the forward feeding the backward: every replay gives the eager bits, with
    eager calls on other data between the replays."""
    T, H = 130, 7168
    s, (w, b) = shape(T, H, "bf16"), params(H, 21)
    x, r, gy = rows(T, H, "bf16", 22), rows(T, H, "bf16", 23), rows(T, H, "bf16", 24)

    def buffers():
        return dict(sm=torch.empty_like(x), y=torch.empty_like(x), mean=torch.empty(T, device="cuda"),
                    rstd=torch.empty(T, device="cuda"), gx=torch.empty_like(x), gw=torch.empty_like(w),
                    gb=torch.empty_like(b), q=torch.empty(T, H, dtype=torch.int8, device="cuda"),
                    sc=torch.empty(T, device="cuda"),
                    ws=torch.empty(moe.moe_layer_norm_backward_workspace_size(s), dtype=torch.uint8, device="cuda"))

    def calls(x_, o):
        moe.moe_layer_norm(s, x_, r, w, b, EPS, o["sm"], o["y"], o["mean"], o["rstd"])
        moe.moe_layer_norm_backward(s, gy, o["sm"], w, o["mean"], o["rstd"], gy, o["gx"], o["gw"], o["gb"], o["ws"])
        moe.moe_layer_norm_quantize(s, x_, r, w, b, EPS, o["sm"], None, o["q"], o["sc"])

    eager, side, graph = buffers(), buffers(), buffers()
    calls(x, eager)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        calls(x, side)
    torch.cuda.synchronize()
    keys = ("sm", "y", "mean", "rstd", "gx", "gw", "gb", "q", "sc")
    for k in keys:
        assert torch.equal(eager[k], side[k]), k
    x2 = x.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls(x2, graph)
    other = buffers()
    for n in range(3):
        x2.copy_(x if n != 1 else r)
        g.replay()
        torch.cuda.synchronize()
        calls(x if n != 1 else r, other)
        torch.cuda.synchronize()
        for k in keys:
            assert torch.equal(other[k], graph[k]), (n, k)


@pytest.mark.parametrize("dtype,H,offset,spread", [("f32", *c) for c in no.OFFSETS] +
                         [("bf16", *c) for c in no.OFFSETS_BF16])
def test_common_offset_costs_no_precision(dtype, H, offset, spread):
    """Rows far from zero, held to bounds that do not grow with the offset; rows of one value give exactly the bias."""
    T = 6
    say(f"norm offset {dtype} H={H} offset={offset}")
    s, (w, b), dt = shape(T, H, dtype), params(H, 40), no.TORCH[dtype]
    x = torch.from_numpy(no.offset_rows(T, H, offset, spread)).cuda().to(dt)
    x[4], x[5] = offset, 1.7e10
    y, mean, rstd = torch.empty_like(x), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    for p in ((w, b), (None, None)):
        moe.moe_layer_norm(s, x, None, *p, EPS, None, y, mean, rstd)
        torch.cuda.synchronize()
        w64, b64 = (f64(w), f64(b)) if p[0] is not None else (np.ones(H), np.zeros(H))
        ref, m64, r64 = no.norm(f64(x), w64, b64, EPS)
        by, bm, br = no.norm_bound_about_mean(f64(x), w64, b64, EPS, dtype)
        within(y[:4], ref[:4], by[:4], "y")
        within(mean, m64, bm, "mean")
        within(rstd[:4], r64[:4], br[:4] * r64[:4], "rstd")
        assert torch.equal(y[4:], (b if p[0] is not None else torch.zeros(H, device="cuda")).to(dt).expand(2, H))
    # the residual form and the quantising form read the same rows
    half, sm, y2 = x * 0.5, torch.empty_like(x), torch.empty_like(x)
    q, sc = torch.empty(T, H, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    moe.moe_layer_norm_quantize(s, half, half, None, None, EPS, sm, y2, q, sc)
    torch.cuda.synchronize()
    assert torch.equal(sm, x) and torch.equal(y2, y)
    quantizes(y, q, sc)


@pytest.mark.parametrize("dtype,H", [("bf16", 320), ("bf16", 2048), ("bf16", 7168), ("f32", 324), ("f32", 2052)])
def test_rows_past_the_range_of_the_sums(dtype, H):
    """Finite rows whose squared distances add up to more than float32 holds give NaN, as rows with an infinity do, and no
    other row changes; just inside the range a row is right."""
    T = 9
    s, (w, b), dt = shape(T, H, dtype), params(H, 41), no.TORCH[dtype]
    x = rows(T, H, dtype, 42)
    sign = 1.0 - 2.0 * (torch.arange(H, device="cuda") % 2)
    big = x.clone()
    edge = (3.4e38 / H) ** 0.5                      # squares of this size just reach the end of the range
    for row, size in ((1, 1e25), (3, 1.25 * edge), (4, 0.5 * edge), (6, 3e38), (7, 1e36)):
        big[row] = (size * sign).to(dt)
    big[7, 1:] = 0.0                                # one value alone
    y, y2 = torch.empty_like(x), torch.empty_like(x)
    st = torch.empty(2, T, device="cuda")
    q, sc = torch.full((T, H), 9, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    moe.moe_layer_norm(s, x, None, w, b, EPS, None, y)
    moe.moe_layer_norm(s, big, None, w, b, EPS, None, y2, st[0], st[1])
    torch.cuda.synchronize()
    for row in range(T):
        if row in (1, 3, 6, 7):
            assert bool(y2[row].isnan().all()) and bool(st[1, row].isnan()), row
        elif row == 4:
            r = f64(big[4:5])
            within(y2[4:5], no.norm(r, f64(w), f64(b), EPS)[0], no.norm_bound(r, f64(w), f64(b), EPS, dtype), "y")
        else:
            assert torch.equal(y2[row], y[row]), row
    moe.moe_layer_norm_quantize(s, big, None, w, b, EPS, None, y, q, sc)
    torch.cuda.synchronize()
    assert torch.equal(y.isnan(), y2.isnan())
    for row in (1, 3, 6, 7):
        assert bool(sc[row].isnan()) and not q[row].any(), row
    assert bool(sc[[0, 2, 4, 5, 8]].isfinite().all())


# rows that a workgroup of the gradient holds at a time (1024 threads of at most 16 values)
GRAD_WIDTHS = [("bf16", 64, 16), ("bf16", 320, 16), ("bf16", 1024, 16), ("f32", 1020, 16), ("bf16", 1088, 8),
               ("bf16", 2048, 8), ("f32", 1028, 8), ("bf16", 4096, 4), ("f32", 4100, 2), ("bf16", 7168, 2),
               ("bf16", 8256, 1), ("f32", 16384, 1)]


@pytest.mark.parametrize("dtype,H,par", GRAD_WIDTHS)
def test_norm_backward_over_several_rows(dtype, H, par):
    """Both sides of one workgroup (twice the rows it holds), of 256 workgroups, and several rows after one another in
    each, the last of them ragged."""
    for T, residual in ((par + 1, False), (2 * par, True), (2 * par + 1, False), (256 * par, True),
                        (256 * par + 1, False), (563 * par + 7, True)):
        say(f"norm_backward {dtype} T={T} H={H}")
        s, dt = shape(T, H, dtype), no.TORCH[dtype]
        x, (w, _) = rows(T, H, dtype, 43, 1.0), params(H, 44)
        gy, gs = rows(T, H, dtype, 45), rows(T, H, dtype, 46) if residual else None
        xd = x.double()
        mean = xd.mean(1)
        rstd = ((xd - mean[:, None]).square().mean(1) + EPS).rsqrt()
        mean, rstd = mean.float(), rstd.float()
        gx = torch.full((T, H), 7.0, dtype=dt, device="cuda")
        wholew, gw = guarded(H, 4, torch.float32, 7.0)
        wholeb, gb = guarded(H, 4, torch.float32, 7.0)
        need = moe.moe_layer_norm_backward_workspace_size(s)
        ws = torch.full((need + 256,), 0xff, dtype=torch.uint8, device="cuda")
        moe.moe_layer_norm_backward(s, gy, x, w, mean, rstd, gs, gx, gw, gb, ws[:need])
        torch.cuda.synchronize()
        args = (f64(gy), f64(x), f64(w), f64(mean), f64(rstd), f64(gs) if residual else None)
        for got, ref, bound, what in zip((gx, gw, gb), no.norm_grad(*args), no.norm_grad_bounds(*args, dtype),
                                         ("grad_x", "grad_weight", "grad_bias")):
            within(got, ref, bound, f"{what} of {T} rows")
        assert bool((wholew[H:] == 7.0).all()) and bool((wholeb[H:] == 7.0).all()) and bool((ws[need:] == 0xff).all())
        gx2, gw2, gb2 = torch.empty_like(gx), torch.empty_like(gw), torch.empty_like(gb)
        ws.fill_(0xa5)
        moe.moe_layer_norm_backward(s, gy, x, w, mean, rstd, gs, gx2, gw2, gb2, ws)
        torch.cuda.synchronize()
        assert torch.equal(gx, gx2) and torch.equal(gw, gw2) and torch.equal(gb, gb2)
