"""The router on the GPU against float64, row by row: ids have to be equal, weights and gradients lie within roundings that
are counted from the kernel's own steps."""
import math

import numpy as np
import pytest
import torch

import block_oracle as bo
import combine_top_route_expert_amd as moe
from gpu_layer import say

pytestmark = pytest.mark.gpu
U = bo.U32
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 0.0, "bf16": 2.0 ** -8}  # of the one rounding to the logits' type
INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.load_library()


def make_logits(T, E, dtype, seed, spread=2.0):
    """Rows with ties, closed experts, a wholly closed row, one with a single open expert, large and small values."""
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(T, E)) * spread
    x[rng.random((T, E)) < 0.15] = -INF
    x[rng.random((T, E)) < 0.1] = 0.0
    x[rng.random((T, E)) < 0.05] = -0.0
    if T > 4:
        x[1] = -INF
        x[2] = -INF
        x[2, E // 2] = -3.0
        x[3] = 1.0
        x[4] = rng.normal(size=E) * 30.0
    return torch.from_numpy(x).to(TYPES[dtype]).cuda()


def route(x, k, G=1, bias=None, score="softmax", limit=0, renorm=True, factor=1.0, stream=None):
    T, E = x.shape
    s = moe.make_shape(T, 64, E, k, 64, G, 1, "bf16")
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), 7.0, device="cuda")
    moe.moe_router_top_k(s, x, bias, score, limit, renorm, factor, idx, w, stream)
    return idx, w


def rel_bound(row, ids, E):
    """Relative rounding of one weight: the exponentials' arguments (a difference of two logits, half a unit of it, in
    numerator and denominator), the exponentials (2 units each), the sigmoid's sum, quotient and product, a sum of E
    terms in at most 16 + 6 steps, the quotient and the factor."""
    fin = row[np.isfinite(row)]
    far = float(np.abs(fin).max() + abs(fin.max() - fin.min())) if len(fin) else 0.0
    return U * (2 * far + 2 * 4 + 6 + 22 + 4)


def check(x, k, G, bias, score, limit, renorm, factor):
    idx, w = route(x, k, G, bias, score, limit, renorm, factor)
    rows, idx, w = x.double().cpu().numpy(), idx.cpu().numpy(), w.double().cpu().numpy()
    b = None if bias is None else bias.double().cpu().numpy()
    for t, row in enumerate(rows):
        ids = bo.route_row(row, b, score, G, limit, k)
        assert idx[t].tolist() == ids, (t, idx[t].tolist(), ids)
        ref = np.array(bo.weights_row(row, ids, score, renorm, factor))
        bound = rel_bound(row, ids, len(row)) * np.abs(ref) + 1e-37
        assert (np.abs(w[t] - ref) <= bound).all(), (t, w[t], ref, bound)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E,k", [(1, 1), (2, 3), (7, 2), (60, 4), (64, 8), (65, 64), (96, 6), (128, 8), (254, 9),
                                 (256, 8), (320, 5), (512, 8), (1000, 3), (1024, 64)])
def test_choice_by_logits(E, k, dtype):
    say(f"router E={E} k={k} {dtype}")
    x = make_logits(37, E, dtype, E * 100 + k)
    for score in ("softmax", "sigmoid"):
        for renorm, factor in ((False, 1.0), (True, 2.5)):
            check(x, k, 1, None, score, 0, renorm, factor)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,limit,k", [(8, 8, 3, 2), (8, 1, 0, 3), (60, 4, 2, 4), (60, 20, 7, 6), (128, 64, 5, 8),
                                         (256, 8, 4, 8), (256, 8, 8, 8), (320, 5, 1, 70 - 6), (1024, 32, 4, 8)])
def test_choice_by_score(E, G, limit, k, score):
    say(f"router E={E} G={G} limit={limit} k={k} {score}")
    rng = np.random.default_rng(E + G)
    bias = rng.normal(size=E) * 0.3
    bias[rng.random(E) < 0.1] = -INF
    bias[rng.random(E) < 0.03] = math.nan
    bias = torch.from_numpy(bias).float().cuda()
    for dtype in ("f32", "bf16"):
        x = make_logits(23, E, dtype, E)
        check(x, k, G, bias, score, limit, True, 2.5)
        check(x, k, G, None, score, limit, False, 1.0)


def test_scores_that_float32_rounds_onto_each_other():
    # sigmoids of 17 .. 18 differ by less than a float32 unit of 1: their order is the logits'
    E = 64
    x = torch.linspace(17.0, 18.0, E, device="cuda").flip(0)[None].contiguous()
    idx, _ = route(x, 8, bias=torch.zeros(E, device="cuda"), score="sigmoid")
    assert idx[0].tolist() == list(range(8))
    idx, _ = route(-x, 8, bias=torch.zeros(E, device="cuda"), score="sigmoid")
    assert idx[0].tolist() == list(range(E - 1, E - 9, -1))


def test_weights_beyond_the_range_of_their_scores():
    # e^-300 and e^-88 leave float32; divided by the chosen ones' sum they are ordinary
    for base in (-300.0, -88.0, 40.0, 300.0):
        x = torch.tensor([[base, base - 1.0, base - 2.0, -INF]], device="cuda")
        want = np.exp([0.0, -1.0, -2.0]) if base < 0 else np.ones(3)
        for score in ("sigmoid", "softmax"):
            ref = (np.exp([0.0, -1.0, -2.0]) if score == "softmax" else want)
            _, w = route(x, 3, score=score)
            # base enters the exponentials' arguments only through exact differences
            assert np.abs(w[0].double().cpu().numpy() - ref / ref.sum()).max() < 32 * U, (base, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bad", [math.nan, INF])
def test_a_token_without_an_order(score, bad):
    for E, k in ((5, 3), (256, 8), (3, 5)):
        x = make_logits(9, E, "f32", 5)
        clean, clean_w = route(x, k, score=score)
        x[6, E - 1] = bad
        for bias in (None, torch.zeros(E, device="cuda")):
            idx, w = route(x, k, bias=bias, score=score)
            assert idx[6].tolist() == [j if j < E else -1 for j in range(k)] and bool(w[6].isnan().all())
        idx, w = route(x, k, score=score)
        others = torch.arange(9, device="cuda") != 6
        assert torch.equal(idx[others], clean[others]) and torch.equal(w[others], clean_w[others])
        grad = backward(x, idx, torch.ones(9, k, device="cuda"), score, True, 1.0)
        assert bool(grad[6].isnan().all()) and not bool(grad[others].isnan().any())


def backward(x, idx, gw, score, renorm, factor, stream=None):
    T, E = x.shape
    s = moe.make_shape(T, 64, E, idx.shape[1], 64, 1, 1, "bf16")
    grad = torch.full((T, E), 7.0, dtype=x.dtype, device="cuda")
    moe.moe_router_top_k_backward(s, x, idx, gw, score, renorm, factor, grad, stream)
    return grad


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,k", [(1, 1), (3, 5), (60, 4), (64, 64), (130, 8), (256, 8), (510, 3), (512, 8), (1024, 9)])
def test_gradient(E, k, renorm, score, dtype):
    say(f"router gradient E={E} k={k} {score} renorm={renorm} {dtype}")
    T = 29
    x = make_logits(T, E, dtype, E + 1)
    idx, _ = route(x, k, score=score, renorm=renorm)
    # ids that the router would not give: outside the experts, twice the same, a closed one
    idx[7, 0] = E
    idx[8, -1] = -5
    if k > 1:
        idx[9, 1] = idx[9, 0]
    gw = torch.randn(T, k, generator=torch.Generator(device="cuda").manual_seed(E), device="cuda")
    factor = 2.5
    got = backward(x, idx, gw, score, renorm, factor).double().cpu().numpy()
    rows, ids, g = x.double().cpu().numpy(), idx.cpu().numpy(), gw.double().cpu().numpy()
    for t, row in enumerate(rows):
        ref, size = bo.route_grad_row(row, ids[t].tolist(), g[t], score, renorm, factor)
        # each term: a weight's roundings, its product with factor and gradient, the sums over k slots and the difference
        err = (rel_bound(row, ids[t], E) + U * (k + 8)) * size + 1e-37
        err = err + HALF[dtype] * (np.abs(ref) + err)
        assert (np.abs(got[t] - ref) <= err).all(), (t, np.abs(got[t] - ref).max())


def test_gradient_takes_the_forwards_weights_back():
    """Together as in a training step: the directional difference of the weights is what the gradient says."""
    E, k, T = 64, 6, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, E, generator=g, device="cuda")
    d = torch.randn(T, E, generator=g, device="cuda")
    gw = torch.randn(T, k, generator=g, device="cuda")
    h = 2.0 ** -10
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            idx, _ = route(x, k, score=score, renorm=renorm)
            grad = backward(x, idx, gw, score, renorm, 1.0)
            side = []
            for sign in (1, -1):
                i2, w2 = route(x + sign * h * d, k, score=score, renorm=renorm)
                # the same experts' weights, whatever order the step left them in
                place = torch.full((T, E), 0.0, device="cuda").scatter_(1, i2.long(), w2)
                same = (torch.sort(i2, 1).values == torch.sort(idx, 1).values).all(1)
                side.append((place.gather(1, idx.long()), same))
            ok = side[0][1] & side[1][1]
            assert int(ok.sum()) >= T // 2
            diff = ((side[0][0] - side[1][0]).double() * gw.double()).sum(1) / (2 * h)
            want = (grad.double() * d.double()).sum(1)
            # weights' roundings (64 units of at most 1, over 2 h) and h^2 / 6 times a third derivative (|d|^3 |gw|)
            bound = gw.abs().double().sum(1) * (64 * U / h + h * h / 6 * d.abs().max().double() ** 3)
            assert bool(((diff - want).abs() <= bound)[ok].all()), (score, renorm)


def test_empty_batch_and_stream():
    x = torch.empty(0, 8, device="cuda")
    idx, w = route(x, 2)
    assert idx.numel() == 0 and backward(x, idx, w, "softmax", True, 1.0).numel() == 0
    x = make_logits(300, 64, "f32", 1)
    want, want_w = route(x, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    idx, w = route(x, 4, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(idx, want) and torch.equal(w, want_w)
