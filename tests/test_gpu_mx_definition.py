"""The layer with 4-bit experts on the GPU against its definition in float64, whatever form a size takes:
  act = rd(silu(g) u),  g, u = x . W,  y = W_down act,  out = rd(sum_j w_j y_j)
on hidden states as the caller gave them and on the values that the packed weights stand for.

Two bounds.  Element by element: float32 sums of exact products, act's and out's rounding to bf16, y's to scaled fp16, all in the
worst case.  And over all elements: roundings are independent, so act's and out's come to the root of the sum of their squares.
One rounding of a bf16 number is off by a uniform part of half a step: 2^-8 / sqrt(3) of a number's power of two, 0.736 of that
of the number itself where its logarithm is uniform, 1.66e-3.  Two of them 2.35e-3, y's 2e-4 adds nothing; a tenth for inputs whose
numbers lie low in their binade."""
import numpy as np
import pytest
import torch

import combine_top_route_expert_amd as moe
import test_gpu_mx_experts as base
from gpu_layer import say
from test_gpu_mx_experts import BF16, HALF, U, Case, few, few_reference, gen, products, swiglu_bound, within

pytestmark = pytest.mark.gpu
TWO_ROUNDINGS = 1.1 * 2.35e-3


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.load_library()


def definition(c: Case, x=None, few_form=None):
    """(values in float64, bound of what the library's float32 sums and roundings may be off); few_form: whether the layer
    takes the form for a few assignments, None for small experts."""
    s = c.shape
    x = c.x if x is None else x
    if few(s) if few_form is None else few_form:
        return few_reference(c, x)
    ref = torch.zeros(s.T, s.H, dtype=torch.float64, device="cuda")
    err = torch.zeros_like(ref)
    idx = c.idx.long()
    for e in range(s.E):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        if t.numel() == 0:
            continue
        p, ep = products(x[t], np.full(t.numel(), e), c.vgu)
        act, ea = swiglu_bound(*p.chunk(2, 1), *ep.chunk(2, 1))
        ea = ea + HALF * (act.abs() + ea) + 1e-37
        v = c.vd[e].double().t().contiguous()
        y = act @ v
        ey = ea @ v.abs() + (act.abs() + ea) @ v.abs() * (s.I / 16 + 16) * 2 * U
        # scaled fp16: half a step, relative; below its normal range half of the smallest step, 2^-25, where the largest
        # magnitude of the row's 64 columns is brought to 2^14 or more
        top = (y.abs() + ey).view(-1, s.H // 64, 64).amax(2).repeat_interleave(64, 1)
        ey = ey + 2.0 ** -11 * (y.abs() + ey) + 2.0 ** -39 * top + 1e-37
        w = c.w[t, j].double()[:, None]
        ref.index_add_(0, t, y * w)
        err.index_add_(0, t, ey * w.abs() + (y.abs() + ey) * w.abs() * (s.k + 1) * U)
    return ref, err + HALF * (ref.abs() + err) + 1e-37


def norm_error(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


def check(c, x=None):
    got = c.forward(x=x)
    ref, err = definition(c, x)
    within(got, ref, err, "out")
    assert norm_error(got, ref) <= TWO_ROUNDINGS, norm_error(got, ref)
    return got


@pytest.mark.parametrize("T,H,E,k,I,N", base.SHAPES)
def test_shapes(T, H, E, k, I, N):  # noqa: E741
    say(f"4-bit experts T={T} H={H} E={E} k={k} I={I} N={N}")
    c = Case(T, H, E, k, I, N, seed=T)
    within(c.forward(), *definition(c), "out")
    assert int(c.err.item()) == 0


@pytest.mark.parametrize("T,H,E,k,I", base.FEW)
def test_few_assignments(T, H, E, k, I):  # noqa: E741
    say(f"4-bit experts T={T} H={H} E={E} k={k} I={I}")
    c = Case(T, H, E, k, I, seed=T + k)
    within(c.forward(), *definition(c), "out")
    c.idx[0, 0], c.idx[T - 1, k - 1] = -3, E
    within(c.forward(), *definition(c), "out")
    assert int(c.err.item()) == (1 if T * k == 1 else 2)


@pytest.mark.parametrize("T,few_form", [(2, True), (5, True), (6, False), (8, False)])
def test_few_assignments_of_large_experts(T, few_form):
    """23 MB an expert: up to 512 MB, 22 assignments, unsorted; of more, whose error shows act's rounding, sorted."""
    H, E, k, I = 7168, 32, 4, 2048  # noqa: E741
    say(f"4-bit experts, {T * k} assignments of large experts")
    c = Case(T, H, E, k, I, seed=T)
    got = c.forward()
    ref, err = definition(c, few_form=few_form)
    within(got, ref, err, "out")
    off = norm_error(got, ref)
    assert off <= (TWO_ROUNDINGS if not few_form else 1.1 * 1.66e-3), off
    assert few_form or off > 1.1 * 1.66e-3, off
    assert int(c.err.item()) == 0


@pytest.mark.parametrize("few_rows", [True, False])
def test_row_counts(few_rows):
    counts = base.EDGES[:9] if few_rows else base.EDGES
    T = int(sum(counts)) // 2 + 5
    say(f"4-bit experts, rows {counts}")
    c = Case(T, 192, len(counts), 2, 128, 1, counts=counts, seed=3)
    within(c.forward(), *definition(c), "out")
    assert int(c.err.item()) == T * 2 - sum(counts)


# rows of experts: tiles of 32 rows (24 an expert at most on average), and tiles of one to four blocks of 32
STREAMED, TILED = [20, 3, 9, 16, 1, 0, 32, 31], [128, 96, 64, 32, 33, 127, 65, 300]


@pytest.mark.parametrize("counts", [STREAMED, TILED])
@pytest.mark.parametrize("H,I", [(64, 128), (192, 256), (320, 384), (384, 768), (448, 512), (512, 2048), (576, 320),
                                 (640, 1088), (704, 192), (768, 384), (2048, 512), (4096 + 320, 64)])
def test_lengths_of_sums(H, I, counts):  # noqa: E741
    """K of one block of 64 columns up to many units of four, whole ones and with one, two or three blocks left over."""
    say(f"4-bit experts H={H} I={I} rows {counts}")
    check(Case(sum(counts), H, len(counts), 1, I, 1, counts=counts, seed=H))


@pytest.mark.parametrize("T", [8, 300, 4500])
def test_magnitudes(T):
    """Rows of every size, with values far above the others, rows of zeros."""
    c = Case(T, 256, 4, 1, 128, 1, seed=11)
    g = gen(12)
    size = torch.exp2(torch.randint(-60, 12, (T, 1), generator=g, device="cuda").float())
    out_of_line = torch.where(torch.rand(T, 256, generator=g, device="cuda") < 0.02, 100.0, 1.0)
    x = (c.x.float() * size * out_of_line).to(BF16)
    x[T // 2] = 0.0
    got = c.forward(x=x)
    within(got, *definition(c, x), "out")
    assert bool((got[T // 2] == 0).all())


@pytest.mark.parametrize("T", [8, 60, 700])
@pytest.mark.parametrize("factor", [100, 300, 1000])
@pytest.mark.parametrize("where", ["x", "act"])
def test_a_large_channel_takes_nothing_from_the_others(where, factor, T):
    """One channel in 32 is far larger and has no weight in the product that reads it: the others decide the result."""
    say(f"4-bit experts, one channel of {where} {factor} times larger, T={T}")
    E, H, I = 16, 512, 256  # noqa: E741
    c = Case(T, H, E, 2, I, 1, seed=factor)
    g = gen(factor)
    wgu = torch.randn(E, 2 * I, H, generator=g, device="cuda") / H ** 0.5
    wd = torch.randn(E, H, I, generator=g, device="cuda") / I ** 0.5
    x = torch.randn(T, H, generator=g, device="cuda")
    if where == "x":
        x[:, 7::32] *= factor
        wgu[:, :, 7::32] = 0.0
    else:
        wgu[:, I + 7::32] *= factor     # rows of up
        wd[:, :, 7::32] = 0.0
    c.wgu, c.wgus, c.vgu = base.packed(wgu.to(BF16))
    c.wd, c.wds, c.vd = base.packed(wd.to(BF16))
    check(c, x.to(BF16))


@pytest.mark.parametrize("k", [1, 3])
def test_one_assignment_more_changes_no_more_than_roundings(k):
    """The rows of 32 assignments (33) alone and in a batch: each as near to the definition as the other."""
    c = Case(200, 1024, 64, k, 512, 1, seed=k)
    ref, _ = definition(c)
    whole = norm_error(c.forward(), ref)
    n = 32 // k + 1
    part = []
    for T in (n - 1, n):
        s = moe.make_shape(T, 1024, 64, k, 512, 1, 1, "bf16")
        part.append(norm_error(c.forward(s, out=torch.empty(T, 1024, dtype=BF16, device="cuda")), ref[:T]))
    say(f"norm errors {part} and {whole}")
    assert max(part + [whole]) <= TWO_ROUNDINGS


def test_one_expert_gets_everything():
    for T in (64, 300, 5000):
        c = Case(T, 256, 16, 1, 128, 1, counts=[0] * 7 + [T] + [0] * 8, seed=T)
        within(c.forward(), *definition(c), "out")


@pytest.mark.parametrize("T", [3, 200, 4200])
def test_dropped_slots_and_what_is_no_number(T):
    c = Case(T, 128, 4, 2, 64, 1, seed=9)
    c.idx[1] = -1                       # a token without experts
    c.idx[2, 0] = 4
    clean = c.forward()
    assert bool((clean[1] == 0).all()) and int(c.err.item()) == 3
    within(clean, *definition(c), "out")
    for bad in (float("nan"), float("inf"), -float("inf")):
        x = c.x.clone()
        x[0, 5] = bad
        x[1, 3] = bad
        got = c.forward(x=x)
        assert torch.equal(got[1:], clean[1:])
        assert not bool(got[0].isfinite().any() if bad != bad else got[0].isfinite().all())


@pytest.mark.parametrize("H,I", [(512, 768), (448, 320)])
def test_both_tilings_give_the_same_bits(H, I):  # noqa: E741
    """Experts that get nothing lower the average of rows that chooses the tiles: 4 of 64 experts, and the same 4 alone."""
    T = 700
    c = Case(T, H, 64, 2, I, 1, counts=[300, 129, 33, 900] + [0] * 60, seed=8)
    want = c.forward()
    c.idx[c.idx >= 4] = -1
    assert torch.equal(c.forward(moe.make_shape(T, H, 4, 2, I, 1, 1, "bf16")), want)
    for n in (2, 3):
        assert torch.equal(c.forward(moe.make_shape(T, H, 4, 2, I, 1, n, "bf16")), want), n


def test_rows_in_another_order_stay_the_same():
    """A token's result does not depend on which tokens it is batched with, nor on where it lies."""
    c = Case(900, 320, 6, 2, 192, 1, seed=21)
    want = c.forward()
    at = torch.randperm(900, generator=torch.Generator().manual_seed(1)).cuda()
    c.idx, c.w = c.idx[at].contiguous(), c.w[at].contiguous()
    assert torch.equal(c.forward(x=c.x[at].contiguous()), want[at])


@pytest.mark.parametrize("T", [8, 60, 700])
def test_the_smallest_weights(T):
    """Groups with the power 2^-127: their values are subnormal numbers of bf16, and as exact as others."""
    E, H, I = 16, 128, 64  # noqa: E741
    c = Case(T, H, E, 2, I, 1, seed=T)
    codes = torch.randint(0, 256, (E * 2 * I * H // 2,), generator=gen(T), device="cuda", dtype=torch.uint8)
    c.wgu, c.wgus = codes, torch.zeros_like(c.wgus)
    moe.moe_dequantize_mx(E * 2 * I, H, "f32", c.wgu, c.wgus, c.vgu)
    assert 0.0 < float(c.vgu.abs().max()) <= 6 * 2.0 ** -127
    x = (c.x.float() * 2.0 ** 125).to(BF16)
    check(c, x)


@pytest.mark.parametrize("T", [4, 60, 2100])
def test_two_layers_at_once(T):
    """Two streams, each with its own rows, workspace and output, over the same weights; eager and as two graphs."""
    c = Case(T, 320, 8, 2, 192, 2, seed=T)
    xs = [c.x, (c.x.float() * 2 + 1).to(BF16)]
    want = [c.forward(x=x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    size = moe.moe_mx_workspace_size(c.shape)
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in xs]
    out = [torch.empty_like(w) for w in want]
    err = [torch.empty(1, dtype=torch.int32, device="cuda") for _ in xs]

    def layer(i, stream=None):
        moe.moe_mx_forward(c.shape, xs[i], c.idx, c.w, c.wgu, c.wgus, c.wd, c.wds, out[i], ws[i], err[i], stream)

    graphs = []
    for i, side in enumerate(streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            layer(i)
        graphs.append(graph)
    for go in (lambda i: layer(i, streams[i]), lambda i: graphs[i].replay()):
        for _ in range(4):
            for o in out:
                o.fill_(float("nan"))
            torch.cuda.synchronize()
            for i, side in enumerate(streams):
                with torch.cuda.stream(side):
                    go(i)
            torch.cuda.synchronize()
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_block_as_it_is_served():
    """Norm, router on its rows, the 4-bit layer, its output into the residual stream; eager, then captured and replayed with other
    rows and with eager work between."""
    T, H, E, k, I = 48, 256, 16, 4, 128  # noqa: E741
    c = Case(T, H, E, k, I, 1, seed=8)
    s = moe.make_shape(T, H, E, k, I, 4, 1, "bf16")
    g = gen(1)
    gate, bias = torch.randn(H, E, generator=g, device="cuda") / 16, 0.1 * torch.randn(E, generator=g, device="cuda")
    x, y = c.x.clone(), torch.empty_like(c.x)
    out, total = torch.empty_like(x), torch.empty_like(x)
    so = torch.tensor([5, 6], device="cuda")
    ws = torch.empty(moe.moe_mx_workspace_size(s), dtype=torch.uint8, device="cuda")
    idx, w, logits = torch.empty_like(c.idx), torch.empty_like(c.w), torch.empty(T, E, device="cuda")

    def block():
        moe.moe_layer_norm(s, x, None, None, None, 1e-5, None, y)
        torch.mm(y.float(), gate, out=logits)
        moe.moe_router_top_k(s, logits, bias, "sigmoid", 2, True, 1.0, idx, w)
        moe.moe_mx_forward(s, y, idx, w, c.wgu, c.wgus, c.wd, c.wds, out, ws)
        moe.moe_dropout_add(s, out, x, 0.1, so, total)

    block()
    c.x, c.idx, c.w = y, idx, w
    within(out, *definition(c), "out")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        block()
    first = x.clone()
    for i in range(4):
        x.copy_(first * (1 + i) + i)
        block()
        want = out.clone(), total.clone()
        out.fill_(float("nan"))
        total.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(total, want[1]), i
