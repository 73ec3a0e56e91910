"""The layer with 4-bit experts on the GPU against float64 on the values that the packed weights stand for.

The reference rounds the activations as the library does (two 6-bit parts) and bounds, element by element, what can differ: float32
sums of exact products (a bound that grows with the number of additions and the sum of the magnitudes), values so close to a
rounding border that those sums decide the side, scaled fp16 of y and one rounding to bf16."""
import numpy as np
import pytest
import torch

import block_oracle as bo
import combine_top_route_expert_amd as moe
from gpu_layer import say

pytestmark = pytest.mark.gpu
U, HALF = bo.U32, 2.0 ** -8
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.load_library()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def packed(x):
    """x [E][rows][cols] (bf16) as packed matrices, and the values that they stand for in float32."""
    E, rows, cols = x.shape
    q = torch.empty(E * rows * cols // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(moe.moe_mx_scale_size(E * rows, cols), dtype=torch.uint8, device="cuda")
    moe.moe_quantize_mx(E * rows, cols, "bf16", x, q, s)
    v = torch.empty(E, rows, cols, device="cuda")
    moe.moe_dequantize_mx(E * rows, cols, "f32", q, s, v)
    return q, s, v


def ids_with_counts(counts, T, k, seed, outside=(-1, 1 << 20)):
    """[T][k] ids in which expert e appears counts[e] times; the rest lie outside the experts."""
    flat = np.concatenate([np.repeat(np.arange(len(counts)), counts),
                           np.resize(np.array(outside), T * k - int(np.sum(counts)))])
    np.random.default_rng(seed).shuffle(flat)
    return torch.from_numpy(flat.astype(np.int32).reshape(T, k)).cuda()


class Case:
    def __init__(self, T, H, E, k, I, N=1, counts=None, seed=0):  # noqa: E741
        g = gen(seed)
        self.shape = s = moe.make_shape(T, H, E, k, I, 1, N, "bf16")
        if counts is None:
            self.idx = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
        else:
            self.idx = ids_with_counts(counts, T, k, seed)
        self.w = torch.rand(T, k, generator=g, device="cuda")
        self.x = torch.randn(T, H, generator=g, device="cuda").to(BF16)
        # groups of very different size, so that a scale of the wrong group shows
        def weights(rows, cols):
            w = torch.randn(E, rows, cols, generator=g, device="cuda")
            size = torch.exp2(torch.randint(-3, 4, (E, rows, cols // 32), generator=g, device="cuda").float())
            return (w * size.repeat_interleave(32, 2) / (2 * cols ** 0.5)).to(BF16)
        self.wgu, self.wgus, self.vgu = packed(weights(2 * I, H))
        self.wd, self.wds, self.vd = packed(weights(H, I))
        i32 = dict(dtype=torch.int32, device="cuda")
        self.counts, self.offsets = torch.empty(N, E, **i32), torch.empty(N, E + 1, **i32)
        self.splits, self.err = torch.empty(N, 1, **i32), torch.empty(1, **i32)
        self.src, self.dst = torch.empty(T * k, **i32), torch.empty(T * k, **i32)
        ws = torch.empty(moe.moe_route_meta_workspace_size(s), dtype=torch.uint8, device="cuda")
        moe.moe_route_meta(s, self.idx, self.counts, self.offsets, self.splits, self.src, self.dst, self.err, ws)
        self.off = self.offsets.cpu().numpy()

    def pair_rows(self, c):
        """Joint rows of pair (c, c + 1) as (part, chunk row, expert) arrays, and the rows that the parts may hold."""
        s = self.shape
        bound = [(b - a) * s.k for a, b in (moe.moe_chunk_range(s, x) for x in (c, c + 1) if x < s.N)]
        o0 = self.off[c]
        o1 = self.off[c + 1] if len(bound) > 1 else np.zeros_like(o0)
        part, row, exp = [], [], []
        for e in range(s.E):
            for p, o in ((0, o0), (1, o1)):
                n = int(o[e + 1] - o[e])
                part += [p] * n
                row += range(o[e], o[e] + n)
                exp += [e] * n
        return np.array(part, int), np.array(row, int), np.array(exp, int), bound + [0] * (2 - len(bound))

    def forward(self, shape=None, ws=None, out=None, x=None, stream=None):
        s = self.shape if shape is None else shape
        ws = torch.full((moe.moe_mx_workspace_size(s),), 0xa5, dtype=torch.uint8, device="cuda") if ws is None else ws
        out = torch.full((s.T, s.H), float("nan"), dtype=BF16, device="cuda") if out is None else out
        moe.moe_mx_forward(s, self.x if x is None else x, self.idx, self.w, self.wgu, self.wgus, self.wd, self.wds, out,
                           ws, self.err, stream)
        return out


def within(got, ref, bound, what):
    off = (got.double() - ref).abs() - bound
    assert not bool(off.isnan().any()), what
    worst = int(off.argmax())
    assert float(off.flatten()[worst]) <= 0, \
        f"{what}[{worst}]: {float(got.flatten()[worst])!r} against {float(ref.flatten()[worst])!r}, " \
        f"bound {float(bound.flatten()[worst]):.3g}"


def products(rows, expert, values):
    """rows @ values[expert].T in float64, and the bound of a float32 sum: matrix instructions add 16 products at a time
    to a running sum, each addition off by at most 2 U of the magnitudes so far."""
    K = rows.shape[1]
    got = torch.empty(rows.shape[0], values.shape[1], dtype=torch.float64, device="cuda")
    size = torch.empty_like(got)
    for e in np.unique(expert):
        at = torch.from_numpy(np.nonzero(expert == e)[0]).cuda()
        v = values[int(e)].double().t().contiguous()
        got[at] = rows[at].double() @ v
        size[at] = rows[at].double().abs() @ v.abs()
    return got, size * (K / 16 + 16) * 2 * U


def swiglu_bound(g, u, eg, eu):
    ref = g * torch.sigmoid(g) * u
    # silu's slope is at most 1.1; the exponential's argument, itself, the reciprocal, the sum and two products
    err = 1.1 * eg * (u.abs() + eu) + (g * torch.sigmoid(g)).abs() * eu + ref.abs() * U * (2 * g.abs() + 12) + 1e-37
    return ref, err


def e2m3(v):
    """Magnitudes up to 7.5 rounded to E2M3 numbers: 1/8 apart up to 2, 1/4 up to 4, 1/2 above; ties to even."""
    a = v.abs()
    gap = torch.where(a < 2.0, 0.125, torch.where(a < 4.0, 0.25, 0.5)).double()
    return torch.round(v / gap) * gap


def e2m3_step(big):
    """2^s, s the least integer (at least -127) with big <= 7.5 2^s."""
    m, e = torch.frexp(big.double())            # big = m 2^e, m in [0.5, 1); 7.5 = 0.9375 2^3
    return torch.exp2((e - 3 + (m > 0.9375).int()).double().clamp_min(-127.0))


def parts_of(g):
    """(h, l, step of h, step of l) of float64 groups [..., 32]."""
    hs = e2m3_step(g.abs().amax(-1, keepdim=True))
    h = e2m3(g / hs) * hs
    ls = e2m3_step((g - h).abs().amax(-1, keepdim=True))
    return h, e2m3((g - h) / ls) * ls, hs, ls


def two_parts(x, delta=None):
    """x [rows][cols] in two 6-bit parts; with delta also how far the parts of a value within delta of x may lie off."""
    g = x.double().view(x.shape[0], -1, 32)
    h, l, hs, ls = parts_of(g)
    v = h + l
    if delta is None:
        return v.view_as(x)
    d = delta.view_as(g)
    big = g.abs().amax(-1, keepdim=True)
    up, down = g + d, g - d
    # a group whose scales or whose h parts depend on the side: any two representations lie within 2^-8.9 of the
    # largest value of what they stand for
    most = (g.abs() + d).amax(-1, keepdim=True)
    least = (g.abs() - d).clamp_min(0.0).amax(-1, keepdim=True)
    unsure = (e2m3_step(most) != hs) | (e2m3_step(least) != hs)
    unsure = unsure | ((e2m3(up / hs) * hs != h) | (e2m3(down / hs) * hs != h)).any(-1, keepdim=True)
    rest = (g - h).abs()
    unsure = unsure | (e2m3_step((rest + d).amax(-1, keepdim=True)) != ls) | \
        (e2m3_step((rest - d).clamp_min(0.0).amax(-1, keepdim=True)) != ls)
    off = torch.maximum((e2m3((up - h) / ls) * ls - l).abs(), (e2m3((down - h) / ls) * ls - l).abs())
    off = torch.where(unsure, d + 2.0 * 2.0 ** -8.9 * (big + d), off)
    return v.view_as(x), off.view_as(x)


def few(s):
    """Whether a layer takes the form for a few assignments: x as it is, act in two bf16 numbers, y in float32."""
    return s.T * s.k <= 32 and (s.T == 1 or s.T * s.k <= s.E)


def few_reference(c: Case, x=None):
    """Float32 sums of exact products: at most K / 2 additions in a row, each off by at most 2 U of the magnitudes so far, then
    at most 32 of partial sums.  act comes as two bf16 numbers, off by 2^-16, and takes twice as many; the slots' weights and
    sums add k + 1 more."""
    s = c.shape
    x = (c.x if x is None else x).double()
    ref = torch.zeros(s.T, s.H, dtype=torch.float64, device="cuda")
    err = torch.zeros_like(ref)
    for t in range(s.T):
        for j in range(s.k):
            e = int(c.idx[t, j])
            if not 0 <= e < s.E:
                continue
            gu = c.vgu[e].double()
            p = gu @ x[t]
            act, ea = swiglu_bound(*p.chunk(2), *((gu.abs() @ x[t].abs()) * (s.H + 64) * U).chunk(2))
            ea = ea + 2.0 ** -16 * act.abs()
            v, w = c.vd[e].double(), float(c.w[t, j])
            ref[t] += v @ act * w
            err[t] += (v.abs() @ ea + v.abs() @ (act.abs() + ea) * (2 * s.I + 66 + s.k) * U) * abs(w)
    return ref, err + HALF * (ref.abs() + err)


def layer_reference(c: Case, x=None):
    s = c.shape
    if few(s):
        return few_reference(c, x)
    x2 = two_parts(c.x if x is None else x)
    ref = torch.zeros(s.T, s.H, dtype=torch.float64, device="cuda")
    err = torch.zeros_like(ref)
    idx = c.idx.long()
    for e in range(s.E):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        if t.numel() == 0:
            continue
        p, ep = products(x2[t], np.full(t.numel(), e), c.vgu)
        act, ea = swiglu_bound(*p.chunk(2, 1), *ep.chunk(2, 1))
        a2, ea = two_parts(act, ea)
        v = c.vd[e].double().t().contiguous()
        y = a2 @ v
        ey = ea @ v.abs() + (a2.abs() + ea) @ v.abs() * (s.I / 16 + 16) * 2 * U
        # scaled fp16: half a step, relative; below its normal range half of the smallest step, 2^-25 where the row's
        # 64 columns have their largest in [2^14, 2^15)
        row = (y.abs() + ey).amax(1, keepdim=True)
        ey = ey + 2.0 ** -11 * (y.abs() + ey) + 2.0 ** -38 * row
        w = c.w[t, j].double()[:, None]
        ref.index_add_(0, t, y * w)
        err.index_add_(0, t, ey * w.abs() + (y.abs() + ey) * w.abs() * (s.k + 1) * U)
    return ref, err + HALF * (ref.abs() + err)


SHAPES = [
    # T, H, E, k, I, N: one row, one expert; K of one block; K off every unit; several chunks, the last ones empty
    (1, 64, 1, 1, 64, 1), (5, 64, 3, 2, 64, 1), (40, 128, 4, 3, 192, 1), (97, 320, 5, 4, 448, 3), (130, 576, 8, 2, 256, 2),
    (3, 256, 4, 2, 128, 5), (700, 192, 7, 6, 320, 2), (1500, 448, 12, 3, 192, 1), (2100, 320, 6, 2, 64, 3),
]


@pytest.mark.parametrize("T,H,E,k,I,N", SHAPES)
def test_against_float64(T, H, E, k, I, N):  # noqa: E741
    say(f"4-bit experts T={T} H={H} E={E} k={k} I={I} N={N}")
    c = Case(T, H, E, k, I, N, seed=T)
    within(c.forward(), *layer_reference(c), "out")
    assert int(c.err.item()) == 0


# one token and a handful: one expert, as many assignments as experts, 32 of them and one more; K of less than a unit of
# columns, of a part of one, of more units than waves
FEW = [(1, 64, 1, 1, 64), (1, 64, 2, 8, 64), (1, 2048, 16, 4, 1024), (2, 320, 8, 3, 448), (8, 192, 32, 4, 576),
       (11, 192, 40, 3, 64), (4, 4096 + 320, 9, 2, 2240), (4, 64, 64, 8, 128), (1, 128, 3, 32, 192),
       (11, 128, 70, 3, 192)]


@pytest.mark.parametrize("T,H,E,k,I", FEW)
def test_few_assignments(T, H, E, k, I):  # noqa: E741
    say(f"4-bit experts T={T} H={H} E={E} k={k} I={I}")
    c = Case(T, H, E, k, I, seed=T + k)
    want = c.forward()
    within(want, *layer_reference(c), "out")
    assert int(c.err.item()) == 0
    for n in (2, 5):
        if not few(c.shape):
            break
        assert torch.equal(c.forward(moe.make_shape(T, H, E, k, I, 1, n, "bf16")), want), n
    c.idx[0, 0], c.idx[T - 1, k - 1] = -3, E
    if T == 1 and k == 1:
        assert bool((c.forward() == 0).all())
    within(c.forward(), *layer_reference(c), "out")
    assert int(c.err.item()) == (1 if T * k == 1 else 2)


# row counts on both sides of every tile limit, an expert without rows, slots that are dropped
EDGES = [0, 1, 31, 32, 33, 63, 65, 96, 127, 129, 160, 161, 192, 224, 255, 256, 257, 300, 511, 513, 1025]


@pytest.mark.parametrize("few", [True, False])
def test_row_counts(few):
    counts = EDGES[:9] if few else EDGES
    T = int(sum(counts)) // 2 + 5
    say(f"4-bit experts, rows {counts}")
    c = Case(T, 192, len(counts), 2, 128, 1, counts=counts, seed=3)
    within(c.forward(), *layer_reference(c), "out")
    assert int(c.err.item()) == T * 2 - sum(counts)


@pytest.mark.parametrize("counts", [[1, 2, 40, 5], [300, 40, 700, 2060], [64, 64, 64, 64], [20, 3, 9, 16]])
def test_long_rows(counts):
    """K of many stages: the ring of stages and of scales turns over several times, for few and for many rows."""
    c = Case(sum(counts), 4096 + 320, len(counts), 1, 1088, 1, counts=counts, seed=1)
    say(f"4-bit experts H={c.shape.H} rows {counts}")
    within(c.forward(), *layer_reference(c), "out")


@pytest.mark.parametrize("T", [8, 300, 4500])
def test_magnitudes(T):
    """Rows of every size, groups with one value far above the others, rows of zeros: each is held to its own scale."""
    c = Case(T, 256, 4, 1, 128, 1, seed=11)
    g = gen(12)
    size = torch.exp2(torch.randint(-60, 12, (T, 1), generator=g, device="cuda").float())
    out_of_line = torch.where(torch.rand(T, 256, generator=g, device="cuda") < 0.02, 100.0, 1.0)
    x = (c.x.float() * size * out_of_line).to(BF16)
    x[T // 2] = 0.0
    got = c.forward(x=x)
    within(got, *layer_reference(c, x), "out")
    assert bool((got[T // 2] == 0).all())


@pytest.mark.parametrize("T,k,N", [(2048, 2, (1, 2, 3, 5)), (90, 3, (1, 2, 4))])
def test_chunks_do_not_change_a_bit(T, k, N):
    c = Case(T, 320, 9, k, 192, 1, seed=5)
    want = c.forward()
    for n in N[1:]:
        assert torch.equal(c.forward(moe.make_shape(T, 320, 9, k, 192, 1, n, "bf16")), want), n


def test_both_tilings_give_the_same_bits():
    """Experts that get nothing lower the average of rows that chooses the tiles: 4 of 64 experts, and the same 4 alone."""
    T, H, I = 700, 448, 320  # noqa: E741
    c = Case(T, H, 64, 2, I, 1, counts=[300, 129, 33, 900] + [0] * 60, seed=8)
    want = c.forward()
    c.idx[c.idx >= 4] = -1
    assert torch.equal(c.forward(moe.make_shape(T, H, 4, 2, I, 1, 1, "bf16")), want)


def test_one_expert_gets_everything():
    for T, k in ((64, 1), (300, 1), (5000, 1)):
        c = Case(T, 256, 16, k, 128, 1, counts=[0] * 7 + [T] + [0] * 8, seed=T)
        within(c.forward(), *layer_reference(c), "out")


@pytest.mark.parametrize("T", [3, 200, 4200])
def test_dropped_slots_and_nan(T):
    c = Case(T, 128, 4, 2, 64, 1, seed=9)
    c.idx[1] = -1                       # a token without experts
    c.idx[2, 0] = 4
    clean = c.forward()
    assert bool((clean[1] == 0).all()) and int(c.err.item()) == 3
    within(clean, *layer_reference(c), "out")
    x = c.x.clone()
    x[0, 5] = float("nan")
    x[1, 3] = float("inf")
    got = c.forward(x=x)
    assert bool(got[0].isnan().all())
    assert torch.equal(got[1:], clean[1:])


def test_a_group_that_is_nan():
    c = Case(300, 128, 3, 1, 64, 1, seed=2)
    clean = c.forward()
    c.wds[5] = 255                      # rows 0..31 of expert 0: entry 1, byte 1 (block 1): a group past K = 64 is not read
    assert torch.equal(c.forward(), clean)
    c.wds[4] = 255                      # row 1, columns 0..31
    got = c.forward()
    hit = (c.idx[:, 0] == 0)
    assert bool(got[hit][:, 1].isnan().all())
    got[hit, 1] = clean[hit, 1]
    assert torch.equal(got, clean)


def test_a_group_that_is_nan_for_few_assignments():
    c = Case(3, 128, 4, 1, 64, 1, seed=2)
    c.idx[:, 0] = torch.tensor([0, 1, 0], dtype=torch.int32)
    clean = c.forward()
    c.wds[5] = 255                      # row 1, columns 64..95: past K, not read
    assert torch.equal(c.forward(), clean)
    c.wds[4] = 255                      # row 1, columns 0..31
    got = c.forward()
    assert bool(got[[0, 2], 1].isnan().all())
    got[[0, 2], 1] = clean[[0, 2], 1]
    assert torch.equal(got, clean)


@pytest.mark.parametrize("T", [2, 70, 2100])
def test_graph_and_stream(T):
    c = Case(T, 256, 8, 2, 128, 2, seed=T)
    want = c.forward()
    ws = torch.empty(moe.moe_mx_workspace_size(c.shape), dtype=torch.uint8, device="cuda")
    out, x = torch.empty(T, 256, dtype=BF16, device="cuda"), c.x.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    c.forward(stream=side, out=out, ws=ws)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        c.forward(ws=ws, out=out, x=x)
    for i in range(4):
        x.copy_(c.x * (i + 1))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, c.forward(x=x.clone())), i


def test_experts_weights_read_where_they_lie():
    """Experts' matrices at any 16-byte address, and buffers larger than needed, of which nothing more is read."""
    c = Case(150, 128, 5, 2, 128, 1, seed=4)
    want = c.forward()
    for name in ("wgu", "wgus", "wd", "wds"):
        t = getattr(c, name)
        big = torch.full((t.numel() + 272,), 255, dtype=torch.uint8, device="cuda")
        big[16:16 + t.numel()] = t
        setattr(c, name, big[16:16 + t.numel()])
        assert getattr(c, name).data_ptr() % 256 == 16
    assert torch.equal(c.forward(), want)


def test_whole_block():
    """As a serving program runs it: norm, router on its rows, the 4-bit layer, all in one captured graph."""
    T, H, E, k, I = 48, 256, 16, 4, 128  # noqa: E741
    c = Case(T, H, E, k, I, 1, seed=8)
    s = moe.make_shape(T, H, E, k, I, 4, 1, "bf16")
    g = gen(1)
    gate, bias = torch.randn(H, E, generator=g, device="cuda") / 16, 0.1 * torch.randn(E, generator=g, device="cuda")
    x, y = c.x.clone(), torch.empty_like(c.x)
    out, ws = torch.empty_like(x), torch.empty(moe.moe_mx_workspace_size(s), dtype=torch.uint8, device="cuda")
    idx, w, logits = torch.empty_like(c.idx), torch.empty_like(c.w), torch.empty(T, E, device="cuda")

    def block():
        moe.moe_layer_norm(s, x, None, None, None, 1e-5, None, y)
        torch.mm(y.float(), gate, out=logits)
        moe.moe_router_top_k(s, logits, bias, "sigmoid", 2, True, 1.0, idx, w)
        moe.moe_mx_forward(s, y, idx, w, c.wgu, c.wgus, c.wd, c.wds, out, ws)

    block()
    for t in range(T):
        assert idx[t].tolist() == bo.route_row(logits[t].double().cpu().numpy(), bias.double().cpu().numpy(), "sigmoid", 4,
                                               2, k)
    c.x, c.idx, c.w = y, idx, w
    within(out, *layer_reference(c), "out")
    eager = out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        block()
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


def test_empty_batch():
    c = Case(4, 64, 2, 1, 64, 1)
    s = moe.make_shape(0, 64, 2, 1, 64, 1, 1, "bf16")
    e = dict(device="cuda")
    ws = torch.empty(moe.moe_mx_workspace_size(s), dtype=torch.uint8, **e)
    moe.moe_mx_forward(s, torch.empty(0, 64, dtype=BF16, **e), torch.empty(0, 1, dtype=torch.int32, **e),
                       torch.empty(0, 1, **e), c.wgu, c.wgus, c.wd, c.wds, torch.empty(0, 64, dtype=BF16, **e), ws, c.err)
    torch.cuda.synchronize()
    assert int(c.err.item()) == 0
