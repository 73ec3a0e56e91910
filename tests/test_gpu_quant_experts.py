"""The layer with 8-bit integer experts on the GPU against float64 (integer sums are exact there).

Each step is held, element by element, to its own inputs' exact result and a bound counted in float32 roundings plus the
one rounding to the output's dtype; the quantised act rows have to be equal; the whole layer has to give the bits of its
steps."""
import numpy as np
import pytest
import torch

import combine_top_route_expert_amd as moe
import norm_oracle as no
from gpu_layer import say

pytestmark = pytest.mark.gpu
U = no.U32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.load_library()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def int8(g, *size):
    """Every value of the type, -128 among them."""
    return torch.randint(-128, 128, size, generator=g, device="cuda", dtype=torch.int8)


def scales(g, *size):
    return (0.25 + torch.rand(size, generator=g, device="cuda")) * 2.0 ** -9


def ids_with_counts(counts, T, k, seed, outside=(-1, 1 << 20)):
    """[T][k] ids in which expert e appears counts[e] times; the rest lie outside the experts."""
    flat = np.concatenate([np.repeat(np.arange(len(counts)), counts),
                           np.resize(np.array(outside), T * k - int(np.sum(counts)))])
    np.random.default_rng(seed).shuffle(flat)
    return torch.from_numpy(flat.astype(np.int32).reshape(T, k)).cuda()


class Case:
    def __init__(self, T, H, E, k, I, N, dtype, counts=None, seed=0):  # noqa: E741
        g = gen(seed)
        self.dt = no.TORCH[dtype]
        self.dtype = dtype
        self.shape = s = moe.make_shape(T, H, E, k, I, 1, N, dtype)
        if counts is None:
            self.idx = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
        else:
            self.idx = ids_with_counts(counts, T, k, seed)
        self.w = torch.rand(T, k, generator=g, device="cuda")
        # activations as rows' quantisation leaves them, now and then with a value that only weights hold
        self.q, self.qs = int8(g, T, H), scales(g, T)
        self.wgu, self.wgus = int8(g, E, 2 * I, H), scales(g, E, 2 * I) / H ** 0.5
        self.wd, self.wds = int8(g, E, H, I), scales(g, E, H)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.counts, self.offsets = torch.empty(N, E, **i32), torch.empty(N, E + 1, **i32)
        self.splits, self.err = torch.empty(N, 1, **i32), torch.empty(1, **i32)
        self.src, self.dst = torch.empty(T * k, **i32), torch.empty(T * k, **i32)
        ws = torch.empty(moe.moe_route_meta_workspace_size(s), dtype=torch.uint8, device="cuda")
        moe.moe_route_meta(s, self.idx, self.counts, self.offsets, self.splits, self.src, self.dst, self.err, ws)
        self.off = self.offsets.cpu().numpy()

    def pair_rows(self, c):
        """Joint rows of pair (c, c + 1) as (joint row, part, chunk row, expert) arrays, and the rows it may hold."""
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

    def forward(self, ws=None, out=None, q=None, qs=None):
        s = self.shape
        ws = torch.full((moe.moe_quant_workspace_size(s),), 0xa5, dtype=torch.uint8, device="cuda") if ws is None else ws
        out = torch.full((s.T, s.H), float("nan"), dtype=self.dt, device="cuda") if out is None else out
        moe.moe_quant_forward(s, self.q if q is None else q, self.qs if qs is None else qs, self.idx, self.w, self.wgu,
                              self.wgus, self.wd, self.wds, out, ws, self.err)
        return out


def within(got, ref, bound, what):
    off = (got.double() - ref).abs() - bound
    assert not bool(off.isnan().any()), what
    worst = int(off.argmax())
    assert float(off.flatten()[worst]) <= 0, \
        f"{what}[{worst}]: {float(got.flatten()[worst])!r} against {float(ref.flatten()[worst])!r}, " \
        f"bound {float(bound.flatten()[worst]):.3g}"


def products(rows, scale, expert, wq, ws):
    """The scaled products of every row with its expert's matrix, in float64: exact integer sums, exact scales' product
    to 53 bits."""
    got = torch.empty(rows.shape[0], wq.shape[1], dtype=torch.float64, device="cuda")
    for e in np.unique(expert):
        at = torch.from_numpy(np.nonzero(expert == e)[0]).cuda()
        got[at] = rows[at].double() @ wq[int(e)].double().t().contiguous() * scale[at].double()[:, None] * \
            ws[int(e)].double()
    return got


def check_gate_up(act, rows, scale, expert, wgu, wgus, dtype, what):
    p = products(rows, scale, expert, wgu, wgus)
    g, u = p.chunk(2, 1)
    ref = g * torch.sigmoid(g) * u
    # g and u: conversion and two products each (3 roundings); silu's relative sensitivity to g is at most 1 + |g|; the
    # exponential's argument is rounded (2 |g| units of its result), it, the reciprocal, the sum and the two products
    # add one or two units each; a result below float32's normal range is off by that range
    err = ref.abs() * U * (3 * (1 + g.abs()) + 3 + 2 * g.abs() + 10) + 1e-37
    within(act, ref, err + no.HALF_STEP[dtype] * (ref.abs() + err), what)


def check_down(y, rows, scale, expert, wd, wds, dtype, what):
    ref = products(rows, scale, expert, wd, wds)
    err = ref.abs() * 3 * U + 1e-37
    within(y, ref, err + no.HALF_STEP[dtype] * (ref.abs() + err), what)


def run_steps(c: Case):
    """All pairs step by step, each step checked; returns the layer's output from the steps."""
    s = c.shape
    out = torch.full((s.T, s.H), float("nan"), dtype=c.dt, device="cuda")
    for chunk in range(0, s.N, 2):
        part, row, exp, bound = c.pair_rows(chunk)
        n, total = len(exp), sum(bound)
        if total == 0:
            continue
        act = torch.full((total, s.I), 7.0, dtype=c.dt, device="cuda")
        moe.moe_quant_gate_up_gather_pair(s, chunk, c.q, c.qs, c.src, c.offsets, c.wgu, c.wgus, act)
        t0 = [moe.moe_chunk_range(s, x)[0] if x < s.N else 0 for x in (chunk, chunk + 1)]
        src = c.src.cpu().numpy()
        token = torch.from_numpy(np.array([src[t0[p] * s.k + r] // s.k for p, r in zip(part, row)], np.int64)).cuda()
        if n:
            check_gate_up(act[:n], c.q[token], c.qs[token], exp, c.wgu, c.wgus, c.dtype, f"act of chunk {chunk}")
        assert bool((act[n:] == 7.0).all()), "rows past the valid ones were written"
        aq = torch.full((total, s.I), 99, dtype=torch.int8, device="cuda")
        asc = torch.full((total,), -7.0, device="cuda")
        moe.moe_quant_act_pair(s, chunk, act, c.offsets, aq, asc)
        if n:
            rq, rs = no.quantize(no.f64(act[:n]))
            assert np.array_equal(aq[:n].cpu().numpy(), rq)
            assert np.array_equal(asc[:n].cpu().numpy(), rs.astype(np.float32))
        assert bool((aq[n:] == 99).all()) and bool((asc[n:] == -7.0).all())
        y = [torch.full((b, s.H), 7.0, dtype=c.dt, device="cuda") for b in bound]
        moe.moe_quant_down_pair(s, chunk, aq, asc, c.offsets, c.wd, c.wds, y[0], y[1] if bound[1] else None)
        for p in (0, 1):
            at = np.nonzero(part == p)[0]
            if len(at):
                joint = torch.from_numpy(at).cuda()
                check_down(y[p][torch.from_numpy(row[at]).cuda()], aq[joint], asc[joint], exp[at], c.wd, c.wds, c.dtype,
                           f"y of chunk {chunk + p}")
            if bound[p]:
                assert bool((y[p][len(at):] == 7.0).all()), "rows past the valid ones were written"
                moe.moe_unpermute_combine(s, chunk + p, y[p], c.dst, c.w, out)
    return out


# counts on both sides of every class of tile (32, 64, 128, 160, 256 rows), none at all, and several tiles
COUNTS = [1, 0, 31, 32, 33, 64, 65, 0, 127, 128, 129, 160, 161, 255, 256, 257, 600]
SMALL = [(1, 64, 1, 1, 64, 1), (1, 320, 8, 4, 192, 1), (3, 192, 16, 8, 64, 4), (7, 448, 5, 3, 320, 2),
         (64, 512, 16, 4, 128, 1), (97, 64, 9, 2, 448, 3), (500, 320, 8, 4, 192, 1), (203, 128, 40, 3, 256, 2)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,E,k,I,N", SMALL)
def test_small(dtype, T, H, E, k, I, N):  # noqa: E741
    say(f"quant {dtype} T={T} H={H} E={E} k={k} I={I} N={N}")
    c = Case(T, H, E, k, I, N, dtype, seed=T)
    steps, out = run_steps(c), c.forward()
    torch.cuda.synchronize()
    assert torch.equal(steps, out)
    assert int(c.err) == 0


@pytest.mark.parametrize("dtype,N", [("bf16", 1), ("bf16", 2), ("f32", 1)])
@pytest.mark.parametrize("H,I", [(128, 128), (320, 384), (512, 192), (64, 640), (576, 256)])
def test_tile_classes(dtype, N, H, I):  # noqa: E741
    """Every class of tile in one launch of more than 4096 rows (the large tile, for bf16 and even I), and of fewer."""
    for T in (1400, 900):
        say(f"quant tiles {dtype} T={T} N={N} H={H} I={I}")
        counts = list(COUNTS) if T * 4 > 4096 else [n // 2 for n in COUNTS]
        c = Case(T, H, len(counts), 4, I, N, dtype, counts, seed=H + I)
        steps, out = run_steps(c), c.forward()
        torch.cuda.synchronize()
        assert torch.equal(steps, out)
        assert int(c.err) == T * 4 - sum(counts)
        gone = (c.idx < 0) | (c.idx >= len(counts))
        assert not out[gone.all(1)].any()            # a token whose slots were all dropped


FEW = [(1, 64, 3, 3, 64, 1), (1, 320, 8, 4, 192, 1), (1, 1088, 40, 32, 2112, 2), (1, 128, 40, 33, 64, 1),
       (4, 448, 64, 4, 320, 3), (8, 2048, 64, 4, 1024, 1), (32, 192, 64, 1, 64, 32), (8, 192, 63, 4, 64, 1),
       (16, 64, 70, 2, 448, 2), (8, 192, 32, 4, 64, 1), (16, 64, 31, 2, 128, 1),
       (1, 64, 9, 8, 8192, 1), (1, 64, 9, 8, 8256, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,E,k,I,N", FEW)
def test_few_assignments(dtype, T, H, E, k, I, N):  # noqa: E741
    """Both sides of the rule for unsorted assignments (at most 32 of them, as many as experts unless they are one
    token's, and 64 KB of quantised rows): the layer gives the bits of the sorted steps, dropped ids and repeated experts
    among them."""
    for kind in ("distinct", "same", "dropped", "all dropped"):
        say(f"few {dtype} T={T} H={H} E={E} k={k} I={I} N={N} {kind}")
        g = np.random.default_rng(T * k)
        if kind == "distinct":
            counts = np.bincount(g.permutation(E)[np.arange(T * k) % E], minlength=E)
        elif kind == "same":
            counts = np.bincount([E - 1] * (T * k), minlength=E)
        else:
            counts = np.bincount(g.integers(0, E, T * k // 2 if kind == "dropped" else 0), minlength=E)
        c = Case(T, H, E, k, I, N, dtype, counts, seed=T)
        c.err.fill_(-7)
        steps, out = run_steps(c), c.forward()
        torch.cuda.synchronize()
        assert torch.equal(steps, out)
        assert int(c.err) == T * k - counts.sum()


def test_few_assignments_bad_token_and_replay():
    T, H, E, k, I = 4, 512, 64, 4, 256  # noqa: E741
    c = Case(T, H, E, k, I, 1, "bf16", seed=40)
    good = c.forward()
    qs = c.qs.clone()
    qs[2] = float("nan")
    out = c.forward(qs=qs)
    torch.cuda.synchronize()
    assert bool(out[2].isnan().all()) and torch.equal(out[[0, 1, 3]], good[[0, 1, 3]])
    ws = torch.empty(moe.moe_quant_workspace_size(c.shape), dtype=torch.uint8, device="cuda")
    idx, got = c.idx.clone(), torch.empty_like(good)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.forward(ws=ws, out=got)
    for n in range(3):
        c.idx.copy_((idx + n) % E if n != 1 else -idx)
        got.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        ref = c.forward()
        torch.cuda.synchronize()
        assert torch.equal(ref, got), n


def test_many_experts_few_active():
    """More experts than the rows can fill: workgroups that take several tiles."""
    E = 1024
    for H, I in ((1024, 512), (832, 384)):  # noqa: E741
        counts = np.zeros(E, int)
        counts[[3, 700, 1023]] = [4000, 90, 6]
        say(f"quant E={E} H={H} I={I}")
        c = Case(1024, H, E, 4, I, 1, "bf16", counts, seed=5)
        steps, out = run_steps(c), c.forward()
        torch.cuda.synchronize()
        assert torch.equal(steps, out)


def test_chunks_and_repeats_give_the_same_bits():
    ref = None
    for N in (1, 2, 3, 4, 7, 2000):
        c = Case(1100, 320, 12, 5, 256, N, "bf16", seed=3)
        out = c.forward()
        again = c.forward()
        torch.cuda.synchronize()
        assert torch.equal(out, again)
        ref = out if ref is None else ref
        assert torch.equal(out, ref), N


def test_same_expert_in_every_slot_and_all_dropped():
    c = Case(300, 128, 4, 8, 128, 1, "bf16", seed=4)
    c.idx.fill_(2)
    c2 = Case(300, 128, 4, 8, 128, 1, "bf16", seed=4)
    c2.idx.fill_(-1)
    out, out2 = c.forward(), c2.forward()
    torch.cuda.synchronize()
    assert bool(out.isfinite().all()) and int(c2.err) == 2400 and not out2.any()


def test_no_tokens():
    c = Case(5, 128, 4, 2, 64, 1, "bf16", seed=6)
    s = moe.make_shape(0, 128, 4, 2, 64, 1, 1, "bf16")
    none = torch.empty(0, device="cuda")
    ws = torch.empty(moe.moe_quant_workspace_size(s), dtype=torch.uint8, device="cuda")
    err = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    moe.moe_quant_forward(s, none.to(torch.int8), none, none.int(), none, c.wgu, c.wgus, c.wd, c.wds,
                          none.bfloat16(), ws, err)
    torch.cuda.synchronize()
    assert int(err) == 0


def test_bad_token_stays_in_its_row():
    for dtype in ("bf16", "f32"):
        c = Case(1030, 192, 6, 4, 128, 1, dtype, seed=7)
        x = torch.randn(1030, 192, generator=gen(8), device="cuda").to(c.dt)
        x[17, 3], x[900, 191], x[41] = float("nan"), float("inf"), 0.0
        q, qs = torch.empty(1030, 192, dtype=torch.int8, device="cuda"), torch.empty(1030, device="cuda")
        moe.moe_quantize_rows(1030, 192, dtype, x, q, qs)
        out = c.forward(q=q, qs=qs)
        x[17], x[900] = 1.0, 1.0
        moe.moe_quantize_rows(1030, 192, dtype, x, q, qs)
        good = c.forward(q=q, qs=qs)
        torch.cuda.synchronize()
        bad = torch.zeros(1030, dtype=torch.bool, device="cuda")
        bad[[17, 900]] = True
        assert bool(out[bad].isnan().all()) and torch.equal(out[~bad], good[~bad])
        assert not out[41].any()


def test_rows_and_weights_past_4_gib():
    """Rows of A beyond 32-bit offsets (the global form of the stage loads), by samples."""
    g = gen(9)
    for T, H, I, k in ((66000, 65536, 128, 1), (66000, 65536 + 64, 64, 1)):  # noqa: E741
        say(f"quant T={T} H={H}: {T * H / 2**30:.1f} GiB of hidden rows")
        s = moe.make_shape(T, H, 2, k, I, 1, 1, "bf16")
        q, qs = torch.empty(T, H, dtype=torch.int8, device="cuda"), scales(g, T) / 256
        for t in range(0, T, 6000):
            q[t:t + 6000] = int8(g, min(6000, T - t), H)
        wgu, wgus = int8(g, 2, 2 * I, H), scales(g, 2, 2 * I)
        src = torch.randperm(T, generator=g, device="cuda").int()
        off = torch.tensor([[0, 40000, T]], dtype=torch.int32, device="cuda")
        act = torch.empty(T, I, dtype=torch.bfloat16, device="cuda")
        moe.moe_quant_gate_up_gather_pair(s, 0, q, qs, src, off, wgu, wgus, act)
        torch.cuda.synchronize()
        at = torch.cat([torch.topk(src, 40).indices, torch.tensor([0, 39999, 40000, T - 1], device="cuda")])
        token = src[at].long()
        check_gate_up(act[at], q[token], qs[token], (at >= 40000).int().cpu().numpy(), wgu, wgus, "bf16", "act")
        # the same bytes as the quantised act of an (H, I)-swapped layer
        sd = moe.make_shape(T, I, 2, k, H, 1, 1, "bf16")
        wd, wds = int8(g, 2, I, H), scales(g, 2, I)
        y = torch.empty(T, I, dtype=torch.bfloat16, device="cuda")
        moe.moe_quant_down_pair(sd, 0, q, qs, off, wd, wds, y, None)
        torch.cuda.synchronize()
        at = torch.tensor([0, 1, 39999, 40000, 65535, 65536, 65537, T - 1], device="cuda")
        check_down(y[at], q[at], qs[at], (at >= 40000).int().cpu().numpy(), wd, wds, "bf16", "y")
        del q


def test_side_stream_and_two_graphs():
    """On a side stream, and two captured layers with a workspace each, replayed in turn with eager calls between."""
    cases = [Case(70, 512, 16, 4, 256, 1, "bf16", seed=10), Case(1300, 320, 8, 4, 128, 2, "bf16", seed=11)]
    ref = [c.forward() for c in cases]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):                     # the buffers are filled, used and freed on st, too
        side = [c.forward() for c in cases]
    torch.cuda.synchronize()
    for a, b in zip(ref, side):
        assert torch.equal(a, b)
    graphs = []
    for c in cases:
        ws = torch.empty(moe.moe_quant_workspace_size(c.shape), dtype=torch.uint8, device="cuda")
        out = torch.empty_like(ref[0] if c is cases[0] else ref[1])
        x = torch.randn(c.shape.T, c.shape.H, generator=gen(12), device="cuda").bfloat16()
        q, qs = torch.empty_like(c.q), torch.empty_like(c.qs)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.moe_quantize_rows(c.shape.T, c.shape.H, "bf16", x, q, qs)
            c.forward(ws=ws, out=out, q=q, qs=qs)
        graphs.append((g, x, out, ws))
    for n in range(3):
        for c, (g, x, out, _) in zip(cases, graphs):
            x.normal_(generator=gen(20 + n))
            out.fill_(7.0)
            g.replay()
        torch.cuda.synchronize()
        for c, (g, x, out, _) in zip(cases, graphs):
            q, qs = torch.empty_like(c.q), torch.empty_like(c.qs)
            moe.moe_quantize_rows(c.shape.T, c.shape.H, "bf16", x, q, qs)
            eager = c.forward(q=q, qs=qs)
            torch.cuda.synchronize()
            assert torch.equal(out, eager), n


def test_norm_then_experts_as_served():
    """Norm with quantised rows, then the layer, against the float64 definition of both: the layer's two rounded
    intermediates (act, and its 8-bit form) may fall to the other side of a rounding, by one unit in few places, so the
    output is held by its rows' largest value, as the bf16 layer is."""
    T, H, E, k, I = 333, 448, 10, 4, 192  # noqa: E741
    c = Case(T, H, E, k, I, 2, "bf16", seed=13)
    x = torch.randn(T, H, generator=gen(14), device="cuda").bfloat16()
    r = torch.randn(T, H, generator=gen(15), device="cuda").bfloat16()
    nw, nb = 1 + 0.1 * torch.randn(H, device="cuda", generator=gen(16)), 0.1 * torch.randn(H, device="cuda", generator=gen(17))
    wgu = (0.05 * torch.randn(E, 2 * I, H, generator=gen(18), device="cuda")).bfloat16()
    wd = (0.05 * torch.randn(E, H, I, generator=gen(19), device="cuda")).bfloat16()
    moe.moe_quantize_rows(E * 2 * I, H, "bf16", wgu, c.wgu, c.wgus)
    moe.moe_quantize_rows(E * H, I, "bf16", wd, c.wd, c.wds)
    sm, y, q, qs = torch.empty_like(x), torch.empty_like(x), torch.empty_like(c.q), torch.empty_like(c.qs)
    moe.moe_layer_norm_quantize(c.shape, x, r, nw, nb, 1e-5, sm, y, q, qs)
    out = c.forward(q=q, qs=qs)
    torch.cuda.synchronize()
    s64 = no.f64((x.float() + r.float()).bfloat16())
    y64 = torch.from_numpy(no.norm(s64, no.f64(nw), no.f64(nb), 1e-5)[0]).bfloat16()
    q64, qs64 = no.quantize(no.f64(y64))
    rows = (torch.from_numpy(q64).double() * torch.from_numpy(qs64)[:, None]).cuda()
    ref = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    plain = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    xy = y64.double().cuda()
    for e in range(E):
        for hid, gu, dn, quant, to in ((rows, c.wgu[e].double() * c.wgus[e].double()[:, None],
                                        c.wd[e].double() * c.wds[e].double()[:, None], True, ref),
                                       (xy, wgu[e].double(), wd[e].double(), False, plain)):
            g, u = (hid @ gu.t().contiguous()).chunk(2, 1)
            act = g * torch.sigmoid(g) * u
            if quant:
                aq, asc = no.quantize(no.f64(act.bfloat16()))
                act = (torch.from_numpy(aq).double() * torch.from_numpy(asc)[:, None]).cuda()
            ye = act @ dn.t().contiguous()
            to += ye * (c.w.double() * (c.idx == e)).sum(1, keepdim=True)
    big = ref.abs().amax(1, keepdim=True)
    assert float(((out.double() - ref).abs() / big).max()) < 2e-2
    # and the 8-bit layer is the layer: its distance from unquantised products is that of 8-bit rounding (each of
    # three quantised factors adds about max / (127 sqrt 12) per value against values of max / 4)
    rel = float((out.double() - plain).norm() / plain.norm())
    assert rel < 3 * 4 / (127 * 12 ** 0.5) * 2


def test_norm_around_the_layer_as_trained():
    """Norm forward, layer forward and backward, norm backward in float32: the gradients against autograd in float64."""
    T, H, E, k, I = 37, 64, 5, 3, 64  # noqa: E741
    s = moe.make_shape(T, H, E, k, I, 1, 2, "f32")
    g = gen(30)
    x, r = (torch.randn(T, H, generator=g, device="cuda") for _ in range(2))
    nw, nb = 1 + 0.1 * torch.randn(H, generator=g, device="cuda"), 0.1 * torch.randn(H, generator=g, device="cuda")
    idx = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    w = torch.rand(T, k, generator=g, device="cuda")
    wgu = 0.2 * torch.randn(E, 2 * I, H, generator=g, device="cuda")
    wd = 0.2 * torch.randn(E, H, I, generator=g, device="cuda")
    go = torch.randn(T, H, generator=g, device="cuda")
    f32 = dict(device="cuda")
    sm, y, out = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(T, **f32), torch.empty(T, **f32)
    moe.moe_layer_norm(s, x, r, nw, nb, 1e-5, sm, y, mean, rstd)
    moe.moe_chunked_forward(s, y, idx, w, wgu, wd, out,
                            torch.empty(moe.moe_workspace_size(s), dtype=torch.uint8, **f32))
    gy, gw, ggu, gd = torch.empty_like(x), torch.empty_like(w), torch.empty_like(wgu), torch.empty_like(wd)
    moe.moe_chunked_backward(s, y, idx, w, wgu, wd, go, gy, gw, ggu, gd,
                             torch.empty(moe.moe_backward_workspace_size(s), dtype=torch.uint8, **f32))
    gx, gnw, gnb = torch.empty_like(x), torch.empty_like(nw), torch.empty_like(nb)
    moe.moe_layer_norm_backward(s, gy, sm, nw, mean, rstd, go, gx, gnw, gnb,
                                torch.empty(moe.moe_layer_norm_backward_workspace_size(s), dtype=torch.uint8, **f32))
    torch.cuda.synchronize()
    # block output = sum + layer(norm(sum)): the residual gradient is grad_out itself
    leaf = [t.double().cpu().requires_grad_() for t in (sm, nw, nb)]
    d = leaf[0] - leaf[0].mean(1, keepdim=True)
    yn = d / ((d * d).mean(1, keepdim=True) + 1e-5).sqrt() * leaf[1] + leaf[2]
    ids, tot = idx.cpu(), leaf[0]
    for e in range(E):
        gg, uu = (yn @ wgu[e].double().cpu().t()).chunk(2, 1)
        ye = (gg * torch.sigmoid(gg) * uu) @ wd[e].double().cpu().t()
        tot = tot + ye * (w.double().cpu() * (ids == e)).sum(1, keepdim=True)
    (tot * go.double().cpu()).sum().backward()
    for got, lf in zip((gx, gnw, gnb), leaf):
        # float32 throughout; the layer's own fp32 backward is held to 1e-5 of its rows' largest value
        err = (got.double().cpu() - lf.grad).abs().max() / lf.grad.abs().max()
        assert float(err) < 2e-5


def test_large_tiles_below_4096_rows():
    """Few experts with many rows each: the large tile for both products, for one of them, and (K too short) for none."""
    for T, H, E, I in ((600, 2048, 32, 2048), (600, 2048, 16, 2048), (640, 1984, 40, 1024)):  # noqa: E741
        say(f"quant T={T} H={H} E={E} I={I}")
        c = Case(T, H, E, 4, I, 1, "bf16", seed=50)
        steps, out = run_steps(c), c.forward()
        torch.cuda.synchronize()
        assert torch.equal(steps, out)


def test_random_shapes():
    rng = np.random.default_rng(60)
    for n in range(16):
        k = int(rng.integers(1, 9))
        E, T = int(rng.integers(max(1, k // 2), 70)), int(np.exp(rng.uniform(0, np.log(1500))))
        H, I = 64 * int(rng.integers(1, 14)), 64 * int(rng.integers(1, 14))  # noqa: E741
        N, dtype = int(rng.integers(1, 5)), ("bf16", "f32")[n % 2]
        say(f"quant random {n}: {dtype} T={T} H={H} E={E} k={k} I={I} N={N}")
        c = Case(T, H, E, k, I, N, dtype, seed=100 + n)
        steps, out = run_steps(c), c.forward()
        torch.cuda.synchronize()
        assert torch.equal(steps, out)


def test_two_layers_at_once():
    """Two streams, a workspace each, twenty layers on either without a wait between them."""
    cases = [Case(900, 320, 12, 5, 256, 1, "bf16", seed=70), Case(3, 512, 16, 4, 256, 1, "bf16", seed=71)]
    ref = [c.forward() for c in cases]
    outs = [[torch.empty_like(r) for _ in range(20)] for r in ref]
    ws = [torch.empty(moe.moe_quant_workspace_size(c.shape), dtype=torch.uint8, device="cuda") for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()                        # every buffer is ready before either stream starts
    for n in range(20):
        for c, st, o, w in zip(cases, streams, outs, ws):
            with torch.cuda.stream(st):
                c.forward(ws=w, out=o[n])
    torch.cuda.synchronize()
    for r, o in zip(ref, outs):
        for t in o:
            assert torch.equal(r, t)


def test_fp32_act_is_exact_to_its_roundings():
    """gate and up are exact in float32 here (integer sums below 2^24, scales that are powers of two), so what is left in
    act is the exponential (within 3 units, 6 half units), the sum, the quotient and the product: 9 half units, and a tenth
    for their products, whatever the size of gate."""
    T, H, E, I = 700, 64, 3, 64  # noqa: E741
    c = Case(T, H, E, 1, I, 1, "f32", seed=80)
    c.qs.fill_(2.0 ** -6)
    c.wgus.fill_(2.0 ** -4)
    c.wgu.copy_(torch.randint(-30, 31, c.wgu.shape, generator=gen(81), device="cuda"))
    act = torch.empty(T, I, device="cuda")
    moe.moe_quant_gate_up_gather_pair(c.shape, 0, c.q, c.qs, c.src, c.offsets, c.wgu, c.wgus, act)
    torch.cuda.synchronize()
    _, _, exp, _ = c.pair_rows(0)
    token = c.src.long()
    p = products(c.q[token], c.qs[token], exp, c.wgu, c.wgus)
    assert torch.equal(p, p.float().double())
    g, u = p.chunk(2, 1)
    assert -80 < float(g.min()) < -30  # no result below float32's normal range
    ref = g * torch.sigmoid(g) * u
    within(act, ref, 10 * U * ref.abs(), "act")
