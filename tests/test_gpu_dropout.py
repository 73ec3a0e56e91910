"""Dropout into the residual stream on the GPU: the mask against Philox on Python integers, values against float64."""
import numpy as np
import pytest
import torch

import block_oracle as bo
import combine_top_route_expert_amd as moe
from gpu_layer import say

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.load_library()


def words(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


def apply(x, res, p, so, out=None, stream=None):
    T, H = x.shape
    s = moe.make_shape(T, H, 1, 1, 64, 1, 1, "bf16" if x.dtype is torch.bfloat16 else "f32")
    out = torch.full_like(x, float("nan")) if out is None else out
    moe.moe_dropout_add(s, x, res, p, so, out, stream)
    return out


@pytest.mark.parametrize("dtype,T,H", [("bf16", 1, 64), ("bf16", 3, 192), ("bf16", 130, 64), ("f32", 1, 4), ("f32", 3, 4),
                                       ("f32", 7, 36), ("f32", 65, 100), ("f32", 2, 1028)])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.99999])
def test_against_float64(dtype, T, H, p):
    say(f"dropout {dtype} T={T} H={H} p={p}")
    g = torch.Generator(device="cuda").manual_seed(T * H)
    x = torch.randn(T, H, generator=g, device="cuda").to(TYPES[dtype])
    res = torch.randn(T, H, generator=g, device="cuda").to(TYPES[dtype])
    seed, offset = -(1 << 61) + 12345, (1 << 62) + T
    kept = torch.from_numpy(bo.kept_mask(T * H, p, seed, offset)).view(T, H).cuda()
    least = min(65535, round(p * 65536))
    scale = 65536.0 / (65536 - least)
    for r in (res, None):
        ref = torch.where(kept, x.double() * scale, 0.0)
        size = ref.abs()
        if r is not None:
            ref = ref + r.double()
        got = apply(x, r, p, words(seed, offset)).double()
        # the factor in float32 (one rounding of the product's size), then one rounding of the sum
        err = bo.U32 * size * (1 + HALF[dtype])
        # (float32 without a residual: a rounded product instead of a rounded sum; both count as the last one)
        assert bool(((got - ref).abs() <= err + HALF[dtype] * (ref.abs() + err) + 1e-37).all())


def test_mask_depends_on_seed_offset_and_place_only():
    n = 64 * 1024
    one = torch.ones(64, 1024, device="cuda")
    a = apply(one, None, 0.3, words(1, 2)) > 0
    assert torch.equal(a, apply(one.bfloat16(), None, 0.3, words(1, 2)) > 0)
    assert torch.equal(a.view(-1), (apply(one.view(4096, 16), None, 0.3, words(1, 2)) > 0).view(-1))
    for other in (words(2, 2), words(1, 3), words(1 + (1 << 32), 2), words(1, 2 + (1 << 32))):
        assert 0.35 < float((apply(one, None, 0.3, other) > 0).eq(a).float().mean()) < 0.75  # 0.58 where independent
    # kept 0.7 of 65536: 8 standard deviations are 0.0144
    assert abs(float(a.float().mean()) - 0.7) < 0.0144
    assert n == a.numel()


def test_a_large_batch_agrees_where_it_is_looked_at():
    """Groups past the first pass of the grid: 2^27 elements, a few stretches against the generator."""
    T, H = 1 << 14, 1 << 13
    x = torch.ones(T, H, dtype=torch.bfloat16, device="cuda")
    got = (apply(x, None, 0.25, words(99, 7)) > 0).view(-1)
    for first in (0, 12345, (T * H) // 16 + 3, T * H // 8 - 40):
        want = bo.kept_mask(320, 0.25, 99, 7, first)
        assert got[8 * first: 8 * first + 320].cpu().numpy().tolist() == want.tolist(), first


def test_dropped_values_leave_nothing():
    T, H, p = 4, 256, 0.5
    kept = torch.from_numpy(bo.kept_mask(T * H, p, 5, 6)).view(T, H).cuda()
    for bad in (float("nan"), float("inf")):
        x = torch.where(kept, 1.0, bad).float()
        for dt in TYPES.values():
            got = apply(x.to(dt), None, p, words(5, 6))
            assert torch.equal(got, torch.where(kept, 2.0, 0.0).to(dt))
            assert torch.equal(apply(x.to(dt), torch.ones_like(got), p, words(5, 6)), got + 1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_in_place_and_gradient(dtype):
    T, H, p = 33, 320, 0.2
    g = torch.Generator(device="cuda").manual_seed(1)
    x, res, gout = (torch.randn(T, H, generator=g, device="cuda").to(TYPES[dtype]) for _ in range(3))
    so = words(11, 12)
    want = apply(x, res, p, so)
    assert torch.equal(apply(x.clone(), res, p, so, out=(buf := x.clone())), want) and buf is not x
    both = x.clone()
    assert torch.equal(apply(both, res, p, so, out=both), want)
    both = res.clone()
    assert torch.equal(apply(x, both, p, so, out=both), want)
    # gradient: the same mask and factor; against the difference of outputs along gout it is linear, so exact in x
    grad = apply(gout, None, p, so).double()
    kept = torch.from_numpy(bo.kept_mask(T * H, p, 11, 12)).view(T, H).cuda()
    scale = 65536.0 / (65536 - round(p * 65536))
    ref = torch.where(kept, gout.double() * scale, 0.0)
    err = ref.abs() * bo.U32 * 2
    assert bool(((grad - ref).abs() <= err + HALF[dtype] * (ref.abs() + err)).all())


def test_graph_that_advances_its_offset():
    """Replays whose offset a captured addition advances give the masks of eager calls with those offsets."""
    T, H, p = 64, 512, 0.1
    x = torch.randn(T, H, device="cuda").bfloat16()
    res, out, so = torch.randn(T, H, device="cuda").bfloat16(), torch.empty_like(x), words(3, 100)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    step = torch.tensor([0, 1], device="cuda")
    with torch.cuda.graph(graph, stream=side):
        apply(x, res, p, so, out=out)
        so.add_(step)
    for i in range(5):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, apply(x, res, p, words(3, 100 + i))), i
        assert so.tolist() == [3, 101 + i]


def test_empty_batch():
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    assert apply(x, None, 0.5, words(1, 1)).numel() == 0
