"""Calls that are run in several launches: tokens of which one launch of a wave for each holds 2^25, dropout of more than 2^30
elements."""
import pytest
import torch

import block_oracle as bo
import combine_top_route_expert_amd as moe
from gpu_layer import say

pytestmark = pytest.mark.gpu
MANY = (1 << 26) + 77


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.load_library()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_router(dtype):
    """Three experts: every token's ids and weights against torch, and the gradient of a weight that is a sigmoid."""
    T, E, k = MANY, 3, 2
    say(f"router of {T} tokens, {dtype}")
    x = torch.randint(-40, 40, (T, E), device="cuda", dtype=torch.int8).to(dtype) / 8
    s = moe.make_shape(T, 64, E, k, 64, 1, 1, "bf16")
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), 7.0, device="cuda")
    moe.moe_router_top_k(s, x, None, "sigmoid", 0, False, 1.0, idx, w)
    top, at = torch.sort(x.float(), dim=1, descending=True, stable=True)
    assert torch.equal(idx, at[:, :k].int())
    want = torch.sigmoid(top[:, :k])
    assert float((w - want).abs().max()) < 8 * 2.0 ** -24
    grad = torch.full_like(x, 7.0)
    moe.moe_router_top_k_backward(s, x, idx, torch.ones_like(w), "sigmoid", False, 1.0, grad)
    ref = torch.zeros_like(top).scatter_(1, at[:, :k], want * (1 - want))
    # one rounding to bf16 of at most 1/4
    assert float((grad.float() - ref).abs().max()) < (2.0 ** -10 if dtype is torch.bfloat16 else 2.0 ** -22)


def test_4bit_layer():
    """One expert whose act is x silu(x) in the first of 64 columns, and whose output is that in each."""
    T, H = MANY, 64
    say(f"4-bit layer of {T} tokens")
    gu = torch.zeros(1, 128, H, device="cuda")
    gu[0, 0, 0] = gu[0, 64, 0] = 1.0
    d = torch.zeros(1, H, 64, device="cuda")
    d[0, :, 0] = 1.0

    def packed(v):
        rows, cols = v.shape[1:]
        q = torch.empty(rows * cols // 2, dtype=torch.uint8, device="cuda")
        sc = torch.empty(moe.moe_mx_scale_size(rows, cols), dtype=torch.uint8, device="cuda")
        moe.moe_quantize_mx(rows, cols, "f32", v, q, sc)
        return q, sc

    s = moe.make_shape(T, H, 1, 1, 64, 1, 2, "bf16")
    value = (torch.arange(T, device="cuda") % 251 - 125).to(torch.bfloat16) / 16
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = value
    idx, w = torch.zeros(T, 1, dtype=torch.int32, device="cuda"), torch.ones(T, 1, device="cuda")
    ws = torch.empty(moe.moe_mx_workspace_size(s), dtype=torch.uint8, device="cuda")
    out = torch.full_like(x, float("nan"))
    moe.moe_mx_forward(s, x, idx, w, *packed(gu), *packed(d), out, ws)
    v = value.float()
    ref = v * v * torch.sigmoid(v)
    # act and out: one rounding to bf16 each
    bound = ref.abs() * (2 * 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -16) + 1e-30
    for c in (0, 63):
        assert bool(((out[:, c].float() - ref).abs() <= bound).all())
    first, last = out[: 1 << 20], out[-(1 << 20):]
    assert bool((first == first[:, :1]).all()) and bool((last == last[:, :1]).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dropout(dtype):
    """The mask goes on where one launch ends: stretches on both sides of it, and the last elements, against the generator."""
    T, H = (1 << 22) + 3, 256
    say(f"dropout of {T} x {H} {dtype}")
    s = moe.make_shape(T, H, 1, 1, 64, 1, 1, "bf16" if dtype is torch.bfloat16 else "f32")
    x = torch.ones(T, H, dtype=dtype, device="cuda")
    so = torch.tensor([99, 7], device="cuda")
    for residual in (None, x):
        out = torch.full_like(x, float("nan"))
        moe.moe_dropout_add(s, x, residual, 0.25, so, out)
        scale = 65536 / (65536 - 16384)
        base = 0.0 if residual is None else 1.0
        # the factor 4/3 is rounded to float32 (U of it) before its product with 1 is added to the base (one rounding)
        half = 2.0 ** -8 if dtype is torch.bfloat16 else bo.U32
        bound = bo.U32 * scale + half * (scale + base)
        got = out.view(-1)
        for first in (0, (1 << 27) - 20, 1 << 27, (1 << 27) + 3, T * H // 8 - 40):
            want = torch.from_numpy(bo.kept_mask(320, 0.25, 99, 7, first)).cuda()
            ref = base + scale * want.double()
            off = (got[8 * first: 8 * first + 320].double() - ref).abs()
            assert bool((off <= torch.where(want, bound, 0.0)).all()), first
        del out, got
