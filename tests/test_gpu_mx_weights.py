"""4-bit matrices on the GPU: quantiser, packing and their inverse have to be equal to the references, bit by bit."""
import numpy as np
import pytest
import torch

import block_oracle as bo
import combine_top_route_expert_amd as moe
from gpu_layer import say

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.load_library()


def buffers(rows, cols, fill=0xA5):
    u8 = dict(dtype=torch.uint8, device="cuda")
    return (torch.full((rows * cols // 2,), fill, **u8),
            torch.full((moe.moe_mx_scale_size(rows, cols),), fill, **u8))


def quantize(x, dtype):
    q, s = buffers(*x.shape)
    moe.moe_quantize_mx(*x.shape, dtype, x, q, s)
    return q, s


def used(scale, rows, cols):
    """The scale bytes that stand for a group (a row of blocks may end in unused ones)."""
    at = bo.pack(np.zeros((rows, cols), np.uint8), np.ones((rows, cols // 32), np.uint8))[1]
    return scale.cpu().numpy()[at == 1]


def awkward(rows, cols, dtype, seed):
    """Groups of every size in the type's range, ties between 4-bit numbers, zeros, subnormals and the largest finite."""
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(rows, cols // 32, 32)) * 2.0 ** rng.integers(-20, 20, size=(rows, cols // 32, 1))
    x[0] *= 2.0 ** -110
    x[1] *= 2.0 ** 100
    x[2] = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -5.0], size=x[2].shape)
    x[3] = 0.0
    x[4] *= 2.0 ** -125
    x[5] = 2.0 ** -149 * rng.integers(-9, 10, size=x[5].shape) if dtype == "f32" else \
        2.0 ** -133 * rng.integers(-9, 10, size=x[5].shape)
    x[6, :, 0] = float(torch.finfo(TYPES[dtype]).max)
    x[7, :, 1] = 6.0 * 2.0 ** 3
    x[8, :, 1] = 6.03125 * 2.0 ** 3
    x[9] = -0.0
    x[10] = 2.0 ** 126 * rng.choice([3.0, 3.25, 3.5, 3.75, -3.5, 0.25], size=x[10].shape)
    return torch.from_numpy(x.reshape(rows, cols)).to(TYPES[dtype]).cuda()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(32, 64), (32, 192), (64, 256), (96, 320), (32, 1088)])
def test_quantize(rows, cols, dtype):
    say(f"4-bit matrix {rows} x {cols} {dtype}")
    x = awkward(rows, cols, dtype, rows + cols)
    codes, bytes_ = bo.quantize_row_major(x.double().cpu().numpy())
    want_q, want_s = bo.pack(codes, bytes_)
    q, s = quantize(x, dtype)
    assert q.cpu().numpy().tolist() == want_q.tolist()
    assert used(s, rows, cols).tolist() == used(torch.from_numpy(want_s), rows, cols).tolist()
    back = torch.full_like(x, float("nan"))
    moe.moe_dequantize_mx(rows, cols, dtype, q, s, back)
    assert np.array_equal(back.double().cpu().numpy(), bo.values(codes, bytes_))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_groups_without_a_number(dtype):
    x = torch.ones(32, 128, dtype=TYPES[dtype], device="cuda")
    x[3, 40], x[5, 0], x[31, 127] = float("inf"), float("nan"), -float("inf")
    q, s = quantize(x, dtype)
    back = torch.zeros_like(x)
    moe.moe_dequantize_mx(32, 128, dtype, q, s, back)
    bad = torch.zeros(32, 4, dtype=torch.bool, device="cuda")
    bad[3, 1] = bad[5, 0] = bad[31, 3] = True
    bad = bad.repeat_interleave(32, 1)
    assert bool(back[bad].isnan().all()) and bool((back[~bad] == 1).all())


@pytest.mark.parametrize("rows,cols", [(32, 64), (64, 448), (160, 512)])
def test_pack_every_code_and_scale(rows, cols):
    rng = np.random.default_rng(rows)
    codes = rng.integers(0, 16, size=(rows, cols)).astype(np.uint8)
    bytes_ = rng.integers(0, 256, size=(rows, cols // 32)).astype(np.uint8)
    want_q, want_s = bo.pack(codes, bytes_)
    row_q = torch.from_numpy(codes[:, 0::2] | codes[:, 1::2] << 4).cuda()
    q, s = buffers(rows, cols)
    moe.moe_pack_mx(rows, cols, row_q, torch.from_numpy(bytes_).cuda(), q, s)
    assert q.cpu().numpy().tolist() == want_q.tolist()
    assert used(s, rows, cols).tolist() == used(torch.from_numpy(want_s), rows, cols).tolist()
    ref = bo.values(codes, bytes_)
    for dtype, dt in TYPES.items():
        back = torch.zeros(rows, cols, dtype=dt, device="cuda")
        moe.moe_dequantize_mx(rows, cols, dtype, q, s, back)
        got = back.double().cpu().numpy()
        over = np.abs(ref) >= 2.0 ** 128
        assert np.array_equal(got[~over], ref[~over], equal_nan=True)
        assert np.array_equal(got[over], np.sign(ref[over]) * np.inf)


def test_several_matrices_in_one_call_or_many():
    """Experts' matrices follow one another: rows of all of them in one call are the experts' own."""
    x = torch.randn(4, 64, 320, device="cuda").bfloat16()
    q, s = quantize(x.view(256, 320), "bf16")
    for e in range(4):
        qe, se = quantize(x[e].contiguous(), "bf16")
        assert torch.equal(q.view(4, -1)[e], qe) and torch.equal(s.view(4, -1)[e], se)


def test_nothing_past_the_matrix_is_written():
    rows, cols = 64, 320
    x = torch.randn(rows, cols, device="cuda")
    q, s = torch.full((rows * cols // 2 + 64,), 7, dtype=torch.uint8, device="cuda"), \
        torch.full((moe.moe_mx_scale_size(rows, cols) + 64,), 7, dtype=torch.uint8, device="cuda")
    moe.moe_quantize_mx(rows, cols, "f32", x, q, s)
    assert bool((q[-64:] == 7).all()) and bool((s[-64:] == 7).all())
    back = torch.full((rows * cols + 64,), 7.0, device="cuda")
    moe.moe_dequantize_mx(rows, cols, "f32", q, s, back)
    assert bool((back[-64:] == 7).all())
