"""The 4-bit layer where act leaves the range of bf16, for a few assignments and for more: the same infinities."""
import pytest
import torch

import combine_top_route_expert_amd as moe
from test_gpu_mx_experts import BF16, Case, packed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.load_library()


@pytest.mark.parametrize("T", [1, 2, 40, 300])
def test_act_past_the_largest_number(T):
    """g and u of 6.4e21 make an act of 4e43, infinite in float32 too; W_down's signs, the same along a row, go on to out."""
    E, H, I = 4, 64, 64  # noqa: E741
    c = Case(T, H, E, 1, I, 1, seed=T)
    c.wgu, c.wgus, c.vgu = packed(torch.ones(E, 2 * I, H, device="cuda").to(BF16))
    sign = torch.where(torch.arange(H, device="cuda") % 3 == 0, -1.0, 1.0)
    c.wd, c.wds, c.vd = packed(sign[:, None].expand(E, H, I).to(BF16).contiguous())
    c.w.fill_(0.5)
    x = torch.full((T, H), 1e20, device="cuda").to(BF16)
    got = c.forward(x=x)
    assert torch.equal(got, (sign * float("inf")).to(BF16).expand(T, H))
    x[0] = 1.0                            # the other rows' infinities stay in their rows
    got = c.forward(x=x)
    assert bool(got[0].isfinite().all()) and bool(got[1:].isinf().all())
