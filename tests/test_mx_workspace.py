"""Workspace of the layer with 4-bit experts (no GPU: every call returns before any HIP call)."""
import combine_top_route_expert_amd as moe
from test_mx_experts_host import TOO_SMALL, forward, shape


def test_rows_of_a_pair():
    """act in bf16, y in fp16 with a byte for 64 columns, and metadata."""
    s = shape(T=1000, H=2048, E=64, k=4, I=1024, N=2)
    need = moe.moe_mx_workspace_size(s)
    rows = 2 * 500 * 4
    assert 0 < need - rows * (2 * 1024 + 2 * 2048 + 2048 // 64) < 1 << 18
    assert forward(s, n=need - 1) == TOO_SMALL


def test_chunks_share_it():
    one, two, four = (moe.moe_mx_workspace_size(shape(T=16384, H=2048, E=128, k=8, I=768, N=n)) for n in (1, 2, 4))
    assert abs(two / one - 1) < 0.01 and abs(four / one - 0.5) < 0.01


def test_few_assignments_take_four_bytes_a_value_of_act():
    """8 tokens in 8 chunks, so that a pair holds fewer rows than there are assignments."""
    need = moe.moe_mx_workspace_size(shape(T=8, H=64, E=32, k=4, I=65536, N=8))
    assert 32 * 65536 * 4 < need < 32 * 65536 * 4 + (1 << 16)
