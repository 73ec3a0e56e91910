"""The router's group limit where experts are closed: a group with an open expert ranks above one without."""
import math

import numpy as np
import pytest
import torch

import block_oracle as bo
import combine_top_route_expert_amd as moe
from gpu_layer import say
from test_gpu_router import INF, backward, make_logits, rel_bound, route

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.load_library()


def ids_of_row(row, bias, score, G, limit, k):
    """Ids of one row by sorting.  Groups: those with more open experts among their two largest keys first, then by the sum
    of these, then by number."""
    E, n = len(row), len(row) // G
    if bias is None and not 0 < limit < G:
        key = row.copy()
    else:
        s = bo.scores(row, score)
        key = np.array([s[e] + (0.0 if bias is None else bias[e])
                        if row[e] > -INF and (bias is None or np.isfinite(bias[e])) else -INF for e in range(E)])
    if 0 < limit < G:
        best = [[v for v in sorted(key[g * n:(g + 1) * n])[-2:] if v > -INF] for g in range(G)]
        kept = sorted(range(G), key=lambda g: (-len(best[g]), -sum(best[g]), g))[:limit]
        key = np.array([key[e] if e // n in kept else -INF for e in range(E)])
    ids = [e for e in sorted(range(E), key=lambda e: (-key[e], e)) if key[e] > -INF][:k]
    return ids + [-1] * (k - len(ids))


def check(x, k, G, bias, score, limit, renorm, factor):
    idx, w = route(x, k, G, bias, score, limit, renorm, factor)
    rows, idx, w = x.double().cpu().numpy(), idx.cpu().numpy(), w.double().cpu().numpy()
    b = None if bias is None else bias.double().cpu().numpy()
    for t, row in enumerate(rows):
        ids = ids_of_row(row, b, score, G, limit, k)
        assert idx[t].tolist() == ids, (t, idx[t].tolist(), ids)
        ref = np.array(bo.weights_row(row, ids, score, renorm, factor))
        assert (np.abs(w[t] - ref) <= rel_bound(row, ids, len(row)) * np.abs(ref) + 1e-37).all(), (t, w[t], ref)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_two_open_experts_in_two_groups(score, dtype):
    x = torch.full((3, 8), -INF, device="cuda", dtype=dtype)
    x[0, 5], x[0, 7] = 1.0, 2.0          # the last expert of each of groups 2 and 3
    x[1, 2], x[1, 5], x[1, 7] = 1.0, 3.0, 2.0
    x[2, 6], x[2, 7], x[2, 0] = -9.0, -9.0, 5.0   # two open experts rank above one
    idx, _ = route(x, 2, 4, None, score, 2)
    assert idx.tolist() == [[7, 5], [5, 7], [0, 6]]
    idx, _ = route(x, 2, 4, None, score, 1)
    assert idx.tolist() == [[7, -1], [5, -1], [6, 7]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,limit,k", [(8, 8, 3, 2), (8, 4, 2, 2), (8, 1, 0, 3), (60, 4, 2, 4), (60, 20, 7, 6),
                                         (60, 30, 11, 7), (128, 64, 5, 8), (128, 64, 60, 8), (256, 8, 4, 8), (256, 8, 8, 8),
                                         (320, 5, 1, 64), (1024, 32, 4, 8)])
def test_choice_by_score(E, G, limit, k, score):
    say(f"router E={E} G={G} limit={limit} k={k} {score}")
    rng = np.random.default_rng(E + G)
    bias = rng.normal(size=E) * 0.3
    bias[rng.random(E) < 0.1] = -INF
    bias[rng.random(E) < 0.03] = math.nan
    bias = torch.from_numpy(bias).float().cuda()
    for dtype in ("f32", "bf16"):
        x = make_logits(23, E, dtype, E)
        x[torch.from_numpy(rng.random((23, E)) < 0.5).cuda() & (torch.arange(23, device="cuda") >= 12)[:, None]] = -INF
        check(x, k, G, bias, score, limit, True, 2.5)
        check(x, k, G, None, score, limit, False, 1.0)


def test_gradient_reaches_the_experts_that_were_left():
    x = torch.full((1, 8), -INF, device="cuda")
    x[0, 5], x[0, 7] = 1.0, 2.0
    idx, w = route(x, 2, 4, None, "softmax", 2)
    grad = backward(x, idx, torch.tensor([[1.0, 0.0]], device="cuda"), "softmax", True, 1.0)
    p = 1 / (1 + math.exp(-1.0))         # of expert 7
    want = torch.zeros(1, 8, dtype=torch.float64)
    want[0, 7], want[0, 5] = p * (1 - p), -p * (1 - p)
    assert float((grad.double().cpu() - want).abs().max()) < 16 * bo.U32


@pytest.mark.parametrize("E,G", [(4, 2), (256, 8), (6, 1), (256, 128)])
def test_all_groups_open_is_no_limit(E, G):
    """With group_limit = num_groups, or none, the key is the logit: it tells sigmoids apart that are the same number in 64
    bits.  With a bias they are equal, and the lower id comes first."""
    x = torch.zeros(1, E, device="cuda")
    x[0, 0], x[0, 1], x[0, 3] = 40.0, 41.0, 42.0
    for limit in (0, G):
        assert route(x, 3, G, None, "sigmoid", limit)[0].tolist() == [[3, 1, 0]]
        assert route(x, 3, G, torch.zeros(E, device="cuda"), "sigmoid", limit)[0].tolist() == [[0, 1, 3]]
