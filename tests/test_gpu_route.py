"""GPU parity: the expert router against float64 (ids equal, weights to f32 rounding)."""
import numpy as np
import pytest
import torch

import fp8_linear_layers_b200 as ql
from tests import _w4

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _run(logits, k, sigmoid=False, bias=None, **kw):
    ids, w = ql.route(logits.cuda(), k, score=ql.ROUTE_SIGMOID if sigmoid else ql.ROUTE_SOFTMAX,
                      bias=None if bias is None else bias.cuda(), **kw)
    rid, rw = _w4.route64(logits, k, sigmoid, bias, **kw)
    ids, w = ids.cpu().numpy(), w.cpu().double().numpy()
    assert np.array_equal(ids, rid), [(t, ids[t], rid[t]) for t in np.nonzero((ids != rid).any(1))[0][:3]]
    # expf, the divisions and sums of up to 32 (or, not renormalized, 1024) terms:
    # 2^-19 relative; the difference of two logits rounds to 2^-24 of itself
    l = np.nan_to_num(logits.double().numpy(), nan=0.0, posinf=3.4e38, neginf=0.0)
    span = np.minimum(np.abs(l).max(1, keepdims=True), 110.0)
    assert (np.abs(w - rw) <= np.abs(rw) * (2.0 ** -19 + 2 * span * 2.0 ** -24) + 1e-37).all()
    return ids, w


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("T,E,k,groups,top_groups,group_top", [
    (1, 1, 1, 1, 1, 1), (1, 8, 2, 1, 1, 1), (3, 33, 5, 1, 1, 1), (5, 64, 8, 1, 1, 1), (130, 128, 8, 1, 1, 1),
    (67, 256, 8, 8, 4, 2), (9, 160, 6, 8, 3, 1), (11, 96, 6, 6, 2, 2), (4, 1024, 32, 32, 8, 2), (7, 512, 10, 4, 1, 1),
    (5, 40, 10, 5, 2, 2), (6, 32, 32, 1, 1, 1), (33, 16, 4, 8, 4, 2)])
def test_route(cuda, dtype, sigmoid, with_bias, T, E, k, groups, top_groups, group_top):
    g = _gen(T * 1000 + E)
    logits = (torch.randn(T, E, generator=g) * 1.5).to(dtype)
    bias = torch.randn(E, generator=g) * 0.05 if with_bias else None
    for renorm, scale in ((True, 1.0), (False, 2.5)):
        _run(logits, k, sigmoid, bias, groups=groups, top_groups=top_groups, group_top=group_top,
             renormalize=renorm, scale=scale)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("groups,top_groups,group_top", [(1, 1, 1), (8, 3, 2), (8, 3, 1)])
def test_near_ties_follow_the_exact_values(cuda, sigmoid, groups, top_groups, group_top):
    """Biases that bring every choice within a few f32 steps of the others: the
    order is that of the exact sums, not of their f32 roundings."""
    T, E = 64, 64
    g = _gen(2)
    base = torch.randn(1, E, generator=g)
    logits = base + torch.randn(T, E, generator=g) * 1e-6
    p = torch.sigmoid(base.double()) if sigmoid else torch.softmax(base.double(), -1)
    bias = (0.75 - p[0]).float()
    _run(logits, 8, sigmoid, bias, groups=groups, top_groups=top_groups, group_top=group_top)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("groups,top_groups,group_top", [(1, 1, 1), (4, 2, 2), (4, 2, 1)])
def test_ties_go_to_the_lower_index(cuda, dtype, with_bias, groups, top_groups, group_top):
    g = _gen(4)
    logits = torch.randint(-2, 3, (50, 64), generator=g).to(dtype) * 0.5
    logits[0] = 0.0
    logits[1, ::2] = -0.0
    bias = torch.randint(0, 2, (64,), generator=g).float() * 0.25 if with_bias else None
    _run(logits, 9, True, bias, groups=groups, top_groups=top_groups, group_top=group_top)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("groups,top_groups,group_top", [(1, 1, 1), (4, 2, 1), (4, 2, 2)])
def test_masked_and_extreme_logits(cuda, sigmoid, with_bias, groups, top_groups, group_top):
    inf, nan = float("inf"), float("nan")
    g = _gen(7)
    logits = torch.randn(9, 32, generator=g)
    logits[0] = -inf                      # nothing left
    logits[1] = nan
    logits[2, 3:] = -inf                  # fewer than k left
    logits[3, ::2] = nan
    logits[4, 5] = inf
    logits[5, [1, 9, 30]] = inf
    logits[6] = -torch.arange(32) * 40.0  # scores underflow, ratios do not
    logits[7] = -3.4e38
    logits[8] *= 1e30
    bias = None
    if with_bias:
        bias = torch.randn(32, generator=g) * 0.1
        bias[[4, 11]] = -inf
        bias[17] = nan
    for renorm in (True, False):
        _run(logits, 6, sigmoid, bias, groups=groups, top_groups=top_groups, group_top=group_top, renormalize=renorm)


def test_stream_graph_and_outputs(cuda):
    logits = torch.randn(37, 64, generator=_gen(1)).cuda()
    ids = torch.full((37, 4), -9, dtype=torch.int32, device="cuda")
    w = torch.full((37, 4), -9.0, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ql.route(logits, 4, ids=ids, weights=w)
    logits.copy_(torch.randn(37, 64, generator=_gen(2)))
    graph.replay()
    torch.cuda.synchronize()
    rid, _ = _w4.route64(logits.cpu(), 4)
    assert np.array_equal(ids.cpu().numpy(), rid)
    empty, _ = ql.route(logits[:0], 4)
    assert empty.shape == (0, 4)
