"""GPU: the router's order with biases at the ends of f32 (masks of the lowest value, infinities,
sums out of range), and with a few choices closer than f32 tells, against float64."""
import numpy as np
import pytest
import torch

import fp8_linear_layers_b200 as ql

pytestmark = pytest.mark.gpu

MIN, INF = torch.finfo(torch.float32).min, float("inf")


def _ids(logits, bias, k, sigmoid, groups, top_groups, group_top):
    """The documented order, token by token, in float64."""
    out = np.full((logits.shape[0], k), -1, np.int32)
    b = bias.double().numpy()
    size = logits.shape[1] // groups
    for t, l in enumerate(logits.double().numpy()):
        p = 1 / (1 + np.exp(-l)) if sigmoid else np.exp(l - l.max()) / np.exp(l - l.max()).sum()
        c = np.where(b > -INF, p + b, -INF)  # (NaN biases are unavailable too)
        if groups > 1:
            value = []
            for g in range(groups):
                v = sorted(c[g * size:(g + 1) * size], reverse=True)[:group_top]
                value.append(-INF if v[-1] == -INF else sum(v))
            keep = sorted(range(groups), key=lambda g: (-value[g], g))[:top_groups]
            c = np.where(np.isin(np.arange(len(c)) // size, keep), c, -INF)
        order = sorted((e for e in range(len(c)) if c[e] > -INF), key=lambda e: (-c[e], e))[:k]
        out[t, :len(order)] = order
    return out


def _check(logits, bias, k, sigmoid, groups=1, top_groups=1, group_top=1):
    ids, w = ql.route(logits.cuda(), k, score=ql.ROUTE_SIGMOID if sigmoid else ql.ROUTE_SOFTMAX, bias=bias.cuda(),
                      groups=groups, top_groups=top_groups, group_top=group_top)
    want = _ids(logits, bias, k, sigmoid, groups, top_groups, group_top)
    got = ids.cpu().numpy()
    assert np.array_equal(got, want), [(t, got[t], want[t]) for t in np.nonzero((got != want).any(1))[0][:3]]
    assert w.isfinite().all()


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E,groups,top_groups,group_top", [(64, 8, 4, 2), (64, 8, 4, 1), (96, 6, 3, 2), (64, 1, 1, 1),
                                                           (40, 5, 3, 2), (256, 8, 5, 2)])
def test_biases_at_the_ends(cuda, sigmoid, E, groups, top_groups, group_top):
    g = torch.Generator().manual_seed(E + groups)
    logits = torch.randn(20, E, generator=g)
    size = E // groups
    plain = torch.randn(E, generator=g) * 0.1
    cases = []
    for masked in {max(m, 0) for m in (groups - 1, groups - 2, groups - top_groups)}:
        b = plain.clone()
        b[torch.randperm(groups, generator=g)[:masked].repeat_interleave(size) * size
          + torch.arange(size).repeat(masked)] = MIN  # whole groups masked by the lowest value
        cases.append(b)
        c = b.clone()
        c[:size] = -INF                               # and the first group unavailable
        cases.append(c)
        c = c.clone()
        c[size // 2] = INF if masked % 2 else 1.0     # or short of a second expert
        cases.append(c)
    big = plain.clone()
    big[torch.randperm(E, generator=g)[:E // 2]] = torch.where(torch.rand(E // 2, generator=g) < 0.5, 3.0e38, -3.0e38)
    cases.append(big)
    cases.append(big * torch.rand(E, generator=g))
    inf = plain.clone()
    inf[torch.randperm(E, generator=g)[:6]] = INF
    inf[torch.randperm(E, generator=g)[:6]] = float("nan")
    cases.append(inf)
    for b in cases:
        _check(logits, b, 6, sigmoid, groups, top_groups, group_top)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E,close,k", [(64, 3, 8), (64, 12, 8), (33, 20, 8), (160, 24, 6), (512, 30, 10), (256, 31, 31)])
@pytest.mark.parametrize("step", [1e-9, 1e-7, 3e-7])
def test_a_few_close_choices(cuda, sigmoid, E, close, k, step):
    """Up to 31 choices a step of 1e-9 .. 3e-7 apart, the rest far below: they are ranked by
    their f64 values, among themselves and against the border of the k best."""
    g = torch.Generator().manual_seed(close)
    logits = torch.randn(50, E, generator=g) * 0.5
    l = logits.double()
    p = torch.sigmoid(l) if sigmoid else torch.softmax(l, -1)
    at = torch.randperm(E, generator=g)[:close]
    bias = torch.full((E,), -0.5)
    # one bias for all tokens: make the close experts' scores alike in every token
    level = 0.75
    bias[at] = (level - p[0, at]).float()
    logits[:] = logits[0]
    logits[:, at] += (torch.randn(50, close, generator=g).double() * step / p[0, at]).float()
    _check(logits, bias, k, sigmoid)
