"""GPU parity: the routed experts' 4-bit products against float64, and a router,
its experts' up rows, the activation and the down rows run together."""
import pytest
import torch

import fp8_linear_layers_b200 as ql
from tests import _w4

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _case(T, k, E, N, K, group, zeros, combine, seed=0):
    g = _gen(seed)
    x = torch.randn(*((T, k, K) if combine else (T, K)), generator=g).bfloat16()
    wq, sw, wz = _w4.make_weights(g, (E, N), K, group, zeros)
    ids = torch.stack([torch.randperm(max(E, k), generator=g)[:k] % E for _ in range(T)]).int() if T else \
        torch.zeros(0, k, dtype=torch.int32)
    wts = torch.rand(T, k, generator=g) if combine else None
    return x, ids, wq, sw, wz, wts


# combine: each pair's product may be rounded to bf16 once before the sum (the
# long-prompt path), and the sum once
def _check(x, ids, wq, sw, wz, wts, group):
    combine = wts is not None
    T, k = ids.shape
    N = wq.shape[1]
    w = ql.W4Weight(wq.cuda(), sw.cuda(), None if wz is None else wz.cuda(), group)
    n = T * N if combine else T * k * N
    buf = torch.full((n + 512,), float("nan"), dtype=torch.bfloat16, device="cuda")
    y = buf[256:256 + n].view((T, N) if combine else (T, k, N))
    ql.experts_w4(x.cuda(), ids.cuda(), w, weights=wts.cuda() if combine else None, y=y)
    assert ql.device_status()[0] == 0
    assert buf[:256].isnan().all() and buf[256 + n:].isnan().all()
    wd, size = _w4.dequantize(wq, sw, wz, group), _w4.magnitudes(wq, sw, wz, group)
    ref, mag = _w4.experts64(x, ids, wd, size, wts)
    lim = _w4.product_limit(ref, mag, x.shape[-1], wz is not None)
    if combine:
        # sum_j |w_j| |y_j| <= the magnitude, but a bf16 rounding is relative to each
        # pair's own value: bound it by the pairs' values
        pairs, _ = _w4.experts64(x.reshape(T * k, -1), ids.reshape(T * k, 1), wd, size)
        lim = lim + 2.0 ** -8 * (pairs.view(T, k, N).abs() * wts.double().abs()[..., None]).sum(1)
    err = (y.double().cpu() - ref).abs()
    assert (err <= lim).all(), (err - lim).max()
    return y


@pytest.mark.parametrize("combine", [False, True])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, False), (128, True)])
@pytest.mark.parametrize("T,k,E,N,K", [(1, 1, 1, 1, 32), (1, 8, 16, 33, 256), (3, 2, 5, 17, 96), (8, 4, 8, 64, 160),
                                       (9, 3, 7, 130, 288), (20, 2, 3, 48, 224), (77, 4, 6, 129, 160)])
def test_experts(cuda, combine, group, zeros, T, k, E, N, K):
    _check(*_case(T, k, E, N, K, group, zeros, combine), group)


@pytest.mark.parametrize("combine", [False, True])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True)])
@pytest.mark.parametrize("T", [2, 7, 9, 16, 17])
def test_large_experts_for_few_tokens(cuda, combine, group, zeros, T):
    x, ids, wq, sw, wz, wts = _case(T, 4, 6, 2056, 1056, group, zeros, combine)
    ids[0, 1], ids[-1, 2] = ids[0, 0], -1  # an expert twice, and none
    _check(x, ids, wq, sw, wz, wts, group)


@pytest.mark.parametrize("combine", [False, True])
@pytest.mark.parametrize("T,k,E,N,K,group,zeros", [
    (16, 32, 64, 40, 64, 32, False), (70, 32, 1024, 8, 32, 32, True), (700, 4, 24, 65, 96, 64, True),
    (1030, 2, 1, 72, 288, 128, False), (650, 4, 40, 264, 2080, 32, False)])
def test_many_pairs(cuda, combine, T, k, E, N, K, group, zeros):
    """The most slots and experts; more pairs than are placed by counting; ids out of
    range among them."""
    x, ids, wq, sw, wz, wts = _case(T, k, E, N, K, group, zeros, combine)
    ids[1, 0], ids[T // 2, 1], ids[-1, :] = E, -1, -5
    _check(x, ids, wq, sw, wz, wts, group)


@pytest.mark.parametrize("combine", [False, True])
@pytest.mark.parametrize("T", [1, 5, 8, 13, 40])
@pytest.mark.parametrize("kind", ["one expert", "same expert twice", "out of range", "nothing"])
def test_uneven_ids(cuda, combine, T, kind):
    x, ids, wq, sw, wz, wts = _case(T, 4, 6, 40, 128, 64, False, combine)
    if kind == "one expert":
        ids[:, :] = 3
    elif kind == "same expert twice":
        ids[:, 1] = ids[:, 0]
    elif kind == "out of range":
        ids[0, 0], ids[-1, 2], ids[T // 2, 1] = -1, 6, 2 ** 31 - 1
    else:
        ids[:, :] = -1
    y = _check(x, ids, wq, sw, wz, wts, 64)
    if kind == "nothing":
        assert not y.any()


@pytest.mark.parametrize("combine", [False, True])
@pytest.mark.parametrize("N", [40, 41])
@pytest.mark.parametrize("counts", [(19,), (39, 1), (18, 33, 3), (1, 2, 31, 32, 64, 5), (17,) * 6, (59, 21)])
def test_pairs_of_an_expert(cuda, combine, N, counts):
    """Experts with one, an odd number of, and more pairs than a token tile holds."""
    x, ids, wq, sw, wz, wts = _case(sum(counts), 1, 24, N, 128, 64, False, combine)
    ids[:, 0] = torch.repeat_interleave(torch.arange(len(counts)) * 3, torch.tensor(counts)).int()
    ids = ids[torch.randperm(len(ids), generator=_gen(1))].contiguous()
    _check(x, ids, wq, sw, wz, wts, 64)


@pytest.mark.parametrize("T", [2, 40])
def test_non_finite_stays_with_its_token(cuda, T):
    """An infinite token, or an expert with an infinite scale, touches no other row."""
    x, ids, wq, sw, wz, wts = _case(T, 2, 4, 40, 128, 64, False, True)
    ids[:] = torch.tensor([0, 1], dtype=torch.int32)
    ids[1] = torch.tensor([2, 3], dtype=torch.int32)
    w = ql.W4Weight(wq.cuda(), sw.cuda(), None, 64)
    clean = ql.experts_w4(x.cuda(), ids.cuda(), w, weights=wts.cuda())
    x[1, 0, 3] = float("nan")
    sw[3, :, 1] = float("inf")
    w = ql.W4Weight(wq.cuda(), sw.cuda(), None, 64)
    y = ql.experts_w4(x.cuda(), ids.cuda(), w, weights=wts.cuda())
    keep = [t for t in range(T) if t != 1]
    assert torch.equal(y[keep], clean[keep]) and not y[1].isfinite().any()


def test_no_tokens(cuda):
    x, ids, wq, sw, wz, wts = _case(1, 2, 4, 40, 128, 64, False, True)
    w = ql.W4Weight(wq.cuda(), sw.cuda(), None, 64)
    assert ql.experts_w4(x[:0].cuda(), ids[:0].cuda(), w, weights=wts[:0].cuda()).shape == (0, 40)


def _layer(logits, x, up, down, k, E, ws_up, ws_down):
    ids, wts = ql.route(logits, k, score=ql.ROUTE_SIGMOID, groups=4, top_groups=2, group_top=2, scale=2.0)
    h = ql.experts_w4(x, ids, up, workspace=ws_up)
    a, b = h.float().chunk(2, -1)
    act = (a * torch.sigmoid(a) * b).bfloat16()
    return ids, wts, h, act, ql.experts_w4(act, ids, down, weights=wts, workspace=ws_down)


@pytest.mark.parametrize("T", [1, 6, 50])
def test_route_up_activation_down(cuda, T):
    """The operators as a decoder layer runs them, eager and captured in a graph:
    every stage against float64 on the stage before it."""
    k, E, H, I = 4, 16, 256, 96
    g = _gen(T)
    x = torch.randn(T, H, generator=g).bfloat16()
    logits = torch.randn(T, E, generator=g)
    up_h, down_h = _w4.make_weights(g, (E, 2 * I), H, 64, False), _w4.make_weights(g, (E, H), I, 32, True)
    up = ql.W4Weight(up_h[0].cuda(), up_h[1].cuda(), None, 64)
    down = ql.W4Weight(*(t.cuda() for t in down_h), 32)
    ws_up = ql.new_workspace(ql.experts_w4_workspace_bytes(T, k, up))
    ws_down = ql.new_workspace(ql.experts_w4_workspace_bytes(T, k, down, combine=True))
    xd, ld = x.cuda(), logits.cuda()

    def verify(out, x, logits):
        ids, wts, h, act, y = (o.cpu() for o in out)
        rid, _ = _w4.route64(logits, k, True, None, groups=4, top_groups=2, group_top=2, scale=2.0)
        assert (ids.numpy() == rid).all()
        ref, mag = _w4.experts64(x, ids, _w4.dequantize(*up_h, 64), _w4.magnitudes(*up_h, 64))
        assert ((h.double() - ref).abs() <= _w4.product_limit(ref, mag, H)).all()
        wd, size = _w4.dequantize(*down_h, 32), _w4.magnitudes(*down_h, 32)
        ref, mag = _w4.experts64(act, ids, wd, size, wts)
        pairs, _ = _w4.experts64(act.reshape(T * k, I), ids.reshape(T * k, 1), wd, size)
        lim = _w4.product_limit(ref, mag, I, True) + 2.0 ** -8 * (pairs.view(T, k, H).abs() * wts.double()[..., None]).sum(1)
        assert ((y.double() - ref).abs() <= lim).all()

    verify(_layer(ld, xd, up, down, k, E, ws_up, ws_down), x, logits)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _layer(ld, xd, up, down, k, E, ws_up, ws_down)
    x2, l2 = torch.randn(T, H, generator=g).bfloat16(), torch.randn(T, E, generator=g)
    xd.copy_(x2)
    ld.copy_(l2)
    graph.replay()
    torch.cuda.synchronize()
    verify(out, x2, l2)
    assert ql.device_status()[0] == 0


def test_two_streams_at_once(cuda):
    """Calls in flight on two streams, each with its own workspace, give what they give
    alone: every kind of tile beside every other."""
    x, ids, wq, sw, wz, wts = _case(300, 4, 6, 520, 1056, 64, True, True)
    experts = ql.W4Weight(wq.cuda(), sw.cuda(), wz.cuda(), 64)
    g = _gen(11)
    dense = ql.W4Weight(*(t.cuda() for t in _w4.make_weights(g, (4096,), 2048, 128, True)), 128)
    xs = [torch.randn(M, 2048, generator=g).bfloat16().cuda() for M in (1, 16, 40, 128, 700)]
    xd, idd, wd = x.cuda(), ids.cuda(), wts.cuda()
    calls = [lambda ws, v=v: ql.forward_w4(v, dense, workspace=ws) for v in xs]
    calls += [lambda ws, T=T: ql.experts_w4(xd[:T], idd[:T], experts, weights=wd[:T], workspace=ws) for T in (5, 60, 300)]
    size = max([ql.forward_w4_workspace_bytes(len(v), dense) for v in xs] +
               [ql.experts_w4_workspace_bytes(300, 4, experts, combine=True)])
    alone = [c(None) for c in calls]
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [ql.new_workspace(size) for _ in streams]
    torch.cuda.synchronize()
    got = [[], []]
    for i in range(2 * len(calls)):
        for n, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[n].append(calls[(i + 3 * n) % len(calls)](spaces[n]))
    torch.cuda.synchronize()
    assert ql.device_status()[0] == 0
    for n in range(2):
        for i, y in enumerate(got[n]):
            assert torch.equal(y, alone[(i + 3 * n) % len(calls)]), (n, i)
