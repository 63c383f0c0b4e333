"""GPU parity: 4-bit weight quantization and the 4-bit product, against float64.

Tolerances are derived in tests/_w4.py (one bf16 rounding, f32 sums of exact
products)."""
import pytest
import torch

import fp8_linear_layers_b200 as ql
from tests import _w4

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _case(M, N, K, group, zeros, seed=0):
    g = _gen(seed)
    x = torch.randn(M, K, generator=g).bfloat16()
    return x, *_w4.make_weights(g, (N,), K, group, zeros)


def _handle(wq, sw, wz, group):
    return ql.W4Weight(wq.cuda(), sw.cuda(), None if wz is None else wz.cuda(), group)


def _guarded(M, N):
    """y inside a larger buffer of NaN, to see a write outside it."""
    buf = torch.full((M * N + 512,), float("nan"), dtype=torch.bfloat16, device="cuda")
    return buf, buf[256:256 + M * N].view(M, N)


def _check(x, wq, sw, wz, group, what=""):
    M, N = x.shape[0], wq.shape[0]
    buf, y = _guarded(M, N)
    out = ql.forward_w4(x.cuda(), _handle(wq, sw, wz, group), y=y)
    assert out is y and ql.device_status()[0] == 0
    assert buf[:256].isnan().all() and buf[256 + M * N:].isnan().all()
    _w4.assert_product(y, x, wq, sw, wz, group, what)
    return y


@pytest.mark.parametrize("group", ql.W4_GROUPS)
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,N,K", [(1, 1, 32), (1, 17, 96), (1, 130, 4128), (2, 16, 128), (7, 33, 288), (8, 64, 512),
                                   (9, 15, 160), (16, 257, 1056), (17, 129, 224), (33, 300, 2080), (64, 128, 256),
                                   (65, 1, 64), (129, 255, 992), (300, 514, 1312)])
def test_product(cuda, group, zeros, M, N, K):
    _check(*_case(M, N, K, group, zeros), group)


@pytest.mark.parametrize("M,N,K,group,zeros", [
    (1, 1024, 4096, 128, False), (3, 4096, 14336, 128, True), (12, 14336, 4096, 64, False), (24, 4096, 4096, 32, True),
    (512, 1024, 4096, 128, False), (1, 4096, 4096, 32, True), (8, 6144, 4096, 64, True), (16, 4096, 4160, 128, True),
    (2, 5003, 4128, 128, False), (9, 14336, 992, 32, False), (300, 14336, 992, 64, True), (1030, 8197, 512, 128, False),
    (400, 20001, 160, 32, True), (130, 4096, 4096, 64, True), (300, 1030, 4128, 32, False),
    (700, 20000, 32, 32, False), (20, 300, 32, 32, True), (900, 20008, 64, 64, True)])
def test_product_layer_sizes(cuda, M, N, K, group, zeros):
    """Decoder layer sizes, and the same call twice in one workspace gives the same bits."""
    x, wq, sw, wz = _case(M, N, K, group, zeros)
    y = _check(x, wq, sw, wz, group)
    w = _handle(wq, sw, wz, group)
    ws = ql.new_workspace(ql.forward_w4_workspace_bytes(M, w))
    ws.fill_(0xA5)  # scratch: its contents before a call do not matter
    assert torch.equal(ql.forward_w4(x.cuda(), w, workspace=ws), y)
    assert torch.equal(ql.forward_w4(x.cuda(), w, workspace=ws), y)


def test_no_tokens(cuda):
    x, wq, sw, wz = _case(1, 64, 64, 32, False)
    y = ql.forward_w4(x[:0].cuda(), _handle(wq, sw, wz, 32))
    assert y.shape == (0, 64)


@pytest.mark.parametrize("M,N,K", [(1, 70, 512), (12, 70, 512), (40, 70, 512), (3, 4096, 4096), (16, 4096, 4096),
                                   (300, 70, 512), (300, 10000, 512)])
def test_wide_range(cuda, M, N, K):
    """Scales 2^-100 .. 2^20 in one row, tokens 2^-60 .. 2^60 apart: nothing is lost
    to the operands' range."""
    group = 64
    g = _gen(3)
    x, wq, sw, _ = _case(M, N, K, group, False, seed=3)
    x = (x.float() * 2.0 ** torch.randint(-60, 60, (M, 1), generator=g)).bfloat16()
    sw = (2.0 ** torch.randint(-12, 20, sw.shape, generator=g)).bfloat16()
    sw[: N // 2] = (sw[: N // 2].float() * 2.0 ** -88).bfloat16()
    _check(x, wq, sw, None, group)


@pytest.mark.parametrize("M", [1, 40])
def test_zero_scales_and_tokens(cuda, M):
    x, wq, sw, wz = _case(M, 96, 256, 64, True)
    sw[:, 1] = 0
    sw[5] = 0
    x[M // 2] = 0
    y = _check(x, wq, sw, wz, 64)
    assert not y[M // 2].any() and not y[:, 5].any()


@pytest.mark.parametrize("M,N,K", [(1, 80, 256), (9, 80, 256), (40, 80, 256), (4, 4096, 4096)])
def test_infinite_and_nan_tokens_stay_in_their_row(cuda, M, N, K):
    x, wq, sw, wz = _case(M + 2, N, K, 128, False)
    clean = ql.forward_w4(x.cuda(), _handle(wq, sw, wz, 128))
    x[0, 7] = float("inf")
    x[1, 9] = float("nan")
    y = ql.forward_w4(x.cuda(), _handle(wq, sw, wz, 128))
    assert torch.equal(y[2:], clean[2:])
    assert y[1].isnan().all() and not y[0].isfinite().any()


def test_row_results_do_not_depend_on_the_batch(cuda):
    """A token's row has the same bits wherever it stands in a batch of one path."""
    x, wq, sw, wz = _case(8, 200, 1024, 128, False)
    w = _handle(wq, sw, wz, 128)
    full = ql.forward_w4(x.cuda(), w)
    perm = torch.tensor([3, 1, 7, 0, 2, 6, 5, 4])
    assert torch.equal(ql.forward_w4(x[perm].cuda(), w), full[perm.cuda()])
    assert torch.equal(ql.forward_w4(x[:1].cuda(), w), full[:1])


@pytest.mark.parametrize("M,N,K", [(1, 144, 384), (16, 144, 384), (50, 144, 384), (5, 4096, 4096), (300, 520, 384),
                                   (300, 10000, 384)])
def test_side_stream_and_graph(cuda, M, N, K):
    """On another stream than the current one, and captured: the replay reads the
    inputs, the weights and the zero points as they are then."""
    x, wq, sw, wz = _case(M, N, K, 64, True)
    xd, w = x.cuda(), _handle(wq, sw, wz, 64)
    ref = ql.forward_w4(xd, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = ql.forward_w4(xd, w, stream=side)
    side.synchronize()
    assert torch.equal(y, ref)
    ws = ql.new_workspace(ql.forward_w4_workspace_bytes(M, w))
    out = torch.empty_like(ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ql.forward_w4(xd, w, workspace=ws, y=out)
    x2, wq2, sw2, wz2 = _case(M, N, K, 64, True, seed=9)
    for d, h in ((xd, x2), (w.wq, wq2), (w.sw, sw2), (w.wz, wz2)):
        d.copy_(h)
    graph.replay()
    torch.cuda.synchronize()
    _w4.assert_product(out, x2, wq2, sw2, wz2, 64)


@pytest.mark.parametrize("M,N,K", [(1, 512, 2048), (40, 512, 2048), (2, 4096, 4096), (200, 512, 2048)])
def test_weights_written_just_before_on_the_stream(cuda, M, N, K):
    """The weights may come from work still in flight on the same stream."""
    x, wq, sw, wz = _case(M, N, K, 128, False)
    w0 = torch.randn(N, K, generator=_gen(5)).bfloat16().cuda()
    xd = x.cuda()
    ref = ql.forward_w4(xd, ql.quantize_weight_w4(w0))
    torch.cuda.synchronize()
    for _ in range(5):
        w = ql.quantize_weight_w4(w0)
        y = ql.forward_w4(xd, w)
        w.sw.zero_()
        assert torch.equal(y, ref)


# ------------------------------------------------------------------ quantization


@pytest.mark.parametrize("group", ql.W4_GROUPS)
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("lead,K", [((1,), 32), ((5,), 96), ((33,), 4128), ((3, 7), 160)])
def test_quantize(cuda, group, zeros, lead, K):
    """Codes, scales and zero points equal the definition bit for bit (f32 IEEE steps)."""
    g = _gen(1)
    w = (torch.randn(*lead, K, generator=g) * 0.02).bfloat16()
    w[..., :2] = 0
    w[0, ..., : min(K, 40)] = 0
    w[-1, ..., 0] = 3.0
    got = ql.quantize_weight_w4(w.cuda(), group, zeros)
    G = -(-K // group)
    wp = torch.nn.functional.pad(w.float(), (0, G * group - K)).view(*lead, G, group)
    lo, hi = wp.amin(-1).clamp(max=0), wp.amax(-1).clamp(min=0)
    s = ((hi - lo) / 15.0 if zeros else torch.maximum(hi, -lo) / 7.0).bfloat16()
    sf = s.float()
    t = torch.where(sf[..., None] > 0, torch.round(wp / sf[..., None]), torch.zeros(()))
    z = torch.full_like(sf, 8.0)
    if zeros:
        z = torch.where(sf > 0, torch.round(-lo / sf).clamp(0, 15), z)
        q = (t + z[..., None]).clamp(0, 15)
        assert torch.equal(got.wz.cpu(), z.to(torch.uint8))
    else:
        q = t.clamp(-7, 7) + 8
    q = q.reshape(*lead, G * group)[..., :K].to(torch.uint8)
    assert torch.equal(got.wq.cpu(), q[..., 0::2] | (q[..., 1::2] << 4))
    assert torch.equal(got.sw.cpu(), s)
    # every weight is within the rounding of its code: half a scale, and what the
    # rounding of the scale to bf16 (2^-8 of it, at most 15 steps) takes from the range
    err = (_w4.dequantize(got.wq.cpu(), got.sw.cpu(), got.wz.cpu() if zeros else None, group) - w.double()).abs()
    step = sf.double().repeat_interleave(group, -1)[..., :K]
    assert (err <= step * (0.5 + 15 * 2.0 ** -8 + (0.5 if zeros else 0)) + 1e-40).all()
