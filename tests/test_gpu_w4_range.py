"""GPU: nothing is lost to the operands' range.  The largest scales (or the largest inputs)
meet weights of zero, so that values far below them decide the outputs: for few tokens, where
operands stay bf16, and for many, where f16 carries them and what it cannot is added apart."""
import pytest
import torch

import fp8_linear_layers_b200 as ql
from tests import _w4

pytestmark = pytest.mark.gpu


def _limit(y, mag, K, rounded):
    """One bf16 rounding of the output (2^-8 of it), f32 sums of exact products (K / 16 tensor-core
    steps and at most 64 further additions, each off by 2^-22 of the magnitudes), and, with zero
    points for more than 16 tokens, 2^-11 of each term for the weight's rounding to f16."""
    return 2.0 ** -8 * y.abs() + ((K / 16 + 64) * 2.0 ** -22 + (2.0 ** -11 if rounded else 0.0)) * mag + 1e-38


def _spread(gen, kind, x, wq, sw, wz, group):
    """Large scales or inputs where the weights are zero.  Returns x, wq, sw."""
    K, G = x.shape[-1], sw.shape[-1]
    q = torch.stack((wq & 15, wq >> 4), -1).flatten(-2)
    zero = torch.full_like(q, 8) if wz is None else wz.repeat_interleave(group, -1)[..., :K]
    off = torch.rand(G, generator=gen) < 0.4  # groups of zero weights, in every row
    off[0], off[-1] = True, G == 1
    at = off.repeat_interleave(group)[:K]
    q = torch.where(at, zero, q)
    wq = (q[..., 0::2] | (q[..., 1::2] << 4)).contiguous()
    if "scales" in kind:  # 2^-60 .. 2^-20 against 2^0 .. 2^20; every third row as it was
        e = torch.where(off, torch.randint(0, 21, sw.shape, generator=gen), torch.randint(-60, -19, sw.shape, generator=gen))
        wide = (sw.float() * 2.0 ** e).bfloat16()
        keep = torch.arange(sw.shape[-2]) % 3 == 1
        sw = torch.where(keep[:, None], sw, wide)
    if "tokens" in kind:
        e = torch.where(at, torch.randint(10, 31, x.shape, generator=gen), torch.randint(-50, -9, x.shape, generator=gen))
        wide = (x.float() * 2.0 ** e).bfloat16()
        rows = torch.arange(x.shape[0]) % 3 != 1
        x = torch.where(rows.view(-1, *[1] * (x.dim() - 1)), wide, x)
    return x, wq, sw


@pytest.mark.parametrize("kind", ["scales", "tokens", "scales and tokens"])
@pytest.mark.parametrize("M,N,K,group,zeros", [
    (3, 70, 512, 64, False), (16, 300, 1056, 32, True), (17, 70, 512, 64, False), (40, 130, 992, 32, True),
    (100, 257, 2080, 128, False), (129, 255, 1312, 64, True), (300, 70, 512, 64, False), (400, 20001, 160, 32, False),
    (260, 10000, 512, 128, True)])
def test_product(cuda, kind, M, N, K, group, zeros):
    g = torch.Generator().manual_seed(M)
    x = torch.randn(M, K, generator=g).bfloat16()
    wq, sw, wz = _w4.make_weights(g, (N,), K, group, zeros)
    x, wq, sw = _spread(g, kind, x, wq, sw, wz, group)
    y = ql.forward_w4(x.cuda(), ql.W4Weight(wq.cuda(), sw.cuda(), wz.cuda() if zeros else None, group))
    assert ql.device_status()[0] == 0
    ref = x.double() @ _w4.dequantize(wq, sw, wz, group).t()
    mag = x.double().abs() @ _w4.magnitudes(wq, sw, wz, group).t()
    err, lim = (y.double().cpu() - ref).abs(), _limit(ref, mag, K, zeros and M > 16)
    assert (err <= lim).all(), (int((err > lim).sum()), (err / lim).max())


@pytest.mark.parametrize("combine", [False, True])
@pytest.mark.parametrize("kind", ["scales", "tokens", "scales and tokens"])
@pytest.mark.parametrize("T,k,E,N,K,group,zeros", [(9, 2, 3, 40, 288, 32, False), (60, 2, 3, 260, 512, 64, False),
                                                   (70, 3, 5, 41, 416, 32, True), (900, 3, 4, 72, 256, 64, False)])
def test_experts(cuda, combine, kind, T, k, E, N, K, group, zeros):
    g = torch.Generator().manual_seed(T)
    x = torch.randn(*((T, k, K) if combine else (T, K)), generator=g).bfloat16()
    wq, sw, wz = _w4.make_weights(g, (E, N), K, group, zeros)
    x, wq, sw = _spread(g, kind, x, wq, sw, wz, group)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    ids[T // 2, 0] = -1
    wts = torch.randn(T, k, generator=g) if combine else None
    w = ql.W4Weight(wq.cuda(), sw.cuda(), wz.cuda() if zeros else None, group)
    y = ql.experts_w4(x.cuda(), ids.cuda(), w, weights=wts.cuda() if combine else None)
    assert ql.device_status()[0] == 0
    ref, mag = _w4.experts64(x, ids, _w4.dequantize(wq, sw, wz, group), _w4.magnitudes(wq, sw, wz, group), wts)
    err, lim = (y.double().cpu() - ref).abs(), _limit(ref, mag, K, zeros and T > 16)
    assert (err <= lim).all(), (int((err > lim).sum()), (err / lim).max())


@pytest.mark.parametrize("M", [16, 17, 300])
def test_the_two_ends_of_the_types(cuda, M):
    """The smallest scale against the largest, the smallest input against the largest."""
    K, group = 128, 32
    x = torch.zeros(M, K).bfloat16()
    x[:, :32] = 3.0
    x[1, 40] = 2.0 ** 127
    x[2] = 2.0 ** -133          # the smallest bf16
    x[3, 32:] = float.fromhex("0x1.fep127")
    q = torch.full((5, K), 8, dtype=torch.uint8)
    q[:, :32] = 9
    q[3, :32] = 0
    sw = torch.ones(5, 4).bfloat16()
    sw[0, 0], sw[0, 1:] = 2.0 ** -133, float.fromhex("0x1.fep127")
    sw[1, 0], sw[1, 1:] = 2.0 ** -60, 2.0 ** 60
    sw[2] = 2.0 ** -133
    wq = (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous()
    y = ql.forward_w4(x.cuda(), ql.W4Weight(wq.cuda(), sw.cuda(), None, group))
    ref = x.double() @ _w4.dequantize(wq, sw, None, group).t()
    assert ((y.double().cpu() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-38).all()
    assert (y[0, 1] != 0) and (y[1, 1] != 0)


def test_rows_longer_than_any_layer(cuda):
    """Over 65536 inputs many tokens run as blocks of few."""
    g = torch.Generator().manual_seed(4)
    K = 65536 + 32
    x = torch.randn(37, K, generator=g).bfloat16()
    wq, sw, wz = _w4.make_weights(g, (2, 24), K, 128, True)
    w = ql.W4Weight(wq[0].cuda(), sw[0].cuda(), wz[0].cuda(), 128)
    assert ql.forward_w4_workspace_bytes(37, w) == 0
    size = _w4.magnitudes(wq, sw, wz, 128)
    wd = _w4.dequantize(wq, sw, wz, 128)
    ref, mag = x.double() @ wd[0].t(), x.double().abs() @ size[0].t()
    assert ((ql.forward_w4(x.cuda(), w).double().cpu() - ref).abs() <= _limit(ref, mag, K, False)).all()
    experts = ql.W4Weight(wq.cuda(), sw.cuda(), wz.cuda(), 128)
    ids = torch.randint(0, 2, (37, 2), generator=g, dtype=torch.int32)
    ref, mag = _w4.experts64(x, ids, wd, size)
    assert ((ql.experts_w4(x.cuda(), ids.cuda(), experts).double().cpu() - ref).abs() <= _limit(ref, mag, K, False)).all()
    xp, wts = x[:36].view(18, 2, K), torch.randn(18, 2, generator=g)
    ref, mag = _w4.experts64(xp, ids[:18], wd, size, wts)
    y = ql.experts_w4(xp.cuda(), ids[:18].cuda(), experts, weights=wts.cuda())
    assert ((y.double().cpu() - ref).abs() <= _limit(ref, mag, K, False)).all()
    assert ql.device_status()[0] == 0
