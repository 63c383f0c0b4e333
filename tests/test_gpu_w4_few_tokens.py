"""GPU: up to 16 tokens nothing is rounded but the output: with zero points as without, and for
combined experts.  (Limits without the terms that the many-token path needs.)"""
import pytest
import torch

import fp8_linear_layers_b200 as ql
from tests import _w4

pytestmark = pytest.mark.gpu


def _limit(y, mag, K):
    """Half a step of bf16, 2^-9 of the rounded value (2^-8 covers the value's own distance
    from it), and f32 sums of exact products: x has 8 significant bits, q - z at most 4, so a
    product has 12; K / 16 tensor-core steps, a scale's product and at most 64 further
    additions, each off by at most 2^-22 of the magnitudes."""
    return 2.0 ** -8 * y.abs() + (K / 16 + 64) * 2.0 ** -22 * mag + 1e-38


@pytest.mark.parametrize("group", ql.W4_GROUPS)
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,N,K", [(1, 130, 4128), (5, 4096, 1024), (8, 64, 512), (9, 15, 160), (16, 257, 1056),
                                   (2, 40, 14336), (13, 5003, 992)])
def test_product(cuda, group, zeros, M, N, K):
    g = torch.Generator().manual_seed(M * 7 + group)
    x = torch.randn(M, K, generator=g).bfloat16()
    wq, sw, wz = _w4.make_weights(g, (N,), K, group, zeros)
    y = ql.forward_w4(x.cuda(), ql.W4Weight(wq.cuda(), sw.cuda(), wz.cuda() if zeros else None, group))
    ref = x.double() @ _w4.dequantize(wq, sw, wz, group).t()
    mag = x.double().abs() @ _w4.magnitudes(wq, sw, wz, group).t()
    assert ((y.double().cpu() - ref).abs() <= _limit(ref, mag, K)).all()


@pytest.mark.parametrize("combine", [False, True])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, True), (64, False), (128, True)])
@pytest.mark.parametrize("T,k,E,N,K", [(1, 8, 16, 33, 256), (5, 4, 6, 2056, 544), (9, 3, 7, 130, 288), (16, 6, 12, 72, 1024)])
def test_experts(cuda, combine, group, zeros, T, k, E, N, K):
    g = torch.Generator().manual_seed(T)
    x = torch.randn(*((T, k, K) if combine else (T, K)), generator=g).bfloat16()
    wq, sw, wz = _w4.make_weights(g, (E, N), K, group, zeros)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    wts = torch.randn(T, k, generator=g) if combine else None
    y = ql.experts_w4(x.cuda(), ids.cuda(), ql.W4Weight(wq.cuda(), sw.cuda(), wz.cuda() if zeros else None, group),
                      weights=wts.cuda() if combine else None)
    ref, mag = _w4.experts64(x, ids, _w4.dequantize(wq, sw, wz, group), _w4.magnitudes(wq, sw, wz, group), wts)
    assert ((y.double().cpu() - ref).abs() <= _limit(ref, mag, K)).all()


@pytest.mark.parametrize("M", [1, 16, 17, 150])
def test_a_weight_of_twelve_bits(cuda, M):
    """15 s - 14 s - s = 0 for s = 255/128, whose fifteenfold has 12 significant bits: nothing
    is left up to 16 tokens; above, where the header rounds a weight to 11, at most half a
    step of 15 s, 2^-11 of it."""
    wq = torch.zeros(3, 32, dtype=torch.uint8)
    wq[:, 0], wq[:, 1] = 0xEF, 0x01  # codes 15, 14, 1
    sw = torch.full((3, 2), 255 / 128).bfloat16()
    x = torch.zeros(M, 64).bfloat16()
    x[:, 0], x[:, 1], x[:, 2] = 1.0, -1.0, -1.0
    w = ql.W4Weight(wq.cuda(), sw.cuda(), torch.zeros(3, 2, dtype=torch.uint8, device="cuda"), 32)
    y = ql.forward_w4(x.cuda(), w).double().abs()
    assert (y <= (0.0 if M <= 16 else 2.0 ** -11 * 15 * 255 / 128)).all()
