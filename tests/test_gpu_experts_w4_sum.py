"""GPU: the combined experts' product sums a token's experts in f32 and rounds once, for few
and for many tokens (where the pairs' products pass through the workspace)."""
import pytest
import torch

import fp8_linear_layers_b200 as ql
from tests import _w4

pytestmark = pytest.mark.gpu


def _limit(y, mag, K):
    """The output's one bf16 rounding (2^-8 of the value covers half a step and its rounding of
    the limit itself), and f32 sums of exact products: K / 16 tensor-core steps, at most 64
    further additions of parts and pairs, each off by at most 2^-22 of the magnitudes.  No
    term for a pair's own rounding: there is none."""
    return 2.0 ** -8 * y.abs() + (K / 16 + 64) * 2.0 ** -22 * mag + 1e-38


@pytest.mark.parametrize("T,k,E,N,K,group", [
    (3, 4, 6, 40, 128, 64), (16, 8, 12, 136, 288, 32), (17, 8, 12, 136, 288, 32), (40, 6, 9, 41, 256, 128),
    (77, 8, 16, 260, 160, 64), (300, 8, 10, 72, 512, 64), (290, 32, 40, 42, 96, 32)])
def test_terms_that_cancel(cuda, T, k, E, N, K, group):
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, k, K, generator=g).bfloat16()
    wq, sw, _ = _w4.make_weights(g, (E, N), K, group, False)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    wts = torch.randn(T, k, generator=g)
    # the second half of a token's pairs almost undoes the first: the same experts on inputs
    # a few bf16 steps away
    h = k // 2
    ids[:, h:2 * h], wts[:, h:2 * h] = ids[:, :h], -wts[:, :h]
    x[:, h:2 * h] = (x[:, :h].float() * (1 + 2.0 ** -6 * torch.randn(T, h, K, generator=g))).bfloat16()
    y = ql.experts_w4(x.cuda(), ids.cuda(), ql.W4Weight(wq.cuda(), sw.cuda(), None, group), weights=wts.cuda())
    assert ql.device_status()[0] == 0
    ref, mag = _w4.experts64(x, ids, _w4.dequantize(wq, sw, None, group), _w4.magnitudes(wq, sw, None, group), wts)
    err = (y.double().cpu() - ref).abs()
    lim = _limit(ref, mag, K)
    assert (err <= lim).all(), ((err - lim).max(), int((err > lim).sum()))
