"""GPU: one workspace for 8-bit and 4-bit calls, as the header allows it: the large-M K split
and the 4-bit calls share a buffer as they are; a small-M call needs it zeroed behind another."""
import numpy as np
import pytest
import torch

import fp8_linear_layers_b200 as ql
from tests import _w4

pytestmark = pytest.mark.gpu


def _quantized(scheme, M, N, K, gen):
    x = torch.randn(M, K, generator=gen).bfloat16().cuda()
    w = (torch.randn(N, K, generator=gen) * 0.02).bfloat16().cuda()
    return ql.quantize_act(scheme, x) + ql.quantize_weight(scheme, w)


def test_large_m_split_and_4_bit_calls_share_a_buffer(cuda):
    """Split products of different numbers of tiles and schemes, and 4-bit calls of both
    kinds, in turn in one buffer that is zeroed once: each gives what it gives in a buffer of
    its own."""
    g = torch.Generator().manual_seed(1)
    products = [(ql.W8A8_INT8_ROW, 512, 4096, 8192), (ql.FP8_E4M3_BLOCK128, 512, 1024, 4096),
                (ql.FP8_E4M3_ROW, 256, 2048, 8192), (ql.FP8_E4M3_BLOCK128, 128, 256, 8192),
                (ql.W8A8_INT8_ROW, 1152, 2048, 8192)]
    calls, sizes = [], []
    for scheme, M, N, K in products:
        n = ql.workspace_bytes(scheme, M, N, K)
        assert n > 0
        args = _quantized(scheme, M, N, K, g)
        calls.append(lambda ws, y, a=args, s=scheme: ql.gemm(s, *a, workspace=ws, y=y))
        sizes.append((n, (M, N)))
    w = ql.W4Weight(*(t.cuda() for t in _w4.make_weights(g, (300,), 2048, 64, True)), 64)
    experts = ql.W4Weight(*(t.cuda() for t in _w4.make_weights(g, (4, 2000), 512, 64, True)), 64)
    x = torch.randn(900, 2048, generator=g).bfloat16().cuda()
    xe = torch.randn(1200, 2, 512, generator=g).bfloat16().cuda()
    ids, wts = torch.randint(0, 4, (1200, 2), generator=g, dtype=torch.int32).cuda(), torch.rand(1200, 2, generator=g).cuda()
    calls.append(lambda ws, y: ql.forward_w4(x, w, workspace=ws, y=y))
    sizes.append((ql.forward_w4_workspace_bytes(900, w), (900, 300)))
    calls.append(lambda ws, y: ql.experts_w4(xe, ids, experts, weights=wts, workspace=ws, y=y))
    sizes.append((ql.experts_w4_workspace_bytes(1200, 2, experts, combine=True), (1200, 2000)))
    new = lambda shape: torch.full(shape, -7.0, dtype=torch.bfloat16, device="cuda")
    alone = [c(ql.new_workspace(n), new(shape)) for c, (n, shape) in zip(calls, sizes)]
    for spare in (0, 1000):  # (a size that is not a multiple of 256 too)
        ws = ql.new_workspace(max(n for n, _ in sizes) + spare)
        order = np.random.default_rng(spare).permutation(np.repeat(np.arange(len(calls)), 3))
        for i in order:
            assert torch.equal(calls[i](ws, new(sizes[i][1])), alone[i]), (i, order)
    assert ql.device_status()[0] == 0


@pytest.mark.parametrize("scheme", [ql.W8A8_INT8_ROW, ql.FP8_E4M3_BLOCK128])
def test_small_m_after_a_4_bit_call(cuda, scheme):
    """Zeroed in between, as the header asks.  int8 sums are whole numbers, so the outputs are
    equal.  E4M3 sums: at most 148 parts of a tile meet in f32 in the order of arrival, so two
    calls differ by up to 148 * 2^-23 < 2^-15 of the magnitudes, and then by one step of bf16,
    2^-7 of the value (the limit's own factor 1 + 2^-6 covers a step up)."""
    g = torch.Generator().manual_seed(2)
    M, N, K = 16, 1024, 4096
    x = torch.randn(M, K, generator=g).bfloat16().cuda()
    w = (torch.randn(N, K, generator=g) * 0.02).bfloat16().cuda()
    wq, sw = ql.quantize_weight(scheme, w)
    w4 = ql.W4Weight(*(t.cuda() for t in _w4.make_weights(g, (N,), K, 128, False)[:2]), group=128)
    x4 = torch.randn(200, K, generator=g).bfloat16().cuda()
    n = max(ql.workspace_bytes(scheme, M, N, K), ql.forward_w4_workspace_bytes(200, w4))
    alone, alone4 = ql.gemm_small(scheme, x, wq, sw, ql.new_workspace(n)), ql.forward_w4(x4, w4)
    mag = x.double().abs() @ w.double().abs().t() * 1.2  # (quantization moves a value by at most 2^-4)
    lim = 0.0 if scheme == ql.W8A8_INT8_ROW else (2.0 ** -7 * alone.double().abs() + 2.0 ** -15 * mag) * (1 + 2.0 ** -6)
    ws = ql.new_workspace(n)
    for _ in range(3):
        assert torch.equal(ql.forward_w4(x4, w4, workspace=ws), alone4)
        ws.zero_()
        y = ql.gemm_small(scheme, x, wq, sw, ws, y=torch.full((M, N), -7.0, dtype=torch.bfloat16, device="cuda"))
        assert ((y.double() - alone.double()).abs() <= lim).all()
    assert ql.device_status()[0] == 0
