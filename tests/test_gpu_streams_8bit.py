"""GPU: 8-bit calls on another stream than the current one take their outputs, and a zeroed
workspace that they make, from that stream's memory and order."""
import pytest
import torch

import fp8_linear_layers_b200 as ql

pytestmark = pytest.mark.gpu


def _calls():
    g = torch.Generator().manual_seed(0)
    N, K, s, b = 2048, 4096, ql.W8A8_INT8_ROW, ql.FP8_E4M3_BLOCK128
    w0 = (torch.randn(N, K, generator=g) * 0.02).bfloat16().cuda()
    x = torch.randn(600, K, generator=g).bfloat16().cuda()
    wq, sw = ql.quantize_weight(s, w0)
    bq, bw = ql.quantize_weight(b, w0)
    qx, sx = ql.quantize_act(s, x)
    qb, sb = ql.quantize_act(b, x)
    ws = [ql.new_workspace(ql.forward_workspace_bytes(s, 600, N, K)) for _ in range(3)]
    small = ql.new_workspace(ql.workspace_bytes(s, 16, N, K))
    torch.cuda.synchronize()
    return {
        "quantize_weight": lambda **k: list(ql.quantize_weight(s, w0, **k)),
        "quantize_act": lambda **k: list(ql.quantize_act(s, x, **k)),
        "gemv": lambda **k: [ql.gemv(s, x[:1], wq, sw, **k)],
        "gemv_grouped": lambda **k: ql.gemv_grouped(s, [(x[:1], wq, sw, None)] * 2, **k),
        "gemv_prequant": lambda **k: [ql.gemv_prequant(s, qx[:1], sx[:1], wq, sw, **k)],
        "gemv_weight_only": lambda **k: [ql.gemv_weight_only(s, x[:1], wq, sw, **k)],
        "gemm_small": lambda **k: [ql.gemm_small(s, x[:16], wq, sw, small, **k)],
        "gemm_small_prequant": lambda **k: [ql.gemm_small_prequant(s, qx[:16], sx[:16], wq, sw, small, **k)],
        "gemm_small_noalloc": lambda **k: [ql.gemm_small_noalloc(s, x[:16], wq, sw, **k)],
        "gemm_small_grouped": lambda **k: ql.gemm_small_grouped(s, x[:16], [(wq, sw, None)], small, **k),
        "gemm": lambda **k: [ql.gemm(s, qx, sx, wq, sw, **k)],
        "gemm_grouped": lambda **k: ql.gemm_grouped(s, qx, sx, [(wq, sw, None)] * 2, **k),
        "gemm_quant_out": lambda **k: list(ql.gemm_quant_out(b, qb, sb, bq, bw, **k)),
        "forward": lambda **k: [ql.forward(s, x, wq, sw, workspace=ws[0], **k)],
    }


@pytest.mark.parametrize("name", ["quantize_weight", "quantize_act", "gemv", "gemv_grouped", "gemv_prequant",
                                  "gemv_weight_only", "gemm_small", "gemm_small_prequant", "gemm_small_noalloc",
                                  "gemm_small_grouped", "gemm", "gemm_grouped", "gemm_quant_out", "forward"])
def test_outputs_belong_to_the_calls_stream(cuda, name):
    call = _calls()[name]
    want = call()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    held = [torch.full_like(t, 7) for t in want for _ in range(2)]  # used and freed on the current stream
    freed = {t.data_ptr() for t in held}
    del held
    got = call(stream=side)
    assert not freed & {t.data_ptr() for t in got}
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert ql.device_status()[0] == 0


def test_weight_only_workspace_is_zeroed_on_the_calls_stream(cuda):
    """While the current stream is busy: the call does not see what the memory held."""
    g = torch.Generator().manual_seed(1)
    s, M, N, K = ql.W8A8_INT8_ROW, 16, 2048, 4096
    x = torch.randn(M, K, generator=g).bfloat16().cuda()
    w = (torch.randn(N, K, generator=g) * 0.02).bfloat16().cuda()
    wq, sw = ql.quantize_weight(s, w)
    want = ql.forward_weight_only(s, x, wq, sw).double()
    mag = x.double().abs() @ w.double().abs().t() * 1.01
    # parts meet in f32 in the order of arrival (at most 148 of them): 148 * 2^-23 < 2^-15 of the
    # magnitudes, then one step of bf16
    lim = (2.0 ** -7 * want.abs() + 2.0 ** -15 * mag) * (1 + 2.0 ** -6)
    nb = ql.weight_only_workspace_bytes(s, M, N, K)
    assert nb > 0
    side = torch.cuda.Stream()
    for _ in range(2):  # kernels loaded, and memory of both streams that is not zero
        warm = [ql.forward_weight_only(s, x, wq, sw, stream=side) for _ in range(4)]
        held = [torch.full((nb,), 0x3F, dtype=torch.uint8, device="cuda") for _ in range(4)]
        with torch.cuda.stream(side):
            dirty = [torch.full((nb,), 0x3F, dtype=torch.uint8, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        del warm, held, dirty
    torch.cuda._sleep(1_000_000_000)  # about half a second of the current stream
    got = [ql.forward_weight_only(s, x, wq, sw, stream=side) for _ in range(4)]
    torch.cuda.synchronize()
    for y in got:
        assert ((y.double() - want).abs() <= lim).all()
    assert ql.device_status()[0] == 0
