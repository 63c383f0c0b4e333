"""GPU: what a call on another stream allocates comes from that stream's memory.  A block
freed on the current stream, which queued work there may still use, is not handed out to it."""
import pytest
import torch

import fp8_linear_layers_b200 as ql
from tests import _w4

pytestmark = pytest.mark.gpu

M, N, K, E, K_TOP = 600, 2304, 1024, 4, 2


def _calls():
    g = torch.Generator().manual_seed(0)
    w0 = (torch.randn(N, K, generator=g) * 0.02).bfloat16().cuda()
    x = torch.randn(M, K, generator=g).bfloat16().cuda()
    w = ql.W4Weight(*(t.cuda() for t in _w4.make_weights(g, (N,), K, 64, True)), 64)
    experts = ql.W4Weight(*(t.cuda() for t in _w4.make_weights(g, (E, N), K, 64, True)), 64)
    logits = torch.randn(40000, 32, generator=g).cuda()
    ids = torch.randint(0, E, (M, K_TOP), generator=g, dtype=torch.int32).cuda()
    xp, wts = torch.randn(M, K_TOP, K, generator=g).bfloat16().cuda(), torch.rand(M, K_TOP, generator=g).cuda()
    return {
        "forward_w4": lambda **s: [ql.forward_w4(x, w, **s)],
        "route": lambda **s: list(ql.route(logits, 8, **s)),
        "experts_w4": lambda **s: [ql.experts_w4(x, ids, experts, **s)],
        "experts_w4 combined": lambda **s: [ql.experts_w4(xp, ids, experts, weights=wts, **s)],
        "quantize_weight_w4": lambda **s: (lambda h: [h.wq, h.sw, h.wz])(ql.quantize_weight_w4(w0, 64, True, **s)),
    }


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", ["forward_w4", "route", "experts_w4", "experts_w4 combined", "quantize_weight_w4"])
def test_outputs_belong_to_the_calls_stream(cuda, name, handle):
    call = _calls()[name]
    want = call()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # blocks of the outputs' sizes, used and freed on the current stream
    held = [torch.full_like(t, 7) for t in want for _ in range(2)]
    freed = {t.data_ptr() for t in held}
    del held
    got = call(stream=side.cuda_stream if handle else side)
    assert not freed & {t.data_ptr() for t in got}
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert ql.device_status()[0] == 0
