"""GPU: a 4-bit weight handle whose tensors are replaced, or get other memory, is refused; one
whose tensors' contents change answers with the new ones."""
import pytest
import torch

import fp8_linear_layers_b200 as ql
from tests import _w4

pytestmark = pytest.mark.gpu


def _handle(lead=(40,), zeros=True):
    g = torch.Generator().manual_seed(0)
    host = _w4.make_weights(g, lead, 128, 64, zeros)
    return host, ql.W4Weight(*(None if t is None else t.cuda() for t in host), 64)


@pytest.mark.parametrize("name", ["wq", "sw", "wz", "group", "N", "_p"])
def test_nothing_is_replaced(cuda, name):
    _, w = _handle()
    with pytest.raises(AttributeError):
        setattr(w, name, getattr(w, name))
    with pytest.raises((AttributeError, TypeError)):
        delattr(w, name)


@pytest.mark.parametrize("name", ["wq", "sw", "wz"])
@pytest.mark.parametrize("M", [2, 40])
def test_other_memory_is_refused(cuda, name, M):
    _, w = _handle()
    _, e = _handle((3, 40))
    x = torch.ones(M, 128, dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(M, 2, dtype=torch.int32, device="cuda")
    ql.forward_w4(x, w)
    for h in (w, e):
        t = getattr(h, name)
        keep = t.data  # (the old memory stays alive)
        t.data = keep.clone()
        with pytest.raises(ValueError, match="memory"):
            ql.forward_w4(x, h) if h is w else ql.experts_w4(x, ids, h)
        t.data = keep
    ql.forward_w4(x, w)
    ql.experts_w4(x, ids, e)
    torch.cuda.synchronize()


def test_contents_may_change(cuda):
    (wq, sw, wz), w = _handle()
    x = torch.randn(3, 128, generator=torch.Generator().manual_seed(1)).bfloat16()
    w.sw.mul_(2.0)
    w.wq.copy_(wq.flip(0))
    _w4.assert_product(ql.forward_w4(x.cuda(), w), x, wq.flip(0), sw * 2.0, wz, 64)
