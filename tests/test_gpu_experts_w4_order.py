"""GPU: the experts' products have the same bits call after call, also where the pairs'
places come from atomic additions (more than 2048 pairs) and an expert has more pairs than
a token tile takes."""
import pytest
import torch

import fp8_linear_layers_b200 as ql
from tests import _w4

pytestmark = pytest.mark.gpu


def _case(T, k, E, N, K, combine, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*((T, k, K) if combine else (T, K)), generator=g).bfloat16().cuda()
    w = ql.W4Weight(*(t.cuda() for t in _w4.make_weights(g, (E, N), K, 64, True)), 64)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32).cuda()
    return x, ids, w, torch.rand(T, k, generator=g).cuda() if combine else None


@pytest.mark.parametrize("combine", [False, True])
@pytest.mark.parametrize("T,k,E,N,K", [(1500, 2, 1, 264, 1312), (1100, 4, 5, 520, 2080), (2100, 3, 24, 264, 800),
                                       (700, 4, 3, 41, 1312)])
def test_same_bits_call_after_call(cuda, combine, T, k, E, N, K):
    x, ids, w, wts = _case(T, k, E, N, K, combine)
    ws = ql.new_workspace(ql.experts_w4_workspace_bytes(T, k, w, combine=combine))
    first = ql.experts_w4(x, ids, w, weights=wts, workspace=ws)
    for i in range(20):
        ws.fill_(0x5A + i)
        assert torch.equal(ql.experts_w4(x, ids, w, weights=wts, workspace=ws), first), i
    assert ql.device_status()[0] == 0


@pytest.mark.parametrize("combine", [False, True])
def test_same_bits_on_two_streams(cuda, combine):
    x, ids, w, wts = _case(1100, 4, 5, 520, 2080, combine, seed=1)
    alone = ql.experts_w4(x, ids, w, weights=wts)
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [ql.new_workspace(ql.experts_w4_workspace_bytes(1100, 4, w, combine=combine)) for _ in streams]
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        for s, ws in zip(streams, spaces):
            with torch.cuda.stream(s):
                got.append(ql.experts_w4(x, ids, w, weights=wts, workspace=ws))
    torch.cuda.synchronize()
    assert all(torch.equal(y, alone) for y in got)
    assert ql.device_status()[0] == 0


def test_a_pair_does_not_see_its_tile(cuda):
    """One token's pair has the same bits among few and among many pairs of its expert, in
    a full tile and in the short last one."""
    x, _, w, _ = _case(1000, 4, 3, 264, 1312, False, seed=2)
    x[:] = x[0]
    ids = torch.tensor([0, 1, 2, 0], dtype=torch.int32, device="cuda").repeat(1000, 1)
    y = ql.experts_w4(x, ids, w)
    assert torch.equal(y, y[:1].expand_as(y)) and torch.equal(y[:, 0], y[:, 3])
    few = ql.experts_w4(x[:20].contiguous(), ids[:20].contiguous(), w)
    assert torch.equal(few, y[:20])
