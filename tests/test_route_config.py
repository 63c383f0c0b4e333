"""The router's configuration is read at each call (CPU only)."""
import numpy as np
import pytest
import torch

import fp8_linear_layers_b200 as ql

FIELDS = dict(experts=64, top_k=8, groups=8, top_groups=4, group_top=2, score=1, renormalize=True, scale=2.5)


def _config(**kw):
    return ql._route_config(*{**FIELDS, **kw}.values())


def test_fields():
    c = _config()
    assert {n: getattr(c, n) for n in FIELDS} == {**FIELDS, "renormalize": 1}
    assert _config() is c  # built once


@pytest.mark.parametrize("make", [lambda v: torch.tensor(v), lambda v: torch.nn.Parameter(torch.tensor(v), requires_grad=False)])
def test_a_tensor_is_read_again(make):
    scale = make(1.0)
    assert _config(scale=scale).scale == 1.0
    scale.fill_(2.0)
    assert _config(scale=scale).scale == 2.0
    for name, dtype in (("top_k", torch.int64), ("top_groups", torch.int64), ("renormalize", torch.bool)):
        t = torch.ones((), dtype=dtype)
        assert getattr(_config(**{name: t}), name) == 1
        t.zero_()
        assert getattr(_config(**{name: t}), name) == 0


def test_an_array_is_read_again():
    scale = np.array(1.0)
    assert _config(scale=scale).scale == 1.0
    scale[...] = 2.0
    assert _config(scale=scale).scale == 2.0


@pytest.mark.parametrize("bad", [dict(top_k=2.5), dict(groups="8"), dict(scale=None), dict(score=None)])
def test_refusals(bad):
    with pytest.raises((TypeError, ValueError)):
        _config(**bad)
