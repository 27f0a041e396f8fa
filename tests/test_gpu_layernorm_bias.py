"""GPU: the gradient of a layer norm's bias where there is no weight."""
import math

import pytest
import torch

import gated_delta_rule_58_amd as kda
from tests import linattn_ref as ref
from tests.gpu_util import DEV, need_gpu, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape, bshape", [((300, 3, 128), (3, 128)), ((300, 3, 128), (128,)),
                                           ((7, 1000), (1000,)), ((0, 64), (64,))])
def test_bias_without_a_weight(shape, bshape):
    """dx and dbias are those of a weight of ones; the bias's values do not matter."""
    need_gpu()
    say("layernorm bias only", shape, bshape)
    gen = torch.Generator().manual_seed(3)
    x, dy = torch.randn(*shape, generator=gen), torch.randn(*shape, generator=gen)
    b = torch.randn(*bshape, generator=gen)
    X, DY, B = x.to(DEV), dy.to(DEV), b.to(DEV)
    dx, dw, db = kda.layernorm_backward(DY, X, bias=B)
    want = kda.layernorm_backward(DY, X, torch.ones_like(B))
    assert dw is None and torch.equal(dx, want[0]) and torch.equal(db, want[2])
    # a sum of rows in fp32: rows u of the values' absolute sum at most
    over = tuple(range(x.dim() - b.dim()))
    err = (db.cpu().double() - dy.double().sum(over)).abs()
    assert (err <= (math.prod(shape[:len(over)]) + 32) * ref.U
            * dy.double().abs().sum(over)).all()
    again = kda.layernorm_backward(DY, X, bias=B * 0)
    assert torch.equal(again[2], db)
    assert kda.layernorm_backward(DY, X, bias=B, want_dbias=False)[1:] == (None, None)
    assert kda.layernorm_backward(DY, X)[1:] == (None, None)
    both = kda.layernorm_backward(DY, X, torch.ones_like(B), bias=B)
    assert torch.equal(both[1], want[1]) and torch.equal(both[2], want[2])
