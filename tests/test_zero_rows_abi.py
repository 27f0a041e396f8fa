"""kda_zero_rows_behind refuses bad arguments on the host before any HIP call (fake device
addresses, never dereferenced)."""
import ctypes

import pytest
import torch

from tests.test_linattn_abi import DEV, _fn, _last


def _call(cu=DEV[0], N=2, T=48, tensors=(DEV[1], DEV[2]), sizes=(256, 12), count=None):
    n = len(tensors)
    p, b = (ctypes.c_void_p * n)(*tensors), (ctypes.c_int64 * n)(*sizes)
    return _fn("kda_zero_rows_behind")(cu, N, T, p, b, n if count is None else count, None)


@pytest.mark.parametrize("bad, status", [
    (dict(N=-1), 1), (dict(T=-1), 1), (dict(count=-1), 1), (dict(T=1 << 31), 4),
    (dict(tensors=(DEV[1],) * 5, sizes=(4,) * 5), 4), (dict(cu=None), 1), (dict(cu=DEV[0] + 2), 5),
    (dict(sizes=(256, 6)), 2), (dict(sizes=(-4, 4)), 2), (dict(tensors=(DEV[1], None)), 1),
    (dict(tensors=(DEV[1] + 2, DEV[2])), 5), (dict(tensors=(DEV[0], DEV[2])), 1),
    (dict(sizes=(1 << 31, 4)), 2),
])
def test_refusals(bad, status):
    assert _call(**bad) == status, _last()
    assert "kda_zero_rows_behind" in _last()


def test_nothing_to_clear_is_nothing():
    assert _call(T=0, tensors=(None, None)) == 0
    assert _call(sizes=(0, 0)) == 0
    assert _fn("kda_zero_rows_behind")(DEV[0], 1, 8, None, None, 0, None) == 0


def test_binding_refuses():
    import gated_delta_rule_58_amd as kda
    with pytest.raises(TypeError, match="int32"):
        kda.zero_rows_behind(torch.zeros(3), torch.zeros(4, 2))
    with pytest.raises(ValueError, match="GPU"):
        kda.zero_rows_behind(torch.zeros(3, dtype=torch.int32), torch.zeros(4, 2))
