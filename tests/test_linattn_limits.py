"""Calls that no launch can hold (2^32 work items or more) are refused on the host with
KDA_ERR_UNSUPPORTED, before anything is launched (fake device addresses, never
dereferenced)."""
import pytest

from tests.test_linattn_abi import _fn, _last

FAR = [(i + 1) << 42 for i in range(16)]  # 4 TiB each


@pytest.mark.parametrize("N, H, dv, dt", [
    (1 << 15, 128, 128, 1),   # 4.2 M pairs x 2 column tiles x 704 threads
    (1 << 17, 64, 64, 1),     # 8.4 M pairs x 704
    (1 << 17, 64, 64, 0),     # fp32: 512 threads
    (3051000, 1, 128, 1),     # 2 x 3,051,008 x 704: just above
])
def test_prefill(N, H, dv, dt):
    T = 48
    st = _fn("kda_linattn_chunk_prefill")(
        FAR[0], H * 128, FAR[1], H * 128, FAR[2], H * dv, dt, FAR[3], T * H, FAR[4], None, N, None,
        None, 0, N, None, FAR[5], 1, T, H, H, 128, dv, 1.0, None, 0, None)
    assert st == 4, _last()
    assert "launch" in _last()


@pytest.mark.parametrize("N, H, dk, dv, dt", [
    (1 << 14, 64, 128, 128, 1),   # 1 M pairs x 6 workgroups x 704 threads
    (1 << 17, 24, 64, 64, 1),     # 3.1 M x 3 x 704
    (1 << 16, 128, 128, 64, 0),   # fp32: 8.4 M x 2 x 512
])
def test_backward(N, H, dk, dv, dt):
    T = 48
    need = _fn("kda_linattn_chunk_prefill_backward_workspace_bytes")(T, N, H, H, dk, dv)
    st = _fn("kda_linattn_chunk_prefill_backward")(
        FAR[0], H * dk, FAR[1], H * dk, FAR[2], H * dv, dt, FAR[3], T * H, FAR[4], None, N, None,
        FAR[5], dt, None, FAR[6], FAR[7], FAR[8], 1, FAR[9], None, T, H, H, dk, dv, 1.0, FAR[10],
        need, None)
    assert st == 4, _last()
    assert "launch" in _last()


@pytest.mark.parametrize("N, H", [(1 << 17, 64), ((1 << 23) - 7, 1), (1 << 14, 16384)])
def test_decode(N, H):
    st = _fn("kda_linattn_recurrent_decode")(
        FAR[0], H * 64, FAR[1], H * 64, FAR[2], H * 64, 1, FAR[3], N * H, FAR[4], 1, 1, FAR[5],
        FAR[6], 1, N, H, H, 64, 64, 1.0, None)
    assert st == 4, _last()
    assert "N*H" in _last()


def test_lengths_that_do_not_fit_are_refused_before_they_are_multiplied():
    T, H = (1 << 62) + 3, 8
    st = _fn("kda_linattn_chunk_prefill")(
        FAR[0], H * 128, FAR[1], H * 128, FAR[2], H * 128, 1, FAR[3], 3 * H, FAR[4], None, 1, None,
        None, 0, 1, None, FAR[5], 1, T, H, H, 128, 128, 1.0, None, 0, None)
    assert st == 4 and "int32" in _last(), _last()
