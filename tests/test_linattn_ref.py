"""CPU: the reference of the linear attention and layer norm gradients against
central differences of its forward in 64 bits, every element."""
import pytest
import torch

from tests import linattn_ref as ref


def _differences(f, x, h=1e-6):
    """d f / d x elementwise by central differences (x is changed in place and put back)."""
    out = torch.zeros_like(x)
    flat, res = x.view(-1), out.view(-1)
    for i in range(flat.numel()):
        keep = flat[i].item()
        flat[i] = keep + h
        up = f()
        flat[i] = keep - h
        down = f()
        flat[i] = keep
        res[i] = (up - down) / (2 * h)
    return out


@pytest.mark.parametrize("per_token", [True, False])
def test_attention_gradients_against_differences(per_token):
    gen = torch.Generator().manual_seed(7)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    cu, H, Hk, dk, dv = [0, 3, 3, 4, 9], 4, 2, 3, 2
    T, N, scale = cu[-1], 4, 0.7
    q, k, v = rnd(T, Hk, dk), rnd(T, Hk, dk), rnd(T, H, dv)
    g = -torch.rand(T, H, generator=gen, dtype=torch.float64) if per_token else \
        -torch.rand(H, generator=gen, dtype=torch.float64)
    S0, do, dS = rnd(N, H, dk, dv), rnd(T, H, dv), rnd(N, H, dk, dv)

    def loss():
        o, S = ref.forward(q, k, v, g, cu, S0, scale)
        return float((o * do).sum() + (S * dS).sum())

    got = ref.backward(q, k, v, g, cu, do, S0, dS, scale)
    for x, w in zip((q, k, v, g, S0), got):
        # second differences of order 1 leave 1e-12, the rounding of the loss 1e-16 * 100 / 1e-6
        assert torch.allclose(_differences(loss, x), w, rtol=1e-7, atol=1e-7)


@pytest.mark.parametrize("wshape", [None, (5,), (3, 5)])
def test_norm_gradients_against_differences(wshape):
    gen = torch.Generator().manual_seed(8)
    x = torch.randn(4, 3, 5, generator=gen, dtype=torch.float64)
    dy = torch.randn(4, 3, 5, generator=gen, dtype=torch.float64)
    w = None if wshape is None else torch.randn(*wshape, generator=gen, dtype=torch.float64)
    b = None if wshape is None else torch.randn(*wshape, generator=gen, dtype=torch.float64)
    loss = lambda: float((ref.norm(x, w, b, 1e-3) * dy).sum())  # noqa: E731
    dx, dw, db = ref.norm_backward(dy, x, w, 1e-3)
    assert torch.allclose(_differences(loss, x), dx, rtol=1e-7, atol=1e-7)
    if w is not None:
        assert torch.allclose(_differences(loss, w), dw, rtol=1e-7, atol=1e-7)
        assert torch.allclose(_differences(loss, b), db, rtol=1e-7, atol=1e-7)
