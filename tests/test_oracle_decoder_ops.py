"""The plain forms of rotary positions and of the vocabulary loss, pinned to independent ones: complex
multiplication, finite differences, torch's own cross entropy and autograd in 64 bits."""
import math

import pytest
import torch

from oracle import decoder_ops as R64


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_is_a_complex_product_and_its_inverse_the_gradient(layout):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(2, 3, 2, 10, generator=g, dtype=torch.float64)
    pos = torch.tensor([[0, 1, 5], [100000, 7, 3]])
    theta, m = R64.rope_frequencies(6)
    y = R64.rope(x, pos, theta, 1.25, layout)
    z = torch.complex(x[..., 0:3], x[..., 3:6]) if layout == "half" else torch.complex(x[..., 0:6:2], x[..., 1:6:2])
    w = z * torch.polar(torch.full((2, 3, 1, 3), 1.25, dtype=torch.float64), pos[..., None, None] * theta)
    got = torch.complex(y[..., 0:3], y[..., 3:6]) if layout == "half" else torch.complex(y[..., 0:6:2], y[..., 1:6:2])
    assert torch.allclose(got, w, atol=1e-12) and torch.equal(y[..., 6:], x[..., 6:])
    dy = torch.randn(y.shape, generator=g, dtype=torch.float64)
    xr = x.clone().requires_grad_()
    R64.rope(xr, pos, theta, 1.25, layout).backward(dy)
    assert torch.allclose(R64.rope(dy, pos, theta, 1.25, layout, inverse=True), xr.grad, atol=1e-12)


def test_rope_frequencies_closed_forms():
    t, m = R64.rope_frequencies(8)
    assert m == 1.0 and torch.allclose(t, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64))
    assert torch.allclose(R64.rope_frequencies(8, scaling="linear", factor=4)[0], t / 4)
    n = R64.rope_frequencies(8, scaling="ntk", factor=4)[0]            # the longest wave is stretched by factor
    assert math.isclose(n[0], 1.0) and math.isclose(n[3], t[3] / 4, rel_tol=1e-12)
    b = R64.rope_frequencies(8, scaling="banded", factor=4, original_length=4096)[0]
    assert b[0] == t[0] and math.isclose(b[3], t[3] / 4, rel_tol=1e-12)   # 652 turns stay, 0.65 are stretched
    y, m = R64.rope_frequencies(8, scaling="yarn", factor=4, original_length=4096)
    assert math.isclose(m, 0.1 * math.log(4) + 1) and y[0] == t[0] and math.isclose(y[3], t[3] / 4, rel_tol=1e-12)


def test_vocab_loss_matches_torch_and_differences():
    g = torch.Generator().manual_seed(2)
    X = torch.randn(7, 5, generator=g, dtype=torch.float64, requires_grad=True)
    W = torch.randn(11, 5, generator=g, dtype=torch.float64)
    y = torch.tensor([0, 10, -100, 3, 3, -100, 7])
    w = torch.rand(7, generator=g, dtype=torch.float64)
    loss, dX = R64.vocab_loss(X.detach(), W, y, w)
    ref = torch.nn.functional.cross_entropy(X @ W.t(), y, reduction="none")
    (ref * w).sum().backward()
    assert torch.allclose(loss, ref.detach(), atol=1e-12) and torch.allclose(dX, X.grad, atol=1e-12)
    for t, k in ((0, 1), (4, 3)):
        e = torch.zeros(7, 5, dtype=torch.float64)
        e[t, k] = 1e-5
        up, dn = (R64.vocab_loss(X.detach() + s * e, W, y)[0] for s in (1, -1))
        assert abs(((up - dn).sum() / 2e-5 * w[t]) - dX[t, k]) < 1e-8
