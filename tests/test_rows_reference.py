"""The plain forms that the norm, rotation and append tests compare with: the gradient against central
differences and against autograd, the rotation against complex products, and planted mistakes."""
import pytest
import torch

from tests import rows_reference as ref


def case(seed, D=32, rot=24, B=2, H=3, S=4):
    g = torch.Generator().manual_seed(seed)
    x, dz = (torch.randn((B, H, S, D), generator=g, dtype=torch.float64) for _ in range(2))
    w = 1 + 0.3 * torch.randn((D,), generator=g, dtype=torch.float64)
    cos, sin = ref.angle_tables(16, rot)
    pos = torch.randint(0, 16, (B, S), generator=g)
    return x, dz, w, cos, sin, pos


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_matches_differences_and_autograd(interleaved):
    x, dz, w, cos, sin, pos = case(1)
    dx, _, dw, _ = ref.backward(x, w, cos, sin, pos, interleaved, 1e-6, dz)

    def loss(x, w):
        return (ref.forward(x, w, cos, sin, pos, interleaved, 1e-6)[0] * dz).sum()

    xa, wa = x.clone().requires_grad_(), w.clone().requires_grad_()
    loss(xa, wa).backward()
    assert torch.allclose(dx, xa.grad, rtol=1e-10, atol=1e-12)
    assert torch.allclose(dw, wa.grad, rtol=1e-10, atol=1e-12)
    h = 1e-5  # central differences: h^2 truncation and 2^-53 / h rounding, both near 1e-10
    for i in (0, 7, 23, 31):
        e = torch.zeros_like(x)
        e[1, 2, 3, i] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[1, 2, 3, i]) < 1e-7
        e = torch.zeros_like(w)
        e[i] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[i]) < 1e-7


def test_rotation_is_a_complex_product():
    x, _, _, cos, sin, pos = case(2)
    z = torch.complex(cos[pos].double(), sin[pos].double())[:, None]
    a, b = ref.pair_index(24, True)
    want = torch.view_as_complex(x[..., :24].reshape(*x.shape[:-1], 12, 2).contiguous()) * z
    got = ref.forward(x, None, cos, sin, pos, True, 0.0)[0]
    assert torch.allclose(torch.stack((got[..., a], got[..., b]), -1), torch.view_as_real(want))
    assert torch.equal(got[..., 24:], x[..., 24:])


@pytest.mark.parametrize("mistake", ["pairs", "sign", "norm", "eps", "weight"])
def test_planted_mistakes_leave_the_bounds(mistake):
    x, dz, w, cos, sin, pos = case(3)
    want, bound = ref.forward(x, w, cos, sin, pos, False, 1e-2)
    if mistake == "pairs":
        got = ref.forward(x, w, cos, sin, pos, True, 1e-2)[0]
    elif mistake == "sign":
        got = ref.forward(x, w, cos, -sin, pos, False, 1e-2)[0]
    elif mistake == "norm":
        got = ref.forward(x, None, cos, sin, pos, False, 1e-2)[0]
    elif mistake == "eps":
        got = ref.forward(x, w, cos, sin, pos, False, 0.0)[0] * 1.01
    else:
        got = ref.forward(x, w + 0.05, cos, sin, pos, False, 1e-2)[0]
    with pytest.raises(AssertionError):
        ref.within(got, want, bound)


def test_append_skips_what_is_no_token():
    B, Hkv, Sq, D, page = 2, 1, 3, 32, 16
    k = torch.randn((B, Hkv, Sq, D))
    table = torch.tensor([[1, 9], [0, -1]])
    pages = torch.zeros((3, Hkv, page, D))
    *_, where = ref.append(pages, pages, None, k, k, None, None, None, None, None, [17, 2], [3, 3], table, False, 0.0)
    assert where == [(0, 0, 1, 14), (0, 1, 1, 15), (1, 1, 0, 0), (1, 2, 0, 1)]  # page 9 and place -1 are left out
