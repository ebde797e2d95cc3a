"""That the bounds the norm's tests use tell where eps goes: planted mistakes in eps alone, on rows whose mean
square is of its size, leave the bounds of the forward, the gradient and the weights' gradient."""
import pytest
import torch

from tests import rows_reference as ref

EPS = 1e-6
MISTAKES = {
    "dropped": lambda x, eps: x.pow(2).mean(-1, keepdim=True).sqrt(),
    "outside the root": lambda x, eps: x.pow(2).mean(-1, keepdim=True).sqrt() + eps,
    "in the sum": lambda x, eps: ((x.pow(2).sum(-1, keepdim=True) + eps) / x.shape[-1]).sqrt(),
    "another value": lambda x, eps: (x.pow(2).mean(-1, keepdim=True) + 1e-5).sqrt(),
}


def rows(seed, scale):
    g = torch.Generator().manual_seed(seed)
    x, dz = (torch.randn((1, 2, 6, 32), generator=g) for _ in range(2))
    w = (1 + 0.3 * torch.randn((32,), generator=g)).to(torch.bfloat16)
    cos, sin = ref.angle_tables(6, 32)
    return (x * scale).to(torch.bfloat16), dz.to(torch.bfloat16), w, cos, sin, torch.arange(6)[None]


@pytest.mark.parametrize("mistake", MISTAKES)
def test_planted_mistakes_in_eps_leave_the_bounds(mistake, monkeypatch):
    x, dz, w, cos, sin, pos = rows(5, 1e-3)
    z, bz = ref.forward(x, w, cos, sin, pos, False, EPS)
    dx, bx, dw, bw = ref.backward(x, w, cos, sin, pos, False, EPS, dz)
    root = MISTAKES[mistake](x.double(), EPS)
    # The same formulas with the mistaken root: eps' = root^2 - mean(x^2), row by row.
    wrong = root.pow(2) - x.double().pow(2).mean(-1, keepdim=True)
    got = ref.forward(x, w, cos, sin, pos, False, wrong)[0]
    gdx, _, gdw, _ = ref.backward(x, w, cos, sin, pos, False, wrong, dz)
    for a, b, bound in ((got, z, bz), (gdx, dx, bx), (gdw, dw, bw)):
        with pytest.raises(AssertionError):
            ref.within(a, b, bound)


def test_at_ordinary_sizes_a_dropped_eps_would_pass():
    """Why the sizes above: beside a mean square near 1, an eps of 1e-6 is far below the rounding to bf16."""
    x, _, w, cos, sin, pos = rows(6, 1.0)
    ref.within(ref.forward(x, w, cos, sin, pos, False, 0.0)[0], *ref.forward(x, w, cos, sin, pos, False, EPS))
