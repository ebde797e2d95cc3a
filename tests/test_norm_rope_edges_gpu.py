"""attn_qk_norm_rope and its gradient where they can go wrong: weights that are not finite, against the plain
64-bit forms with the error bounds of tests/rows_reference.py."""
import pytest
import torch

from causal_attention_attn_b200 import attn, build
from tests import rows_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    if torch.cuda.get_device_capability(0) != (10, 0):
        pytest.skip("needs an sm_100 device")
    build.build()
    attn.load_library()
    yield
    torch.cuda.synchronize()


def make(B, Hq, Hkv, S, D, rot, seed):
    """q, k, their weights and gradients (on the CPU), and the tables."""
    g = torch.Generator().manual_seed(seed)
    x = [torch.randn((B, H, S, D), generator=g).to(torch.bfloat16) for H in (Hq, Hkv)]
    dz = [torch.randn((B, H, S, D), generator=g).to(torch.bfloat16) for H in (Hq, Hkv)]
    w = [(1 + 0.2 * torch.randn((D,), generator=g)).to(torch.bfloat16) for _ in range(2)]
    return x, dz, w, *ref.angle_tables(S + 3, rot)


@pytest.mark.parametrize("D,interleaved", [(32, False), (64, True), (128, False), (128, True)])
def test_rows_without_a_position_are_zeros_whatever_the_weights(D, interleaved):
    """A weight of infinity or NaN reaches the rows that have a position, and no other."""
    B, Hq, Hkv, S = 2, 5, 2, 9
    x, dz, w, cos, sin = make(B, Hq, Hkv, S, D, D // 2, seed=D)
    for t in w:
        t[1], t[D - 2] = float("inf"), float("nan")
    pos = torch.arange(S, dtype=torch.int32).repeat(B, 1)
    pos[0, ::2], pos[1, 3] = -1, S + 3
    gone = (pos < 0) | (pos >= S + 3)
    cu = lambda t: t.cuda()  # noqa: E731
    kw = dict(q_weight=w[0].cuda(), k_weight=w[1].cuda(), positions=pos.cuda(), interleaved=interleaved)
    out = attn.attn_qk_norm_rope(*map(cu, x), cos.cuda(), sin.cuda(), **kw)
    back = attn.attn_qk_norm_rope_bwd(*map(cu, x), cos.cuda(), sin.cuda(), *map(cu, dz), **kw)
    for t in (*out, *back[:2]):
        rows = t.cpu().transpose(1, 2)  # [B, S, H, D]
        assert torch.all(rows[gone] == 0)
        assert torch.isnan(rows[~gone]).any(-1).all()
    for i, (a, b) in enumerate(zip(x, dz)):  # the weights' gradient does not read the weights
        _, _, dw, bw = ref.backward(a, w[i], cos, sin, pos, interleaved, 1e-6, b)
        ref.within(back[2 + i], dw, bw)
