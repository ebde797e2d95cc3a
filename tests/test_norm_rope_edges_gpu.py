"""attn_qk_norm_rope and its gradient where they can go wrong: weights that are not finite, rows of eps's
size, gradients written over the inputs, against the plain 64-bit forms with the error bounds of tests/rows_reference.py."""
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


@pytest.mark.parametrize("scale,eps", [(1e-3, 1e-6), (1.0, 0.5), (3e-2, 1e-5), (1e-3, 1e-2)])
@pytest.mark.parametrize("D,interleaved", [(32, False), (64, True), (128, False)])
def test_rows_of_the_size_of_eps(D, interleaved, scale, eps):
    """mean(x^2) next to eps or below it, and rows of zeros (0 / sqrt(eps) = 0; their gradient is w dy / sqrt(eps)).
    That these sizes tell where eps goes: tests/test_rows_eps.py."""
    B, Hq, Hkv, S = 2, 6, 3, 21
    x, dz, w, cos, sin = make(B, Hq, Hkv, S, D, D, seed=D + int(1 / eps))
    x = [(t.float() * scale).to(torch.bfloat16) for t in x]
    for t in x:
        t[0, 1, 3] = 0
        t[1, :, 20] = 0
    at = torch.arange(S).expand(B, S)
    cu = lambda t: t.cuda()  # noqa: E731
    kw = dict(q_weight=w[0].cuda(), k_weight=w[1].cuda(), interleaved=interleaved, eps=eps)
    out = attn.attn_qk_norm_rope(*map(cu, x), cos.cuda(), sin.cuda(), **kw)
    back = attn.attn_qk_norm_rope_bwd(*map(cu, x), cos.cuda(), sin.cuda(), *map(cu, dz), **kw)
    for i in range(2):
        ref.within(out[i], *ref.forward(x[i], w[i], cos, sin, at, interleaved, eps), f"forward {i}")
        assert torch.all(out[i][0, 1, 3] == 0) and torch.all(out[i][1, :, 20] == 0)
        dx, bx, dw, bw = ref.backward(x[i], w[i], cos, sin, at, interleaved, eps, dz[i])
        ref.within(back[i], dx, bx, f"backward {i}")
        ref.within(back[2 + i], dw, bw, f"weight {i}")


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("scale,eps", [(1e-3, 1e-6), (1.0, 0.5)])
def test_append_of_rows_of_the_size_of_eps(scale, eps, fp8):
    B, Hq, Hkv, S, D, page = 2, 4, 2, 16, 128, 16
    x, _, w, cos, sin = make(B, Hq, Hkv, S, D, D, seed=77)
    q, k = ((t.float() * scale).to(torch.bfloat16) for t in x)
    k[0, 1, 3] = 0
    table = torch.arange(B, dtype=torch.int32).view(B, 1).cuda()
    lens = torch.full((B,), S, dtype=torch.int32).cuda()
    pages = [torch.zeros((B, Hkv, page, D), dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda") for _ in range(2)]
    coef = 2.0 ** -4
    scales = [torch.full((Hkv, D), coef).cuda() for _ in range(2)] if fp8 else []
    fn = attn.attn_append_paged_fp8 if fp8 else attn.attn_append_paged
    q_out = fn(k.cuda(), k.cuda(), cos.cuda(), sin.cuda(), *pages, *scales, table, lens, q=q.cuda(), q_weight=w[0].cuda(),
               k_weight=w[1].cuda(), eps=eps)
    at = torch.arange(S).expand(B, S)
    ref.within(q_out, *ref.forward(q, w[0], cos, sin, at, False, eps), "q")
    kz, kb = ref.forward(k, w[1], cos, sin, at, False, eps)
    if not fp8:
        ref.within(pages[0], kz, kb, "k")
        return
    # Half a step of e4m3 (2^-4 of the binade's start, 2^-10 among its subnormals), the quotient's rounding (u) and
    # the fp32 error of x (the bound without its bf16 part).
    t = kz / coef
    step = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6))) - 4)
    ref.within(pages[0].view(torch.float8_e4m3fn).float(), t.clamp(-448, 448),
               step + 2 * (kb - ref.BF16 * kz.abs()) / coef + ref.U * t.abs(), "k codes")


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("D,interleaved", [(32, False), (64, True), (128, False)])
def test_gradients_written_over_the_inputs(D, interleaved, norm):
    """dq may be q (and dk k) as well as dq_out: the same bits as in memory of their own."""
    B, Hq, Hkv, S = 3, 7, 2, 210
    x, dz, w, cos, sin = make(B, Hq, Hkv, S, D, D, seed=D + 1)
    q, k, dqo, dko = (t.cuda() for t in (*x, *dz))
    kw = dict(q_weight=w[0].cuda() if norm else None, k_weight=w[1].cuda() if norm else None, interleaved=interleaved)
    want = attn.attn_qk_norm_rope_bwd(q, k, cos.cuda(), sin.cuda(), dqo, dko, **kw)
    fused = torch.cat((q, k), dim=1).transpose(1, 2).contiguous()  # token-major, as a projection leaves it
    qv, kv = fused[:, :, :Hq].transpose(1, 2), fused[:, :, Hq:].transpose(1, 2)
    over = attn.attn_qk_norm_rope_bwd(qv, kv, cos.cuda(), sin.cuda(), dqo, dko, dq=qv, dk=kv, **kw)
    assert over[0] is qv and over[1] is kv
    for a, b in zip(over, want):
        assert a is None and b is None or torch.equal(a, b)
