"""Element offsets past 2^32: rows, heads and sequences 2^31 + 64 elements apart, so that the third lies behind
2^32 elements, for every tensor with strides; and cache pages behind 2^32 elements. Signed or unsigned 32-bit
index arithmetic would wrap. The tensors are columns of one buffer of 8.6 GB, of which only their rows are set."""
import pytest
import torch

from causal_attention_attn_b200 import attn, build
from tests import rows_reference as ref

pytestmark = pytest.mark.gpu
EPS = 1e-6
STEP = (1 << 31) + 64
WIDTH = 4096  # elements that the columns take


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
    torch.cuda.empty_cache()


@pytest.fixture(scope="module")
def big():
    return torch.empty((2 * STEP + WIDTH,), dtype=torch.bfloat16, device="cuda")


class Columns:
    """Tensors of three entries along `axis` (0 batch, 1 head, 2 row), STEP elements apart, side by side."""

    def __init__(self, big, axis, D):
        self.big, self.axis, self.D, self.at = big, axis, D, 0

    def take(self, other=1, values=None):
        """[B, H, S, D]: three along the axis, `other` heads (rows where the axis is the heads)."""
        shape, stride = [1, 1, 1, self.D], [8, 8, 8, 1]
        shape[self.axis], stride[self.axis] = 3, STEP
        second = 2 if self.axis == 1 else 1
        shape[second], stride[second] = other, self.D
        t = torch.as_strided(self.big, shape, stride, self.at)
        self.at += other * self.D
        assert self.at <= WIDTH
        if values is None:
            t.fill_(float("nan"))
        else:
            t.copy_(values(shape))
        return t


@pytest.mark.parametrize("axis", [0, 1, 2], ids=["batch", "head", "row"])
@pytest.mark.parametrize("D,interleaved", [(32, True), (64, False), (128, False)])
def test_norm_and_rotation_and_its_gradient(big, axis, D, interleaved):
    g = torch.Generator().manual_seed(D + axis)
    draw = lambda shape: torch.randn(shape, generator=g).to(torch.bfloat16)  # noqa: E731
    cols = Columns(big, axis, D)
    x, dz = [cols.take(2, draw) for _ in range(2)], [cols.take(2, draw) for _ in range(2)]
    out, dx = [cols.take(2) for _ in range(2)], [cols.take(2) for _ in range(2)]
    w = [(1 + 0.2 * draw((D,)).float()).to(torch.bfloat16) for _ in range(2)]
    cos, sin = ref.angle_tables(8, D)
    kw = dict(q_weight=w[0].cuda(), k_weight=w[1].cuda(), interleaved=interleaved, eps=EPS)
    attn.attn_qk_norm_rope(*x, cos.cuda(), sin.cuda(), q_out=out[0], k_out=out[1], **kw)
    back = attn.attn_qk_norm_rope_bwd(*x, cos.cuda(), sin.cuda(), *dz, dq=dx[0], dk=dx[1], **kw)
    B, _, S, _ = x[0].shape
    at = torch.arange(S).expand(B, S)
    for i in range(2):
        xc, dc = x[i].cpu(), dz[i].cpu()
        ref.within(out[i], *ref.forward(xc, w[i], cos, sin, at, interleaved, EPS), f"forward {i}")
        want, bound, dw, bw = ref.backward(xc, w[i], cos, sin, at, interleaved, EPS, dc)
        ref.within(dx[i], want, bound, f"backward {i}")
        ref.within(back[2 + i], dw, bw, f"weight {i}")


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("axis", [0, 1, 2], ids=["batch", "head", "row"])
def test_append(big, axis, fp8):
    """Strided q, k, v and q_out, to pages the last of which lie behind 2^32 elements of the cache."""
    D, page, g = 128, 128, torch.Generator().manual_seed(axis)
    draw = lambda shape: torch.randn(shape, generator=g).to(torch.bfloat16)  # noqa: E731
    cols = Columns(big, axis, D)
    q, k, v = (cols.take(2, draw) for _ in range(3))
    q_out = cols.take(2)
    B, Hkv, S, _ = k.shape
    n_pages = (1 << 32) // (Hkv * page * D) + 4
    pages = [torch.empty((n_pages, Hkv, page, D), dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda") for _ in range(2)]
    for t in pages:
        t[-4:] = 3
    table = torch.tensor([[n_pages - 4 + b] for b in range(B)], dtype=torch.int32)
    lens = [page - b for b in range(B)]
    cos, sin = ref.angle_tables(page, D)
    w = (1 + 0.2 * draw((D,)).float()).to(torch.bfloat16)
    coef = 2.0 ** -3
    scales = [torch.full((Hkv, D), coef).cuda() for _ in range(2)] if fp8 else []
    fn = attn.attn_append_paged_fp8 if fp8 else attn.attn_append_paged
    fn(k, v, cos.cuda(), sin.cuda(), *pages, *scales, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), q=q,
       q_out=q_out, q_weight=w.cuda(), k_weight=w.cuda(), eps=EPS)
    last = [t[-4:].cpu() for t in pages]
    fresh = [torch.full_like(t, 3) for t in last]
    near = table - (n_pages - 4)
    qz, qb, kz, kb, vz, where = ref.append(fresh[0], fresh[1], q.cpu(), k.cpu(), v.cpu(), w, w, cos, sin, None, lens, None, near,
                                           False, EPS)
    ref.within(q_out, qz, qb, "q_out")
    assert len(where) == B * S
    for n, (b, i, pg, slot) in enumerate(where):
        if fp8:
            # Half a step of e4m3 (2^-4 of the binade's start, 2^-10 among its subnormals), the quotient's
            # rounding (u) and, for a key, the fp32 error of x. A value's code is exact.
            t = kz[n] / coef
            step = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6))) - 4)
            ref.within(last[0][pg, :, slot].view(torch.float8_e4m3fn).float(), t.clamp(-448, 448),
                       step + 2 * (kb[n] - ref.BF16 * kz[n].abs()) / coef + ref.U * t.abs(), "k")
            code = (vz[n].float() / coef).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            assert torch.equal(last[1][pg, :, slot], code)
        else:
            ref.within(last[0][pg, :, slot], kz[n], kb[n], "k")
            assert torch.equal(last[1][pg, :, slot], vz[n])
        last[0][pg, :, slot] = last[1][pg, :, slot] = 3
    assert all(torch.equal(t, f) for t, f in zip(last, fresh)), "a slot that no token names has changed"
