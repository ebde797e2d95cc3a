"""attn_qk_norm_rope and its gradient on the GPU against the plain 64-bit forms, with the error bounds
derived in tests/rows_reference.py."""
import pytest
import torch

import oracle
from causal_attention_attn_b200 import attn, build
from tests import rows_reference as ref

pytestmark = pytest.mark.gpu
EPS = 1e-6


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


def make(B, Hq, Hkv, S, D, rot, seed, norm=True, max_pos=None, positions=False):
    """Head slices of one fused token-major projection (on the GPU), their gradients heads-major."""
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn((B, S, Hq + 2 * Hkv, D), generator=g).to(torch.bfloat16)
    qkv[..., ::5] *= 8
    w = [(1 + 0.2 * torch.randn((D,), generator=g)).to(torch.bfloat16) if norm else None for _ in range(2)]
    max_pos = max_pos or S + 3
    cos, sin = ref.angle_tables(max_pos, rot) if rot else (None, None)
    pos = torch.randint(0, max_pos, (B, S), generator=g).to(torch.int32) if positions else None
    dz = [torch.randn((B, H, S, D), generator=g).to(torch.bfloat16) for H in (Hq, Hkv)]
    return qkv, w, cos, sin, pos, dz


def cuda(t):
    return None if t is None else t.cuda()


def default_positions(pos, B, S):
    return pos if pos is not None else torch.arange(S).expand(B, S)


CASES = [
    # B, Hq, Hkv, S, D, rot, interleaved, norm, positions
    (2, 8, 2, 37, 128, 128, False, True, False),
    (2, 8, 2, 37, 128, 128, True, True, True),
    (1, 1, 1, 1, 128, 128, False, True, True),       # one row of q and one of k
    (16, 32, 8, 1, 128, 128, False, True, True),     # a decode step
    (3, 5, 3, 17, 64, 64, True, True, False),        # heads that do not divide, odd counts
    (3, 10, 2, 77, 64, 32, False, True, True),       # half of each head rotated
    (2, 7, 1, 19, 32, 32, False, True, False),
    (2, 3, 2, 33, 32, 16, True, True, True),         # one lane of two rotated
    (1, 4, 4, 65, 128, 80, False, True, False),      # five lanes of eight
    (2, 4, 2, 21, 128, 16, False, True, False),      # one lane of eight
    (2, 6, 2, 25, 128, 128, False, False, True),     # rotation only
    (2, 6, 2, 25, 64, 0, False, True, False),        # norm only
    (1, 2, 2, 9, 32, 0, True, False, False),         # neither: a copy
    (1, 32, 8, 1500, 128, 128, False, True, False),  # many blocks
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "b{}_hq{}_hkv{}_s{}_d{}_rot{}_il{:d}_n{:d}_p{:d}".format(*c))
def test_forward_and_backward(case):
    B, Hq, Hkv, S, D, rot, il, norm, positions = case
    qkv, w, cos, sin, pos, dz = make(B, Hq, Hkv, S, D, rot, seed=S + D + rot, norm=norm, positions=positions)
    dev = qkv.cuda()
    q, k = dev[:, :, :Hq].transpose(1, 2), dev[:, :, Hq:Hq + Hkv].transpose(1, 2)
    kw = dict(q_weight=cuda(w[0]), k_weight=cuda(w[1]), positions=cuda(pos), interleaved=il, eps=EPS)
    got = attn.attn_qk_norm_rope(q, k, cuda(cos), cuda(sin), **kw)
    grad = torch.full_like(dev, 7.0)  # dq and dk land in slices of a fused gradient; v's slice stays
    dq, dk = grad[:, :, :Hq].transpose(1, 2), grad[:, :, Hq:Hq + Hkv].transpose(1, 2)
    back = attn.attn_qk_norm_rope_bwd(q, k, cuda(cos), cuda(sin), dz[0].cuda(), dz[1].cuda(), dq=dq, dk=dk, **kw)
    torch.cuda.synchronize()
    at = default_positions(pos, B, S)
    for i, (lo, hi) in enumerate(((0, Hq), (Hq, Hq + Hkv))):
        x = qkv[:, :, lo:hi].transpose(1, 2)
        ref.within(got[i], *ref.forward(x, w[i], cos, sin, at, il, EPS), f"forward {i}")
        dx, bx, dw, bw = ref.backward(x, w[i], cos, sin, at, il, EPS, dz[i])
        ref.within(back[i], dx, bx, f"backward {i}")
        if norm:
            ref.within(back[2 + i], dw, bw, f"weight {i}")
        else:
            assert back[2 + i] is None
    assert torch.all(grad[:, :, Hq + Hkv:] == 7)
    if not norm and not rot:
        assert torch.equal(got[0].cpu(), qkv[:, :, :Hq].transpose(1, 2))


def test_positions_outside_the_tables_give_zeros():
    B, Hq, Hkv, S, D = 2, 4, 2, 12, 64
    qkv, w, cos, sin, _, dz = make(B, Hq, Hkv, S, D, D, seed=4, max_pos=10)
    pos = torch.arange(S, dtype=torch.int32).repeat(B, 1)  # 10 and 11 lie behind the tables
    pos[1, 3], pos[1, 4], pos[0, 0] = -1, 2 ** 31 - 1, -2 ** 31
    dev = qkv.cuda()
    q, k = dev[:, :, :Hq].transpose(1, 2), dev[:, :, Hq:Hq + Hkv].transpose(1, 2)
    # eps = 0 as well: a row that is left out must not bring 0 / 0 into the weight's sum.
    kw = dict(q_weight=w[0].cuda(), k_weight=w[1].cuda(), positions=pos.cuda(), eps=0.0)
    got = attn.attn_qk_norm_rope(q, k, cos.cuda(), sin.cuda(), **kw)
    back = attn.attn_qk_norm_rope_bwd(q, k, cos.cuda(), sin.cuda(), dz[0].cuda(), dz[1].cuda(), **kw)
    for i, (lo, hi) in enumerate(((0, Hq), (Hq, Hq + Hkv))):
        x = qkv[:, :, lo:hi].transpose(1, 2)
        ref.within(got[i], *ref.forward(x, w[i], cos, sin, pos, False, 0.0))
        dx, bx, dw, bw = ref.backward(x, w[i], cos, sin, pos, False, 0.0, dz[i])
        ref.within(back[i], dx, bx)
        ref.within(back[2 + i], dw, bw)
        assert torch.all(got[i][:, :, 10:] == 0) and torch.all(got[i][1, :, 3:5] == 0) and torch.all(got[i][0, :, 0] == 0)


def test_infinities_and_nans_stay_in_their_rows_and_channels():
    qkv, w, cos, sin, _, _ = make(1, 4, 2, 8, 128, 64, seed=5, norm=False)
    qkv[0, 2, 1, 100] = float("inf")    # behind rot_dim: passed through, its neighbours as well
    qkv[0, 3, 4, 5] = float("nan")      # turned with channel 37
    dev = qkv.cuda()
    q, k = dev[:, :, :4].transpose(1, 2), dev[:, :, 4:6].transpose(1, 2)
    got = attn.attn_qk_norm_rope(q, k, cos.cuda(), sin.cuda())
    clean = torch.nan_to_num(qkv, nan=0.0, posinf=0.0).cuda()
    want = attn.attn_qk_norm_rope(clean[:, :, :4].transpose(1, 2), clean[:, :, 4:6].transpose(1, 2), cos.cuda(), sin.cuda())
    assert torch.isinf(got[0][0, 1, 2, 100]) and torch.isnan(got[1][0, 0, 3, [5, 37]]).all()
    got[0][0, 1, 2, 100] = 0
    got[1][0, 0, 3, [5, 37]] = want[1][0, 0, 3, [5, 37]]
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # With a norm, an infinite element takes its own row with it and no other.
    ww = torch.ones((128,), dtype=torch.bfloat16).cuda()
    got = attn.attn_qk_norm_rope(q, k, cos.cuda(), sin.cuda(), q_weight=ww, k_weight=ww)
    want = attn.attn_qk_norm_rope(clean[:, :, :4].transpose(1, 2), clean[:, :, 4:6].transpose(1, 2), cos.cuda(), sin.cuda(),
                                  q_weight=ww, k_weight=ww)
    keep = torch.ones((1, 4, 8), dtype=torch.bool)
    keep[0, 1, 2] = False
    assert torch.equal(got[0].cpu()[keep], want[0].cpu()[keep])


def test_in_place_and_repeatable():
    B, Hq, Hkv, S, D = 2, 8, 2, 300, 128
    qkv, w, cos, sin, pos, dz = make(B, Hq, Hkv, S, D, D, seed=6, positions=True)
    dev = qkv.cuda()
    q, k = dev[:, :, :Hq].transpose(1, 2), dev[:, :, Hq:Hq + Hkv].transpose(1, 2)
    kw = dict(q_weight=w[0].cuda(), k_weight=w[1].cuda(), positions=pos.cuda())
    want = attn.attn_qk_norm_rope(q, k, cos.cuda(), sin.cuda(), **kw)
    again = dev.clone()
    qa, ka = again[:, :, :Hq].transpose(1, 2), again[:, :, Hq:Hq + Hkv].transpose(1, 2)
    attn.attn_qk_norm_rope(qa, ka, cos.cuda(), sin.cuda(), q_out=qa, k_out=ka, **kw)
    assert torch.equal(qa, want[0]) and torch.equal(ka, want[1])
    dqo, dko = dz[0].cuda(), dz[1].cuda()
    first = attn.attn_qk_norm_rope_bwd(q, k, cos.cuda(), sin.cuda(), dqo, dko, **kw)
    for _ in range(3):
        b = attn.attn_qk_norm_rope_bwd(q, k, cos.cuda(), sin.cuda(), dqo, dko, **kw)
        assert all(torch.equal(x, y) for x, y in zip(first, b))
    inplace = attn.attn_qk_norm_rope_bwd(q, k, cos.cuda(), sin.cuda(), dqo, dko, dq=dqo, dk=dko, **kw)
    assert all(torch.equal(x, y) for x, y in zip(first, inplace))


def test_strides_past_32_bits():
    """Rows more than 2^32 bytes apart: element offsets do not fit 32 bits."""
    D, S = 64, 3
    step = (1 << 31) // 2 + 64  # elements between rows
    big = torch.empty((2 * step + 2 * D,), dtype=torch.bfloat16, device="cuda")
    q = torch.as_strided(big, (1, 2, S, D), (8, D, step, 1))
    g = torch.Generator().manual_seed(8)
    x = torch.randn((1, 2, S, D), generator=g).to(torch.bfloat16)
    q.copy_(x)
    cos, sin = ref.angle_tables(S, D)
    w = torch.ones((D,), dtype=torch.bfloat16)
    got = attn.attn_qk_norm_rope(q, q, cos.cuda(), sin.cuda(), q_weight=w.cuda(), k_weight=w.cuda())
    for t in got:
        ref.within(t, *ref.forward(x, w, cos, sin, torch.arange(S)[None], False, EPS))


def test_other_stream_and_graph_replay():
    B, Hq, Hkv, S, D = 2, 8, 2, 64, 128
    qkv, w, cos, sin, pos, dz = make(B, Hq, Hkv, S, D, D, seed=9)
    dev, other = qkv.cuda(), (qkv * 2 + 1).cuda()
    cos, sin, wq, wk, dqo, dko = cos.cuda(), sin.cuda(), w[0].cuda(), w[1].cuda(), dz[0].cuda(), dz[1].cuda()

    def step(x, stream=None):
        q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hkv].transpose(1, 2)
        kw = dict(q_weight=wq, k_weight=wk, stream=stream)
        return (*attn.attn_qk_norm_rope(q, k, cos, sin, **kw),
                *attn.attn_qk_norm_rope_bwd(q, k, cos, sin, dqo, dko, **kw))

    want, want_other = step(dev), step(other)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(dev, stream=side)  # the current stream stays the default one
    both = step(other)            # overlaps it: each call has a workspace of its own
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a, b) for a, b in zip(both, want_other))
    static = dev.clone()
    graphs, outs = [], []
    with torch.cuda.stream(side):
        for _ in range(2):  # two graphs, replayed in turn and out of order
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=side):
                outs.append(step(static))
            graphs.append(gr)
    side.synchronize()
    for x, expect in ((other, want_other), (dev, want)):
        static.copy_(x)
        torch.cuda.synchronize()
        for i in (1, 0, 1):
            graphs[i].replay()
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(a, b) for a, b in zip(o, expect))


def test_training_step_with_attention():
    """Norm and rotation, attention, its gradient, and the gradient back to the projection, against the
    64-bit chain. The tolerance is the attention gradients' own (1e-2 and 1e-3 of the largest value),
    which the bf16 rounding of the rotated q, k (2^-8) and of dq, dk adds to: twice it."""
    B, Hq, Hkv, S, D = 1, 4, 2, 200, 128
    qkv, w, cos, sin, _, _ = make(B, Hq, Hkv, S, D, D, seed=10)
    qkv[..., ::5] /= 8
    dout = torch.randn((B, Hq, S, D), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    dev = qkv.cuda()
    q, k, v = (dev[:, :, a:b].transpose(1, 2) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    kw = dict(q_weight=w[0].cuda(), k_weight=w[1].cuda())
    qr, kr = attn.attn_qk_norm_rope(q, k, cos.cuda(), sin.cuda(), **kw)
    vc = v.contiguous()
    o, lse = attn.attn_fwd(qr, kr, vc, causal=True)
    dqr, dkr, _ = attn.attn_bwd(qr, kr, vc, o, lse, dout.cuda(), causal=True)
    dq, dk, dwq, dwk = attn.attn_qk_norm_rope_bwd(q, k, cos.cuda(), sin.cuda(), dqr, dkr, **kw)
    at = torch.arange(S)[None]
    xs = [qkv[:, :, a:b].transpose(1, 2) for a, b in ((0, Hq), (Hq, Hq + Hkv))]
    z = [ref.forward(x, ww, cos, sin, at, False, EPS)[0].to(torch.bfloat16) for x, ww in zip(xs, w)]
    rdq, rdk, _ = oracle.attention_bwd(z[0], z[1], qkv[:, :, Hq + Hkv:].transpose(1, 2).contiguous(), dout, D ** -0.5, True)
    for x, ww, dzz, got, gw in ((xs[0], w[0], rdq, dq, dwq), (xs[1], w[1], rdk, dk, dwk)):
        want, _, wantw, _ = ref.backward(x, ww, cos, sin, at, False, EPS, torch.from_numpy(dzz))
        for a, b in ((got, want), (gw, wantw)):
            err, top = (a.cpu().double() - b).abs(), b.abs().max()
            assert err.max() <= 2e-2 * top and err.mean() <= 2e-3 * top


def test_refusals():
    x = torch.zeros((1, 4, 8, 64), dtype=torch.bfloat16, device="cuda")
    cos, sin = (t.cuda() for t in ref.angle_tables(8, 64))
    with pytest.raises(ValueError, match="tables rotate"):
        attn.attn_qk_norm_rope(x[..., :32].contiguous(), x[..., :32].contiguous(), cos, sin)
    with pytest.raises(ValueError, match="positions"):
        attn.attn_qk_norm_rope(x, x, cos, sin, positions=torch.zeros((1, 7), dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="contiguous last"):
        attn.attn_qk_norm_rope(x.transpose(2, 3), x, cos, sin)
    with pytest.raises(ValueError, match="live on"):
        attn.attn_qk_norm_rope(x, x, cos, sin.cpu())
    with pytest.raises(attn.AttnError) as e:
        attn.attn_qk_norm_rope(x, x, cos[:, :30].contiguous(), sin[:, :30].contiguous())
    assert e.value.status == -14
    with pytest.raises(attn.AttnError) as e:
        attn.attn_qk_norm_rope(x[:, :1].expand(1, 4, 8, 64), x, cos, sin)  # a broadcast head: stride 0
    assert e.value.status == -5
    with pytest.raises(attn.AttnError) as e:
        attn.attn_qk_norm_rope(x, x, cos, sin, q_weight=torch.ones(64, dtype=torch.bfloat16, device="cuda"))
    assert e.value.status == -1
    for one in ("q_weight", "k_weight"):
        with pytest.raises(attn.AttnError) as e:
            attn.attn_qk_norm_rope_bwd(x, x, cos, sin, x, x, **{one: torch.ones(64, dtype=torch.bfloat16, device="cuda")})
        assert e.value.status == -1
