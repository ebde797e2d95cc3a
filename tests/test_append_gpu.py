"""attn_append_paged and attn_append_paged_fp8 on the GPU against the plain 64-bit form
(tests/rows_reference.py): the rows written, the rows left alone, and the attention that reads them."""
import pytest
import torch

import oracle
from causal_attention_attn_b200 import attn, build
from tests import rows_reference as ref
from tests.compare import compare

pytestmark = pytest.mark.gpu
EPS = 1e-6
D = 128


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
    assert attn.device_status() == 0


def cuda(t):
    return None if t is None else t.cuda()


def e4m3(codes):
    return codes.cpu().view(torch.float8_e4m3fn).float().double()


def make(B, Hq, Hkv, Sq, page, per, seed, norm, rot, fp8, max_pos):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn((B, Sq, Hq + 2 * Hkv, D), generator=g).to(torch.bfloat16)
    qkv[..., ::7] *= 6
    w = [(1 + 0.2 * torch.randn((D,), generator=g)).to(torch.bfloat16) if norm else None for _ in range(2)]
    n_pages = B * per + 2
    table = torch.randperm(n_pages, generator=g)[:B * per].view(B, per).to(torch.int32)
    if fp8:
        pages = [torch.randint(0, 127, (n_pages, Hkv, page, D), generator=g).to(torch.uint8) for _ in range(2)]
        coef = [(0.5 + torch.rand((Hkv, D), generator=g)) / 64 for _ in range(2)]
        coef[1][:, :4] /= 64  # some channels saturate
    else:
        pages = [torch.randn((n_pages, Hkv, page, D), generator=g).to(torch.bfloat16) for _ in range(2)]
        coef = [None, None]
    cos, sin = ref.angle_tables(max_pos, rot) if rot else (None, None)
    return qkv, w, pages, coef, table, cos, sin, g


def check(k_pages, v_pages, pages, coef, expect):
    """The pages after the call: the rows `expect` names as computed, every other byte as it was."""
    _, _, kz, kb, vz, where = expect
    new = [k_pages.cpu(), v_pages.cpu()]
    fp8 = coef[0] is not None
    keep = torch.ones(pages[0].shape[:1] + pages[0].shape[2:3], dtype=torch.bool)
    for n, (b, i, pg, slot) in enumerate(where):
        keep[pg, slot] = False
        if fp8:
            # Half a step of e4m3 (2^-4 of the binade's start, 2^-10 among its subnormals), the quotient's
            # 2 units in the last place (4 u) and, for a key, the fp32 error of x.
            for x, err, cf, now, what in ((kz[n], kb[n] - ref.BF16 * kz[n].abs(), coef[0], new[0], "k"),
                                          (vz[n].double(), torch.zeros_like(kz[n]), coef[1], new[1], "v")):
                t = x / cf.double()
                step = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6))) - 4)
                ref.within(e4m3(now[pg, :, slot]), t.clamp(-448, 448), step + 2 * err.clamp(min=0) / cf + 4 * ref.U * t.abs(),
                           f"{what} row {n}")
        else:
            ref.within(new[0][pg, :, slot], kz[n], kb[n], f"k row {n}")
            assert torch.equal(new[1][pg, :, slot], vz[n]), f"v row {n}"
    for old, now in zip(pages, new):
        m = keep[:, None, :, None].expand(old.shape)
        assert torch.equal(old[m].view(torch.uint8), now[m].view(torch.uint8)), "a slot that no token names has changed"


CASES = [
    # B, Hq, Hkv, Sq, page, pages_per_seq, lengths, new_lens, norm, rot, interleaved, positions
    (4, 32, 8, 1, 64, 5, [1, 64, 65, 320], None, True, 128, False, False),     # decode, page borders
    (3, 8, 8, 1, 16, 4, [17, 1, 64], None, False, 128, True, False),
    (3, 6, 2, 20, 16, 6, [20, 96, 50], [20, 7, 0], True, 128, False, False),   # ragged: one brings nothing
    (2, 4, 1, 33, 128, 2, [33, 10], None, True, 64, False, True),              # a length below Sq
    (2, 4, 2, 9, 256, 1, [9, 250], [100, -3], False, 0, False, False),         # new_lens out of range
    (5, 16, 4, 3, 32, 2, [3, 66, 64, 0, -7], None, True, 128, True, False),    # past the table, empty, negative
    (2, 0, 3, 40, 16, 8, [40, 128], None, True, 128, False, True),             # keys and values only
    (1, 1, 1, 700, 64, 16, [1000], None, True, 128, False, False),
]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "b{}_hq{}_hkv{}_sq{}_page{}".format(*c[:5]))
def test_append(case, fp8):
    B, Hq, Hkv, Sq, page, per, lens, new, norm, rot, il, positions = case
    qkv, w, pages, coef, table, cos, sin, g = make(B, Hq, Hkv, Sq, page, per, sum(map(abs, lens)) + Sq, norm, rot, fp8,
                                                   max_pos=page * per)
    pos = torch.randint(0, page * per, (B, Sq), generator=g).to(torch.int32) if positions else None
    if positions:
        pos[0, 1], pos[-1, -1] = -1, page * per  # no row of the tables: left out
    q, k, v = (qkv[:, :, a:b].transpose(1, 2) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    dev = qkv.cuda()
    dq, dk, dv = (dev[:, :, a:b].transpose(1, 2) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    kp, vp = pages[0].cuda(), pages[1].cuda()
    kw = dict(q=dq if Hq else None, q_weight=cuda(w[0]) if Hq else None, k_weight=cuda(w[1]), positions=cuda(pos),
              new_lens=None if new is None else torch.tensor(new, dtype=torch.int32).cuda(), interleaved=il, eps=EPS)
    lens_t = torch.tensor(lens, dtype=torch.int32).cuda()
    if fp8:
        got = attn.attn_append_paged_fp8(dk, dv, cuda(cos), cuda(sin), kp, vp, coef[0].cuda(), coef[1].cuda(),
                                         table.cuda(), lens_t, **kw)
    else:
        got = attn.attn_append_paged(dk, dv, cuda(cos), cuda(sin), kp, vp, table.cuda(), lens_t, **kw)
    torch.cuda.synchronize()
    expect = ref.append(pages[0], pages[1], q if Hq else None, k, v, w[0], w[1], cos, sin, pos, lens, new, table, il, EPS)
    check(kp, vp, pages, coef, expect)
    if Hq:
        ref.within(got, expect[0], expect[1], "q_out")
    else:
        assert got is None


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_bad_table_entries_write_nothing(fp8):
    B, Hq, Hkv, Sq, page, per = 2, 4, 8, 40, 16, 3
    qkv, w, pages, coef, table, cos, sin, _ = make(B, Hq, Hkv, Sq, page, per, 3, True, 128, fp8, 64)
    table[0, 1], table[1, 0], table[1, 2] = -1, pages[0].shape[0], (1 << 29) + 3  # the last wraps onto page 3
    lens = [40, 48]
    dev = qkv.cuda()
    q, k, v = (qkv[:, :, a:b].transpose(1, 2) for a, b in ((0, 4), (4, 12), (12, 20)))
    dq, dk, dv = (dev[:, :, a:b].transpose(1, 2) for a, b in ((0, 4), (4, 12), (12, 20)))
    kp, vp = pages[0].cuda(), pages[1].cuda()
    args = (table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    kw = dict(q=dq, q_weight=w[0].cuda(), k_weight=w[1].cuda())
    if fp8:
        got = attn.attn_append_paged_fp8(dk, dv, cos.cuda(), sin.cuda(), kp, vp, coef[0].cuda(), coef[1].cuda(), *args, **kw)
    else:
        got = attn.attn_append_paged(dk, dv, cos.cuda(), sin.cuda(), kp, vp, *args, **kw)
    expect = ref.append(pages[0], pages[1], q, k, v, w[0], w[1], cos, sin, None, lens, None, table, False, EPS)
    assert 0 < len(expect[5]) < B * Sq
    check(kp, vp, pages, coef, expect)
    ref.within(got, expect[0], expect[1], "q_out")


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_two_tokens_of_one_slot(fp8):
    """Two sequences that share a page: every 16 bytes (e4m3: 8) of the slot are one token's or the other's."""
    B, Hkv, page = 2, 8, 16
    qkv, w, pages, coef, table, cos, sin, g = make(B, 0, Hkv, 1, page, 1, 31, True, 128, fp8, max_pos=page)
    k, v = qkv[:, :, :Hkv].transpose(1, 2).cuda(), qkv[:, :, Hkv:].transpose(1, 2).cuda()
    fn = attn.attn_append_paged_fp8 if fp8 else attn.attn_append_paged
    scales = [c.cuda() for c in coef] if fp8 else []
    lens = torch.tensor([4, 4], dtype=torch.int32).cuda()

    def append(tab):
        kp, vp = pages[0].cuda(), pages[1].cuda()
        fn(k, v, cos.cuda(), sin.cuda(), kp, vp, *scales, torch.tensor(tab, dtype=torch.int32).cuda(), lens, k_weight=w[1].cuda())
        return kp.cpu(), vp.cpu()

    apart, same = append([[0], [1]]), append([[1], [1]])
    for one, two in zip(apart, same):
        a, b, c = (t.contiguous().view(torch.uint8).view(Hkv, -1, 8 if fp8 else 16) for t in (one[0, :, 3], one[1, :, 3], two[1, :, 3]))
        assert torch.all((c == a).all(-1) | (c == b).all(-1))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_padding_may_hold_anything(fp8):
    B, Hq, Hkv, Sq, page = 3, 4, 2, 12, 16
    qkv, w, pages, coef, table, cos, sin, g = make(B, Hq, Hkv, Sq, page, 2, 32, True, 128, fp8, max_pos=32)
    new = [5, 0, 12]
    fn = attn.attn_append_paged_fp8 if fp8 else attn.attn_append_paged
    scales = [c.cuda() for c in coef] if fp8 else []
    res = []
    for fill in (float("nan"), 1.0):
        t = qkv.clone()
        for b in range(B):
            t[b, :Sq - new[b]] = fill
        t = t.cuda()
        q, k, v = (t[:, :, a:b].transpose(1, 2) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
        kp, vp = pages[0].cuda(), pages[1].cuda()
        q_out = fn(k, v, cos.cuda(), sin.cuda(), kp, vp, *scales, table.cuda(), torch.tensor([20, 12, 31], dtype=torch.int32).cuda(),
                   q=q, q_weight=w[0].cuda(), k_weight=w[1].cuda(), new_lens=torch.tensor(new, dtype=torch.int32).cuda())
        for b in range(B):
            assert torch.all(q_out[b, :, :Sq - new[b]] == 0)
        res.append([x.cpu().view(torch.uint8) for x in (q_out, kp, vp)])
    assert all(torch.equal(a, b) for a, b in zip(*res))


def test_e4m3_special_values():
    """NaN stays NaN, infinities and large values saturate, ties go to the even code."""
    k = torch.zeros((1, 1, 1, D), dtype=torch.bfloat16)
    vals = torch.tensor([float("nan"), float("inf"), float("-inf"), 1e30, 448.0, 464.0, 465.0, 17.0, 19.0, 2.0 ** -10,
                         3 * 2.0 ** -10, 0.0, -0.0, -2.0 ** -9], dtype=torch.bfloat16)
    k[0, 0, 0, :len(vals)] = vals
    kp = torch.zeros((1, 1, 16, D), dtype=torch.uint8, device="cuda")
    vp = kp.clone()
    one = torch.ones((1, D), device="cuda")
    attn.attn_append_paged_fp8(k.cuda(), k.cuda(), None, None, kp, vp, one, one,
                               torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                               torch.ones((1,), dtype=torch.int32, device="cuda"))
    want = [float("nan"), 448, -448, 448, 448, 448, 448, 16, 20, 0, 2.0 ** -8, 0, 0, -2.0 ** -9]
    for p in (kp, vp):
        got = e4m3(p[0, 0, 0, :len(vals)])
        assert torch.isnan(got[0]) and got[1:].tolist() == want[1:], got


def test_slots_past_32_bits():
    """A cache of more than 2^32 bytes: page offsets do not fit 32 bits."""
    Hkv, page, n_pages = 8, 128, 17000  # 4.46 GB of bf16 each
    kp = torch.empty((n_pages, Hkv, page, D), dtype=torch.bfloat16, device="cuda")
    vp = torch.empty((n_pages, Hkv, page, D), dtype=torch.bfloat16, device="cuda")
    kp[-2:], vp[-2:] = 1.0, 2.0
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn((1, Hkv, 3, D), generator=g).to(torch.bfloat16) for _ in range(2))
    table = torch.tensor([[n_pages - 2, n_pages - 1]], dtype=torch.int32, device="cuda")
    attn.attn_append_paged(k.cuda(), v.cuda(), None, None, kp, vp, table, torch.tensor([130], dtype=torch.int32, device="cuda"))
    assert torch.equal(kp[-2, :, 127].cpu(), k[0, :, 0]) and torch.equal(kp[-1, :, :2].cpu(), k[0, :, 1:])
    assert torch.equal(vp[-2, :, 127].cpu(), v[0, :, 0]) and torch.equal(vp[-1, :, :2].cpu(), v[0, :, 1:])
    assert torch.all(kp[-2, :, :127] == 1) and torch.all(kp[-1, :, 2:] == 1)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_decode_steps_through_a_graph(fp8):
    """Prompt appended and attended to, then five decode steps (append, attention) replayed from one
    graph with the lengths advanced on the device, against the oracle over the cache's own rows."""
    B, Hq, Hkv, page, per, prompt = 2, 8, 2, 16, 5, 37
    qkv, w, pages, coef, table, cos, sin, g = make(B, Hq, Hkv, prompt, page, per, 21, True, 128, fp8, page * per)
    if fp8:
        coef = [torch.full((Hkv, D), 2.0 ** -4) for _ in range(2)]
    kp, vp, tab = pages[0].cuda(), pages[1].cuda(), table.cuda()
    cosd, sind, wq, wk = cos.cuda(), sin.cuda(), w[0].cuda(), w[1].cuda()
    cd = [cuda(c) for c in coef]
    lens = torch.full((B,), prompt, dtype=torch.int32, device="cuda")

    def append(x):
        q, k, v = (x[:, :, a:b].transpose(1, 2) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
        kw = dict(q=q, q_weight=wq, k_weight=wk)
        if fp8:
            return attn.attn_append_paged_fp8(k, v, cosd, sind, kp, vp, *cd, tab, lens, **kw)
        return attn.attn_append_paged(k, v, cosd, sind, kp, vp, tab, lens, **kw)

    def decode(q):
        if fp8:
            return attn.attn_decode_paged_fp8(q, kp, vp, *cd, tab, lens, page * per)
        return attn.attn_decode_paged(q, kp, vp, tab, lens, page * per)

    append(qkv.cuda())
    x = torch.zeros((B, 1, Hq + 2 * Hkv, D), dtype=torch.bfloat16, device="cuda")
    decode(append(x))  # the attention's workspace is in place before the capture
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        lens.add_(1)
        qo = append(x)
        o, lse = decode(qo)
    for step in range(5):
        x.copy_(torch.randn(x.shape, generator=g).to(torch.bfloat16))
        gr.replay()
        torch.cuda.synchronize()
        n = prompt + 1 + step
        assert lens.tolist() == [n] * B
        for b in range(B):
            rows = [(kp if not fp8 else kp.view(torch.float8_e4m3fn)), (vp if not fp8 else vp.view(torch.float8_e4m3fn))]
            kk, vv = (r.cpu().float()[table[b].long()].transpose(0, 1).reshape(Hkv, -1, D)[:, :n] for r in rows)
            if fp8:
                kk, vv = kk * coef[0][:, None], vv * coef[1][:, None]
            kk, vv = kk.to(torch.bfloat16)[None], vv.to(torch.bfloat16)[None]  # exact: codes times a power of two
            rep = compare(o[b:b + 1], lse[b:b + 1], *oracle.attention(qo[b:b + 1].cpu(), kk, vv, D ** -0.5, True))
            # The bounds of tests/compare.py, O's relative to the values it averages.
            assert rep.lse_max_abs <= 1e-3 and rep.o_max_abs <= 1e-2 * max(1.0, float(vv.float().abs().max())), rep


def test_a_dense_cache_is_one_page_a_sequence():
    """Tokens appended one by one to [B, Hkv, S, 128], then attn_fwd over it."""
    B, Hq, Hkv, S, steps = 3, 8, 2, 256, 3
    g = torch.Generator().manual_seed(41)
    cache = [torch.randn((B, Hkv, S, D), generator=g).to(torch.bfloat16) for _ in range(2)]
    dev = [t.cuda() for t in cache]
    table = torch.arange(B, dtype=torch.int32).view(B, 1).cuda()
    for n in range(steps):
        new = torch.randn((B, Hq + 2 * Hkv, 1, D), generator=g).to(torch.bfloat16)
        q, k, v = new.split((Hq, Hkv, Hkv), dim=1)
        at = S - steps + n
        lens = torch.full((B,), at + 1, dtype=torch.int32)
        attn.attn_append_paged(k.cuda(), v.cuda(), None, None, dev[0], dev[1], table, lens.cuda())
        cache[0][:, :, at], cache[1][:, :, at] = k[:, :, 0], v[:, :, 0]
    for old, now in zip(cache, dev):
        assert torch.equal(old, now.cpu())
    o, lse = attn.attn_fwd(q.cuda().contiguous(), dev[0], dev[1])
    torch.cuda.synchronize()
    assert compare(o.cpu(), lse.cpu(), *oracle.attention(q, *cache, D ** -0.5, True)).ok()


def test_in_place_queries_and_another_stream():
    B, Hq, Hkv, Sq, page, per = 2, 8, 2, 50, 64, 2
    qkv, w, pages, coef, table, cos, sin, _ = make(B, Hq, Hkv, Sq, page, per, 12, True, 128, False, 128)
    lens = torch.tensor([50, 90], dtype=torch.int32).cuda()
    res = []
    for inplace, stream in ((False, None), (True, torch.cuda.Stream())):
        dev = qkv.cuda()
        q, k, v = (dev[:, :, a:b].transpose(1, 2) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
        kp, vp, tab, wq, wk, c, s = (t.cuda() for t in (*pages, table, *w, cos, sin))
        torch.cuda.synchronize()
        out = attn.attn_append_paged(k, v, c, s, kp, vp, tab, lens, q=q, q_out=q if inplace else None, q_weight=wq,
                                     k_weight=wk, stream=stream)
        torch.cuda.synchronize()
        res.append((out.clone(), kp, vp))
    assert all(torch.equal(a, b) for a, b in zip(*res))


def test_refusals():
    z = torch.zeros((2, 2, 3, D), dtype=torch.bfloat16, device="cuda")
    pages = torch.zeros((4, 2, 16, D), dtype=torch.bfloat16, device="cuda")
    table, lens = torch.zeros((2, 2), dtype=torch.int32, device="cuda"), torch.ones((2,), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="expected k, v"):
        attn.attn_append_paged(z, z, None, None, pages[:, :1].contiguous(), pages[:, :1].contiguous(), table, lens)
    with pytest.raises(TypeError, match="k_pages"):
        attn.attn_append_paged(z, z, None, None, pages.to(torch.uint8), pages, table, lens)
    with pytest.raises(ValueError, match="one row"):
        attn.attn_append_paged(z, z, None, None, pages, pages, table[:1], lens)
    with pytest.raises(ValueError, match="new_lens"):
        attn.attn_append_paged(z, z, None, None, pages, pages, table, lens, new_lens=lens[:1])
    with pytest.raises(ValueError, match="k_scale"):
        codes = pages.to(torch.uint8)
        attn.attn_append_paged_fp8(z, z, None, None, codes, codes, torch.ones((1, D), device="cuda"),
                                   torch.ones((2, D), device="cuda"), table, lens)
    with pytest.raises(attn.AttnError) as e:
        p = torch.zeros((4, 2, 48, D), dtype=torch.bfloat16, device="cuda")
        attn.attn_append_paged(z, z, None, None, p, p, table, lens)
    assert e.value.status == -2
