"""attn_decode_prefix on the GPU against the fp64 oracle: each sequence's token attends to the shared
prefix's keys and its own suffix's, both paged. Unused cache slots hold NaN. Tolerance: tests/compare.py's
for attention (O 1e-2 and 1e-3, LSE 1e-3)."""
import numpy as np
import pytest
import torch

import oracle
from causal_attention_attn_b200 import attn, build, inputs
from tests.compare import compare

pytestmark = pytest.mark.gpu
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
    assert attn.device_status() == 0, "a kernel-side wait ran out during the shared-prefix tests"


def make(B, Hq, Hkv, plen, lens, page, seed):
    """q, the dense prefix and suffixes, and the same keys scattered over random pages (NaN elsewhere)."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((B, Hq, 1, D), generator=g).to(torch.bfloat16)
    pre = [torch.randn((Hkv, plen, D), generator=g).to(torch.bfloat16) for _ in range(2)]
    cap = max(max(lens), 1)
    suf = [torch.randn((B, Hkv, cap, D), generator=g).to(torch.bfloat16) for _ in range(2)]
    n_pre, per = max(-(-plen // page), 1), -(-cap // page)
    n_pages = n_pre + B * per + 3
    perm = torch.randperm(n_pages, generator=g)
    pages = [torch.full((n_pages, Hkv, page, D), float("nan"), dtype=torch.bfloat16) for _ in range(2)]
    ptab, table = perm[:n_pre].to(torch.int32), perm[n_pre:n_pre + B * per].view(B, per).to(torch.int32)
    for which in range(2):
        for n in range(-(-plen // page)):
            part = pre[which][:, n * page:(n + 1) * page]
            pages[which][ptab[n], :, :part.shape[1]] = part
        for b in range(B):
            for n in range(-(-lens[b] // page)):
                part = suf[which][b, :, n * page:min((n + 1) * page, lens[b])]
                pages[which][table[b, n], :, :part.shape[1]] = part
    return q, pre, suf, pages, ptab, table


def expect(q, pre, suf, lens, b, scale, plen=None):
    plen = pre[0].shape[1] if plen is None else plen
    k, v = (torch.cat((p[:, :plen], s[b, :, :lens[b]]), dim=1)[None] for p, s in zip(pre, suf))
    return oracle.attention(q[b:b + 1], k, v, scale, True)


def call(q, pages, ptab, plen, table, lens, **kw):
    o, lse = attn.attn_decode_prefix(q.cuda(), pages[0].cuda(), pages[1].cuda(), ptab.cuda(),
                                     torch.tensor([plen], dtype=torch.int32).cuda(), table.cuda(),
                                     torch.tensor(lens, dtype=torch.int32).cuda(), **kw)
    torch.cuda.synchronize()
    return o.cpu(), lse.cpu()


CASES = [
    # B, Hq, Hkv, prefix, suffix lengths (int: that many at most, drawn), page
    (1, 1, 1, 1, [0], 16),                    # one key
    (2, 4, 1, 127, [1, 0], 16),
    (4, 32, 8, 512, [100, 1, 64, 0], 64),
    (3, 8, 8, 300, [0, 0, 0], 32),            # group 1, no suffixes
    (16, 32, 8, 4096, 256, 64),
    (33, 32, 8, 700, 70, 16),                 # one sequence in the second tile
    (5, 16, 1, 129, [128, 129, 127, 1, 300], 128),
    (70, 18, 6, 1000, 40, 128),               # groups of three: 126 rows to a tile, two tiles
    (100, 14, 2, 260, 20, 256),               # groups of seven
    (200, 8, 8, 640, 10, 64),                 # 128 sequences to a tile
    (140, 10, 2, 385, 5, 32),                 # six tiles: three lists a head
    (3, 130, 1, 200, [3, 0, 60], 16),         # a group above 128 heads, in two parts
    (2, 131, 1, 140, [7, 0], 16),             # a prime group: one head to a part
    (300, 4, 1, 64, 3, 16),                   # fewer units than CTAs
    (6, 32, 2, 5000, 33, 64),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "b{}_hq{}_hkv{}_p{}_page{}".format(*c[:4], c[5]))
def test_matches_oracle(case):
    B, Hq, Hkv, plen, lens, page = case
    if isinstance(lens, int):
        lens = [int(x) for x in np.random.RandomState(B).randint(0, lens + 1, size=B)]
    q, pre, suf, pages, ptab, table = make(B, Hq, Hkv, plen, lens, page, seed=B + plen)
    o, lse = call(q, pages, ptab, plen, table, lens, max_prefix_len=plen, max_seq_len=max(lens))
    for b in range(B):
        rep = compare(o[b:b + 1], lse[b:b + 1], *expect(q, pre, suf, lens, b, D ** -0.5))
        assert rep.ok(), f"sequence {b} (suffix {lens[b]}): {rep}"


def widen(t, entries):
    """A table with room for far more pages than there are; the entries behind the real ones name page 0."""
    return torch.cat((t, t.new_zeros(t.shape[:-1] + (entries - t.shape[-1],))), dim=-1)


@pytest.mark.parametrize("case", CASES + [
    (150, 8, 2, 900, [0, 300, 1, 17, 0] * 30, 16),   # short and long suffixes side by side, and none
    (40, 20, 1, 1500, [250, 3, 0, 90] * 10, 64),     # more than eight heads to a pair
    (1, 8, 8, 9000, [5000], 128),
    (9, 32, 8, 0, [40] * 9, 16),
], ids=lambda c: "b{}_hq{}_hkv{}_p{}_page{}".format(*c[:4], c[5]))
def test_lengths_far_below_the_bounds(case):
    """Such a call's split between prefix and suffixes is worked out on the device, from its real lengths."""
    B, Hq, Hkv, plen, lens, page = case
    if isinstance(lens, int):
        lens = [int(x) for x in np.random.RandomState(B).randint(0, lens + 1, size=B)]
    q, pre, suf, pages, ptab, table = make(B, Hq, Hkv, plen, lens, page, seed=B + plen)
    big = 4 << 20
    o, lse = call(q, pages, widen(ptab, big // page), plen, widen(table, 65536 // page), lens, max_prefix_len=big,
                  max_seq_len=65536)
    for b in range(B):
        rep = compare(o[b:b + 1], lse[b:b + 1], *expect(q, pre, suf, lens, b, D ** -0.5))
        assert rep.ok(), f"sequence {b} (suffix {lens[b]}): {rep}"


def test_empty_prefix_and_empty_sequences():
    B, Hq, Hkv, lens, page = 3, 8, 2, [70, 0, 5], 16
    q, pre, suf, pages, ptab, table = make(B, Hq, Hkv, 64, lens, page, seed=1)
    for plen, bound in ((0, 64), (-3, 64), (0, 0)):
        o, lse = call(q, pages, ptab, plen, table, lens, max_prefix_len=bound, max_seq_len=70)
        assert torch.all(o[1] == 0) and torch.all(torch.isneginf(lse[1]))
        for b in (0, 2):
            rep = compare(o[b:b + 1], lse[b:b + 1], *expect(q, pre, suf, lens, b, D ** -0.5, plen=0))
            assert rep.ok(), rep
    o, lse = call(q, pages, ptab, 0, table, [0, 0, 0], max_prefix_len=64, max_seq_len=0)
    assert torch.all(o == 0) and torch.all(torch.isneginf(lse))


def test_lengths_beyond_the_tables_and_bounds_are_clamped():
    B, Hq, Hkv, lens, page = 2, 8, 2, [48, 20], 16
    q, pre, suf, pages, ptab, table = make(B, Hq, Hkv, 96, lens, page, seed=2)
    o, lse = call(q, pages, ptab, 10 ** 9, table, [10 ** 9, 20], max_prefix_len=10 ** 9, max_seq_len=10 ** 9)
    o2, lse2 = call(q, pages, ptab, 96, table, [48, 20], max_prefix_len=50, max_seq_len=30)
    for b in range(B):
        assert compare(o[b:b + 1], lse[b:b + 1], *expect(q, pre, suf, [48, 20], b, D ** -0.5)).ok()
        assert compare(o2[b:b + 1], lse2[b:b + 1], *expect(q, pre, suf, [30, 20], b, D ** -0.5, plen=50)).ok()


def test_a_shorter_prefix_than_the_bound():
    """The plan is made for the bound; the length is read on the device (some CTAs then have no unit)."""
    B, Hq, Hkv, page = 9, 32, 8, 64
    lens = [3] * B
    q, pre, suf, pages, ptab, table = make(B, Hq, Hkv, 200, lens, page, seed=3)
    o, lse = call(q, pages, ptab, 200, table, lens, max_prefix_len=100000, max_seq_len=1000)
    for b in range(B):
        rep = compare(o[b:b + 1], lse[b:b + 1], *expect(q, pre, suf, lens, b, D ** -0.5))
        assert rep.ok(), rep


def test_table_entries_outside_the_pages_read_as_zeros():
    B, Hq, Hkv, page, lens = 2, 8, 4, 64, [100, 64]
    q, pre, suf, pages, ptab, table = make(B, Hq, Hkv, 300, lens, page, seed=4)
    ptab[1], ptab[3], table[0, 1] = -1, (1 << 30) + 1, pages[0].shape[0]
    o, lse = call(q, pages, ptab, 300, table, lens, max_prefix_len=300, max_seq_len=100)
    for t in pre:
        t[:, 64:128], t[:, 192:256] = 0, 0
    for t in suf:
        t[0, :, 64:100] = 0
    for b in range(B):
        rep = compare(o[b:b + 1], lse[b:b + 1], *expect(q, pre, suf, lens, b, D ** -0.5))
        assert rep.ok(), rep


def test_scales_and_outliers():
    """Keys that dominate late in the prefix, or only in a suffix; scales other than 1/sqrt(D). V is
    scaled by 1/4, so that half a bf16 step of O stays below the bound."""
    B, Hq, Hkv, page, lens = 8, 8, 2, 32, [40] * 8
    q, pre, suf, pages, ptab, table = make(B, Hq, Hkv, 900, lens, page, seed=5)
    pages[1] /= 4
    pre[1], suf[1] = pre[1] / 4, suf[1] / 4
    for j in (0, 500, 899):
        pre[0][:, j] *= 8
        pages[0][ptab[j // page], :, j % page] *= 8
    suf[0][3, :, 39] *= 8
    pages[0][table[3, 1], :, 7] *= 8
    for scale in (0.02, 0.3, 1.5):
        o, lse = call(q, pages, ptab, 900, table, lens, max_prefix_len=900, max_seq_len=40, scale=scale)
        for b in range(B):
            rep = compare(o[b:b + 1], lse[b:b + 1], *expect(q, pre, suf, lens, b, scale))
            assert rep.ok(), (scale, rep)


def test_one_sequences_nan_stays_its_own():
    B, Hq, Hkv, page, lens = 6, 8, 2, 16, [20] * 6
    q, pre, suf, pages, ptab, table = make(B, Hq, Hkv, 200, lens, page, seed=6)
    want, want_l = call(q, pages, ptab, 200, table, lens, max_prefix_len=200, max_seq_len=20)
    q[2, 1] = float("nan")                       # a query: its own row
    pages[1][table[4, 0], 1, 3] = float("inf")   # a value of a suffix: its sequence and kv head
    pages[0][table[5, 1], 0, 2] = float("nan")
    o, lse = call(q, pages, ptab, 200, table, lens, max_prefix_len=200, max_seq_len=20)
    keep = torch.ones((B, Hq), dtype=torch.bool)
    keep[2, 1], keep[4, 4:], keep[5, :4] = False, False, False
    assert torch.equal(o[keep], want[keep]) and torch.equal(lse[keep], want_l[keep])
    assert torch.isnan(o[2, 1]).all() and torch.isnan(o[5, :4]).all() and not torch.isfinite(o[4, 4:]).any()


def test_keys_of_score_minus_infinity():
    """Keys with -inf where every query is positive have scores of -inf: weight 0. A whole KV tile of the
    prefix, a whole unit of a suffix, and in one sequence every key there is but the prefix's."""
    B, Hq, Hkv, page, lens = 3, 8, 2, 64, [40, 16, 33]
    q, pre, suf, pages, ptab, table = make(B, Hq, Hkv, 300, lens, page, seed=12)
    q[..., 0] = 1.0
    inf = float("-inf")
    drop_pre = range(0, 128)
    drop_suf = {0: range(16, 32), 1: range(0, 16)}
    for j in drop_pre:
        pages[0][ptab[j // page], :, j % page, 0] = inf
    for b, keys in drop_suf.items():
        for j in keys:
            pages[0][table[b, j // page], :, j % page, 0] = inf
    o, lse = call(q, pages, ptab, 300, table, lens, max_prefix_len=300, max_seq_len=40)
    for b in range(B):
        keep = [j for j in range(lens[b]) if j not in drop_suf.get(b, ())]
        k, v = (torch.cat((p[:, 128:], s[b, :, keep]), dim=1)[None] for p, s in zip(pre, suf))
        rep = compare(o[b:b + 1], lse[b:b + 1], *oracle.attention(q[b:b + 1], k, v, D ** -0.5, True))
        assert rep.ok(), (b, rep)


def test_agrees_with_the_paged_decode_and_repeats():
    """The same keys through attn_decode_paged, with the prefix's pages in every sequence's table."""
    B, Hq, Hkv, page, plen = 12, 32, 8, 64, 640
    lens = [int(x) for x in np.random.RandomState(7).randint(0, 200, size=B)]
    q, pre, suf, pages, ptab, table = make(B, Hq, Hkv, plen, lens, page, seed=7)
    o, lse = call(q, pages, ptab, plen, table, lens, max_prefix_len=plen, max_seq_len=200)
    again, lse_again = call(q, pages, ptab, plen, table, lens, max_prefix_len=plen, max_seq_len=200)
    assert torch.equal(o, again) and torch.equal(lse, lse_again)
    whole = torch.cat((ptab[None].expand(B, -1), table), dim=1).contiguous()
    o2, lse2 = attn.attn_decode_paged(q.cuda(), pages[0].cuda(), pages[1].cuda(), whole.cuda(),
                                      torch.tensor([plen + n for n in lens], dtype=torch.int32).cuda(), plen + 200)
    rep = compare(o, lse, o2.cpu().double().numpy(), lse2.cpu().double().numpy())
    assert rep.ok(), rep


def test_pages_past_32_bits():
    """Prefix pages behind the first 2^32 bytes of the cache."""
    Hq, Hkv, page, n_pages = 8, 8, 128, 17000
    q, pre, suf, pages, ptab, table = make(2, Hq, Hkv, 200, [30, 0], page, seed=8)
    big = [torch.zeros((n_pages, Hkv, page, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    n = pages[0].shape[0]
    for b, p in zip(big, pages):
        b[n_pages - n:] = p.cuda()
    args = [t.cuda() for t in (q, *big, ptab + (n_pages - n), torch.tensor([200], dtype=torch.int32),
                               table + (n_pages - n), torch.tensor([30, 0], dtype=torch.int32))]
    o, lse = attn.attn_decode_prefix(*args, max_prefix_len=200, max_seq_len=30)
    for b in range(2):
        rep = compare(o[b:b + 1].cpu(), lse[b:b + 1].cpu(), *expect(q, pre, suf, [30, 0], b, D ** -0.5))
        assert rep.ok(), rep


def test_streams_and_graphs():
    """Two calls at once on two streams (a workspace each), and a serving loop in a graph: append to the
    suffixes, decode over prefix and suffixes, lengths advanced on the device; a larger eager call
    between replays must not disturb the captured one."""
    B, Hq, Hkv, page, plen, per = 4, 8, 2, 16, 100, 4
    lens = [10, 1, 20, 0]
    q, pre, suf, pages, ptab, table = make(B, Hq, Hkv, plen, lens, page, seed=9)
    n_pages = pages[0].shape[0]
    spare = torch.arange(n_pages, n_pages + B * per, dtype=torch.int32).view(B, per)
    pages = [torch.cat((p, torch.full((B * per, Hkv, page, D), float("nan"), dtype=p.dtype))) for p in pages]
    table = torch.cat((table, spare), dim=1).contiguous()
    cap = table.shape[1] * page
    kp, vp, pt, tab = pages[0].cuda(), pages[1].cuda(), ptab.cuda(), table.cuda()
    plen_t, lens_t = torch.tensor([plen], dtype=torch.int32).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    qc, q2 = q.cuda(), (q * 0.5).cuda()
    ref1 = attn.attn_decode_prefix(qc, kp, vp, pt, plen_t, tab, lens_t, plen, cap)
    ref2 = attn.attn_decode_prefix(q2, kp, vp, pt, plen_t, tab, lens_t, plen, cap)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        a = attn.attn_decode_prefix(qc, kp, vp, pt, plen_t, tab, lens_t, plen, cap, stream=s1)
        b = attn.attn_decode_prefix(q2, kp, vp, pt, plen_t, tab, lens_t, plen, cap, stream=s2)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, ref1)) and all(torch.equal(x, y) for x, y in zip(b, ref2))

    ws = attn.decode_prefix_workspace(B, Hq, Hkv, plen, cap)
    cos, sin = (t.cuda() for t in (torch.ones((plen + cap, 64)), torch.zeros((plen + cap, 64))))  # no turn
    x = torch.zeros((B, Hq + 2 * Hkv, 1, D), dtype=torch.bfloat16, device="cuda")
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        lens_t.add_(1)
        pos = (plen + lens_t - 1).view(B, 1)
        qo = attn.attn_append_paged(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], cos, sin, kp, vp, tab, lens_t, q=x[:, :Hq],
                                    positions=pos)
        o, lse = attn.attn_decode_prefix(qo, kp, vp, pt, plen_t, tab, lens_t, plen, cap, workspace=ws)
    dense = [[s[b, :, :lens[b]] for s in suf] for b in range(B)]
    big = make(64, 32, 8, 500, [5] * 64, 16, seed=10)
    for step in range(3):
        new = torch.randn(x.shape, generator=torch.Generator().manual_seed(step)).to(torch.bfloat16)
        x.copy_(new)
        gr.replay()
        call(big[0], big[3], big[4], 500, big[5], [5] * 64, max_prefix_len=500, max_seq_len=5)
        torch.cuda.synchronize()
        for b in range(B):
            dense[b] = [torch.cat((d, new[b, h:h + Hkv]), dim=1) for d, h in zip(dense[b], (Hq, Hq + Hkv))]
            k, v = (torch.cat((p, d), dim=1)[None] for p, d in zip(pre, dense[b]))
            rep = compare(o[b:b + 1].cpu(), lse[b:b + 1].cpu(), *oracle.attention(new[b:b + 1, :Hq], k, v, D ** -0.5, True))
            assert rep.ok(), (step, b, rep)


def test_one_workspace_for_smaller_calls():
    """A workspace for the largest batch and lengths serves every smaller call, whatever plan that takes."""
    Hq, Hkv = 8, 2
    ws = attn.decode_prefix_workspace(40, Hq, Hkv, 5000, 600)
    for B, plen, longest in ((1, 1, 1), (3, 130, 17), (17, 2000, 600), (40, 5000, 64), (33, 300, 300)):
        need = attn.decode_prefix_workspace(B, Hq, Hkv, plen, longest).numel()
        assert need <= ws.numel()
        lens = [int(x) for x in np.random.RandomState(B).randint(0, longest + 1, size=B)]
        q, pre, suf, pages, ptab, table = make(B, Hq, Hkv, plen, lens, 64, seed=B)
        o, lse = call(q, pages, ptab, plen, table, lens, max_prefix_len=plen, max_seq_len=longest, workspace=ws)
        for b in range(0, B, 5):
            rep = compare(o[b:b + 1], lse[b:b + 1], *expect(q, pre, suf, lens, b, D ** -0.5))
            assert rep.ok(), rep


def test_refusals():
    B, Hq, Hkv, page, lens = 2, 8, 2, 16, [5, 6]
    q, pre, suf, pages, ptab, table = make(B, Hq, Hkv, 40, lens, page, seed=11)
    ok = dict(max_prefix_len=40, max_seq_len=6)
    small = torch.empty((1024,), dtype=torch.uint8, device="cuda")
    with pytest.raises(attn.AttnError) as e:
        call(q, pages, ptab, 40, table, lens, workspace=small, **ok)
    assert e.value.status == -8
    need = attn.decode_prefix_workspace(B, Hq, Hkv, 40, 6)
    with pytest.raises(attn.AttnError) as e:
        call(q, pages, ptab, 40, table, lens, workspace=need[:-1], **ok)
    assert e.value.status == -8
    with pytest.raises(attn.AttnError) as e:
        call(q, pages, ptab, 40, table, lens, scale=-1.0, **ok)
    assert e.value.status == -11
    with pytest.raises(ValueError, match="expected q"):
        call(q[..., :64].contiguous(), pages, ptab, 40, table, lens, **ok)
    with pytest.raises(ValueError, match="one row"):
        call(q, pages, ptab, 40, table, lens[:1], **ok)
    with pytest.raises(ValueError, match="out must"):
        call(q, pages, ptab, 40, table, lens, out=torch.empty((B, Hq, 2, D), dtype=torch.bfloat16, device="cuda"), **ok)
