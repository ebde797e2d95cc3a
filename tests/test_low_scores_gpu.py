"""Scores far below anything a softmax meets in earnest but inside fp32 (a mask written into the keys as a large
negative number): the largest still takes all the weight, over a paged cache as over a dense one. Every key has
one channel that is not zero, and scores 2^100 apart and more, so that the weights are 0 and 1 exactly."""
import pytest
import torch

from causal_attention_attn_b200 import attn, build

pytestmark = pytest.mark.gpu
B, HQ, HKV, D, PAGE = 2, 8, 2, 128, 16


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


def cache(n, best, seed):
    """Keys with -2^50 in channel 0, the `best`-th with -2^49, and their values: [HKV, n, D]."""
    v = torch.randn((HKV, n, D), generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)
    k = torch.zeros((HKV, n, D), dtype=torch.bfloat16)
    k[:, :, 0] = -2.0 ** 50
    k[:, best, 0] = -2.0 ** 49
    return k, v


def paged(t):
    """[HKV, n, D] in pages, the rows behind n NaN."""
    n = t.shape[1]
    pages = torch.full((-(-n // PAGE), HKV, PAGE, D), float("nan"), dtype=torch.bfloat16)
    for j in range(n):
        pages[j // PAGE, :, j % PAGE] = t[:, j]
    return pages


@pytest.mark.parametrize("where", ["prefix", "suffix"])
@pytest.mark.parametrize("far", [False, True], ids=["near", "far"])
def test_decode_prefix(where, far):
    n, own = 300, 37
    pk, pv = cache(n, 200, 1)
    suf = [cache(own, 20, 2 + b) for b in range(B)]
    if where == "prefix":
        for k, _ in suf:
            k[:, :, 0] = -2.0 ** 52
    else:
        pk[:, :, 0] = -2.0 ** 52
    parts = [[pk, *(k for k, _ in suf)], [pv, *(v for _, v in suf)]]
    kp, vp = (torch.cat([paged(t) for t in ts]).cuda() for ts in parts)
    n_pre, per = -(-n // PAGE), -(-own // PAGE)
    ptab = torch.arange(n_pre, dtype=torch.int32)
    table = (n_pre + torch.arange(B * per, dtype=torch.int32)).view(B, per)
    bounds = (n, own)
    if far:
        bounds = (1 << 22, 1 << 16)
        ptab = torch.cat((ptab, ptab.new_zeros(bounds[0] // PAGE - n_pre)))
        table = torch.cat((table, table.new_zeros((B, bounds[1] // PAGE - per))), dim=1).contiguous()
    q = torch.zeros((B, HQ, 1, D), dtype=torch.bfloat16)
    q[..., 0] = 2.0 ** 60
    lens = torch.full((B,), own, dtype=torch.int32)
    o, lse = attn.attn_decode_prefix(q.cuda(), kp, vp, ptab.cuda(), torch.tensor([n], dtype=torch.int32).cuda(), table.cuda(),
                                     lens.cuda(), *bounds)
    for b in range(B):
        want = (pv[:, 200] if where == "prefix" else suf[b][1][:, 20]).repeat_interleave(HQ // HKV, dim=0)
        assert torch.equal(o[b, :, 0].cpu(), want)
    best = -(2.0 ** 109) * D ** -0.5
    assert torch.all((lse.cpu().double() / best - 1).abs() < 1e-5)  # log2 units and back, in fp32


@pytest.mark.parametrize("causal", [False, True])
def test_prefill_paged(causal):
    n, Sq = 300, 130
    ks, vs = zip(*(cache(n, 100, 5 + b) for b in range(B)))
    kp, vp = (torch.cat([paged(t) for t in ts]).cuda() for ts in (ks, vs))
    per = -(-n // PAGE)
    table = torch.arange(B * per, dtype=torch.int32).view(B, per).cuda()
    q = torch.zeros((B, HQ, Sq, D), dtype=torch.bfloat16)
    q[..., 0] = 2.0 ** 60
    o, lse = attn.attn_prefill_paged(q.cuda(), kp, vp, table, torch.full((B,), n, dtype=torch.int32).cuda(), n, causal=causal)
    dense = attn.attn_fwd(q.cuda(), torch.stack(ks).cuda(), torch.stack(vs).cuda(), causal=causal)
    want = torch.stack(vs)[:, :, 100].repeat_interleave(HQ // HKV, dim=1)[:, :, None].expand_as(q)
    assert torch.equal(o.cpu(), want) and torch.equal(dense[0], o) and torch.equal(dense[1], lse)
