"""attn_decode_prefix at the edges of its sizes against the fp64 oracle: the largest batch, groups of exactly one
tile and of several, more lists than blocks, pages named twice. Tolerance: tests/compare.py's for attention."""
import numpy as np
import pytest
import torch

from causal_attention_attn_b200 import attn, build
from tests.compare import compare
from tests.test_prefix_gpu import D, call, expect, make, widen

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
    assert attn.device_status() == 0


def check(q, pre, suf, lens, o, lse, every=1, plen=None):
    for b in range(0, len(lens), every):
        rep = compare(o[b:b + 1], lse[b:b + 1], *expect(q, pre, suf, lens, b, D ** -0.5, plen=plen))
        assert rep.ok(), f"sequence {b} (suffix {lens[b]}): {rep}"


CASES = [
    # B, Hq, Hkv, prefix, suffixes up to, page
    (1024, 8, 2, 300, 4, 16),      # the largest batch
    (3, 128, 1, 300, 70, 64),      # a group that fills a tile: a sequence each
    (5, 256, 1, 200, 33, 32),      # two parts of 128 heads
    (4, 192, 2, 130, 17, 16),      # groups of 96, one sequence to a tile and rows to spare
    (300, 64, 64, 220, 3, 16),     # a block and a bit to each kv head, an odd last tile
    (270, 160, 160, 140, 2, 16),   # more kv heads than blocks: cut end to end
]


@pytest.mark.parametrize("far", [False, True], ids=["near", "far"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "b{}_hq{}_hkv{}_p{}_page{}".format(*c[:4], c[5]))
def test_sizes(case, far):
    """`far`: bounds far above the lengths, so that the split is worked out on the device."""
    B, Hq, Hkv, plen, longest, page = case
    lens = [int(x) for x in np.random.RandomState(B).randint(0, longest + 1, size=B)]
    q, pre, suf, pages, ptab, table = make(B, Hq, Hkv, plen, lens, page, seed=B)
    if far:
        ptab, table = widen(ptab, (1 << 20) // page), widen(table, 8192 // page)
    o, lse = call(q, pages, ptab, plen, table, lens, max_prefix_len=1 << 20 if far else plen,
                  max_seq_len=8192 if far else max(lens))
    check(q, pre, suf, lens, o, lse, every=max(1, B // 40))
    again, lse_again = call(q, pages, ptab, plen, table, lens, max_prefix_len=1 << 20 if far else plen,
                            max_seq_len=8192 if far else max(lens))
    assert torch.equal(o, again) and torch.equal(lse, lse_again)


def test_pages_named_twice():
    """A page that the prefix's table names twice, and one that two sequences share: read twice."""
    B, Hq, Hkv, page, lens = 3, 8, 2, 16, [20, 20, 7]
    q, pre, suf, pages, ptab, table = make(B, Hq, Hkv, 64, lens, page, seed=3)
    ptab[2], table[1] = ptab[0], table[0]
    for t in pre:
        t[:, 32:48] = t[:, :16]
    for t in suf:
        t[1] = t[0]
    o, lse = call(q, pages, ptab, 64, table, lens, max_prefix_len=64, max_seq_len=20)
    check(q, pre, suf, lens, o, lse)


def test_each_bound_alone_clamps():
    B, Hq, Hkv, lens, page = 2, 8, 2, [48, 20], 16
    q, pre, suf, pages, ptab, table = make(B, Hq, Hkv, 96, lens, page, seed=2)
    big = 10 ** 9
    for plen, pmax, own, omax, want_p, want in (
            (big, big, [big, 20], big, 96, [48, 20]),    # the tables
            (96, 50, [48, 20], 48, 50, [48, 20]),        # the prefix's bound
            (96, 96, [48, 20], 30, 96, [30, 20]),        # the suffixes' bound
            (big, 50, [big, -1], 30, 50, [30, 0])):
        o, lse = call(q, pages, ptab, plen, table, own, max_prefix_len=pmax, max_seq_len=omax)
        check(q, pre, suf, want, o, lse, plen=want_p)
