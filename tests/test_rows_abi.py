"""Argument errors of attn_qk_norm_rope, its gradient and the paged appends: every case is rejected on
the host before any CUDA call (fake, aligned addresses; no GPU needed), and the binding's own checks."""
import ctypes

import pytest
import torch

from causal_attention_attn_b200 import attn, build

A = [0x10000 * (i + 1) for i in range(20)]
S3 = ctypes.c_longlong * 3
GOOD_STRIDES = (4096, 128, 1024)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return attn.load_library()


def strides(over, names):
    return [None if over.get(n, 0) is None else S3(*over.get(n, GOOD_STRIDES)) for n in names]


def forward(lib, **kw):
    p = dict(q=A[0], k=A[1], qw=A[2], kw=A[3], cos=A[4], sin=A[5], pos=A[6], qo=A[7], ko=A[8])
    a = dict(B=2, Hq=4, Hkv=2, S=8, D=64, rot=64, max_pos=8, il=0, eps=1e-6)
    p.update({k: v for k, v in kw.items() if k in p})
    a.update({k: v for k, v in kw.items() if k in a})
    st = strides(kw, ("qs", "ks", "qos", "kos"))
    return lib.attn_qk_norm_rope(*p.values(), a["B"], a["Hq"], a["Hkv"], a["S"], a["D"], *st, a["rot"], a["max_pos"],
                                 a["il"], a["eps"], None)


@pytest.mark.parametrize("name,over,expected", [
    ("null q", dict(q=None), -1),
    ("null k_out", dict(ko=None), -1),
    ("one weight", dict(kw=None), -1),
    ("null cos", dict(cos=None), -1),
    ("null strides", dict(qos=None), -1),
    ("zero tokens", dict(S=0), -2),
    ("too many rows", dict(B=1 << 16, S=1 << 14), -2),
    ("flag 2", dict(il=2), -2),
    ("head dim 96", dict(D=96), -4),
    ("misaligned q_out", dict(qo=A[7] + 8), -5),
    ("misaligned weight", dict(qw=A[2] + 2), -5),
    ("misaligned positions", dict(pos=A[6] + 2), -5),
    ("stride of 4", dict(ks=(4096, 4, 1024)), -5),
    ("stride of 0", dict(qs=(0, 128, 1024)), -5),
    ("rot_dim 24", dict(rot=24), -14),
    ("rot_dim above D", dict(rot=80), -14),
    ("negative rot_dim", dict(rot=-16), -14),
    ("no table rows", dict(max_pos=0), -14),
    ("negative eps", dict(eps=-1.0), -15),
    ("nan eps", dict(eps=float("nan")), -15),
])
def test_forward_argument_errors(lib, name, over, expected):
    assert forward(lib, **over) == expected, name


def backward(lib, **kw):
    names = ("q", "k", "qw", "kw", "cos", "sin", "pos", "dqo", "dko", "dq", "dk", "dqw", "dkw", "ws")
    p = dict(zip(names, A))
    p.update({k: v for k, v in kw.items() if k in p})
    st = strides(kw, ("qs", "ks", "dqos", "dkos", "dqs", "dks"))
    return lib.attn_qk_norm_rope_bwd(*p.values(), 2, 4, 2, 8, kw.get("D", 64), *st, 64, 8, 0, kw.get("eps", 1e-6), None)


@pytest.mark.parametrize("name,over,expected", [
    ("null dq_out", dict(dqo=None), -1),
    ("null dk", dict(dk=None), -1),
    ("null q with a norm", dict(q=None), -1),
    ("no workspace", dict(ws=None), -1),
    ("weight gradients without weights", dict(qw=None, kw=None), -1),
    ("null strides", dict(dqos=None), -1),
    ("misaligned workspace", dict(ws=A[13] + 4), -5),
    ("bad dq stride", dict(dqs=(4096, 128, 1025)), -5),
    ("head dim 80", dict(D=80), -4),
    ("infinite eps", dict(eps=float("inf")), -15),
])
def test_backward_argument_errors(lib, name, over, expected):
    assert backward(lib, **over) == expected, name


def append(lib, fp8=False, **kw):
    names = ("q", "k", "v", "qw", "kw", "cos", "sin", "pos", "lens", "new", "table", "qo", "kp", "vp")
    p = dict(zip(names, A))
    if fp8:
        p.update(ksc=A[14], vsc=A[15])
    a = dict(B=2, Hq=8, Hkv=2, Sq=4)
    b = dict(num_pages=4, page_size=64, pages_per_seq=2, rot=128, max_pos=128, il=0, eps=1e-6)
    for d in (p, a, b):
        d.update({k: v for k, v in kw.items() if k in d})
    st = strides(kw, ("qs", "ks", "vs", "qos"))
    fn = lib.attn_append_paged_fp8 if fp8 else lib.attn_append_paged
    return fn(*p.values(), *a.values(), *st, *b.values(), None)


def test_backward_without_a_norm_takes_no_inputs(lib):
    """No q, k or strides of theirs: the arguments pass, and the call fails only where there is no GPU."""
    if torch.cuda.is_available():
        pytest.skip("would reach the device with fake pointers")
    none = dict(q=None, k=None, qw=None, kw=None, dqw=None, dkw=None, ws=None)
    assert backward(lib, qs=None, ks=None, **none) in (-12, -7)
    assert backward(lib, qs=None, ks=None, dqs=None, **none) == -1


@pytest.mark.parametrize("name,over,expected", [
    ("null v", dict(v=None), -1),
    ("null lengths", dict(lens=None), -1),
    ("null table", dict(table=None), -1),
    ("q without q_out", dict(qo=None), -1),
    ("q_out without q", dict(q=None), -1),
    ("q weight without q", dict(q=None, qo=None, Hq=0), -1),
    ("one weight", dict(qw=None), -1),
    ("null q strides", dict(qs=None), -1),
    ("heads without q", dict(q=None, qo=None, qw=None), -2),
    ("zero new tokens", dict(Sq=0), -2),
    ("page size 48", dict(page_size=48), -2),
    ("no pages", dict(num_pages=0), -2),
    ("pages past 32 bits", dict(num_pages=1 << 30, Hkv=4), -2),
    ("misaligned v", dict(v=A[2] + 4), -5),
    ("misaligned table", dict(table=A[10] + 1), -5),
    ("bad v stride", dict(vs=(4096, 12, 1024)), -5),
    ("rot_dim 20", dict(rot=20), -14),
    ("eps -inf", dict(eps=float("-inf")), -15),
])
@pytest.mark.parametrize("fp8", [False, True])
def test_append_argument_errors(lib, fp8, name, over, expected):
    assert append(lib, fp8, **over) == expected, name


def test_append_fp8_needs_its_coefficients(lib):
    assert append(lib, True, ksc=None) == -1
    assert append(lib, True, vsc=A[15] + 4) == -5


def test_binding_rejects_cpu_tensors_and_wrong_types():
    q = torch.zeros((1, 4, 8, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        attn.attn_qk_norm_rope(q, q, None, None)
    with pytest.raises(TypeError, match="q must be"):
        attn.attn_qk_norm_rope(q.float(), q, None, None)
    with pytest.raises(TypeError, match="k must be"):
        attn.attn_append_paged(q.half(), q, None, None, q, q, q, q)
    with pytest.raises(TypeError, match="k_scale"):
        attn.attn_append_paged_fp8(q, q, None, None, q, q, None, None, q, q)


def prefix(lib, **kw):
    names = ("q", "kp", "vp", "ptab", "plen", "tab", "lens", "o", "lse", "ws")
    p = dict(zip(names, A))
    a = dict(ws_bytes=1 << 40, B=2, Hq=8, Hkv=2, num_pages=9, page=64, prefix_pages=3, max_prefix=150, per=2, max_seq=100,
             scale=0.1)
    for d in (p, a):
        d.update({k: v for k, v in kw.items() if k in d})
    return lib.attn_decode_prefix(*p.values(), *a.values(), None)


@pytest.mark.parametrize("name,over,expected", [
    ("null prefix table", dict(ptab=None), -1),
    ("null prefix length", dict(plen=None), -1),
    ("null workspace", dict(ws=None), -1),
    ("batch 1025", dict(B=1025), -2),
    ("too many rows", dict(B=1024, Hq=8192, Hkv=1), -2),
    ("negative bound", dict(max_prefix=-1), -2),
    ("no prefix pages", dict(prefix_pages=0), -2),
    ("page size 80", dict(page=80), -2),
    ("pages past 32 bits", dict(num_pages=1 << 30), -2),
    ("prefix past 32 bits", dict(prefix_pages=1 << 26), -2),
    ("last tile past 31 bits", dict(prefix_pages=(1 << 25) - 1, page=64, max_prefix=(1 << 31) - 1), -2),
    ("gqa not divisible", dict(Hq=7), -3),
    ("misaligned workspace", dict(ws=A[9] + 16), -5),
    ("misaligned lse", dict(lse=A[8] + 4), -5),
    ("misaligned prefix length", dict(plen=A[4] + 2), -5),
    ("nan scale", dict(scale=float("nan")), -11),
])
def test_prefix_argument_errors(lib, name, over, expected):
    assert prefix(lib, **over) == expected, name


def test_prefix_workspace_argument_errors(lib):
    assert lib.attn_decode_prefix_workspace(0, 8, 2, 10, 10) == -2
    assert lib.attn_decode_prefix_workspace(2, 7, 2, 10, 10) == -3
    assert lib.attn_decode_prefix_workspace(2, 8, 2, 10, -1) == -2
