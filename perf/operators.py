"""Cases for the operators around the attention kernels: the norm and rotation of queries and keys
(and its gradient), appending to a paged cache, and decode over a shared prefix.

``run`` computes an operator in plain torch operations, or, with ``own`` true, through this
package's binding. ``exact`` restates each operator in 64 bits, apart from the plain form.

An ``op`` is one of

- ``norm_rope``: q and k of a fused projection, token-major, each head normalised (RMS, a weight per
  channel) and rotated, written heads-major as the attention kernels take them;
- ``norm_rope_bwd``: its gradient, dq and dk written into the fused projection's gradient;
- ``append``: the new tokens' q, k normalised and rotated and their k, v written to a paged cache in
  bf16, or (``fp8``) as e4m3 codes with a coefficient per (kv head, channel);
- ``prefix``: one new token per sequence over a prefix that all sequences share and a suffix of
  their own, both in the same pages.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------------------------------ cases


def _norm_rope(name, bwd, B, Hq, Hkv, S, D, rot=None, interleaved=False, packed=False, norm=True):
    return {"name": name, "op": "norm_rope_bwd" if bwd else "norm_rope", "B": B, "Hq": Hq, "Hkv": Hkv, "S": S, "D": D,
            "rot": D if rot is None else rot, "interleaved": interleaved, "packed": packed, "norm": norm}


def _append(name, B, Hq, Hkv, S, page, past, fp8, norm=True, ragged=False, rot=128, interleaved=False):
    return {"name": name, "op": "append", "B": B, "Hq": Hq, "Hkv": Hkv, "S": S, "D": 128, "page": page, "past": past,
            "fp8": fp8, "norm": norm, "ragged": ragged, "rot": rot, "interleaved": interleaved}


def _prefix(name, B, Hq, Hkv, prefix, suffix, page):
    return {"name": name, "op": "prefix", "B": B, "Hq": Hq, "Hkv": Hkv, "D": 128, "prefix": prefix, "suffix": suffix,
            "page": page}


def listed():
    return [
        # The prefill of the 8B layer (32 query heads, 8 kv heads, 4096 tokens).
        _norm_rope("norm_rope 8B layer", False, 1, 32, 8, 4096, 128),
        # Token-by-token use on a dense cache: 16 sequences, one token each.
        _norm_rope("norm_rope one token", False, 16, 32, 8, 1, 128),
        # The training step of the same layer: several documents packed into each row.
        _norm_rope("norm_rope_bwd 8B layer", True, 1, 32, 8, 4096, 128, packed=True),
        # A small model's odd length, neighbouring channels rotated together, half of each head rotated.
        _norm_rope("norm_rope_bwd odd small", True, 3, 10, 2, 777, 64, rot=32, interleaved=True),
        # The long layer's gradient, 32768 tokens.
        _norm_rope("norm_rope_bwd long", True, 1, 32, 8, 32768, 128),
        # One decode step of 16 sequences around a 4096-token context.
        _append("append decode", 16, 32, 8, 1, 64, 4096, False),
        # Chunked prefill: 8 sequences bring 256 new tokens each over past lengths up to 768.
        _append("append chunk", 8, 32, 8, 256, 64, 768, False, ragged=True),
        # A decode step of many sequences on an e4m3 cache with small pages, keys not normalised.
        _append("append decode e4m3", 61, 32, 8, 1, 16, 4096, True, norm=False),
        # A long prompt written to an e4m3 cache.
        _append("append prompt e4m3", 2, 32, 8, 8192, 128, 0, True),
        # A few sequences after a short system prompt.
        _prefix("prefix short", 4, 32, 8, 512, 100, 64),
        # 16 sequences at a 4096-token common context, up to 256 tokens of their own.
        _prefix("prefix 4K", 16, 32, 8, 4096, 256, 64),
        # Many samples of one long document, up to 768 tokens of their own, a group of three heads
        # and an odd prefix that ends inside a page.
        _prefix("prefix long", 125, 18, 6, 32749, 768, 128),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    case = _draw(rng, log_int)
    del case["name"]
    return case


def _draw(rng, log_int):
    op = rng.choice(["norm_rope", "norm_rope_bwd", "append", "append", "prefix", "prefix"])
    heads = [(32, 8), (18, 6), (10, 2), (8, 8), (16, 1), (28, 4)]
    Hq, Hkv = rng.choice(heads)
    if op in ("norm_rope", "norm_rope_bwd"):
        D = rng.choice([32, 64, 128, 128])
        B = log_int(1, 16)
        S = log_int(1, min(32768, 32768 * 40 * 128 // (B * (Hq + Hkv) * D)))
        rot = rng.choice([D, D, D // 2])
        return _norm_rope("", op == "norm_rope_bwd", B, Hq, Hkv, S, D, rot, rng.random() < 0.4, rng.random() < 0.5,
                          rng.random() < 0.8)
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "append":
        B = log_int(1, 128)
        S = 1 if rng.random() < 0.4 else log_int(1, max(2, min(8192, 16384 // B)))
        return _append("", B, Hq, Hkv, S, page, log_int(1, 4096), rng.random() < 0.5, rng.random() < 0.7,
                       rng.random() < 0.4, rng.choice([128, 128, 64]), rng.random() < 0.4)
    B = log_int(1, 125)
    longest = int(32749 * min(1.0, 125 * 18 / (B * Hq), 6 / Hkv))
    return _prefix("", B, Hq, Hkv, log_int(64, longest), log_int(1, min(768, 125 * 6 * 768 // (B * Hkv))), page)


# ------------------------------------------------------------------------------------------ inputs


def _tables(max_pos, rot):
    """cos and sin of the rotation's angles, fp32 [max_pos, rot / 2], computed in 64 bits."""
    inv = torch.pow(10000.0, -torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    a = torch.arange(max_pos, device=DEV, dtype=torch.float64)[:, None] * inv[None]
    return a.cos().float(), a.sin().float()


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _randint(g, lo, hi, n):
    return torch.randint(lo, hi, (n,), generator=g, device=DEV, dtype=torch.int32)


def _weight(g, D, norm):
    return (1.0 + 0.1 * torch.randn((D,), generator=g, device=DEV)).to(torch.bfloat16) if norm else None


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = {"case": case}
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    if case["op"] in ("norm_rope", "norm_rope_bwd"):
        S, rot = case["S"], case["rot"]
        # Weights and channels of real projections differ in size: a few channels are larger.
        qkv = _randn(g, B, S, Hq + 2 * Hkv, D)
        qkv[..., ::17] *= 4
        st["q"], st["k"] = qkv[:, :, :Hq].transpose(1, 2), qkv[:, :, Hq:Hq + Hkv].transpose(1, 2)
        st["wq"], st["wk"] = _weight(g, D, case["norm"]), _weight(g, D, case["norm"])
        if S == 1:  # decode: each sequence at its own position
            st["pos"] = _randint(g, 0, 4096, B).view(B, 1)
            st["cos"], st["sin"] = _tables(4096, rot)
        elif case["packed"]:  # documents end to end: the position starts again at each
            starts = torch.rand((B, S), generator=g, device=DEV) < 4.0 / S
            starts[:, 0] = True
            at = torch.arange(S, device=DEV).expand(B, S)
            st["pos"] = (at - torch.where(starts, at, 0).cummax(dim=1).values).to(torch.int32).contiguous()
            st["cos"], st["sin"] = _tables(S, rot)
        else:
            st["pos"] = None
            st["cos"], st["sin"] = _tables(S, rot)
        if case["op"] == "norm_rope_bwd":
            st["dqo"], st["dko"] = _randn(g, B, Hq, S, D), _randn(g, B, Hkv, S, D)
            dqkv = torch.zeros_like(qkv)
            st["dq"], st["dk"] = dqkv[:, :, :Hq].transpose(1, 2), dqkv[:, :, Hq:Hq + Hkv].transpose(1, 2)
        else:
            st["qo"] = torch.empty((B, Hq, S, D), dtype=torch.bfloat16, device=DEV)
            st["ko"] = torch.empty((B, Hkv, S, D), dtype=torch.bfloat16, device=DEV)
        return st
    page = case["page"]
    if case["op"] == "append":
        S, past, rot = case["S"], case["past"], case["rot"]
        qkv = _randn(g, B, S, Hq + 2 * Hkv, D)
        qkv[..., ::17] *= 4
        st["q"], st["k"], st["v"] = (t.transpose(1, 2) for t in (qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]))
        st["wq"], st["wk"] = _weight(g, D, case["norm"]), _weight(g, D, case["norm"])
        new = _randint(g, 1, S + 1, B) if case["ragged"] else torch.full((B,), S, dtype=torch.int32, device=DEV)
        st["lens"] = _randint(g, 0, past + 1, B) + new
        st["new"] = new if case["ragged"] else None
        per = -(-(past + S) // page)
        # The pages that new tokens can fall into; those of the past belong to no read or write of this step.
        first = ((st["lens"] - new) // page).cpu().tolist()
        last = ((st["lens"] - 1) // page).cpu().tolist()
        n_pages = B * ((S - 1) // page + 2)
        perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
        table = torch.full((B, per), n_pages, dtype=torch.int32, device=DEV)
        at = 0
        for b in range(B):
            n = last[b] - first[b] + 1
            table[b, first[b]:last[b] + 1] = perm[at:at + n]
            at += n
        st["table"] = table
        st["cos"], st["sin"] = _tables(past + S, rot)
        st["qo"] = torch.empty((B, Hq, S, D), dtype=torch.bfloat16, device=DEV)
        shape = (n_pages, Hkv, page, D)
        if case["fp8"]:
            st["kp"], st["vp"] = ((torch.randn(shape, generator=g, device=DEV) * 60).to(torch.float8_e4m3fn).view(torch.uint8) for _ in range(2))
            # Coefficients that put most channels into the top binades and let the largest saturate.
            st["ks"], st["vs"] = ((3.0 + torch.rand((Hkv, D), generator=g, device=DEV)) / 448.0 for _ in range(2))
            st["ks"][:, ::17] *= 4
            st["vs"][:, ::17] *= 4
        else:
            st["kp"], st["vp"] = _randn(g, *shape), _randn(g, *shape)
        return st
    # prefix: shared pages first in the caller's order, then each sequence's own, all in random places
    Lp, Ls = case["prefix"], case["suffix"]
    st["q"] = _randn(g, B, Hq, 1, D)
    st["plen"] = torch.tensor([Lp], dtype=torch.int32, device=DEV)
    st["lens"] = _randint(g, 0, Ls + 1, B)
    st["lens"][0] = Ls
    np_, ns = -(-Lp // page), -(-Ls // page)
    n_pages = np_ + B * ns
    perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    st["ptab"], st["table"] = perm[:np_].contiguous(), perm[np_:].view(B, ns).contiguous()
    st["kp"], st["vp"] = _randn(g, n_pages, Hkv, page, D), _randn(g, n_pages, Hkv, page, D)
    # A few keys of the prefix stand out, as the first tokens of a prompt do.
    st["kp"][st["ptab"][0].long(), :, :2] *= 4
    st["o"] = torch.empty((B, Hq, 1, D), dtype=torch.bfloat16, device=DEV)
    st["lse"] = torch.empty((B, Hq, 1), dtype=torch.float32, device=DEV)
    if own:
        from causal_attention_attn_b200 import attn

        st["ws"] = attn.decode_prefix_workspace(B, Hq, Hkv, Lp, Ls, device=DEV)
    return st


# ------------------------------------------------------------------------------------------ plain forms


def _positions(st, B, S):
    if st.get("pos") is not None:
        return st["pos"].long()
    return torch.arange(S, device=DEV).expand(B, S)


def _rotate(y, c, s, rot, interleaved, back=False):
    """The rotation of the first `rot` channels of y [B, H, S, D] by the angles' c, s [B, 1, S, rot / 2]."""
    if back:
        s = -s
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
    z = y.clone()
    if interleaved:
        z[..., 0:rot:2], z[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        z[..., :rot // 2], z[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    return z


def _plain_norm(x, w):
    if w is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _plain_norm_bwd(x, w, dy):
    if w is None:
        return dy, None
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xh = x * r
    gr = dy * w.float()
    dx = r * (gr - xh * (gr * xh).mean(-1, keepdim=True))
    return dx, (dy * xh).sum(dim=(0, 1, 2), dtype=torch.float64).float()


def _slots(st, case):
    """For each new token: whether it is real, its position, and its page and slot."""
    B, S, page = case["B"], case["S"], case["page"]
    i = torch.arange(S, device=DEV)[None]
    pos = st["lens"].long()[:, None] - S + i
    live = pos >= 0
    if st["new"] is not None:
        live = live & (i >= S - st["new"].long()[:, None])
    b, n = live.nonzero(as_tuple=True)
    p = pos[b, n]
    return b, n, p, st["table"].long()[b, p // page], p % page, pos, live


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "norm_rope":
        pos = _positions(st, case["B"], case["S"])
        c, s = st["cos"][pos][:, None], st["sin"][pos][:, None]
        out = []
        for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
            out.append(_rotate(_plain_norm(x.float(), w), c, s, case["rot"], case["interleaved"]).to(torch.bfloat16))
        return out
    if op == "norm_rope_bwd":
        pos = _positions(st, case["B"], case["S"])
        c, s = st["cos"][pos][:, None], st["sin"][pos][:, None]
        out, dws = [], []
        for x, w, dz, dx in ((st["q"], st["wq"], st["dqo"], st["dq"]), (st["k"], st["wk"], st["dko"], st["dk"])):
            dy = _rotate(dz.float(), c, s, case["rot"], case["interleaved"], back=True)
            d, dw = _plain_norm_bwd(x.float(), w, dy)
            dx.copy_(d)
            out.append(dx)
            dws += [] if dw is None else [dw]
        return out + dws
    if op == "append":
        b, n, p, pg, slot, pos, live = _slots(st, case)
        at = pos.clamp(min=0)
        c, s = st["cos"][at][:, None], st["sin"][at][:, None]
        z = []
        for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
            z.append(_rotate(_plain_norm(x.float(), w), c, s, case["rot"], case["interleaved"]))
        st["qo"].copy_(torch.where(live[:, None, :, None], z[0], 0.0))
        k, v = z[1][b, :, n], st["v"][b, :, n].float()  # [tokens, Hkv, D]
        if case["fp8"]:
            k, v = ((x / f).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for x, f in ((k, st["ks"]), (v, st["vs"])))
        st["kp"][pg, :, slot] = k.to(st["kp"].dtype)
        st["vp"][pg, :, slot] = v.to(st["vp"].dtype)
        return _cache(st)
    # prefix
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    G, Lp, Ls, page = Hq // Hkv, case["prefix"], case["suffix"], case["page"]
    q = st["q"].float().view(B, Hkv, G, D) * (D ** -0.5)
    kp, vp = (t[st["ptab"].long()].transpose(0, 1).reshape(Hkv, -1, D)[:, :Lp].float() for t in (st["kp"], st["vp"]))
    ks, vs = (t[st["table"].long()].permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)[:, :, :Ls].float() for t in (st["kp"], st["vp"]))
    sp = (q.transpose(0, 1).reshape(Hkv, B * G, D) @ kp.transpose(1, 2)).view(Hkv, B, G, Lp).transpose(0, 1)
    ss = q @ ks.transpose(2, 3)
    ss = ss.masked_fill(torch.arange(Ls, device=DEV) >= st["lens"].long()[:, None, None, None], float("-inf"))
    m = torch.maximum(sp.amax(-1, keepdim=True), ss.amax(-1, keepdim=True))
    ep, es = (sp - m).exp(), (ss - m).exp()
    total = ep.sum(-1, keepdim=True) + es.sum(-1, keepdim=True)
    op_ = (ep.transpose(0, 1).reshape(Hkv, B * G, Lp) @ vp).view(Hkv, B, G, D).transpose(0, 1)
    o = (op_ + es @ vs) / total
    st["o"].copy_(o.reshape(B, Hq, 1, D))
    st["lse"].copy_((m + total.log()).reshape(B, Hq, 1))
    return [st["o"], st["lse"]]


def _cache(st):
    kp, vp = st["kp"], st["vp"]
    if st["case"]["fp8"]:
        kp, vp = kp.view(torch.float8_e4m3fn), vp.view(torch.float8_e4m3fn)
    return [st["qo"], kp, vp]


# ------------------------------------------------------------------------------------------ the framework's calls


def _run_own(st):
    from causal_attention_attn_b200 import attn

    case = st["case"]
    op = case["op"]
    if op == "norm_rope":
        return list(attn.attn_qk_norm_rope(st["q"], st["k"], st["cos"], st["sin"], q_weight=st["wq"], k_weight=st["wk"],
                                           positions=st["pos"], interleaved=case["interleaved"], eps=EPS, q_out=st["qo"],
                                           k_out=st["ko"]))
    if op == "norm_rope_bwd":
        got = attn.attn_qk_norm_rope_bwd(st["q"], st["k"], st["cos"], st["sin"], st["dqo"], st["dko"], q_weight=st["wq"],
                                         k_weight=st["wk"], positions=st["pos"], interleaved=case["interleaved"], eps=EPS,
                                         dq=st["dq"], dk=st["dk"])
        return [t for t in got if t is not None]
    if op == "append":
        kw = dict(q=st["q"], q_out=st["qo"], q_weight=st["wq"], k_weight=st["wk"], new_lens=st["new"],
                  interleaved=case["interleaved"], eps=EPS)
        if case["fp8"]:
            attn.attn_append_paged_fp8(st["k"], st["v"], st["cos"], st["sin"], st["kp"], st["vp"], st["ks"], st["vs"],
                                       st["table"], st["lens"], **kw)
        else:
            attn.attn_append_paged(st["k"], st["v"], st["cos"], st["sin"], st["kp"], st["vp"], st["table"], st["lens"], **kw)
        return _cache(st)
    return list(attn.attn_decode_prefix(st["q"], st["kp"], st["vp"], st["ptab"], st["plen"], st["table"], st["lens"],
                                        max_prefix_len=case["prefix"], max_seq_len=case["suffix"], out=st["o"],
                                        lse=st["lse"], workspace=st["ws"]))


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------------------------ 64 bits


def _turn(y, ang_c, ang_s, rot, interleaved, sign):
    """The rotation as a product with complex numbers of modulus one, in 64 bits."""
    w = torch.complex(ang_c.double(), sign * ang_s.double())
    head = y[..., :rot]
    h = rot // 2
    z = torch.complex(head[..., 0::2], head[..., 1::2]) if interleaved else torch.complex(head[..., :h], head[..., h:])
    z = z * w
    turned = torch.stack((z.real, z.imag), -1).flatten(-2) if interleaved else torch.cat((z.real, z.imag), -1)
    return torch.cat((turned, y[..., rot:]), -1)


def _unit(x, w):
    if w is None:
        return x
    return x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double()


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    if op in ("norm_rope", "norm_rope_bwd"):
        S, rot, il = case["S"], case["rot"], case["interleaved"]
        pos = st["pos"].long() if st["pos"] is not None else torch.arange(S, device=DEV).repeat(B, 1)
        c, s = st["cos"][pos].unsqueeze(1), st["sin"][pos].unsqueeze(1)
        if op == "norm_rope":
            return [_turn(_unit(x.double(), w), c, s, rot, il, 1.0) for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"]))]
        out, dws = [], []
        for x, w, dz in ((st["q"], st["wq"], st["dqo"]), (st["k"], st["wk"], st["dko"])):
            # Head by head, so that the 64-bit temporaries stay small; dw sums over the heads.
            dx, dw = torch.empty(x.shape, dtype=torch.float64, device=DEV), torch.zeros(D, dtype=torch.float64, device=DEV)
            for h in range(x.shape[1]):
                xh = x[:, h:h + 1].double()
                dy = _turn(dz[:, h:h + 1].double(), c, s, rot, il, -1.0)
                if w is None:
                    dx[:, h:h + 1] = dy
                    continue
                n2 = xh.pow(2).sum(-1, keepdim=True) / D + EPS
                inv = n2.pow(-0.5)
                gy = dy * w.double()
                dx[:, h:h + 1] = gy * inv - xh * (gy * xh).sum(-1, keepdim=True) * inv.pow(3) / D
                dw += torch.einsum("bhsd,bhsd->d", dy, xh * inv)
            out.append(dx)
            dws += [] if w is None else [dw]
        return out + dws
    if op == "append":
        S, page, rot, il = case["S"], case["page"], case["rot"], case["interleaved"]
        lens, table = st["lens"].cpu().tolist(), st["table"].cpu()
        new = st["new"].cpu().tolist() if st["new"] is not None else [S] * B
        qo = torch.zeros((B, Hq, S, D), dtype=torch.float64, device=DEV)
        kp, vp = ((t.view(torch.float8_e4m3fn) if case["fp8"] else t).double() for t in (st["kp"], st["vp"]))
        for b in range(B):
            lo = max(S - new[b], S - lens[b], 0)
            p = torch.arange(lens[b] - S + lo, lens[b], device=DEV)
            c, s = st["cos"][p][None], st["sin"][p][None]
            qo[b, :, lo:] = _turn(_unit(st["q"][b, :, lo:].double(), st["wq"]), c, s, rot, il, 1.0)
            k = _turn(_unit(st["k"][b, :, lo:].double(), st["wk"]), c, s, rot, il, 1.0)
            v = st["v"][b, :, lo:].double()
            if case["fp8"]:  # before the rounding to a code
                k = (k / st["ks"].double()[:, None]).clamp(-448, 448)
                v = (v / st["vs"].double()[:, None]).clamp(-448, 448)
            pg = table[b][(p // page).cpu()].long().to(DEV)
            kp[pg, :, p % page] = k.transpose(0, 1)
            vp[pg, :, p % page] = v.transpose(0, 1)
        return [qo, kp, vp]
    Lp, Ls = case["prefix"], case["suffix"]
    G = Hq // Hkv
    o = torch.zeros((B, Hq, 1, D), dtype=torch.float64, device=DEV)
    lse = torch.zeros((B, Hq, 1), dtype=torch.float64, device=DEV)
    lens = st["lens"].cpu().tolist()
    for h in range(Hkv):
        kpre, vpre = (t[st["ptab"].long(), h].reshape(-1, D)[:Lp].double() for t in (st["kp"], st["vp"]))
        for b in range(B):
            own_k, own_v = (t[st["table"][b].long(), h].reshape(-1, D)[:lens[b]].double() for t in (st["kp"], st["vp"]))
            k, v = torch.cat((kpre, own_k)), torch.cat((vpre, own_v))
            s = st["q"][b, h * G:(h + 1) * G, 0].double() @ k.T / math.sqrt(D)
            l = torch.logsumexp(s, -1, keepdim=True)
            o[b, h * G:(h + 1) * G, 0] = torch.exp(s - l) @ v
            lse[b, h * G:(h + 1) * G, 0] = l[:, 0]
    return [o, lse]


# ------------------------------------------------------------------------------------------ work


def work(case):
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    if case["op"] in ("norm_rope", "norm_rope_bwd"):
        S = case["S"]
        rows = B * S * (Hq + Hkv)
        tables = (B if S == 1 else S) * case["rot"] * 4
        if case["op"] == "norm_rope":
            return {"bytes": rows * D * 4 + tables, "flops": rows * D * 8}
        return {"bytes": rows * D * 6 + tables, "flops": rows * D * 16}
    if case["op"] == "append":
        # Half of a ragged chunk's rows are new, on average; the rows before them are only cleared.
        live = (case["S"] + 1) / 2 if case["ragged"] else case["S"]
        elem = 1 if case["fp8"] else 2
        new = B * live * D * (Hq * 2 + Hkv * 2 * 2 + Hkv * 2 * elem) + B * case["S"] * Hq * D * 2
        return {"bytes": new, "flops": B * live * (Hq + Hkv) * D * 8}
    # The suffixes' lengths are drawn evenly up to the longest.
    own_keys = B * case["suffix"] / 2
    keys = case["prefix"] + own_keys
    return {"bytes": keys * Hkv * D * 4 + B * Hq * D * 4 + B * Hq * 4,
            "flops": 4 * D * Hq * (B * case["prefix"] + own_keys)}
