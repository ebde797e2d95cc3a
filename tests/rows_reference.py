"""Plain 64-bit forms of the per-head norm and rotation, its gradient and the paged append, with the
magnitudes their rounding errors scale with. Torch on the CPU; shares no code with the library.

Bounds. u = 2^-24 (half a step of fp32), bf16 output half a step: 2^-8 of the value (2^-7 is bf16's
eps). Forward, y = x r w: the sum of squares goes through chains of 4 + 1 + 4 additions and as many
products (<= 10 u, halved by the root), mean and eps 2 u, rsqrtf 4 u, two products 2 u: <= 14 u of |y|;
the rotation adds two products, one addition: 3 u of |y_a c| + |y_b s|. Together 17 u of that sum;
FORWARD_U = 20. Backward: dy 3 u, g 1 u, the sum of g x 10 u + 2, r three times 14 u in r^3 (f has r^2,
the factor outside r), four more roundings: below 64 u of the sum of magnitudes; BACKWARD_U = 64.
dw: a term is off by at most 3 + 14 + 2 u. The sum runs through chains of: the rows of one lane (n),
the 32 / (D / 16) lane groups of a warp (at most 4 additions), 8 warps, the blocks' partials 128 apart (at most
5 of 592), 2 shuffles and 32 warps: n + 51 u. A lane takes two rows of each unit of its warp, and there are
min(2 per SM, 592) blocks of 8 warps: 6 rows for 1,500 tokens of 32 heads of 128, and at most 88 up to
830,000 rows of a side. So below 19 + 51 + 90 u; WEIGHT_U = 160 of the sum of the terms' magnitudes.
"""
import torch

U = 2.0 ** -24
BF16 = 2.0 ** -8
FORWARD_U, BACKWARD_U, WEIGHT_U = 20, 64, 160


def angle_tables(max_pos, rot, base=10000.0):
    inv = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * inv
    return a.cos().float(), a.sin().float()


def pair_index(rot, interleaved):
    j = torch.arange(rot // 2)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)


def turn(y, c, s, interleaved, sign=1.0):
    """y [..., D] with its first 2 * c.shape[-1] channels turned; c, s broadcast against y[..., :rot/2]."""
    a, b = pair_index(2 * c.shape[-1], interleaved)
    z = y.clone()
    z[..., a] = y[..., a] * c - sign * y[..., b] * s
    z[..., b] = y[..., b] * c + sign * y[..., a] * s
    return z


def turn_magnitude(y, c, s, interleaved):
    a, b = pair_index(2 * c.shape[-1], interleaved)
    z = y.abs().clone()
    z[..., a] = (y[..., a] * c).abs() + (y[..., b] * s).abs()
    z[..., b] = (y[..., b] * c).abs() + (y[..., a] * s).abs()
    return z


def angles(cos, sin, positions):
    """c, s [B, 1, S, rot / 2] and whether each position has a row, [B, 1, S, 1]."""
    ok = (positions >= 0) & (positions < cos.shape[0])
    at = positions.long().clamp(0, cos.shape[0] - 1)
    return cos.double()[at][:, None], sin.double()[at][:, None], ok[:, None, :, None]


def norm(x, w, eps):
    if w is None:
        return x
    return x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w.double()


def forward(x, w, cos, sin, positions, interleaved, eps):
    """z and the bound of its error (bf16 output) for x [B, H, S, D]."""
    y = norm(x.double(), w, eps)
    if cos is None:
        return y, BF16 * y.abs() + FORWARD_U * U * y.abs()
    c, s, ok = angles(cos, sin, positions)
    z = torch.where(ok, turn(y, c, s, interleaved), 0.0)
    mag = torch.where(ok, turn_magnitude(y, c, s, interleaved), 0.0)
    return z, BF16 * z.abs() + FORWARD_U * U * mag * (1 + BF16)


def backward(x, w, cos, sin, positions, interleaved, eps, dz):
    """dx with its bound, dw with its bound (None without w)."""
    x, dz = x.double(), dz.double()
    if cos is None:
        dy, ady = dz, dz.abs()
    else:
        c, s, ok = angles(cos, sin, positions)
        dy = torch.where(ok, turn(dz, c, s, interleaved, -1.0), 0.0)
        ady = torch.where(ok, turn_magnitude(dz, c, s, interleaved), 0.0)
    if w is None:
        return dy, BF16 * dy.abs() + BACKWARD_U * U * ady, None, None
    w = w.double()
    r = (x.pow(2).mean(-1, keepdim=True) + eps).rsqrt()
    g, ag = w * dy, w.abs() * ady
    dx = r * (g - x * r * r * (g * x).mean(-1, keepdim=True))
    adx = r * (ag + x.abs() * r * r * (ag * x.abs()).mean(-1, keepdim=True))
    dims = (0, 1, 2)
    dw, adw = (dy * x * r).sum(dims), (ady * x.abs() * r).sum(dims)
    return dx, BF16 * dx.abs() + BACKWARD_U * U * adx * (1 + BF16), dw, WEIGHT_U * U * adw


def within(got, want, bound, what=""):
    err = (got.detach().cpu().double() - want).abs()
    bad = ~(err <= bound + 1e-300)
    if bad.any():
        i = tuple(int(t[0]) for t in bad.nonzero(as_tuple=True))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds, first at {i}: got "
                             f"{float(got[i])}, want {float(want[i])}, bound {float(bound[i])}")


def append(k_pages, v_pages, q, k, v, qw, kw, cos, sin, positions, seq_lens, new_lens, table, interleaved, eps):
    """For a bf16 or fp32-valued cache: (q_out, its bound, k rows, their bound, v rows, where), with
    `where` the list of (b, i, page, slot) of the rows that are appended, rows [len(where), Hkv, D]."""
    B, Hkv, Sq, D = k.shape
    num_pages, _, page, _ = k_pages.shape
    where = []
    live = torch.zeros((B, Sq), dtype=torch.bool)
    place = torch.zeros((B, Sq), dtype=torch.int64)
    for b in range(B):
        fresh = Sq if new_lens is None else min(max(int(new_lens[b]), 0), Sq)
        for i in range(Sq):
            p = int(seq_lens[b]) - Sq + i
            if i < Sq - fresh or p < 0 or p >= table.shape[1] * page:
                continue
            pg = int(table[b, p // page])
            rp = p if positions is None else int(positions[b, i])
            if pg < 0 or pg >= num_pages or (cos is not None and not 0 <= rp < cos.shape[0]):
                continue
            live[b, i], place[b, i] = True, rp
            where.append((b, i, pg, p % page))
    at = place if cos is not None else None
    kz, kb = forward(k, kw, cos, sin, at, interleaved, eps)
    qz = qb = None
    if q is not None:
        qz, qb = forward(q, qw, cos, sin, at, interleaved, eps)
        qz, qb = (torch.where(live[:, None, :, None], t, 0.0) for t in (qz, qb))
    pick = lambda t: torch.stack([t[b, :, i] for b, i, _, _ in where]) if where else t.new_zeros((0, Hkv, D))  # noqa: E731
    return qz, qb, pick(kz), pick(kb), pick(v), where
