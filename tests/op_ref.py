"""64-bit forms of the operators around the sparse attention, with the error
bounds that their fp32 arithmetic and one rounding of the output allow.

Rotation.  The angle in turns is reduced in 64 bits and rounded once to fp32
(at most 2^-26 of a turn: 2^-23.3 rad); its sine and cosine are within 2 ulp
(2^-23 for values up to 1); the two products and their sum add 2^-23 of the
terms.  So y is within 2^-21 (|z0| + |z1|) of the exact rotation, and the angle
itself carries |p| 2^-51 of the frequency's rounding (one on each side).
Norm: the sum of up to 128 squares (8 terms in a row, then 4 levels of a tree),
the division, the root (2 ulp) and two products stay below 2^-20 of z.
An output rounded to type t adds eps_t / 2 of itself, and half the least
subnormal."""
import torch

U = 2.0 ** -24  # one fp32 rounding, relative


def half_ulp(y, dtype):
    f = torch.finfo(dtype)
    return y.abs() * (f.eps / 2) + f.smallest_normal * f.eps / 2


def angles(split, theta, N, grid=None, positions=None, device="cpu"):
    """[B or 1, 1, N, D/2] angles in 64 bits."""
    if positions is None:
        T, Hh, W = grid
        n = torch.arange(N, device=device)
        pos = torch.stack([n // (Hh * W), (n // W) % Hh, n % W], -1)
    else:
        pos = positions
    if pos.dim() == 2:
        pos = pos[None]
    parts = []
    for a, d in enumerate(split):
        i = torch.arange(d // 2, dtype=torch.float64, device=device)
        parts.append(pos[..., a, None].double() * theta ** (-2.0 * i / max(d, 1)))
    return torch.cat(parts, -1)[:, None]


def turn(z, a, sign=1.0):
    z0, z1 = z[..., 0::2], z[..., 1::2]
    c, s = torch.cos(a), sign * torch.sin(a)
    return torch.stack([z0 * c - z1 * s, z0 * s + z1 * c], -1).flatten(-2)


def pair_sum(z):
    """|z0| + |z1| of each element's pair."""
    t = z.abs().unflatten(-1, (-1, 2)).sum(-1, keepdim=True)
    return t.expand(*t.shape[:-1], 2).flatten(-2)


def norm(x, w, eps):
    r = (x.pow(2).mean(-1, keepdim=True) + eps).rsqrt()
    return x * r * w


def angle_slack(positions):
    """2^-51 |p| for explicit positions (grids: nothing to speak of)."""
    return 0.0 if positions is None else float(positions.double().abs().max()) * 2.0 ** -51


def rope_bound(x, y, dtype, normed, slack=0.0, w=None, eps=0.0):
    z = x if not normed else norm(x, w, eps)
    return pair_sum(z) * ((2.0 ** -21 if not normed else 2.0 ** -19) + slack) + half_ulp(y, dtype)


def rope_grads(dy, x, a, w, eps):
    """(dx, dw) by the formula."""
    dz = turn(dy, a, -1.0)
    r = (x.pow(2).mean(-1, keepdim=True) + eps).rsqrt()
    g = dz * w
    dx = r * (g - x * r * r * (g * x).mean(-1, keepdim=True))
    return dx, (dz * x * r).sum((0, 1, 2))


def rope_grad_bounds(dy, x, a, w, eps, dx, dw, dtype, w_dtype, slack=0.0):
    """dz is off by e = 2^-21 of its pair; m = mean(g x) r^2 by the mean of
    |w x| e and 2^-18 of mean |g x| (sum, r^2); dx = r (g - x m) adds 2^-20 of
    both terms.  dw sums at most `rows` terms, each off by 2^-20 and its e."""
    dz = turn(dy, a, -1.0)
    e = pair_sum(dy) * (2.0 ** -21 + slack)
    r = (x.pow(2).mean(-1, keepdim=True) + eps).rsqrt()
    g = dz * w
    em = r * r * ((w * x).abs() * e + 2.0 ** -18 * (g * x).abs()).mean(-1, keepdim=True)
    m = r * r * (g * x).mean(-1, keepdim=True)
    bdx = r * (w.abs() * e + x.abs() * em + 2.0 ** -20 * (g.abs() + (x * m).abs())) + half_ulp(dx, dtype)
    rows = x.shape[0] * x.shape[1] * x.shape[2]
    bdw = ((dz.abs() * (2.0 ** -20 + rows * U) + e) * (x * r).abs()).sum((0, 1, 2)) + half_ulp(dw, w_dtype)
    return bdx, bdw


def within(got, want, bound, what):
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err - bound).max()):.3e} above the bound"


# ---------------------------------------------------------------- cross attention
def allowed_keys(Bk, M, kv_len=None, kv_mask=None, device="cpu"):
    if kv_mask is not None:
        return kv_mask.bool()
    if kv_len is not None:
        return torch.arange(M, device=device)[None] < kv_len[:, None]
    return torch.ones((Bk, M), dtype=torch.bool, device=device)


def cross(q, k, v, allowed, scale, dtype, do=None):
    """Values and bounds of o, lse (and with do: dq, dk, dv) in 64 bits.

    es: scores are fp32 sums of D exact products; a sum of n terms is off by at
    most n 2^-23 of the sum of absolute values (adders that cut off: one whole
    step a term).  ep, relative to p: es; 2^-22 of the largest score (scale
    times log2 e, and the row's lse, are each rounded); the fused scale and
    shift, and the exponential's 2 ulp, 2^-18 where p > 2^-64.  For the
    normalised p once more the same, for the sum.
    P is rounded to `dtype`: h of itself, or f (half the least subnormal)
    against a row maximum of 1; products with P sum 16 exact products a step.
    """
    B, H, N, D = q.shape
    Bk, Hk, M, _ = k.shape
    G, fi = H // Hk, torch.finfo(dtype)
    h, f = fi.eps / 2, fi.smallest_normal * fi.eps / 2
    dev = q.device
    z = lambda *s: torch.zeros(s, dtype=torch.float64, device=dev)  # noqa: E731
    r = dict(o=z(B, H, N, D), lse=torch.full((B, H, N), -torch.inf, dtype=torch.float64, device=dev))
    b = dict(o=z(B, H, N, D), lse=z(B, H, N))
    if do is not None:
        for t in (r, b):
            t.update(dq=z(B, H, N, D), dk=z(Bk, Hk, M, D), dv=z(Bk, Hk, M, D))
    q, k, v = q.double(), k.double(), v.double()
    do = None if do is None else do.double()
    for bi in range(B):
        kb = bi if Bk == B else 0
        on = allowed[kb].nonzero()[:, 0]
        if len(on) == 0:
            continue
        for hi in range(H):
            hk = hi // G
            Q, K, V = q[bi, hi], k[kb, hk][on], v[kb, hk][on]
            s = scale * Q @ K.T
            es = D * 2.0 ** -23 * scale * (Q.abs() @ K.abs().T)
            ep = es + s.abs().amax(-1, keepdim=True) * 2.0 ** -22 + 2.0 ** -18
            lse = torch.logsumexp(s, -1, keepdim=True)
            p = torch.exp(s - lse)
            epn = ep + (p * ep).sum(-1, keepdim=True)
            o = p @ V
            acc = (len(on) / 16 + 16) * 2.0 ** -23
            bo = (p * (h + epn + acc) + f) @ V.abs()
            r["o"][bi, hi], b["o"][bi, hi] = o, bo
            r["lse"][bi, hi] = lse[:, 0]
            b["lse"][bi, hi] = (p * ep).sum(-1) + acc + 2.0 ** -21 * (1 + lse[:, 0].abs())
            if do is None:
                continue
            dO = do[bi, hi]
            dp = dO @ V.T
            Dl = (dO * o).sum(-1, keepdim=True)
            ds = p * (dp - Dl)
            edp = D * 2.0 ** -23 * (dO.abs() @ V.abs().T)
            eD = (dO.abs() * (bo + half_ulp(o, dtype) + o.abs() * D * 2.0 ** -23)).sum(-1, keepdim=True)
            pb = b["lse"][bi, hi][:, None] + ep  # p from the stored lse
            bds = ds.abs() * (h + pb + 2.0 ** -22) + p * (edp + eD) * (1 + pb) + f
            rows = ((B * G if Bk < B else G) * N / 16 + 16) * 2.0 ** -23
            r["dq"][bi, hi] = scale * ds @ K
            b["dq"][bi, hi] = scale * ((bds + ds.abs() * acc) @ K.abs())
            r["dk"][kb, hk].index_add_(0, on, scale * ds.T @ Q)
            b["dk"][kb, hk].index_add_(0, on, scale * (bds + ds.abs() * rows).T @ Q.abs())
            r["dv"][kb, hk].index_add_(0, on, p.T @ dO)
            b["dv"][kb, hk].index_add_(0, on, (p * (h + pb + rows) + f).T @ dO.abs())
    for n in r:
        if n != "lse":
            b[n] = b[n] + half_ulp(r[n], dtype)
    return r, b


def check_cross(got, r, b, names):
    for n in names:
        if n == "lse":
            none = torch.isinf(r[n])
            assert (got[n][none] == -torch.inf).all(), "lse of rows without keys"
            within(got[n][~none], r[n][~none], b[n][~none], n)
        else:
            within(got[n], r[n], b[n], n)
