"""What the 16-bit softmax weights of cross attention's products may cost, and no more: flat rows over long keys, whose
weights lie far below f16's smallest normal number, and values and keys with a common offset, where the given o's rounding
would fill ds.  Bounds tighter than op_ref.py's:

Each weight is within h (half a step of the type, relative) + pb of itself, whatever its size.  With the given o,
x = dp - do . o differs from dp - D by eD = |do . (o given - o)| at most (and the fp32 sum of do . o).  t = p x is held in
16 bits, so off by (h + pb) |t|, p edp for dp's own sum, and half the least subnormal f.  The kernel takes D - do . o back as
the sum of the unrounded t: edelta = sum over keys of p (|x| (pb + acc) + edp).  dq = scale (sum t k - (D - do . o) sum p k);
dk's ds uses the corrected D, off by edelta and 2^-23 of |D|.  pb, edp, acc as in op_ref.cross; each result is rounded once."""
import pytest
import torch

import cluster_guided_sparse_b200 as scope
import op_ref as R
from test_gpu_cross import BF16, DEV, F16, rand
from test_gpu_cross_bwd import grads

pytestmark = pytest.mark.gpu


def tight(q, k, v, do, o, scale, dtype):
    """(values, bounds, values with D = do . o uncorrected) of dq, dk, dv of one head in 64 bits; o: the kernel's."""
    D, M, N = q.shape[-1], k.shape[0], q.shape[0]
    fi = torch.finfo(dtype)
    h, f = fi.eps / 2, fi.smallest_normal * fi.eps / 2
    q, k, v, do, o = (t.double() for t in (q, k, v, do, o))
    s = scale * q @ k.T
    ep = D * 2.0 ** -23 * scale * (q.abs() @ k.abs().T) + s.abs().amax(-1, keepdim=True) * 2.0 ** -22 + 2.0 ** -18
    p = torch.softmax(s, -1)
    acc = (M / 16 + 16) * 2.0 ** -23
    pb = ep + (p * ep).sum(-1, keepdim=True) + acc + 2.0 ** -21 * (1 + torch.logsumexp(s, -1, keepdim=True).abs())
    dp, exact_o = do @ v.T, p @ v
    Dl = (do * exact_o).sum(-1, keepdim=True)
    edp = D * 2.0 ** -23 * (do.abs() @ v.abs().T)
    off = (do * (o - exact_o)).sum(-1, keepdim=True)
    eD = off.abs() + D * 2.0 ** -23 * (do.abs() * o.abs()).sum(-1, keepdim=True)
    x = (dp - Dl).abs() + eD
    edelta = (p * (x * (pb + acc) + edp)).sum(-1, keepdim=True)
    et = p * (x * (h + pb + 2.0 ** -22) + edp) + f
    ds = p * (dp - Dl)
    rows = (N / 16 + 16) * 2.0 ** -23
    eds = p * (((dp - Dl).abs() + edelta) * (h + pb + 2.0 ** -22) + edp + edelta + 2.0 ** -23 * Dl.abs()) + f
    val = dict(dq=scale * ds @ k, dk=scale * ds.T @ q, dv=p.T @ do)
    bound = dict(dq=scale * ((et + p * x * acc) @ k.abs() + edelta * (p @ k.abs()) + eD * ((p * (h + pb + acc)) @ k.abs())),
                 dk=scale * (eds + ds.abs() * rows).T @ q.abs(), dv=(p * (h + pb + rows)).T @ do.abs())
    for n in val:
        bound[n] = bound[n] + R.half_ulp(val[n], dtype)
    ds = p * (dp - Dl - off)
    return val, bound, dict(dq=scale * ds @ k, dk=scale * ds.T @ q)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("M", [65408, 260112])  # p is 256.5 and 64.5 steps of f16's subnormal numbers
@pytest.mark.parametrize("N", [6, 130])
def test_flat_rows_over_long_keys(M, N, D):
    """Every weight is 1 / M: the scores are exactly zero, their exponentials' sums exact, so p is within 2^-17 of itself
    (its lse of some 12 and its shift are rounded to 24 bits) before h for its 16 bits."""
    q, do = torch.zeros((1, 1, N, D), dtype=F16, device=DEV), rand((1, 1, N, D), F16, 4, gain=500.0).abs()
    k, v = rand((1, 1, M, D), F16, 2), rand((1, 1, M, D), F16, 3)
    got = grads(q, k, v, do)
    scope.ops_sync_status()
    dv = do.double().sum(2, keepdim=True) / M
    bound = dv * (2.0 ** -11 + 2.0 ** -17 + N * 2.0 ** -23) + R.half_ulp(dv, F16)
    R.within(got["dv"], dv, bound, "dv")
    val, b, _ = tight(q[0, 0], k[0, 0], v[0, 0], do[0, 0], got["o"][0, 0], D ** -0.5, F16)
    R.within(got["dq"][0, 0], val["dq"], b["dq"], "dq")
    assert (got["dk"] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("N,M", [(8, 300), (8, 3000), (700, 129)])  # whole, split keys, rows over many tiles
@pytest.mark.parametrize("D", [64, 128])
def test_values_and_keys_with_a_common_offset(dtype, N, M, D):
    c, q, do = 16.0, rand((1, 2, N, D), dtype, 1), rand((1, 2, N, D), dtype, 4, gain=0.5)
    g = torch.Generator(device=DEV).manual_seed(9)
    v = (c + 0.125 * torch.randint(-8, 9, (1, 2, M, D), generator=g, device=DEV)).to(dtype)
    k = rand((1, 2, M, D), dtype, 2, gain=0.5) + 2
    got = grads(q, k, v, do)
    scope.ops_sync_status()
    caught = dict(dq=False, dk=False)
    for h in range(2):
        val, b, wrong = tight(q[0, h], k[0, h], v[0, h], do[0, h], got["o"][0, h], D ** -0.5, dtype)
        for n in val:
            R.within(got[n][0, h], val[n], b[n], n)
        for n in caught:  # a kernel that kept do . o of the rounded o would be seen
            caught[n] |= bool(((wrong[n] - val[n]).abs() > b[n]).any())
    assert caught["dq"] and (caught["dk"] or N > 8), caught


@pytest.mark.parametrize("N", [5, 200])
@pytest.mark.parametrize("M", [200, 4096])
def test_a_tail_of_small_weights_behind_a_large_one(M, N):
    """Forward: one key of weight 1 and value 0, the others of weight P = 16.5 2^-24 and value 1 (16.5 of
    f16's subnormal steps): o = T / (1 + T), T the tail's sum.  P is known to 2^-18 (its exponent's scale is
    rounded, 2^-23 of 20 and less, and the exponential 2^-22), its 16 bits add h = 2^-11, the sums acc.  The
    row's sum is four fp32 sums of a quarter of the weights each; the one with the large weight rounds each
    addition to 2^-24 of itself, at most, so lse is off by M / 4 of those and 2^-21 of itself."""
    H, D = 150, 64  # more items than CTAs: the keys are not split
    q, k = (torch.zeros((1, H, n, D), dtype=F16, device=DEV) for n in (N, M))
    q[..., 0], k[..., 0, 0] = 1.0, 1.0
    v = torch.ones((1, H, M, D), dtype=F16, device=DEV)
    v[:, :, 0] = 0.0
    P = 16.5 * 2.0 ** -24
    scale = -float(torch.log(torch.tensor(P, dtype=torch.float64)))
    o, lse = scope.cross_attn(q, k, v, scale=scale, return_lse=True)
    scope.ops_sync_status()
    T = (M - 1) * P
    want = torch.full_like(o, T / (1 + T), dtype=torch.float64)
    acc = (M / 16 + 16) * 2.0 ** -23
    R.within(o, want, want * (2.0 ** -11 + 2.0 ** -17 + 2 * acc) + R.half_ulp(want, F16), "o")
    want = torch.full_like(lse, scale, dtype=torch.float64) + torch.log1p(torch.tensor(T, dtype=torch.float64))
    R.within(lse, want, 2.0 ** -21 * want + M / 4 * 2.0 ** -24, "lse")
