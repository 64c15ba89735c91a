"""The operators as a video transformer block uses them, forward and backward: norm and rotation of q
and k, self-attention (planned sparse attention, and dense with gradients), cross attention to a prompt."""
import pytest
import torch

import cluster_guided_sparse_b200 as scope
from cluster_guided_sparse_b200 import synth

pytestmark = pytest.mark.gpu
DEV = "cuda"
GRID, D, H, B = (4, 16, 16), 64, 2, 1
N = GRID[0] * GRID[1] * GRID[2]


def ref_norm_rope(x, w, eps=1e-6):
    """[B, H, N, D] in 64 bits, differentiable."""
    n = torch.arange(N, device=DEV)
    pos = (n // (GRID[1] * GRID[2]), (n // GRID[2]) % GRID[1], n % GRID[2])
    a = torch.cat([p[:, None].double() * 10000.0 ** (-torch.arange(0, d, 2, device=DEV, dtype=torch.float64) / d)
                   for p, d in zip(pos, (16, 24, 24))], -1)
    z = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w
    c, s, z0, z1 = torch.cos(a), torch.sin(a), z[..., 0::2], z[..., 1::2]
    return torch.stack([z0 * c - z1 * s, z0 * s + z1 * c], -1).flatten(-2)


def ref_attn(q, k, v, allowed=None):
    s = q @ k.transpose(-1, -2) * D ** -0.5
    if allowed is not None:
        s = s.masked_fill(~allowed[:, None, None], -torch.inf)
    return torch.softmax(s, -1) @ v


def inputs():
    g = torch.Generator(device=DEV).manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g, device=DEV).bfloat16()  # noqa: E731
    qkv = r(3, B, N, H, D).transpose(2, 3)  # as a projection lays them out
    ctx = r(2, B, 77, H, D).transpose(2, 3)
    w = 1.0 + 0.2 * torch.randn(2, D, generator=g, device=DEV)
    return qkv, ctx, w, torch.rand((B, 77), generator=g, device=DEV) < 0.8, r(B, H, N, D)


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def test_block_forward_and_backward():
    (q, k, v), (ck, cv), w, mask, do = inputs()
    p, grid = scope.make_params(d_t=16, d_h=24, d_w=24, theta=10000.0, grid=GRID)
    qr, kr = scope.rope(q, p, grid, weight=w[0]), scope.rope(k, p, grid, weight=w[1])
    x, lse = scope.cross_attn(qr, kr, v, return_lse=True)  # M = N: dense self-attention
    y, clse = scope.cross_attn(x, ck, cv, kv_mask=mask, return_lse=True)
    dx, dck, dcv = scope.cross_attn_backward(do, x, ck, cv, y, clse, kv_mask=mask)
    dqr, dkr, dv = scope.cross_attn_backward(dx, qr, kr, v, x, lse)
    dq, dw0 = scope.rope_backward(dqr, q, p, grid, weight=w[0])
    dk, dw1 = scope.rope_backward(dkr, k, p, grid, weight=w[1])
    scope.ops_sync_status()

    leaves = [t.double().requires_grad_() for t in (q, k, v, ck, cv, w)]
    Q, K, V, CK, CV, W = leaves
    X = ref_attn(ref_norm_rope(Q, W[0]), ref_norm_rope(K, W[1]), V)
    Y = ref_attn(X, CK, CV, mask)
    G = torch.autograd.grad(Y, leaves, do.double())
    # Each stage rounds its results to 2^-8 of themselves at most; a stage's sums weigh its inputs' errors no more
    # than their values, up to the factor by which attention's difference of dp and D cancels.  Eight stages in a
    # row lie between q and dq, with independent roundings: 8 * 2^-8 in norm.
    for name, got, want in (("y", y, Y), ("dck", dck, G[3]), ("dcv", dcv, G[4]), ("dv", dv, G[2]), ("dq", dq, G[0]),
                            ("dk", dk, G[1]), ("dw q", dw0, G[5][0]), ("dw k", dw1, G[5][1])):
        assert rel(got, want) <= 8 * 2.0 ** -8, (name, rel(got, want))


def test_sparse_attention_of_rotated_rows_and_a_prompt():
    """Sparse self-attention on the operators' rows: the plan that rotates by itself reads the same
    values that scope.rope gives (each within half a step of the exact one, and 2^-18 of the pair's
    length for the angle), and cross attention takes the sparse output."""
    w = synth.WORKLOADS["small"]
    q, k, v = (t.cuda() for t in synth.make_inputs(w))
    params, grid = scope.make_params(w)
    pl = scope.plan(q, k, params, grid)
    o = scope.attn(q, k, v, pl)
    pl.sync_status()
    for x, name in ((q, "qr"), (k, "kr")):
        mine, its = scope.rope(x, params, grid), pl.view(name).view(x.shape)
        length = its.double().unflatten(-1, (-1, 2)).pow(2).sum(-1, keepdim=True).sqrt().expand(-1, -1, -1, -1, 2)
        bound = 2.0 ** -7 * its.double().abs() + 2.0 ** -17 * length.flatten(-2)
        assert ((mine.double() - its.double()).abs() <= bound).all()
    B, H, N, D = q.shape
    ctx = torch.randn((2, 1, H, 50, D), device=DEV).to(q.dtype)
    y = scope.cross_attn(o, ctx[0], ctx[1])
    scope.ops_sync_status()
    s = o.double() @ ctx[0].double().transpose(-1, -2) * D ** -0.5
    # p, v's product and y are rounded once each
    assert rel(y, torch.softmax(s, -1) @ ctx[1].double()) <= 3 * 2.0 ** -8
