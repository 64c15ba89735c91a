"""The operators' rows as the input of the planned sparse attention: norm and rotation by scope.rope, then scope.plan
without a grid (which takes its rows as they are), scope.attn and cross attention; each stage against 64 bits on its own
inputs (parity.py's checks and bounds)."""
import numpy as np
import pytest
import torch

import cluster_guided_sparse_b200 as scope
import parity as P
from cluster_guided_sparse_b200 import synth
from test_gpu_parity import lists_fn

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("positions", ["grid", "packed"])
@pytest.mark.parametrize("D,split", [(64, (16, 24, 24)), (128, (16, 56, 56))])
def test_normed_and_rotated_rows_through_a_plan_without_grid(D, split, positions):
    w, (q, k, v) = synth.tiny_case(N=320, D=D, H=2, grid=(0, 0, 0), d_split=split, c_q=8, c_sub=(4, 4, 4), top_p=0.6)
    q, k, v = (t.to(DEV).bfloat16() for t in (q, k, v))
    g = torch.Generator(device=DEV).manual_seed(2)
    wq, wk = (1 + 0.2 * torch.randn(D, generator=g, device=DEV) for _ in range(2))
    params, none = scope.make_params(w)
    if positions == "grid":
        where = dict(grid=scope.ScopeGrid(4, 8, 10))
    else:  # two clips of other sizes, one after another
        n = torch.arange(320, device=DEV)
        a, b = n < 200, torch.clamp(n - 200, min=0)
        where = dict(positions=torch.stack([torch.where(a, n // 50, b // 40), torch.where(a, n // 10 % 5, b // 8 % 5),
                                            torch.where(a, n % 10, b % 8)], -1).int())
    qr, kr = scope.rope(q, params, weight=wq, **where), scope.rope(k, params, weight=wk, **where)
    pl = scope.plan(qr, kr, params, none)
    o = scope.attn(qr, kr, v, pl)
    pl.sync_status()
    assert torch.equal(pl.view("qr").view(qr.shape), qr) and torch.equal(pl.view("kr").view(kr.shape), kr)
    tc = P.TieCounter()
    for h in range(w.H):
        lab, get = pl.view("q_labels")[0, h].cpu().numpy(), lists_fn(pl, w, h)
        P.check_selection(pl.view("lut")[0, h].cpu().numpy(), [pl.view("k_codes")[s, 0, h].cpu().numpy() for s in range(3)],
                          pl.view("q_sizes")[0, h].cpu().numpy(), pl.view("r")[0, h].cpu().numpy(),
                          pl.view("kh")[0, h].item(), pl.view("n")[0, h].cpu().numpy(), get, w, w.N, D, range(w.c_q), tc)
        P.check_attention(P.np64(qr[0, h]), P.np64(kr[0, h]), P.np64(v[0, h]), lab, get, P.np64(o[0, h]), np.arange(w.N))
    tc.assert_ok("lists")
    ctx = torch.randn((2, 1, w.H, 50, D), generator=g, device=DEV).bfloat16()
    y = scope.cross_attn(o, ctx[0], ctx[1], kv_len=torch.tensor([41], dtype=torch.int32, device=DEV))
    scope.ops_sync_status()
    s = o.double() @ ctx[0, :, :, :41].double().transpose(-1, -2) * D ** -0.5
    want = torch.softmax(s, -1) @ ctx[1, :, :, :41].double()
    # p, v's product and y are rounded once each
    assert float((y.double() - want).norm() / want.norm()) <= 3 * 2.0 ** -8
