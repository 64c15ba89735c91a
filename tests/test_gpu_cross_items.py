"""Cross attention where every CTA of the forward and dq kernels runs three work items or more (148 CTAs,
more than 444 items): buffers that come round again, results that leave while the next item runs, items
without keys or without a second row tile between others, steps that run on over item borders.  Against
64 bits (bounds in op_ref.py)."""
import pytest
import torch

import cluster_guided_sparse_b200 as scope
import op_ref as R
from test_gpu_cross import BF16, DEV, F16, rand
from test_gpu_cross_bwd import grads

pytestmark = pytest.mark.gpu

# dtype, D, layout, B, Bk, H, Hk, N, M, mask ("0": every third entry reads nothing); forward items: 256 rows of a key
# set, dq items: 128 rows
CASES = [
    (BF16, 128, "bhnd", 8, 8, 60, 60, 100, 60, "all"),      # 480 of one row tile and one key tile
    (F16, 64, "bnhd", 8, 8, 60, 60, 100, 60, "len0"),
    (BF16, 64, "bhnd", 8, 8, 28, 28, 300, 130, "mask0"),    # 448, two row tiles and one in turn
    (BF16, 128, "bnhd", 8, 8, 28, 28, 300, 130, "len0"),
    (F16, 128, "bhnd", 8, 8, 224, 56, 61, 150, "len0"),     # 448, folded heads
    (BF16, 64, "bnhd", 8, 8, 120, 60, 61, 150, "mask0"),    # 480 of one folded row tile
    (BF16, 128, "bhnd", 1, 1, 150, 150, 700, 200, "all"),   # 450, the last of a head with two row tiles
    (F16, 64, "bhnd", 150, 150, 3, 3, 40, 70, "len0"),
    (F16, 64, "slice", 8, 8, 60, 60, 129, 300, "mask0"),    # second row tiles of one row
    (BF16, 64, "bhnd", 3, 1, 150, 150, 200, 100, "len"),    # states shared by the batch, folded over it
    (BF16, 128, "slice", 8, 8, 60, 60, 128, 64, "mask0"),   # tiles that end with their rows and keys
]


def keys_kw(mask, Bk, M):
    g = torch.Generator(device=DEV).manual_seed(5)
    if mask.startswith("len"):
        n = (torch.rand(Bk, generator=g, device=DEV) * M).ceil().int()
        if mask == "len0":
            n[1::3] = 0
        return dict(kv_len=n)
    if mask.startswith("mask"):
        m = torch.rand((Bk, M), generator=g, device=DEV) < 0.6
        if mask == "mask0":
            m[1::3] = False
        return dict(kv_mask=m)
    return {}


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_many_items_against_64_bits(case):
    dtype, D, layout, B, Bk, H, Hk, N, M, mask = case
    q, do = rand((B, H, N, D), dtype, 1, layout), rand((B, H, N, D), dtype, 4, "bnhd", 0.5)
    k, v = rand((Bk, Hk, M, D), dtype, 2, layout), rand((Bk, Hk, M, D), dtype, 3, layout)
    kw = keys_kw(mask, Bk, M)
    got = grads(q, k, v, do, **kw)
    scope.ops_sync_status()
    r, b = R.cross(q, k, v, R.allowed_keys(Bk, M, device=DEV, **kw), D ** -0.5, dtype, do)
    R.check_cross(got, r, b, ("o", "lse", "dq", "dk", "dv"))
    for _ in range(3):
        again = grads(q, k, v, do, **kw)
        for n in got:
            assert torch.equal(got[n], again[n]), n
    scope.ops_sync_status()


@pytest.mark.parametrize("D", [64, 128])
def test_long_runs_of_short_items(D):
    """12000 items of one row tile and one key tile (81 a CTA): the row tile that has no rows keeps
    step with the other by barriers alone."""
    q, k, v = (rand((50, 240, n, D), BF16, s) for n, s in ((9, 1), (20, 2), (20, 3)))
    o, lse = scope.cross_attn(q, k, v, return_lse=True)
    scope.ops_sync_status()
    s = q.double() @ k.double().transpose(-1, -2) * D ** -0.5
    want = torch.logsumexp(s, -1)
    assert ((lse - want).abs() <= 2.0 ** -16 * (1 + want.abs())).all()
    p = torch.softmax(s, -1)
    # P and o are rounded once each; the scores' fp32 sums add less than 2^-14
    bound = (p @ v.double().abs()) * (2.0 ** -8 + 2.0 ** -14) + (p @ v.double()).abs() * 2.0 ** -8
    assert ((o.double() - p @ v.double()).abs() <= bound).all()
    for _ in range(20):
        assert torch.equal(o, scope.cross_attn(q, k, v))
    scope.ops_sync_status()
