"""scope.cross_attn and its gradients with up to four rows a key set (single tokens, query heads
of a group), on both sides of the sizes where other kernels take over; bounds in op_ref.py."""
import pytest
import torch

import cluster_guided_sparse_b200 as scope
import op_ref as R
from test_gpu_cross import BF16, DEV, F16, keys_kw, rand
from test_gpu_cross_bwd import grads

pytestmark = pytest.mark.gpu

CASES = [  # dtype, D, layout, B, Bk, H, Hk, N, M, mask
    (BF16, 128, "bhnd", 1, 1, 1, 1, 1, 2, "all"),
    (F16, 64, "bhnd", 3, 3, 2, 2, 1, 127, "len"),
    (BF16, 64, "bnhd", 2, 2, 5, 5, 1, 128, "mask none"),
    (BF16, 128, "slice", 2, 2, 3, 3, 1, 129, "len none"),
    (BF16, 128, "bhnd", 2, 2, 4, 2, 1, 257, "mask"),  # two heads of a group
    (F16, 128, "bhnd", 1, 1, 6, 2, 1, 513, "all"),    # three
    (BF16, 64, "bnhd", 2, 2, 8, 2, 1, 1000, "len"),   # four
    (F16, 64, "bhnd", 1, 1, 3, 3, 3, 1025, "mask"),   # three queries
    (BF16, 128, "bnhd", 2, 2, 4, 2, 2, 700, "mask"),  # two queries of two heads
    (BF16, 128, "bhnd", 4, 1, 3, 3, 1, 400, "len"),   # four entries share the states
    (F16, 64, "slice", 2, 1, 4, 2, 1, 600, "mask none"),
    (BF16, 64, "bhnd", 1, 1, 4, 1, 1, 16384, "all"),  # the most keys
    (BF16, 64, "bhnd", 1, 1, 4, 1, 1, 16385, "mask"),
    (BF16, 64, "bhnd", 1, 1, 1, 1, 5, 300, "all"),    # a row more than four
    (BF16, 128, "bhnd", 1, 1, 8, 8, 1, 9700, "len"),  # long keys of few heads
    (F16, 128, "bhnd", 8, 8, 40, 10, 1, 2100, "len"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_few_rows_against_64_bits(case):
    dtype, D, layout, B, Bk, H, Hk, N, M, mask = case
    q, do = rand((B, H, N, D), dtype, 1, layout), rand((B, H, N, D), dtype, 4, "bnhd", 0.5)
    k, v = rand((Bk, Hk, M, D), dtype, 2, layout), rand((Bk, Hk, M, D), dtype, 3, layout)
    kw = keys_kw(mask, Bk, M)
    got = grads(q, k, v, do, **kw)
    scope.ops_sync_status()
    r, b = R.cross(q, k, v, R.allowed_keys(Bk, M, device=DEV, **kw), D ** -0.5, dtype, do)
    R.check_cross(got, r, b, ("o", "lse", "dq", "dk", "dv"))
    again = grads(q, k, v, do, **kw)
    for n in got:
        assert torch.equal(got[n], again[n]), n


@pytest.mark.parametrize("N", [1, 2, 4])
def test_masked_keys_may_hold_anything(N):
    q, k, v = rand((2, 2, N, 128), BF16, 1), rand((2, 2, 700, 128), BF16, 2), rand((2, 2, 700, 128), BF16, 3)
    do = rand((2, 2, N, 128), BF16, 4)
    for mask in ("len", "mask"):
        kw = keys_kw(mask, 2, 700)
        ref = grads(q, k, v, do, **kw)
        off = ~R.allowed_keys(2, 700, device=DEV, **kw)
        for bad in (float("nan"), float("inf"), torch.finfo(BF16).min):
            k2, v2 = (torch.where(off[:, None, :, None], torch.tensor(bad, dtype=BF16, device=DEV), t) for t in (k, v))
            got = grads(q, k2, v2, do, **kw)
            for n in ref:
                assert torch.equal(got[n], ref[n]), n
        assert (ref["dk"].transpose(1, 2)[off] == 0).all() and (ref["dv"].transpose(1, 2)[off] == 0).all()


def test_a_bad_row_stays_in_its_row():
    q, k, v = rand((1, 4, 1, 64), F16, 1), rand((1, 1, 300, 64), F16, 2), rand((1, 1, 300, 64), F16, 3)
    ref = scope.cross_attn(q, k, v)
    q[0, 2, 0, 5] = float("nan")
    o = scope.cross_attn(q, k, v)
    assert torch.isnan(o[0, 2]).all()
    for h in (0, 1, 3):
        assert torch.equal(o[0, h], ref[0, h])


def test_outputs_given_and_only_they_are_written():
    q, do = rand((2, 4, 1, 64), BF16, 1), rand((2, 4, 1, 64), BF16, 4)
    k, v = rand((2, 2, 333, 64), BF16, 2), rand((2, 2, 333, 64), BF16, 3)
    m = keys_kw("mask", 2, 333)
    ref = grads(q, k, v, do, **m)
    big = torch.full((2, 4, 9, 64), 7.0, dtype=BF16, device=DEV)
    kv = torch.full((2, 336, 6, 64), 7.0, dtype=BF16, device=DEV)
    o, dq = big[:, 1:2, 1:9:2].transpose(1, 2), big[:, 2:3, 1:9:2].transpose(1, 2)
    dk, dv = (kv[:, 1:334, i:i + 4:2].transpose(1, 2) for i in (1, 2))
    scope.cross_attn(q, k, v, out=o, **m)
    scope.cross_attn_backward(do, q, k, v, ref["o"], ref["lse"], dq=dq, dk=dk, dv=dv, **m)
    for n, t in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
        assert torch.equal(t, ref[n]), n
        t.fill_(7.0)
    assert (big == 7.0).all() and (kv == 7.0).all()


def test_two_graphs_and_another_stream():
    q, do = rand((3, 4, 1, 128), BF16, 1), rand((3, 4, 1, 128), BF16, 4)
    k, v = rand((3, 4, 900, 128), BF16, 2), rand((3, 4, 900, 128), BF16, 3)
    ref = grads(q, k, v, do)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(grads(q, k, v, do))
        graphs.append(g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graphs[1].replay()
    graphs[0].replay()
    torch.cuda.synchronize()
    for out in outs:
        for n in ref:
            assert torch.equal(out[n], ref[n]), n
    del graphs
