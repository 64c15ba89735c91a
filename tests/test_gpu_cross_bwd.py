"""scope.cross_attn_backward against the formula in 64 bits (bounds in op_ref.py) and against
differences of the forward kernel."""
import pytest
import torch

import cluster_guided_sparse_b200 as scope
import op_ref as R
from test_gpu_cross import BF16, CASES, DEV, F16, keys_kw, rand

pytestmark = pytest.mark.gpu

MORE = [  # rows of one key set over many tiles, keys over many tiles, and both
    (BF16, 128, "bhnd", 1, 1, 2, 2, 2100, 60, "all"),
    (F16, 64, "bnhd", 1, 1, 1, 1, 1500, 1300, "len"),
    (BF16, 64, "bhnd", 2, 1, 6, 2, 900, 200, "mask"),
    (BF16, 128, "slice", 1, 1, 30, 30, 700, 400, "mask"),
]


def grads(q, k, v, do, scale=None, **kw):
    o, lse = scope.cross_attn(q, k, v, return_lse=True, scale=scale, **kw)
    dq, dk, dv = scope.cross_attn_backward(do, q, k, v, o, lse, scale=scale, **kw)
    return dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv)


@pytest.mark.parametrize("case", CASES + MORE, ids=lambda c: "-".join(map(str, c)))
def test_backward_against_64_bits(case):
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


@pytest.mark.parametrize("N,M", [(0, 5), (5, 0), (0, 0)])
def test_no_rows_or_no_keys(N, M):
    q, k = rand((2, 4, N, 64), BF16, 1), rand((2, 2, M, 64), BF16, 2)
    for kw in ({}, dict(kv_len=torch.full((2,), M, dtype=torch.int32, device=DEV)),
               dict(kv_mask=torch.ones((2, M), dtype=torch.bool, device=DEV))):
        got = grads(q, k, k, q, **kw)
        scope.ops_sync_status()
        assert (got["dq"] == 0).all() and (got["dk"] == 0).all() and (got["dv"] == 0).all()
        assert got["dk"].shape == k.shape


def test_backward_against_differences_of_the_kernel():
    """<do, o> along a direction, f16: the kernel's difference may be off by the forward's bounds,
    weighed with |do|, on both sides over 2h; the same difference in 64 bits has to meet the
    gradients' slope within h^2 / 6 of the third derivative and the gradients' bounds.  The third
    derivative is estimated in 64 bits from differences of the formula's slope at both ends."""
    B, H, Hk, N, M, D, h = 2, 4, 2, 70, 90, 64, 2.0 ** -5
    q, k, v = rand((B, H, N, D), F16, 1), rand((B, Hk, M, D), F16, 2), rand((B, Hk, M, D), F16, 3)
    do = rand((B, H, N, D), F16, 4)
    u = [rand(t.shape, F16, s, gain=0.25) for t, s in ((q, 5), (k, 6), (v, 7))]
    on = R.allowed_keys(B, M, device=DEV)
    ends = {s: [(t + s * h * d).to(F16) for t, d in zip((q, k, v), u)] for s in (1, -1)}
    # the steps that the rounded ends make
    steps = [(ends[1][i].double() - ends[-1][i].double()) / 2 for i in range(3)]
    mid = [(ends[1][i].double() + ends[-1][i].double()) / 2 for i in range(3)]
    got = exact = slack = 0.0
    slope = {}
    for s in (1, -1):
        r, b = R.cross(*ends[s], on, D ** -0.5, F16, do)
        o = scope.cross_attn(*ends[s])
        got += s * float((o.double() * do.double()).sum()) / 2
        exact += s * float((r["o"] * do.double()).sum()) / 2
        slack += float((b["o"] * do.double().abs()).sum()) / 2
        slope[s] = sum(float((r[n] * d).sum()) for n, d in zip(("dq", "dk", "dv"), steps))
    assert abs(got - exact) <= slack
    r0, _ = R.cross(*mid, on, D ** -0.5, F16, do)
    s0 = sum(float((r0[n] * d).sum()) for n, d in zip(("dq", "dk", "dv"), steps))
    third = abs(slope[1] + slope[-1] - 2 * s0)  # step^3 f''' to the next order, which doubling covers
    assert abs(exact - s0) <= 2 * third / 6 + 1e-9 * abs(s0)
    m16 = [t.to(F16) for t in mid]
    rm, bm = R.cross(*m16, on, D ** -0.5, F16, do)
    g = grads(*m16, do)
    sk = sum(float((g[n].double() * d).sum()) for n, d in zip(("dq", "dk", "dv"), steps))
    sm = sum(float((rm[n] * d).sum()) for n, d in zip(("dq", "dk", "dv"), steps))
    bound = sum(float((bm[n] * d.abs()).sum()) for n, d in zip(("dq", "dk", "dv"), steps))
    assert abs(sk - sm) <= bound


@pytest.mark.parametrize("mask", ["len", "mask"])
def test_masked_keys_may_hold_anything(mask):
    q, k, v = rand((2, 2, 300, 64), BF16, 1), rand((2, 2, 200, 64), BF16, 2), rand((2, 2, 200, 64), BF16, 3)
    do, kw = rand((2, 2, 300, 64), BF16, 4), keys_kw(mask, 2, 200)
    ref = grads(q, k, v, do, **kw)
    off = ~R.allowed_keys(2, 200, device=DEV, **kw)
    for bad in (float("nan"), float("-inf"), torch.finfo(BF16).min):
        for t in (k, v):
            t.copy_(torch.where(off[:, None, :, None], torch.tensor(bad, dtype=BF16, device=DEV), t))
        got = grads(q, k, v, do, **kw)
        for n in ref:
            assert torch.equal(got[n], ref[n]), n
    assert (ref["dk"].transpose(1, 2)[off] == 0).all() and (ref["dv"].transpose(1, 2)[off] == 0).all()


@pytest.mark.parametrize("N,M", [(150, 200), (1, 2000)])
def test_outputs_given_and_only_they_are_written(N, M):
    q, do = rand((2, 4, N, 128), BF16, 1), rand((2, 4, N, 128), BF16, 4)
    k, v = rand((2, 2, M, 128), BF16, 2), rand((2, 2, M, 128), BF16, 3)
    m = keys_kw("mask", 2, M)
    ref = grads(q, k, v, do, **m)
    big = torch.full((2, N + 5, 9, 128), 7.0, dtype=BF16, device=DEV)
    kv = torch.full((2, M + 3, 6, 128), 7.0, dtype=BF16, device=DEV)
    dq = big[:, 2:N + 2, 1:9:2].transpose(1, 2)
    dk, dv = (kv[:, 1:M + 1, i:i + 4:2].transpose(1, 2) for i in (1, 2))
    scope.cross_attn_backward(do, q, k, v, ref["o"], ref["lse"], dq=dq, dk=dk, dv=dv, **m)
    for n, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        assert torch.equal(t, ref[n]), n
        t.fill_(7.0)
    assert (big == 7.0).all() and (kv == 7.0).all()


def test_other_stream_and_graph():
    q, do = rand((2, 4, 100, 64), BF16, 1), rand((2, 4, 100, 64), BF16, 4)
    k, v = rand((1, 2, 300, 64), BF16, 2), rand((1, 2, 300, 64), BF16, 3)
    kw = keys_kw("mask", 1, 300)
    ref = grads(q, k, v, do, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = scope.cross_attn_backward(do, q, k, v, ref["o"], ref["lse"], stream=side, **kw)
    side.synchronize()
    for t, n in zip(got, ("dq", "dk", "dv")):
        assert torch.equal(t, ref[n])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = grads(q, k, v, do, **kw)
    q.copy_(rand((2, 4, 100, 64), BF16, 11))
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    ref = grads(q, k, v, do, **kw)
    for n in ref:
        assert torch.equal(out[n], ref[n]), n
    del g


def test_shared_states_equal_repeated_ones():
    """Gradients of states shared by the batch and of shared key heads: the sums of those that
    repeated states get (each of which is rounded once)."""
    q, do = rand((3, 4, 130, 64), BF16, 1), rand((3, 4, 130, 64), BF16, 4)
    k, v = rand((1, 2, 150, 64), BF16, 2), rand((1, 2, 150, 64), BF16, 3)
    got = grads(q, k, v, do)
    rep = lambda t: t.repeat(3, 1, 1, 1).repeat_interleave(2, 1).contiguous()  # noqa: E731
    one = grads(q, rep(k), rep(v), do)
    assert torch.equal(got["o"], one["o"]) and torch.equal(got["lse"], one["lse"])
    on = R.allowed_keys(1, 150, device=DEV)
    r, b = R.cross(q, k, v, on, 0.125, BF16, do)
    _, bo = R.cross(q, rep(k), rep(v), on.repeat(3, 1), 0.125, BF16, do)
    for n in ("dk", "dv"):
        s = one[n].double().view(3, 2, 2, 150, 64).sum((0, 2))[None]
        R.within(got[n], s, b[n] + bo[n].view(3, 2, 2, 150, 64).sum((0, 2))[None], n)


def test_refusals_on_the_device():
    q, k = rand((2, 2, 8, 64), BF16, 1), rand((2, 2, 9, 64), BF16, 2)
    o, lse = scope.cross_attn(q, k, k, return_lse=True)
    with pytest.raises(ValueError, match="lse"):
        scope.cross_attn_backward(q, q, k, k, o, lse[:, :1])
    with pytest.raises(ValueError, match="lse"):
        scope.cross_attn_backward(q, q, k, k, o, lse.double())
    with pytest.raises(scope.ScopeError, match="overlap"):
        scope.cross_attn_backward(q, q, k, k, o, lse, dq=q)


@pytest.mark.parametrize("N", [1, 3, 40, 300])
@pytest.mark.parametrize("M,mask", [(1, "all"), (300, "len"), (300, "mask"), (5000, "len")])
def test_a_single_key_has_no_gradient_through_its_score(N, M, mask):
    """p is 1 whatever the score: dq and dk are zero, not what roundings leave; dv is the sum of do,
    rounded once after a sum in 32 bits of p and do within 2^-18 + 2^-8 of themselves (p next to 1
    may round to its 16-bit neighbour)."""
    q, do = rand((2, 2, N, 64), BF16, 1), rand((2, 2, N, 64), BF16, 4)
    k, v = rand((2, 2, M, 64), BF16, 2), rand((2, 2, M, 64), BF16, 3)
    kw = {}
    if mask == "len":
        kw = dict(kv_len=torch.ones(2, dtype=torch.int32, device=DEV))
    elif mask == "mask":
        kw = dict(kv_mask=torch.zeros((2, M), dtype=torch.bool, device=DEV))
        kw["kv_mask"][:, 123] = True
    got = grads(q, k, v, do, **kw)
    scope.ops_sync_status()
    at = 123 if mask == "mask" else 0
    assert (got["dq"] == 0).all() and (got["dk"] == 0).all()
    want, size = do.double().sum(2), do.double().abs().sum(2)
    assert ((got["dv"][:, :, at].double() - want).abs() <= size * (2.0 ** -18 + 2.0 ** -8) + want.abs() * 2.0 ** -8).all()
    assert torch.equal(got["o"], v[:, :, at:at + 1].expand_as(q))
