"""scope.cross_attn against its 64-bit form (bounds in op_ref.py): types,
layouts, lengths from none and one to long ones on either side, key lists,
shared keys and key heads, rows without keys."""
import pytest
import torch

import cluster_guided_sparse_b200 as scope
import op_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F16 = torch.bfloat16, torch.float16


def rand(shape, dtype, seed, layout="bhnd", gain=1.3):
    B, H, N, D = shape
    g = torch.Generator(device=DEV).manual_seed(seed)
    if layout == "bnhd":
        return (gain * torch.randn((B, N, H, D), generator=g, device=DEV)).to(dtype).transpose(1, 2)
    if layout == "slice":
        return (gain * torch.randn((B, 2 * H, N + 3, D), generator=g, device=DEV)).to(dtype)[:, ::2, 2:N + 2]
    return (gain * torch.randn(shape, generator=g, device=DEV)).to(dtype)


def keys_kw(mask, Bk, M, seed=5):
    """kv_len / kv_mask of a kind; the first entry may read nothing for kinds with 'none'."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    if mask == "len":
        return dict(kv_len=(torch.rand(Bk, generator=g, device=DEV) * M).ceil().int())
    if mask == "len none":
        n = (torch.rand(Bk, generator=g, device=DEV) * M).ceil().int()
        n[0] = 0
        return dict(kv_len=n)
    if mask == "mask":
        return dict(kv_mask=torch.rand((Bk, M), generator=g, device=DEV) < 0.6)
    if mask == "mask none":
        m = torch.rand((Bk, M), generator=g, device=DEV) < 0.6
        m[0] = False
        return dict(kv_mask=m)
    return {}


CASES = [  # dtype, D, layout, B, Bk, H, Hk, N, M, mask
    (BF16, 128, "bhnd", 1, 1, 1, 1, 1, 1, "all"),
    (F16, 64, "bhnd", 2, 2, 2, 2, 1, 7, "len"),
    (BF16, 64, "bnhd", 3, 3, 4, 2, 5, 128, "all"),
    (BF16, 128, "bnhd", 2, 2, 4, 4, 127, 129, "mask"),
    (F16, 128, "slice", 2, 2, 3, 3, 128, 127, "len none"),
    (BF16, 64, "slice", 2, 2, 3, 1, 129, 256, "mask none"),
    (F16, 64, "bnhd", 4, 1, 8, 2, 61, 333, "len"),
    (BF16, 128, "bhnd", 3, 1, 6, 3, 200, 77, "mask"),
    (BF16, 128, "bhnd", 2, 1, 2, 2, 33, 50, "len none"),
    (BF16, 128, "bhnd", 1, 1, 2, 2, 700, 513, "all"),
    (F16, 128, "bnhd", 1, 1, 2, 1, 257, 1000, "mask"),
    (BF16, 64, "bhnd", 1, 1, 1, 1, 3, 9001, "all"),
    (BF16, 128, "bhnd", 2, 2, 4, 2, 1, 4097, "mask"),
    (F16, 64, "bhnd", 2, 2, 3, 3, 77, 2500, "len"),
    (BF16, 64, "bhnd", 5, 5, 24, 24, 1, 300, "len"),
    (BF16, 128, "bnhd", 1, 1, 40, 40, 1030, 130, "all"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_cross_against_64_bits(case):
    dtype, D, layout, B, Bk, H, Hk, N, M, mask = case
    q = rand((B, H, N, D), dtype, 1, layout)
    k, v = rand((Bk, Hk, M, D), dtype, 2, layout), rand((Bk, Hk, M, D), dtype, 3, layout)
    kw = keys_kw(mask, Bk, M)
    o, lse = scope.cross_attn(q, k, v, return_lse=True, **kw)
    scope.ops_sync_status()
    r, b = R.cross(q, k, v, R.allowed_keys(Bk, M, device=DEV, **kw), D ** -0.5, dtype)
    R.check_cross(dict(o=o, lse=lse), r, b, ("o", "lse"))
    o2, lse2 = scope.cross_attn(q, k, v, return_lse=True, **kw)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert torch.equal(o, scope.cross_attn(q, k, v, **kw))


@pytest.mark.parametrize("N,M", [(0, 5), (5, 0), (0, 0)])
def test_no_rows_or_no_keys(N, M):
    q, k = rand((2, 4, N, 64), BF16, 1), rand((2, 2, M, 64), BF16, 2)
    for kw in ({}, dict(kv_len=torch.full((2,), M, dtype=torch.int32, device=DEV)),
               dict(kv_mask=torch.ones((2, M), dtype=torch.bool, device=DEV))):
        o, lse = scope.cross_attn(q, k, k, return_lse=True, **kw)
        scope.ops_sync_status()
        assert o.shape == q.shape and (o == 0).all() and (lse == -torch.inf).all()


def test_lengths_outside_the_keys_are_held_to_them():
    q, k, v = rand((3, 2, 9, 64), BF16, 1), rand((3, 2, 140, 64), BF16, 2), rand((3, 2, 140, 64), BF16, 3)
    n = torch.tensor([-5, 141, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    o = scope.cross_attn(q, k, v, kv_len=n)
    assert (o[0] == 0).all() and torch.equal(o[1:], scope.cross_attn(q, k, v)[1:])


@pytest.mark.parametrize("mask", ["len", "mask"])
@pytest.mark.parametrize("N,M", [(300, 200), (2, 3000)])
def test_masked_keys_may_hold_anything(mask, N, M):
    q, k, v = rand((2, 2, N, 64), F16, 1), rand((2, 2, M, 64), F16, 2), rand((2, 2, M, 64), F16, 3)
    kw = keys_kw(mask, 2, M)
    ref = scope.cross_attn(q, k, v, **kw)
    off = ~R.allowed_keys(2, M, device=DEV, **kw)
    assert off.any()
    for bad in (float("nan"), float("inf"), torch.finfo(F16).min):
        for t in (k, v):
            t.copy_(torch.where(off[:, None, :, None], torch.tensor(bad, dtype=F16, device=DEV), t))
        assert torch.equal(scope.cross_attn(q, k, v, **kw), ref)


def test_a_bad_row_stays_in_its_row():
    q, k, v = rand((1, 2, 200, 128), BF16, 1), rand((1, 2, 300, 128), BF16, 2), rand((1, 2, 300, 128), BF16, 3)
    ref = scope.cross_attn(q, k, v)
    q[0, 1, 50, 3] = float("nan")
    o = scope.cross_attn(q, k, v)
    assert torch.isnan(o[0, 1, 50]).all()
    o[0, 1, 50] = ref[0, 1, 50]
    assert torch.equal(o, ref)


def test_scores_far_apart():
    """Scores that grow along the keys by far more than the range of an exponential: the running
    maximum moves in every tile."""
    M = 1024
    q = torch.ones((1, 1, 130, 64), dtype=BF16, device=DEV)
    k = (torch.arange(M, device=DEV).float()[:, None] / 8).expand(M, 64)[None, None].to(BF16).contiguous()
    v = rand((1, 1, M, 64), BF16, 3)
    for kk in (k, k.flip(2).contiguous(), -k):
        o, lse = scope.cross_attn(q, kk, v, return_lse=True, scale=1.0)
        r, b = R.cross(q, kk, v, R.allowed_keys(1, M, device=DEV), 1.0, BF16)
        R.check_cross(dict(o=o, lse=lse), r, b, ("o", "lse"))


@pytest.mark.parametrize("scale", [1e-30, 1e-3, 1.0])
def test_scale(scale):
    q, k, v = rand((1, 2, 70, 64), F16, 1, gain=0.5), rand((1, 2, 150, 64), F16, 2, gain=0.5), rand((1, 2, 150, 64), F16, 3)
    o, lse = scope.cross_attn(q, k, v, scale=scale, return_lse=True, kv_len=torch.tensor([149], dtype=torch.int32, device=DEV))
    r, b = R.cross(q, k, v, torch.arange(150, device=DEV)[None] < 149, scale, F16)
    R.check_cross(dict(o=o, lse=lse), r, b, ("o", "lse"))


def test_only_the_given_rows_are_written():
    big = torch.full((2, 7, 60, 128), 7.0, dtype=BF16, device=DEV)
    out = big[:, 1:7:2, 11:48]
    q, k, v = rand((2, 3, 37, 128), BF16, 1), rand((2, 3, 90, 128), BF16, 2), rand((2, 3, 90, 128), BF16, 3)
    scope.cross_attn(q, k, v, out=out)
    assert torch.equal(out, scope.cross_attn(q, k, v))
    out.fill_(7.0)
    assert (big == 7.0).all()


def test_one_mask_row_for_the_batch():
    q, k, v = rand((3, 2, 20, 64), BF16, 1), rand((3, 2, 90, 64), BF16, 2), rand((3, 2, 90, 64), BF16, 3)
    m = torch.rand((1, 90), device=DEV) < 0.5
    assert torch.equal(scope.cross_attn(q, k, v, kv_mask=m.expand(3, -1)), scope.cross_attn(q, k, v, kv_mask=m.repeat(3, 1)))
    assert torch.equal(scope.cross_attn(q, k, v, kv_mask=m.expand(3, -1)),
                       scope.cross_attn(q, k, v, kv_mask=m.repeat(3, 1).to(torch.uint8) * 255))


def test_long_mask_lists():
    """A mask over more keys than a block scans at once, against the kept keys alone."""
    M = 40000
    q, k, v = rand((1, 2, 33, 64), BF16, 1), rand((1, 2, M, 64), BF16, 2), rand((1, 2, M, 64), BF16, 3)
    m = torch.rand((1, M), generator=torch.Generator(device=DEV).manual_seed(4), device=DEV) < 0.01
    on = m[0].nonzero()[:, 0]
    o, lse = scope.cross_attn(q, k, v, kv_mask=m, return_lse=True)
    r, b = R.cross(q, k[:, :, on], v[:, :, on], R.allowed_keys(1, len(on), device=DEV), 64 ** -0.5, BF16)
    R.check_cross(dict(o=o, lse=lse), r, b, ("o", "lse"))


def test_other_stream_and_two_graphs():
    q, k, v = rand((2, 3, 50, 64), BF16, 1), rand((2, 3, 1500, 64), BF16, 2), rand((2, 3, 1500, 64), BF16, 3)
    m = keys_kw("mask", 2, 1500)["kv_mask"]
    ref = scope.cross_attn(q, k, v, kv_mask=m)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = scope.cross_attn(q, k, v, kv_mask=m, stream=side)
    side.synchronize()
    assert torch.equal(o, ref)
    graphs, outs = [], []
    q2 = rand((2, 3, 50, 64), BF16, 8)
    for x in (q, q2):  # each graph holds a workspace of its own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(scope.cross_attn(x, k, v, kv_mask=m))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], ref) and torch.equal(outs[1], scope.cross_attn(q2, k, v, kv_mask=m))
    del graphs, g


def test_offsets_past_32_bits():
    """Key rows whose element offset passes 2^32 (a head of a long, interleaved cache)."""
    M, H, D = 70000, 512, 128
    cache = torch.empty((1, M, H, D), dtype=BF16, device=DEV)  # 9.2 GB
    part = cache[:, :, -2:].transpose(1, 2)
    k = rand((1, 2, M, D), BF16, 2)
    part.copy_(k)
    q = rand((1, 2, 5, D), BF16, 1)
    assert part.stride(2) * M > 2 ** 32
    assert torch.equal(scope.cross_attn(q, part, part), scope.cross_attn(q, k, k))


def test_refusals_on_the_device():
    q, k = rand((2, 2, 8, 64), BF16, 1), rand((2, 2, 9, 64), BF16, 2)
    with pytest.raises(scope.ScopeError, match="overlap"):
        scope.cross_attn(q, k[:1].expand(2, -1, -1, -1), k)
    with pytest.raises(ValueError, match="cpu"):
        scope.cross_attn(q, k, k, kv_len=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(scope.ScopeError, match="overlap"):
        scope.cross_attn(q, k, k, out=q)
