"""scope.rope and scope.rope_backward against their 64-bit forms (bounds in
op_ref.py): types, head dims, layouts, axis splits, grids and positions, one
token to many, in place, on another stream, captured in a graph."""
import pytest
import torch

import cluster_guided_sparse_b200 as scope
import op_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
SPLITS = {64: (16, 24, 24), 128: (16, 56, 56)}
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def rand(shape, dtype, seed, layout="bhnd", gain=1.5):
    B, H, N, D = shape
    g = torch.Generator(device=DEV).manual_seed(seed)
    if layout == "bnhd":
        return (gain * torch.randn((B, N, H, D), generator=g, device=DEV)).to(dtype).transpose(1, 2)
    if layout == "slice":  # every second head of a larger tensor
        return (gain * torch.randn((B, 2 * H, N, D), generator=g, device=DEV)).to(dtype)[:, ::2]
    return (gain * torch.randn(shape, generator=g, device=DEV)).to(dtype)


def params(split, theta=1e4):
    return scope.make_params(d_t=split[0], d_h=split[1], d_w=split[2], theta=theta)[0]


def grid_of(g):
    return scope.ScopeGrid(*g)


CASES = [  # dtype, D, layout, B, H, grid or (positions kind, N)
    (F32, 64, "bhnd", 1, 1, (1, 1, 1)),
    (BF16, 128, "bhnd", 1, 1, (1, 1, 1)),
    (F32, 128, "bnhd", 2, 5, (3, 5, 7)),
    (F16, 64, "slice", 3, 2, (1, 1, 17)),
    (BF16, 64, "bnhd", 1, 40, (2, 3, 5)),
    (BF16, 128, "slice", 2, 7, (5, 1, 33)),
    (F16, 128, "bnhd", 1, 24, (4, 9, 16)),
    (F32, 64, "bhnd", 2, 3, ("batch", 1)),
    (BF16, 64, "bhnd", 8, 24, ("batch", 1)),
    (F16, 128, "bnhd", 2, 6, ("shared", 211)),
    (F32, 128, "slice", 3, 4, ("batch", 67)),
    (BF16, 128, "bnhd", 1, 9, ("batch", 4097)),
]


def where(spec, B):
    """(N, grid, positions) of a case."""
    if isinstance(spec[0], int):
        return spec[0] * spec[1] * spec[2], spec, None
    g = torch.Generator(device=DEV).manual_seed(7)
    kind, N = spec
    p = torch.randint(-300, 100000, (B if kind == "batch" else 1, N, 3), generator=g, device=DEV, dtype=torch.int32)
    return N, None, p if kind == "batch" else p[0]


def call_kw(grid, pos):
    return dict(grid=grid_of(grid) if grid else None, positions=pos)


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("weight", [None, F32, BF16, F16], ids=["plain", "norm32", "normbf16", "normf16"])
def test_rope_against_64_bits(case, weight):
    dtype, D, layout, B, H, spec = case
    N, grid, pos = where(spec, B)
    x = rand((B, H, N, D), dtype, 1, layout)
    w = None if weight is None else (1 + 0.3 * torch.randn(D, generator=torch.Generator(device=DEV).manual_seed(2),
                                                           device=DEV)).to(weight)
    y = scope.rope(x, params(SPLITS[D]), weight=w, eps=1e-5, **call_kw(grid, pos))
    a = R.angles(SPLITS[D], 1e4, N, grid, pos, DEV)
    xd, wd = x.double(), None if w is None else w.double()
    want = R.turn(xd if w is None else R.norm(xd, wd, 1e-5), a)
    assert y.shape == x.shape and y.dtype == dtype
    R.within(y, want, R.rope_bound(xd, want, dtype, w is not None, R.angle_slack(pos), wd, 1e-5), "y")
    if w is None:
        back = scope.rope(x, params(SPLITS[D]), inverse=True, **call_kw(grid, pos))
        want = R.turn(xd, a, -1.0)
        R.within(back, want, R.rope_bound(xd, want, dtype, False, R.angle_slack(pos)), "inverse")


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("weight", [F32, BF16])
def test_rope_backward_against_64_bits(case, weight):
    dtype, D, layout, B, H, spec = case
    N, grid, pos = where(spec, B)
    x, dy = rand((B, H, N, D), dtype, 1, layout), rand((B, H, N, D), dtype, 3, "bhnd", 0.5)
    w = (1 + 0.3 * torch.randn(D, generator=torch.Generator(device=DEV).manual_seed(2), device=DEV)).to(weight)
    kw = call_kw(grid, pos)
    dx, dw = scope.rope_backward(dy, x, params(SPLITS[D]), weight=w, eps=1e-5, **kw)
    a = R.angles(SPLITS[D], 1e4, N, grid, pos, DEV)
    args = (dy.double(), x.double(), a, w.double(), 1e-5)
    wx, ww = R.rope_grads(*args)
    bx, bw = R.rope_grad_bounds(*args, wx, ww, dtype, weight, R.angle_slack(pos))
    R.within(dx, wx, bx, "dx")
    R.within(dw, ww, bw, "dw")
    assert dw.dtype == weight and dx.dtype == dtype
    dx2, dw2 = scope.rope_backward(dy, x, params(SPLITS[D]), weight=w, eps=1e-5, **kw)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_rope_gradient_against_differences_of_the_kernel():
    """Along a direction, <dx, u> + <dw, v> against central differences of the
    forward kernel in fp32.  With h = 2^-6 the difference of the exact function
    is taken in 64 bits for the same h, so only the kernel's error is left:
    the bound of y weighed with |dy|, twice, over 2h; and the exact difference
    has to meet the exact gradient within its h^2 (third derivatives are O(1)
    a row: the norm's second-order factors stay below 10 for rows of norm
    sqrt(D) and unit entries)."""
    D, N, H = 64, 24, 2
    x, dy, u = (rand((1, H, N, D), F32, s) for s in (1, 2, 3))
    u = u / u.pow(2).sum(-1, keepdim=True).sqrt()
    w = 1 + 0.3 * torch.randn(D, generator=torch.Generator(device=DEV).manual_seed(4), device=DEV)
    p, g, h = params(SPLITS[D]), (2, 3, 4), 2.0 ** -6
    a = R.angles(SPLITS[D], 1e4, N, g, None, DEV)
    dx, _ = scope.rope_backward(dy, x, p, grid_of(g), weight=w)
    got, exact, slack = 0.0, 0.0, 0.0
    for s in (1, -1):
        xs = x + s * h * u
        y = scope.rope(xs, p, grid_of(g), weight=w)
        z = R.turn(R.norm(xs.double(), w.double(), 1e-6), a)
        got += s * float((y.double() * dy.double()).sum()) / (2 * h)
        exact += s * float((z * dy.double()).sum()) / (2 * h)
        slack += float((R.rope_bound(xs.double(), z, F32, True, 0.0, w.double(), 1e-6) * dy.double().abs()).sum()) / (2 * h)
        slack += float((2.0 ** -24 * xs.double().abs() * dy.double().abs()).sum()) / (2 * h)  # xs itself is rounded
    assert abs(got - exact) <= slack
    slope = float((dx.double() * u.double()).sum())
    r3 = float((dy.double().norm(dim=-1) * x.double().pow(2).mean(-1).rsqrt() * 10).sum())
    assert abs(slope - exact) <= h * h / 6 * r3 + slack


@pytest.mark.parametrize("split", [(64, 0, 0), (0, 64, 0), (0, 0, 64), (2, 30, 32), (0, 2, 62)])
def test_axis_splits(split):
    x, g = rand((1, 2, 60, 64), F32, 5), (3, 4, 5)
    y = scope.rope(x, params(split, 500.0), grid_of(g))
    want = R.turn(x.double(), R.angles(split, 500.0, 60, g, None, DEV))
    R.within(y, want, R.rope_bound(x.double(), want, F32, False), "y")


def test_positions_at_the_ends_of_32_bits():
    pos = torch.tensor([[2 ** 31 - 1, -2 ** 31, 0], [-1, 2 ** 31 - 1, -2 ** 31], [0, 0, 0]], dtype=torch.int32, device=DEV)
    x = rand((2, 3, 3, 128), F32, 6)
    y = scope.rope(x, params(SPLITS[128]), positions=pos)
    want = R.turn(x.double(), R.angles(SPLITS[128], 1e4, 3, positions=pos, device=DEV))
    R.within(y, want, R.rope_bound(x.double(), want, F32, False, R.angle_slack(pos)), "y")
    assert torch.equal(y[:, :, 2], x[:, :, 2])


def test_positions_of_a_grid_equal_the_grid():
    g = (3, 5, 7)
    n = torch.arange(105, device=DEV)
    pos = torch.stack([n // 35, (n // 7) % 5, n % 7], -1).int()
    x = rand((2, 4, 105, 64), BF16, 8)
    assert torch.equal(scope.rope(x, params(SPLITS[64]), grid_of(g)), scope.rope(x, params(SPLITS[64]), positions=pos))


def test_rope_equals_the_plans_rotation():
    """The rotated q of a plan: the same definition (fp32 sines here, a table there), so at most
    one rounding step of bf16 apart."""
    from cluster_guided_sparse_b200 import synth
    w = synth.WORKLOADS["small"]
    q, k, _ = (t.cuda() for t in synth.make_inputs(w))
    p, g = scope.make_params(w)
    qr = scope.plan(q, k, p, g).view("qr")
    y = scope.rope(q, p, g).double()
    step = R.half_ulp(y, BF16) * 2 + R.pair_sum(q.double()) * 2.0 ** -20
    assert ((qr.double() - y).abs() <= step * 1.001).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_in_place(dtype):
    x, dy = rand((2, 5, 37, 128), dtype, 9, "bnhd"), rand((2, 5, 37, 128), dtype, 10, "bnhd")
    w = torch.rand(128, device=DEV) + 0.5
    p, kw = params(SPLITS[128]), dict(grid=grid_of((1, 1, 37)))
    ref, ref_n = scope.rope(x, p, **kw), scope.rope(x, p, weight=w, **kw)
    dx, dw = scope.rope_backward(dy, x, p, weight=w, **kw)
    for over in (0, 1):
        a, b = dy.clone(), x.clone()
        dx2, dw2 = scope.rope_backward(a, b, p, weight=w, out=(a, b)[over], **kw)
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    y = x.clone()
    assert scope.rope(y, p, out=y, **kw) is y and torch.equal(y, ref)
    y = x.clone()
    scope.rope(y, p, weight=w, out=y, **kw)
    assert torch.equal(y, ref_n)


def test_only_the_given_rows_are_written():
    big = torch.full((2, 9, 50, 64), 7.0, dtype=BF16, device=DEV)
    out = big[:, 1:8:2, 3:40]
    x = rand((2, 4, 37, 64), BF16, 11)
    scope.rope(x, params(SPLITS[64]), grid_of((1, 37, 1)), out=out)
    assert torch.equal(out, scope.rope(x, params(SPLITS[64]), grid_of((1, 37, 1))))
    out.fill_(7.0)
    assert (big == 7.0).all()


def test_no_rows():
    x = torch.empty((2, 3, 0, 64), dtype=BF16, device=DEV)
    pos = torch.empty((0, 3), dtype=torch.int32, device=DEV)
    assert scope.rope(x, params(SPLITS[64]), positions=pos).shape == x.shape
    dx, dw = scope.rope_backward(x, x, params(SPLITS[64]), positions=pos, weight=torch.ones(64, device=DEV))
    assert dx.shape == x.shape and (dw == 0).all()


def test_zero_rows_infinities_and_nan_stay_in_their_rows():
    x = rand((1, 2, 8, 64), F32, 12)
    x[0, 0, 1] = 0
    x[0, 0, 2, 5] = float("inf")
    x[0, 1, 3, 9] = float("nan")
    w = torch.ones(64, device=DEV)
    y = scope.rope(x, params(SPLITS[64]), grid_of((1, 1, 8)), weight=w)
    ok = torch.ones(1, 2, 8, dtype=torch.bool, device=DEV)
    ok[0, 0, 2] = ok[0, 1, 3] = False
    assert torch.isfinite(y[ok]).all() and (y[0, 0, 1] == 0).all() and torch.isnan(y[0, 1, 3]).any()
    dx, _ = scope.rope_backward(torch.ones_like(x), x, params(SPLITS[64]), grid_of((1, 1, 8)), weight=w)
    assert torch.isfinite(dx[ok]).all()


def test_other_stream_and_graph():
    x, dy = rand((2, 6, 77, 64), BF16, 13), rand((2, 6, 77, 64), BF16, 14)
    w = torch.rand(64, device=DEV) + 0.5
    p, kw = params(SPLITS[64]), dict(grid=grid_of((7, 11, 1)), weight=w)
    y, (dx, dw) = scope.rope(x, p, **kw), scope.rope_backward(dy, x, p, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2 = scope.rope(x, p, stream=side, **kw)
    dx2, dw2 = scope.rope_backward(dy, x, p, stream=side, **kw)
    side.synchronize()
    assert torch.equal(y, y2) and torch.equal(dx, dx2) and torch.equal(dw, dw2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y3 = scope.rope(x, p, **kw)
        dx3, dw3 = scope.rope_backward(dy, x, p, **kw)
    x.copy_(rand((2, 6, 77, 64), BF16, 15))
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    y, (dx, dw) = scope.rope(x, p, **kw), scope.rope_backward(dy, x, p, **kw)
    assert torch.equal(y, y3) and torch.equal(dx, dx3) and torch.equal(dw, dw3)
    del g


def test_refusals_on_the_device():
    x = rand((2, 2, 8, 64), BF16, 16)
    with pytest.raises(ValueError, match="cpu"):
        scope.rope(x, params(SPLITS[64]), positions=torch.zeros(8, 3, dtype=torch.int32))
    with pytest.raises(scope.ScopeError, match="overlap"):
        scope.rope(x[:1].expand(2, -1, -1, -1), params(SPLITS[64]), grid_of((2, 2, 2)))
    with pytest.raises(scope.ScopeError, match="workspace|aligned"):
        ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)[16:]
        scope.rope_backward(x, x, params(SPLITS[64]), grid_of((2, 2, 2)), weight=torch.ones(64, device=DEV), workspace=ws)
