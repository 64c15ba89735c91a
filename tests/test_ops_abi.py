"""Host-only checks of the operators around the sparse attention: every refusal
comes from the argument checks, which run before any CUDA call (the pointers
are fake), and the 64-bit forms that the GPU tests use agree with their own
differences."""
import ctypes

import pytest
import torch

import cluster_guided_sparse_b200 as scope
import op_ref as R
from cluster_guided_sparse_b200 import build, ops

FAKE = 0x7F0000000000  # aligned, never dereferenced
EINVAL, ESHAPE, EDTYPE, EALIGN, EWORKSPACE = 1, 2, 3, 4, 5
by = ctypes.byref


@pytest.fixture(scope="module")
def L():
    build.build()
    return ops._functions()


def T(B=1, H=2, N=256, D=64, dtype=scope.SCOPE_BF16, ptr=FAKE, strides=None):
    return scope.ScopeTensor(ptr, dtype, B, H, N, D, (ctypes.c_int64 * 4)(*(strides or (0, 0, 0, 0))))


def prm(**kw):
    return scope.make_params(**{**dict(d_t=16, d_h=24, d_w=24, theta=10000.0), **kw})[0]


def rope_status(L, x=None, y=None, grid=(4, 8, 8), p=None, pos=None, w=None, eps=1e-6, inverse=0):
    g = scope.ScopeGrid(*grid)
    st = L.scope_rope(by(x or T()), by(g), by(p or prm()), pos and by(pos), w and by(w), eps, inverse,
                      by(y or T(ptr=FAKE + 4096)), None)
    return st, L.scope_last_error().decode()


@pytest.mark.parametrize("kw,code,msg", [
    (dict(p=prm(d_t=15, d_h=25)), ESHAPE, "even"),
    (dict(p=prm(d_t=16, d_h=24, d_w=26)), ESHAPE, "equal D"),
    (dict(p=prm(theta=0.0)), EINVAL, "theta"),
    (dict(p=prm(theta=float("inf"))), EINVAL, "theta"),
    (dict(p=prm(theta=float("nan"))), EINVAL, "theta"),
    (dict(grid=(4, 8, 7)), ESHAPE, "grid"),
    (dict(grid=(4, 0, 64)), ESHAPE, "grid"),
    (dict(grid=(-4, -8, 8)), ESHAPE, "grid"),
    (dict(grid=(1, 65536, 65537)), ESHAPE, "grid"),  # the product passes 32 bits
    (dict(grid=(0, 0, 0)), EINVAL, "grid or positions"),
    (dict(pos=ops.ScopePositions(FAKE, 1)), EINVAL, "not both"),
    (dict(grid=(0, 0, 0), pos=ops.ScopePositions(0, 1)), EINVAL, "null"),
    (dict(grid=(0, 0, 0), pos=ops.ScopePositions(FAKE + 2, 1)), EALIGN, "4-byte"),
    (dict(grid=(0, 0, 0), pos=ops.ScopePositions(FAKE, 3)), ESHAPE, "positions"),
    (dict(w=ops.ScopeVector(0, 0)), EINVAL, "null"),
    (dict(w=ops.ScopeVector(FAKE, 2)), EDTYPE, "weight"),
    (dict(w=ops.ScopeVector(FAKE + 2, 0)), EALIGN, "weight"),
    (dict(w=ops.ScopeVector(FAKE, 0), eps=-1.0), EINVAL, "eps"),
    (dict(w=ops.ScopeVector(FAKE, 0), eps=float("nan")), EINVAL, "eps"),
    (dict(w=ops.ScopeVector(FAKE, 0), inverse=1), EINVAL, "inverse"),
    (dict(inverse=2), EINVAL, "inverse"),
    (dict(x=T(ptr=0)), EINVAL, "null"),
    (dict(x=T(ptr=FAKE + 8)), EALIGN, "aligned"),
    (dict(x=T(D=96)), ESHAPE, "head dim"),
    (dict(x=T(dtype=scope.SCOPE_I32)), EDTYPE, "dtype"),
    (dict(x=T(strides=(0, 64, 0, 1))), ESHAPE, "overlap"),
    (dict(x=T(strides=(0, 64 * 256, 68, 1))), ESHAPE, "16 bytes"),
    (dict(x=T(strides=(0, 64 * 256, 128, 2))), ESHAPE, "strides[3]"),
    (dict(y=T(N=255)), ESHAPE, "differ"),
    (dict(y=T(dtype=scope.SCOPE_F32)), EDTYPE, "differ"),
    (dict(y=T(strides=(0, 64, 128, 1))), EINVAL, "same memory"),
])
def test_rope_refusals(L, kw, code, msg):
    st, err = rope_status(L, **kw)
    assert st == code and msg in err, (st, err)


def test_rope_without_rows_needs_no_device(L):
    x = T(N=0, ptr=0, dtype=ops.SCOPE_F16)
    assert rope_status(L, x=x, y=x, grid=(0, 0, 0), pos=ops.ScopePositions(0, 1))[0] == 0


def rope_backward_status(L, w, dw, ws=FAKE, ws_bytes=1 << 30, dx=None):
    x, g = T(), scope.ScopeGrid(4, 8, 8)
    st = L.scope_rope_backward(by(T()), by(x), by(g), by(prm()), None, w and by(w), 1e-6, by(dx or T()),
                               dw and by(dw), ws, ws_bytes, None)
    return st, L.scope_last_error().decode()


@pytest.mark.parametrize("kw,code,msg", [
    (dict(w=None, dw=None), EINVAL, "inverse"),
    (dict(w=ops.ScopeVector(FAKE, 0), dw=None), EINVAL, "dw"),
    (dict(w=ops.ScopeVector(FAKE, 0), dw=ops.ScopeVector(FAKE + 512, 1)), EDTYPE, "differ"),
    (dict(w=ops.ScopeVector(FAKE, 0), dw=ops.ScopeVector(FAKE, 0)), EINVAL, "overlap"),
    (dict(w=ops.ScopeVector(FAKE, 0), dw=ops.ScopeVector(FAKE + 512, 0), ws=None), EWORKSPACE, "null"),
    (dict(w=ops.ScopeVector(FAKE, 0), dw=ops.ScopeVector(FAKE + 512, 0), ws=FAKE + 16), EALIGN, "256"),
    (dict(w=ops.ScopeVector(FAKE, 0), dw=ops.ScopeVector(FAKE + 512, 0), ws_bytes=64), EWORKSPACE, "small"),
    (dict(w=ops.ScopeVector(FAKE, 0), dw=ops.ScopeVector(FAKE + 512, 0), dx=T(H=3)), ESHAPE, "differ"),
    (dict(w=ops.ScopeVector(FAKE, 0), dw=ops.ScopeVector(FAKE + 512, 0), dx=T(strides=(0, 64, 128, 1))), EINVAL,
     "same memory"),
])
def test_rope_backward_refusals(L, kw, code, msg):
    st, err = rope_backward_status(L, **kw)
    assert st == code and msg in err, (st, err)


def test_bindings_refuse_cpu_tensors_and_wrong_shapes():
    x = torch.zeros(1, 2, 256, 64)
    with pytest.raises(ValueError, match="CUDA"):
        scope.rope(x, prm(), scope.ScopeGrid(4, 8, 8))
    with pytest.raises(ValueError, match="B, H, N, D"):
        ops._tensor(x[0], "x")
    with pytest.raises(ValueError, match="dtype"):
        ops._tensor(x.double(), "x")
    with pytest.raises(ValueError, match="int32"):
        ops._positions(torch.zeros(256, 3, dtype=torch.int64), x)
    with pytest.raises(ValueError, match="positions must be"):
        ops._positions(torch.zeros(2, 256, 3, dtype=torch.int32), x)
    with pytest.raises(ValueError, match="vector"):
        ops._vector(torch.zeros(65), 64, "weight")
    with pytest.raises(ValueError, match="vector"):
        ops._vector(torch.zeros(128)[::2], 64, "weight")


def test_rope_formula_gradients_agree_with_differences():
    g = torch.Generator().manual_seed(0)
    x, dy = (torch.randn(2, 3, 5, 64, generator=g, dtype=torch.float64) for _ in range(2))
    w = 1 + 0.3 * torch.randn(64, generator=g, dtype=torch.float64)
    pos = torch.randint(-50, 50, (2, 5, 3), generator=g, dtype=torch.int32)
    a = R.angles((16, 24, 24), 1e4, 5, positions=pos)
    dx, dw = R.rope_grads(dy, x, a, w, 1e-6)
    u, v = torch.randn(x.shape, generator=g, dtype=torch.float64), torch.randn(64, generator=g, dtype=torch.float64)
    f = lambda s: (R.turn(R.norm(x + s * u, w + s * v, 1e-6), a) * dy).sum()  # noqa: E731
    h = 1e-5  # truncation h^2 of O(1) third derivatives, cancellation 1e-16 * 1e3 / h
    want = (f(h) - f(-h)) / (2 * h)
    assert abs((dx * u).sum() + (dw * v).sum() - want) < 1e-6


def cross_status(L, q=None, k=None, v=None, keys=None, scale=0.0, o=None, ws=FAKE, ws_bytes=1 << 40, lse=None):
    k = k or T(N=77, ptr=FAKE + (1 << 20))
    q = q or T()
    o = o or T(q.B, q.H, q.N, q.D, q.dtype, FAKE + (3 << 20))
    v = v or T(k.B, k.H, k.N, k.D, k.dtype, FAKE + (2 << 20))
    st = L.scope_cross_attn(by(q), by(k), by(v), keys and by(keys), scale, by(o), lse, ws, ws_bytes, None)
    return st, L.scope_last_error().decode()


CROSS_REFUSALS = [
    (dict(q=T(dtype=scope.SCOPE_F32)), EDTYPE, "bf16 or f16"),
    (dict(k=T(N=77, dtype=ops.SCOPE_F16)), EDTYPE, "differ"),
    (dict(k=T(N=77, D=128)), ESHAPE, "head dims"),
    (dict(q=T(B=4), k=T(B=2, N=77)), ESHAPE, "B must be 1"),
    (dict(q=T(H=6), k=T(H=4, N=77)), ESHAPE, "divide"),
    (dict(q=T(H=2), k=T(H=4, N=77)), ESHAPE, "divide"),
    (dict(q=T(B=64, H=3, N=1 << 23), k=T(B=64, H=1, N=77)), ESHAPE, "2^30"),
    (dict(v=T(N=76)), ESHAPE, "differ"),
    (dict(v=T(N=77, dtype=ops.SCOPE_F16)), EDTYPE, "differ"),
    (dict(k=T(N=77, strides=(0, 0, 64, 1))), ESHAPE, "overlap"),
    (dict(k=T(N=77, ptr=0)), EINVAL, "null"),
    (dict(keys=ops.ScopeKeys(FAKE, FAKE, 77)), EINVAL, "not both"),
    (dict(keys=ops.ScopeKeys(FAKE + 1, None, 0)), EALIGN, "len"),
    (dict(keys=ops.ScopeKeys(None, FAKE, -1)), ESHAPE, "mask_stride"),
    (dict(scale=-1.0), EINVAL, "scale"),
    (dict(scale=float("nan")), EINVAL, "scale"),
    (dict(scale=float("inf")), EINVAL, "scale"),
    (dict(scale=1e-38), EINVAL, "scale"),
    (dict(o=T(N=255)), ESHAPE, "differ"),
    (dict(o=T(dtype=ops.SCOPE_F16)), EDTYPE, "differ"),
    (dict(o=T()), EINVAL, "overlap"),
    (dict(lse=FAKE + 2), EALIGN, "lse"),
    (dict(ws=None), EWORKSPACE, "null"),
    (dict(ws=FAKE + 16), EALIGN, "256"),
    (dict(ws_bytes=0), EWORKSPACE, "small"),
]


@pytest.mark.parametrize("kw,code,msg", CROSS_REFUSALS)
def test_cross_attn_refusals(L, kw, code, msg):
    st, err = cross_status(L, **kw)
    assert st == code and msg in err, (st, err)


def test_cross_attn_workspace(L):
    size = lambda q, k, m=0: L.scope_cross_attn_workspace_bytes(by(q), by(k), m)  # noqa: E731
    assert size(T(H=24, N=118800, D=128), T(H=24, N=256, D=128)) == 256  # rows enough: keys are not split
    k = T(B=2, N=1000)
    assert size(T(B=2, N=118800), k, 1) >= size(T(B=2, N=118800), k) + 2 * 1000 * 4
    one = size(T(H=1, N=1), T(H=1, N=118800))  # a single row: ranges of keys with fp32 outputs
    assert one > 256 + 100 * 64 * 4
    assert size(T(dtype=scope.SCOPE_F32), T(dtype=scope.SCOPE_F32)) == 0


def test_cross_bindings_refuse_wrong_masks():
    k = torch.zeros(2, 3, 77, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="kv_len"):
        ops._keys(k, torch.zeros(2, dtype=torch.int64), None)
    with pytest.raises(ValueError, match="kv_len"):
        ops._keys(k, torch.zeros(3, dtype=torch.int32), None)
    with pytest.raises(ValueError, match="kv_mask"):
        ops._keys(k, None, torch.zeros(2, 76, dtype=torch.bool))
    with pytest.raises(ValueError, match="kv_mask"):
        ops._keys(k, None, torch.zeros(2, 77))
    with pytest.raises(ValueError, match="kv_mask"):
        ops._keys(k, None, torch.zeros(77, 2, dtype=torch.bool).T)
    with pytest.raises(ValueError, match="scale"):
        ops._scale(0.0)
    with pytest.raises(ValueError, match="CUDA"):
        scope.cross_attn(k, k, k)


def test_cross_formula_gradients_agree_with_differences():
    g = torch.Generator().manual_seed(1)
    q = torch.randn(2, 4, 5, 64, generator=g, dtype=torch.float64)
    k, v = (torch.randn(1, 2, 7, 64, generator=g, dtype=torch.float64) for _ in range(2))
    do = torch.randn(q.shape, generator=g, dtype=torch.float64)
    on = torch.tensor([[1, 0, 1, 1, 0, 1, 1]], dtype=torch.bool)
    r, _ = R.cross(q, k, v, on, 0.125, torch.bfloat16, do)
    dirs = [torch.randn(t.shape, generator=g, dtype=torch.float64) for t in (q, k, v)]

    def f(s):
        return (R.cross(q + s * dirs[0], k + s * dirs[1], v + s * dirs[2], on, 0.125, torch.bfloat16)[0]["o"] * do).sum()

    h = 1e-5  # h^2 times third derivatives of order 1e2, and cancellation
    want = (f(h) - f(-h)) / (2 * h)
    got = sum((r[n] * d).sum() for n, d in zip(("dq", "dk", "dv"), dirs))
    assert abs(got - want) < 1e-6
    assert (r["dk"][0, :, ~on[0]] == 0).all() and (r["dv"][0, :, ~on[0]] == 0).all()


def cross_backward_status(L, **over):
    at = iter(range(FAKE, FAKE + (64 << 20), 1 << 20))
    t = {n: T(N=256, ptr=next(at)) for n in ("d_o", "q", "o", "dq")}
    t.update({n: T(N=77, ptr=next(at)) for n in ("k", "v", "dk", "dv")})
    rest = dict(lse=FAKE, keys=None, scale=0.0, ws=FAKE, ws_bytes=1 << 40)
    for n, x in over.items():
        (t if n in t else rest)[n] = x
    keys = rest["keys"]
    st = L.scope_cross_attn_backward(by(t["d_o"]), by(t["q"]), by(t["k"]), by(t["v"]), by(t["o"]), rest["lse"],
                                     keys and by(keys), rest["scale"], by(t["dq"]), by(t["dk"]), by(t["dv"]),
                                     rest["ws"], rest["ws_bytes"], None)
    return st, L.scope_last_error().decode()


@pytest.mark.parametrize("kw,code,msg", [
    (dict(d_o=T(N=255)), ESHAPE, "d_o and q"),
    (dict(o=T(dtype=ops.SCOPE_F16)), EDTYPE, "o and q"),
    (dict(dq=T(H=4)), ESHAPE, "dq and q"),
    (dict(dk=T(N=76)), ESHAPE, "dk and k"),
    (dict(dv=T(N=77, dtype=ops.SCOPE_F16)), EDTYPE, "dv and k"),
    (dict(dv=T(N=77, strides=(0, 0, 64, 1))), ESHAPE, "overlap"),
    (dict(dk=T(N=77, ptr=FAKE), dv=T(N=77, ptr=FAKE)), EINVAL, "overlap"),
    (dict(dq=T(ptr=FAKE)), EINVAL, "overlap"),
    (dict(lse=None), EINVAL, "lse"),
    (dict(lse=FAKE + 1), EALIGN, "lse"),
    (dict(scale=-1.0), EINVAL, "scale"),
    (dict(keys=ops.ScopeKeys(FAKE, FAKE, 77)), EINVAL, "not both"),
    (dict(ws=None), EWORKSPACE, "null"),
    (dict(ws=FAKE + 128), EALIGN, "256"),
    (dict(ws_bytes=256), EWORKSPACE, "small"),
])
def test_cross_attn_backward_refusals(L, kw, code, msg):
    st, err = cross_backward_status(L, **kw)
    assert st == code and msg in err, (st, err)


def test_cross_attn_backward_without_rows_and_keys_needs_no_device(L):
    none = {n: T(N=0, ptr=0) for n in ("d_o", "q", "o", "dq", "k", "v", "dk", "dv")}
    assert cross_backward_status(L, lse=None, **none)[0] == 0
