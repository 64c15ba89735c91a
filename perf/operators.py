"""Measured cases of the operators around the sparse self-attention of a video transformer block: rotary positions on
(t, h, w) axes, the same behind a per-head RMS norm, and cross attention to states of another length, each with its
gradients.

`run` computes an operator in its plain form from elementary torch operations, or (`own`) through this repository's
package.  `exact` gives the same outputs from the definitions in 64 bits."""
import functools
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
SPLITS = {64: (16, 24, 24), 128: (16, 56, 56)}  # head dim -> widths of the t, h, w blocks
THETA, EPS = 10000.0, 1e-6


def listed():
    return [
        # A test-sized call: latency of one rotation, fp32.
        dict(name="rope tiny f32", op="rope", B=1, H=2, D=64, T=4, Hh=8, W=8, dtype="f32", layout="bhnd",
             positions="grid", train=False),
        # One of q, k of a 720p video layer.
        dict(name="rope 720p", op="rope", B=1, H=24, D=128, T=33, Hh=45, W=80, dtype="bf16", layout="bhnd",
             positions="grid", train=False),
        # Packed clips with positions of their own, as a projection lays them out, trained in fp32.
        dict(name="rope packed train", op="rope", B=3, H=8, D=64, T=1, Hh=1, W=4097, dtype="f32", layout="bnhd",
             positions="list", train=True),
        # QK norm and rotation of a 480p video layer's q, as a projection lays it out.
        dict(name="norm_rope 480p", op="norm_rope", B=1, H=40, D=128, T=21, Hh=30, W=52, dtype="bf16", layout="bnhd",
             positions="grid", train=False),
        # The same in training, a short clip at 720p.
        dict(name="norm_rope train", op="norm_rope", B=2, H=24, D=128, T=9, Hh=45, W=80, dtype="bf16", layout="bhnd",
             positions="grid", train=True),
        # One streamed token for each of 8 requests against its prompt.
        dict(name="cross one token", op="cross", B=8, Bk=8, H=24, Hk=24, N=1, M=512, D=128, dtype="bf16",
             layout="bhnd", mask="len", train=False),
        # A small clip conditioned on a short prompt with holes, trained.
        dict(name="cross small train", op="cross", B=2, Bk=2, H=8, Hk=8, N=2048, M=77, D=128, dtype="bf16",
             layout="bhnd", mask="mask", train=True),
        # 480p video tokens to a padded prompt of 512 states.
        dict(name="cross 480p", op="cross", B=1, Bk=1, H=40, Hk=40, N=32760, M=512, D=128, dtype="bf16",
             layout="bhnd", mask="none", train=False),
        # 720p video tokens to 256 states, projections' own layout.
        dict(name="cross 720p", op="cross", B=1, Bk=1, H=24, Hk=24, N=118800, M=256, D=128, dtype="bf16",
             layout="bnhd", mask="none", train=False),
        # The other direction: a prompt's tokens reading all video states, few rows and a long axis.
        dict(name="cross long keys", op="cross", B=1, Bk=1, H=24, Hk=24, N=77, M=118800, D=128, dtype="bf16",
             layout="bhnd", mask="none", train=False),
        # 480p video tokens to a prompt, trained.
        dict(name="cross 480p train", op="cross", B=1, Bk=1, H=40, Hk=40, N=32760, M=512, D=128, dtype="bf16",
             layout="bhnd", mask="none", train=True),
        # Grouped key heads and one prompt shared by the batch, fp16, odd lengths, trained.
        dict(name="cross shared train f16", op="cross", B=4, Bk=1, H=16, Hk=4, N=1531, M=333, D=64, dtype="f16",
             layout="bnhd", mask="len", train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "norm_rope", "cross", "cross"])
    D = rng.choice([64, 128])
    layout = rng.choice(["bhnd", "bnhd"])
    if op != "cross":
        dtype = rng.choice(["f32", "bf16", "f16"])
        train = rng.random() < 0.5
        B, H = rng.choice([1, 1, 2, 3]), rng.randint(1, 40)
        most = 24 * 118800 * 128 // (4 if train or dtype == "f32" else 1)
        room = max(1, most // (B * H * D))
        if rng.random() < 0.5:
            T, Hh, W = rng.randint(1, 33), _log(rng, 1, 64), _log(rng, 1, 100)
            while T * Hh * W > room:
                T, Hh, W = max(1, T // 2), max(1, Hh - Hh // 8), max(1, W - W // 8)
            positions = "grid"
        else:
            T, Hh, W = 1, 1, min(room, _log(rng, 1, 60000))
            positions = "list"
        return dict(op=op, B=B, H=H, D=D, T=T, Hh=Hh, W=W, dtype=dtype, layout=layout, positions=positions, train=train)
    dtype = rng.choice(["bf16", "bf16", "f16"])
    train = rng.random() < 0.5
    Hk = rng.choice([1, 2, 3, 4, 8, 12, 24])
    H = Hk * rng.choice([1, 1, 1, 2, 4])
    B = rng.choice([1, 1, 2, 3, 5])
    Bk = rng.choice([B, B, 1])
    most = 24 * 118800 * 256 // (2 if train else 1)
    N, M = _log(rng, 1, 60000), _log(rng, 1, 1500)
    if rng.random() < 0.25:
        N, M = M, N
    while B * H * N * M > most:
        N, M = max(1, N - N // 8), max(1, M - M // 8)
    return dict(op="cross", B=B, Bk=Bk, H=H, Hk=Hk, N=N, M=M, D=D, dtype=dtype, layout=layout,
                mask=rng.choice(["none", "len", "mask"]), train=train)


def _randn(shape, layout, dtype, gen, gain=1.0):
    """Values of logical shape [B, H, N, D], held as [B, H, N, D] or as a projection lays them out, [B, N, H, D]."""
    B, H, N, D = shape
    if layout == "bnhd":
        return (torch.randn((B, N, H, D), generator=gen, device="cuda") * gain).to(dtype).transpose(1, 2)
    return (torch.randn(shape, generator=gen, device="cuda") * gain).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, lay, D = DTYPES[case["dtype"]], case["layout"], case["D"]
    s = {"case": case}
    if case["op"] != "cross":
        B, H, N = case["B"], case["H"], case["T"] * case["Hh"] * case["W"]
        s["x"] = _randn((B, H, N, D), lay, dt, g, 1.7)
        s["grid"] = (case["T"], case["Hh"], case["W"])
        s["positions"] = None
        if case["positions"] == "list":  # clips anywhere on a long timeline
            s["grid"] = (0, 0, 0)
            top = torch.tensor([20000, 128, 128], device="cuda")
            s["positions"] = (torch.rand((B, N, 3), generator=g, device="cuda") * top).to(torch.int32)
        s["weight"] = None
        if case["op"] == "norm_rope":
            s["weight"] = 1.0 + 0.3 * torch.randn(D, generator=g, device="cuda")
        if case["train"]:
            s["dy"] = _randn((B, H, N, D), lay, dt, g, 0.5)
        return s
    B, Bk, H, Hk, N, M = (case[k] for k in ("B", "Bk", "H", "Hk", "N", "M"))
    s["q"] = _randn((B, H, N, D), lay, dt, g, 1.5)
    s["k"] = _randn((Bk, Hk, M, D), lay, dt, g, 1.5)
    s["v"] = _randn((Bk, Hk, M, D), lay, dt, g)
    s["kv_len"] = s["kv_mask"] = None
    if case["mask"] == "len":  # padded prompts: at least a quarter full
        s["kv_len"] = (M - (torch.rand(Bk, generator=g, device="cuda") * (M - M // 4)).floor()).to(torch.int32)
    elif case["mask"] == "mask":  # a quarter of the states dropped
        s["kv_mask"] = torch.rand((Bk, M), generator=g, device="cuda") < 0.75
    if case["train"]:
        s["do"] = _randn((B, H, N, D), lay, dt, g, 0.5)
    return s


@functools.lru_cache(maxsize=None)
def _params(D, grid):
    import cluster_guided_sparse_b200 as scope

    d_t, d_h, d_w = SPLITS[D]
    return scope.make_params(d_t=d_t, d_h=d_h, d_w=d_w, theta=THETA, grid=grid)


def run(s):
    c = s["case"]
    if c["op"] == "cross":
        return (_own_cross if own else _cross)(s)
    return (_own_rope if own else _rope)(s)


# ---------------------------------------------------------------- the framework's calls
def _own_rope(s):
    import cluster_guided_sparse_b200 as scope

    c = s["case"]
    params, grid = _params(c["D"], s["grid"])
    kw = dict(positions=s["positions"])
    if s["weight"] is None:
        y = scope.rope(s["x"], params, grid, **kw)
        return {"y": y, "dx": scope.rope(s["dy"], params, grid, inverse=True, **kw)} if c["train"] else y
    y = scope.rope(s["x"], params, grid, weight=s["weight"], eps=EPS, **kw)
    if not c["train"]:
        return y
    dx, dw = scope.rope_backward(s["dy"], s["x"], params, grid, weight=s["weight"], eps=EPS, **kw)
    return {"y": y, "dx": dx, "dw": dw}


def _own_cross(s):
    import cluster_guided_sparse_b200 as scope

    kw = dict(kv_len=s["kv_len"], kv_mask=s["kv_mask"])
    if not s["case"]["train"]:
        return scope.cross_attn(s["q"], s["k"], s["v"], **kw)
    o, lse = scope.cross_attn(s["q"], s["k"], s["v"], return_lse=True, **kw)
    dq, dk, dv = scope.cross_attn_backward(s["do"], s["q"], s["k"], s["v"], o, lse, **kw)
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


# ---------------------------------------------------------------- plain forms
def _angles(s):
    """cos and sin of each pair's angle, [B or 1, 1, N, D/2], the angle in 64 bits."""
    D, pos = s["case"]["D"], s["positions"]
    dev = s["x"].device
    if pos is None:
        T, Hh, W = s["grid"]
        n = torch.arange(T * Hh * W, device=dev)
        pos = torch.stack([n // (Hh * W), (n // W) % Hh, n % W], -1)[None]
    parts = [pos[..., a, None].double() * THETA ** (-torch.arange(0, d, 2, device=dev, dtype=torch.float64) / d)
             for a, d in enumerate(SPLITS[D])]
    a = torch.cat(parts, -1)[:, None]
    return torch.cos(a).float(), torch.sin(a).float()


def _turn(x, cos, sin):
    x0, x1 = x[..., 0::2], x[..., 1::2]
    return torch.stack([x0 * cos - x1 * sin, x0 * sin + x1 * cos], -1).flatten(-2)


def _rope(s):
    x, w, dt, train = s["x"].float(), s["weight"], s["x"].dtype, s["case"]["train"]
    cos, sin = _angles(s)
    if w is None:
        y = _turn(x, cos, sin).to(dt)
        return {"y": y, "dx": _turn(s["dy"].float(), cos, -sin).to(dt)} if train else y
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    y = _turn(x * r * w, cos, sin).to(dt)
    if not train:
        return y
    dz = _turn(s["dy"].float(), cos, -sin)
    g = dz * w
    dx = r * (g - x * (r * r * (g * x).mean(-1, keepdim=True)))
    return {"y": y, "dx": dx.to(dt), "dw": (dz * x * r).double().sum((0, 1, 2)).float()}


def _allowed(s):
    M = s["case"]["M"]
    if s["kv_mask"] is not None:
        return s["kv_mask"][:, None, None, :]
    if s["kv_len"] is not None:
        return torch.arange(M, device=s["q"].device)[None, None, None, :] < s["kv_len"][:, None, None, None]
    return None


def _cross(s):
    c, dt = s["case"], s["q"].dtype
    B, Bk, H, Hk, N, D = (c[k] for k in ("B", "Bk", "H", "Hk", "N", "D"))
    G, scale = H // Hk, D ** -0.5
    fold = lambda t: t.float().reshape(B, Hk, G * N, D)  # noqa: E731  the group's query heads read one key head
    q, k, v = fold(s["q"]), s["k"].float(), s["v"].float()
    p = torch.matmul(q, k.transpose(-1, -2)) * scale
    allowed = _allowed(s)
    if allowed is not None:
        p = p.masked_fill(~allowed, -math.inf)
    top = p.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)  # rows that may read nothing
    p = torch.exp(p - top)
    total = p.sum(-1, keepdim=True)
    lse = top + torch.log(total)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    o = torch.matmul(p, v)
    if not c["train"]:
        return o.reshape(B, H, N, D).to(dt)
    do = fold(s["do"])
    dp = torch.matmul(do, v.transpose(-1, -2))
    ds = p * (dp - (do * o).sum(-1, keepdim=True))
    dq = torch.matmul(ds, k) * scale
    dk = torch.matmul(ds.transpose(-1, -2), q) * scale
    dv = torch.matmul(p.transpose(-1, -2), do)
    if Bk < B:
        dk, dv = dk.sum(0, keepdim=True), dv.sum(0, keepdim=True)
    back = lambda t: t.reshape(B, H, N, D).to(dt)  # noqa: E731
    return {"o": back(o), "lse": lse.reshape(B, H, N), "dq": back(dq), "dk": dk.to(dt), "dv": dv.to(dt)}


# ---------------------------------------------------------------- work and the definitions in 64 bits
def work(case):
    size, D = BYTES[case["dtype"]], case["D"]
    if case["op"] != "cross":
        n = case["B"] * case["H"] * case["T"] * case["Hh"] * case["W"] * D
        tensors = 4 if case["train"] else 2  # x, y (and dy, dx)
        flops = (3 if case["op"] == "rope" else 7) * n * (2 if case["train"] else 1)
        return {"bytes": tensors * n * size, "flops": flops}
    rows = case["B"] * case["H"] * case["N"]
    part = {"none": 1.0, "len": 0.625, "mask": 0.75}[case["mask"]]  # of the keys are read
    keys = case["Bk"] * case["Hk"] * case["M"]
    n_bytes = 2 * rows * D * size + 2 * part * keys * D * size
    flops = 4.0 * D * rows * case["M"] * part
    if case["train"]:
        n_bytes += 2 * rows * D * size + 2 * keys * D * size + 4 * rows
        flops *= 3.5
    return {"bytes": n_bytes, "flops": flops}


def exact(case, seed):
    s = prepare(case, seed)
    return (_exact_cross if case["op"] == "cross" else _exact_rope)(s, case)


def _exact_rope(s, case):
    """Pairs as complex numbers, turned by exp(i angle); gradients by differentiating the definition."""
    D, out = case["D"], {"y": [], "dx": []}
    B, H, N, _ = s["x"].shape
    n = torch.arange(N, device="cuda")
    T, Hh, W = s["grid"]
    rest = n % max(1, Hh * W)
    raster = (torch.div(n, max(1, Hh * W), rounding_mode="floor"), torch.div(rest, max(1, W), rounding_mode="floor"),
              rest % max(1, W))
    w = None if s["weight"] is None else s["weight"].double().requires_grad_(case["train"])
    dw = 0
    for b in range(B):
        axes = raster if s["positions"] is None else s["positions"][b].unbind(-1)
        phase = torch.empty((N, D // 2), dtype=torch.float64, device="cuda")
        at = 0
        for d, p in zip(SPLITS[D], axes):
            for i in range(d // 2):
                phase[:, at] = p.double() * math.exp(-2.0 * i / d * math.log(THETA))
                at += 1
        e = torch.polar(torch.ones_like(phase), phase)
        for h in range(H):
            x = s["x"][b, h].double().contiguous().requires_grad_(case["train"])
            z = x if w is None else x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / D + EPS) * w
            y = torch.view_as_real(torch.view_as_complex(z.reshape(N, D // 2, 2)) * e).reshape(N, D)
            if case["train"]:
                got = torch.autograd.grad(y, [x] + ([] if w is None else [w]), s["dy"][b, h].double())
                out["dx"].append(got[0].float() if s["x"].dtype != torch.float32 else got[0])
                dw = dw + got[1] if w is not None else 0
            # 16-bit results need no more than 32 bits here, and the largest case half the memory
            out["y"].append(y.detach().float() if s["x"].dtype != torch.float32 else y.detach())
    out = {name: torch.stack(v).reshape(B, H, N, D) for name, v in out.items() if v}
    if not case["train"]:
        return out["y"]
    return out if w is None else {**out, "dw": dw}


def _exact_cross(s, case):
    """Head by head, the softmax over the allowed keys alone; gradients by differentiating the definition."""
    B, Bk, H, Hk, N, M, D = (case[k] for k in ("B", "Bk", "H", "Hk", "N", "M", "D"))
    train = case["train"]
    zeros = lambda *shape: torch.zeros(shape, dtype=torch.float64, device="cuda")  # noqa: E731
    o, lse = zeros(B, H, N, D), torch.full((B, H, N), -math.inf, dtype=torch.float64, device="cuda")
    dq, dk, dv = (zeros(B, H, N, D), zeros(Bk, Hk, M, D), zeros(Bk, Hk, M, D)) if train else (None, None, None)
    for b in range(B):
        kb = b if Bk == B else 0
        if s["kv_mask"] is not None:
            keys = s["kv_mask"][kb].nonzero()[:, 0]
        else:
            keys = torch.arange(M if s["kv_len"] is None else int(s["kv_len"][kb]), device="cuda")
        if not len(keys):
            continue
        for h in range(H):
            hk = h // (H // Hk)
            q, k, v = (t.double().requires_grad_(train) for t in (s["q"][b, h], s["k"][kb, hk][keys], s["v"][kb, hk][keys]))
            logits = q @ k.T / math.sqrt(D)
            lse[b, h] = torch.logsumexp(logits, -1).detach()
            r = torch.softmax(logits, -1) @ v
            o[b, h] = r.detach()
            if train:
                gq, gk, gv = torch.autograd.grad(r, [q, k, v], s["do"][b, h].double())
                dq[b, h] = gq
                dk[kb, hk].index_add_(0, keys, gk)
                dv[kb, hk].index_add_(0, keys, gv)
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv} if train else o
