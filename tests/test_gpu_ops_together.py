"""Calls of the operators at the same time, and the first call of a process inside a capture."""
import subprocess
import sys
import textwrap
import threading

import pytest
import torch

import cluster_guided_sparse_b200 as scope
from conftest import ROOT
from test_gpu_cross import BF16, DEV, F16, keys_kw, rand
from test_gpu_cross_bwd import grads

pytestmark = pytest.mark.gpu


def test_calls_of_several_threads_on_streams_of_their_own():
    cases = [(BF16, 64, 2, 2, 6, 3, 500, 300, "mask"), (F16, 128, 1, 1, 8, 8, 700, 200, "len"),
             (BF16, 128, 3, 3, 4, 4, 1, 900, "len"), (F16, 64, 4, 1, 8, 2, 61, 333, "mask")]
    jobs = []
    for dtype, D, B, Bk, H, Hk, N, M, mask in cases:
        t = [rand(s, dtype, i) for i, s in enumerate(((B, H, N, D), (Bk, Hk, M, D), (Bk, Hk, M, D), (B, H, N, D)))]
        jobs.append((t, keys_kw(mask, Bk, M)))
    p = [scope.make_params(d_t=16, d_h=D // 2 - 8, d_w=D // 2 - 8, theta=t)[0] for D, t in ((64, 1e4), (128, 500.0))]

    def work(t, kw):
        q, k, v, do = t
        D, g = q.shape[-1], scope.ScopeGrid(1, 1, q.shape[2])
        one = torch.ones(D, device=DEV)
        r = scope.rope(q, p[D // 128], g, weight=one)
        out = grads(r, k, v, do, **kw)
        out["dx"], out["dw"] = scope.rope_backward(out["dq"], q, p[D // 128], g, weight=one)
        return out

    refs = [work(*j) for j in jobs]
    torch.cuda.synchronize()
    bad = []

    def run(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(25):
                got = work(*jobs[i])
                s.synchronize()
                bad.extend((i, n) for n in got if not torch.equal(got[n], refs[i][n]))
    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    scope.ops_sync_status()
    assert not bad, bad[:5]


def test_first_calls_of_a_process_inside_a_capture():
    """No call sets up anything that a capture would not take."""
    code = """
        import torch, cluster_guided_sparse_b200 as scope
        g = torch.Generator(device="cuda").manual_seed(1)
        r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
        p, grid = scope.make_params(d_t=16, d_h=24, d_w=24, theta=1e4, grid=(1, 10, 10))
        w, m = torch.ones(64, device="cuda"), torch.rand((2, 90), generator=g, device="cuda") < 0.6
        x, k, v, do, one = r(2, 4, 100, 64), r(2, 2, 90, 64), r(2, 2, 90, 64), r(2, 4, 100, 64), r(2, 2, 1, 64)
        def work():
            q = scope.rope(x, p, grid, weight=w)
            o, lse = scope.cross_attn(q, k, v, kv_mask=m, return_lse=True)
            dq, dk, dv = scope.cross_attn_backward(do, q, k, v, o, lse, kv_mask=m)
            o1, lse1 = scope.cross_attn(one, k, v, return_lse=True)
            return (o, lse, dq, dk, dv, o1, *scope.cross_attn_backward(one, one, k, v, o1, lse1),
                    *scope.rope_backward(dq, x, p, grid, weight=w))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = work()
        graph.replay()
        want = work()
        scope.ops_sync_status()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del graph
        print("same")
    """
    r = subprocess.run([sys.executable, "-c", textwrap.dedent(code)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
