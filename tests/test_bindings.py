"""Host-only checks of what the Python bindings hand to the library."""
import ctypes

import pytest
import torch

import cluster_guided_sparse_b200 as scope
from cluster_guided_sparse_b200 import ops


def test_an_expanded_element_is_not_taken_for_a_contiguous_tensor():
    """Strides of zero throughout mean the contiguous layout to the library; of a tensor they mean
    that all of it is one element, as the gradient of a sum is: no memory lies behind the rest."""
    x = torch.zeros(2, 3, 5, 64, requires_grad=True)
    (dx,) = torch.autograd.grad(x.sum(), x)
    assert dx.stride() == (0, 0, 0, 0)
    for t in (dx, torch.ones(()).bfloat16().expand(1, 1, 1, 64), torch.ones(()).expand(4, 2, 256, 128)):
        with pytest.raises(ValueError, match="expanded"):
            ops._tensor(t, "do")
        with pytest.raises(ValueError, match="expanded"):
            scope.as_tensor(t)
        ops._tensor(t.contiguous(), "do")
        scope.as_tensor(t.contiguous())


@pytest.mark.parametrize("ws", [torch.zeros(1, dtype=torch.uint8).expand(1 << 30),  # one byte
                                torch.zeros(1 << 12, 2, dtype=torch.uint8)[:, 0]])   # every second one
def test_a_workspace_with_gaps_or_repeats_is_refused(ws):
    call = object.__new__(ops._Launch)
    with pytest.raises(ValueError, match="contiguous"):
        call.workspace(ws, ws, 256)
    assert call.workspace(ws, ws.reshape(-1)[:4096].clone(), 256).numel() == 4096
    q = torch.zeros(1, 1, 256, 64, dtype=torch.bfloat16)
    p, g = scope.make_params(d_t=16, d_h=24, d_w=24, theta=1e4, c_q=8, c_t=4, c_h=4, c_w=4, iters=2, top_p=0.5,
                             grid=(4, 8, 8))
    with pytest.raises(ValueError, match="contiguous"):
        scope.plan(q, q, p, g, workspace=ws)
    with pytest.raises(ValueError, match="contiguous"):
        scope.dense_attn(q, q, q, p, g, workspace=ws)


def test_the_operators_selftest_checks_its_arguments():
    L = ops._functions()
    for backward, cycles, msg in ((2, 2_000_000, "backward"), (-1, 2_000_000, "backward"), (0, 10, "wait_cycles"),
                                  (1, 5_000_000_000, "wait_cycles")):
        assert L.scope_ops_selftest_wait_timeout(backward, cycles, None) == 1
        assert msg in L.scope_last_error().decode()


def test_packed_arguments_equal_the_structures():
    """The operators hand tensors, vectors, positions and keys over as packed bytes; the structures are the
    header's layouts, which the refusal tests use."""
    x = torch.zeros(3, 5, 7, 64, dtype=torch.float16).transpose(1, 2)
    for t in (x, x.bfloat16(), torch.zeros(2, 3, 4, 128), torch.zeros(1, 1, 0, 64)):
        dt = {torch.float16: ops.SCOPE_F16, torch.bfloat16: scope.SCOPE_BF16, torch.float32: scope.SCOPE_F32}[t.dtype]
        s = scope.ScopeTensor(t.data_ptr(), dt, *t.shape, (ctypes.c_int64 * 4)(*t.stride()))
        assert ops._tensor(t, "x") == bytes(s)
    w = torch.zeros(64, dtype=torch.bfloat16)
    assert ops._vector(w, 64, "w") == bytes(ops.ScopeVector(w.data_ptr(), scope.SCOPE_BF16))
    pos = torch.zeros(3, 5, 3, dtype=torch.int32)
    assert ops._positions(pos, torch.zeros(3, 2, 5, 64)) == bytes(ops.ScopePositions(pos.data_ptr(), 3))
    assert ops._positions(pos[0], torch.zeros(3, 2, 5, 64)) == bytes(ops.ScopePositions(pos.data_ptr(), 1))
    k, n, m = torch.zeros(3, 2, 9, 64), torch.zeros(3, dtype=torch.int32), torch.ones(3, 12, dtype=torch.bool)[:, 2:11]
    assert ops._keys(k, n, None) == bytes(ops.ScopeKeys(n.data_ptr(), None, 0))
    assert ops._keys(k, None, m) == bytes(ops.ScopeKeys(None, m.data_ptr(), 12))
    assert ops._keys(k, None, None) is None
