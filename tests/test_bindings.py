"""Host-only checks of what the Python bindings hand to the library."""
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
