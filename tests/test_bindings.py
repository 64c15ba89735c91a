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
