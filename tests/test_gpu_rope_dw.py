"""dw of scope.rope_backward where rows hold infinities: only the rows themselves count, not the lanes that
follow the last token and the last head without a row of their own."""
import pytest
import torch

import cluster_guided_sparse_b200 as scope
import op_ref as R
from test_gpu_rope import BF16, DEV, F16, F32, SPLITS, grid_of, params, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H", [1, 5, 8, 33])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_an_infinite_gradient_of_the_last_row_counts_once(dtype, D, H):
    """An infinite dy leaves +-inf in the two columns of its pair (as the sum of dz x r does); 0 * inf of
    a lane without a row would leave NaN."""
    N = 37
    x, dy = rand((1, H, N, D), dtype, 1), rand((1, H, N, D), dtype, 2)
    dy[0, H - 1, N - 1, 10] = float("inf")  # pair 5, on the t axis
    w = torch.ones(D, device=DEV)
    pos = torch.zeros((N, 3), dtype=torch.int32, device=DEV)
    pos[:-1, 1] = torch.arange(N - 1, device=DEV)
    pos[-1, 0] = 1  # turns by 1 rad and less on the t axis (pairs 0 to 7): both halves of the pair are infinite
    _, dw = scope.rope_backward(dy, x, params(SPLITS[D]), positions=pos, weight=w)
    a = R.angles(SPLITS[D], 1e4, N, positions=pos, device=DEV)
    _, want = R.rope_grads(dy.double(), x.double(), a, w.double(), 1e-6)
    assert torch.isinf(want[10:12]).all() and torch.isfinite(want[:10]).all() and torch.isfinite(want[12:]).all()
    assert torch.equal(dw[10:12].double(), want[10:12]) and torch.isfinite(dw[:10]).all() and torch.isfinite(dw[12:]).all()


@pytest.mark.parametrize("over", [0, 1])
@pytest.mark.parametrize("H,D,N", [(3, 64, 5), (40, 128, 37), (64, 64, 1), (17, 128, 321)])
def test_in_place_where_dx_overflows(H, D, N, over):
    """Small f16 rows: r is large and dx passes f16's range while dw is finite.  Lanes without a row see
    dx where it replaces x or dy; dw is the same as out of place, every time."""
    x, dy = rand((1, H, N, D), F16, 3, gain=2.0 ** -13), rand((1, H, N, D), F16, 4, gain=1000.0)
    w = torch.ones(D, device=DEV)
    p, g = params(SPLITS[D]), grid_of((1, 1, N))
    dx, dw = scope.rope_backward(dy, x, p, g, weight=w, eps=0.0)
    assert torch.isinf(dx[:, :, -1]).any() and torch.isfinite(dw).all()
    for _ in range(20):
        a = (dy.clone(), x.clone())
        dx2, dw2 = scope.rope_backward(*a, p, g, weight=w, eps=0.0, out=a[over])
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
