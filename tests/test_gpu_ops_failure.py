"""The operators' failure report without a GPU fault: a bounded wait that runs out (the library's own, on a barrier that
nothing completes, after about a millisecond) is reported once by ops_sync_status, from either error word and from another
stream, and the calls after it run clean."""
import pytest
import torch

import cluster_guided_sparse_b200 as scope
from test_gpu_cross import BF16, rand
from test_gpu_cross_bwd import grads

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("words", [(0,), (1,), (0, 1)])
def test_a_wait_that_ran_out_is_reported_once(words):
    q, do = rand((1, 2, 300, 64), BF16, 1), rand((1, 2, 300, 64), BF16, 4)
    k, v = rand((1, 2, 200, 64), BF16, 2), rand((1, 2, 200, 64), BF16, 3)
    ref = grads(q, k, v, do)
    scope.ops_sync_status()
    for w in words:
        scope.ops_selftest_wait_timeout(2_000_000, backward=bool(w))
    with pytest.raises(scope.ScopeError, match="wait gave up.*0x7e") as e:
        scope.ops_sync_status()
    assert e.value.status == 8
    scope.ops_sync_status()  # cleared by the report
    again = grads(q, k, v, do)
    scope.ops_sync_status()
    for n in ref:
        assert torch.equal(ref[n], again[n]), n


def test_a_wait_on_another_stream_is_reported_there():
    side = torch.cuda.Stream()
    scope.ops_selftest_wait_timeout(2_000_000, stream=side)
    with pytest.raises(scope.ScopeError, match="wait gave up"):
        scope.ops_sync_status(side)
    scope.ops_sync_status(side)
    scope.ops_sync_status()
