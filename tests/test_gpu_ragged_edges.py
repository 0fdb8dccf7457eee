"""GPU tests of the calls on ragged packed caches at the ends of what they
accept: budgets and caches of nothing, full rows, capacities far beyond the
sequences."""
import pytest
import torch

import turboquant_kv_cache_tq_gb300 as tq
from tests import ragged_common as rc
from tests.gpu_common import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _int(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def test_cutting_to_nothing():
    cache = rc.to_gpu(rc.random_cache(2, 3, 20, 128, 8, True, 3, 1))
    w = torch.rand((2, 3, 20), device="cuda")
    for t_cap in (None, 4):
        cut, cw, length = tq.evict_rows(cache, w, 20, 0, 0, lens=_int([20, 7]), t_cap=t_cap)
        assert length.tolist() == [0, 0]
        assert cut["k_codes"].shape[2] == cw.shape[2] == (t_cap or 0)


def test_cutting_a_cache_without_room():
    cache = tq.alloc_cache(2, 3, 0, 128, 8, 3)
    w = torch.zeros((2, 3, 0), device="cuda")
    index, count = tq.tq_evict_select(w, 0, 5, 2)
    assert (index == -1).all() and count.tolist() == [0, 0]
    cut, cw, length = tq.evict_rows(cache, w, 0, 5, 2)
    assert length.tolist() == [0, 0] and cut["k_codes"].shape[2] == 5 and (cw == 0).all()
