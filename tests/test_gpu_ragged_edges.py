"""GPU tests of the calls on ragged packed caches at the ends of what they
accept: budgets and caches of nothing, full rows, capacities far beyond the
sequences."""
import numpy as np
import pytest
import torch

import turboquant_kv_cache_tq_gb300 as tq
from tests import ragged_common as rc
from tests.gpu_common import cache_to_numpy, require_gpu

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


def test_a_path_that_does_not_fit_into_its_row():
    """What fits is appended, new - lens tokens; with that as n_path the weight
    sums see the same observers at the same tokens as a reference of the kept
    part of the path."""
    B, Hkv, G, N, D, cap = 3, 2, 2, 6, 128, 40
    main = rc.random_cache(B, Hkv, cap, D, 8, True, 3, 1)
    draft = rc.random_cache(B, Hkv, N, D, 8, True, 3, 2)
    dm, dt = rc.to_gpu(main), rc.to_gpu(draft)
    lens, path, n_path = [38, 40, 20], [[0, 1, 3, 5], [0, 2, 3, 4], [1, 2, 4, 5]], [4, 3, 4]
    sums = torch.ones((B, Hkv, cap), device="cuda")
    new = tq.commit_path(dm, _int(lens), dt, _int(path), _int(n_path), weights=sums)
    assert new.tolist() == [40, 40, 24]
    after, ow, _ = rc.gather_reference(draft, main, np.array(path), n_path, lens, None, np.ones((B, Hkv, cap), np.float32))
    for k, v in cache_to_numpy(dm).items():
        assert np.array_equal(v, after[k]), k
    assert np.array_equal(sums.cpu().numpy(), ow)
    q = torch.randn((B, Hkv * G, N, D), generator=torch.Generator().manual_seed(3)).bfloat16()
    lse = torch.full((B, Hkv * G, N), 4.0)
    appended = new - _int(lens)
    assert appended.tolist() == [2, 0, 4]
    got = tq.tq_attention_weights(q.cuda(), lse.cuda(), dm, cap, 8, True, path=_int(path), n_path=appended, lens=new,
                                  weights=sums)
    rc.check_weights(got, rc.weights_reference(q, lse, after, cap, 8, True, path, [2, 0, 4], [40, 40, 24], None, None,
                                               torch.tensor(ow), cap))
