"""GPU tests of the window and prefix attention at the ends of their arguments, against
references in 64 bits."""
import sys

import pytest
import torch

import turboquant_kv_cache_tq_gb300 as tq
from tests import step_common as sc
from tests.gpu_common import require_gpu
from tests.test_gpu_span_attention import window

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    assert tq.lib().tq_device_status(None) == 0


@pytest.mark.parametrize("sinks", [sys.maxsize, sys.maxsize - 300, 2 ** 31, 300, 299])
@pytest.mark.parametrize("G,N", [(1, 1), (4, 3), (4, 20), (3, 70)])
@pytest.mark.parametrize("D", [128, 512])
def test_first_tokens_of_any_number(sinks, G, N, D):
    """A window shorter than the sequences and first tokens that are all of them: few rows
    and many give what a window as wide as the sequences gives."""
    args = dict(lens=[300, 133], left_pad=[0, 17])
    out, lse, q, c = window(2, 2, G, N, 300, D, 8, True, 3, 7, sinks, torch.float32, **args)
    if sinks >= 300:
        ref = sc.reference(q, c, 300, 8, True, 3, [300, 133], [0, 17], None, sys.maxsize >> 1, 0)
        sc.check(out, lse, ref, "whole window")
