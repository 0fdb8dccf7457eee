"""GPU tests of the rows that tq_append_kv refuses: nothing that the call was given to write is
touched."""
import pytest
import torch

import turboquant_kv_cache_tq_gb300 as tq
from tests import step_common as sc
from tests.gpu_common import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    assert tq.lib().tq_device_status(None) == 0


def _held(t):
    """t as it is now, to compare with later."""
    return t.clone().view(torch.uint8)


def _every_second(shape, dtype, seed):
    """Rows of which only every second element belongs to the tensor."""
    return sc.normal((*shape[:3], 2 * shape[3]), seed, dtype=dtype)[..., ::2]


def _columns(shape, dtype, seed):
    """Rows that lie across the memory's rows."""
    return sc.normal((*shape[:2], shape[3], shape[2]), seed, dtype=dtype).transpose(2, 3)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("broken", [_every_second, _columns])
def test_append_refuses_rows_that_are_not_contiguous(dtype, broken):
    B, Hq, Hkv, N, D, cap = 2, 4, 2, 8, 64, 32
    shapes = dict(q=(B, Hq, N, D), k=(B, Hkv, N, D), v=(B, Hkv, N, D))
    x = {name: sc.normal(s, i, dtype=dtype) for i, (name, s) in enumerate(shapes.items())}
    cos, sin = tq.rope_tables(D, 64)
    lens = sc.ints([3, 9])

    def call(x, cache, q_out, new):
        return tq.tq_append_kv(x["k"], x["v"], cache, lens, 8, True, 3, cos=cos, sin=sin, q=x["q"], q_out=q_out, new_lens=new)

    cache = sc.cache(B, Hkv, cap, D, 8, True, 3, 1)
    q_out, new = torch.full(shapes["q"], 7.0, dtype=dtype, device="cuda"), sc.ints([-7, -7])
    written = [*cache.values(), q_out, new]
    before = [_held(t) for t in written]
    for name in shapes:
        bad = dict(x)
        bad[name] = broken(shapes[name], dtype, 9)
        assert bad[name].shape == x[name].shape and bad[name].stride(-1) != 1
        with pytest.raises(ValueError, match="%s must be .* contiguous rows" % name):
            call(bad, cache, q_out, new)
        torch.cuda.synchronize()
        assert all(torch.equal(_held(t), b) for t, b in zip(written, before)), name
    call(x, cache, q_out, new)  # the same tensors with contiguous rows
    after, qt, lengths = sc.append_reference(x["k"], x["v"], sc.cache(B, Hkv, cap, D, 8, True, 3, 1), [3, 9], 8, True, 3,
                                             cos, sin, q=x["q"])
    assert sc.same_bytes(cache, after) and torch.equal(q_out.float().cpu(), qt.to(dtype).float()) and new.tolist() == lengths
