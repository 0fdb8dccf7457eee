"""GPU tests of refused window and prefix attention: nothing that a call was given to write is
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


@pytest.mark.parametrize("N", [3, 40])
def test_refused_attention_writes_nothing(N):
    B, Hq, Hkv, D, T = 2, 8, 2, 128, 100
    c, pre = sc.cache(B, Hkv, T, D, 8, True, 8, 1), sc.cache(1, Hkv, 90, D, 8, True, 8, 5)
    q = sc.normal((B, Hq, N, D), 1)
    out, lse = torch.empty_like(q), torch.empty((B, Hq, N), device="cuda")
    other = {k: v.cpu() for k, v in c.items()}
    for call, need, status in (
            (lambda q=q, c=c, T=T, window=30, sinks=2, kb=8, **kw: tq.tq_window_attention(q, c, T, kb, True, 8, window, sinks, **kw),
             tq.tq_window_attention_workspace_size(B, Hq, Hkv, N, D), (dict(window=0), dict(sinks=-1))),
            (lambda q=q, c=c, T=T, P=90, kb=8, **kw: tq.tq_prefix_attention(q, pre, P, c, T, kb, True, 8, **kw),
             tq.tq_prefix_attention_workspace_size(1, B, Hq, Hkv, N, D), (dict(P=91), dict(P=-1)))):
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        want, log = (t.clone() for t in call())
        for kw, error in (
                *((x, tq.TQError) for x in status), (dict(T=T + 1), tq.TQError), (dict(T=-1), tq.TQError),
                (dict(workspace=ws[:need - 16]), tq.TQError), (dict(workspace=ws[:0]), tq.TQError),
                (dict(workspace=ws[8:]), tq.TQError), (dict(workspace=ws.cpu()), ValueError),
                (dict(workspace=out.view(torch.uint8)), tq.TQError),
                (dict(lens=sc.ints([1, 2, 3])), ValueError), (dict(lens=sc.ints([1, 2]).float()), ValueError),
                (dict(count=sc.ints([1, 2]).long()), ValueError), (dict(count=sc.ints([1])), ValueError),
                (dict(left_pad=sc.ints([1, 2], "cpu")), ValueError), (dict(left_pad=sc.ints([1, 0, 2, 0])[::2]), ValueError),
                (dict(q=q.transpose(0, 1)), ValueError), (dict(q=q.float()), ValueError), (dict(q=q[0]), ValueError),
                (dict(c=other), ValueError), (dict(c=pre), ValueError), (dict(kb=4), ValueError),
                (dict(out_dtype=torch.float32), ValueError), (dict(out_dtype=torch.float16), ValueError),
                (dict(lse=lse.double()), ValueError), (dict(lse=out.view(torch.float32).flatten()[:lse.numel()].view(lse.shape)),
                                                       tq.TQError)):
            out.fill_(7.0)
            lse.fill_(7.0)
            ws.fill_(7)
            given = dict(dict(out=out, lse=lse, workspace=ws), **kw)
            with pytest.raises(error):
                call(**given)
            torch.cuda.synchronize()
            assert (out == 7.0).all() and (lse == 7.0).all() and (ws == 7).all(), kw
        for bad in (torch.full((B, Hq, N, D), 7.0, device="cuda"), torch.full((1, Hq, N, D), 7.0, device="cuda").bfloat16(),
                    torch.full((B, Hq, N, 2 * D), 7.0, device="cuda").bfloat16()[..., ::2]):
            lse.fill_(7.0)
            with pytest.raises(ValueError):
                call(out=bad, lse=lse, workspace=ws)
            torch.cuda.synchronize()
            assert (bad == 7.0).all() and (lse == 7.0).all()
        got = call(out=out, lse=lse, workspace=ws)  # and what is accepted is written
        assert got[0] is out and got[1] is lse and torch.equal(out, want) and torch.equal(lse, log)
