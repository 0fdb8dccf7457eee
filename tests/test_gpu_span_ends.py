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


@pytest.mark.parametrize("sinks", [2 ** 64, sys.maxsize, sys.maxsize - 300, 2 ** 31, 300, 299])
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


@pytest.mark.parametrize("S,N,D", [(8, 1, 128), (64, 1, 128), (3, 40, 64), (2, 1, 256), (4, 3, 512)])
def test_passes_side_by_side_read_what_was_just_written(S, N, D):
    """Queries, caches and lengths that the kernel before the call has written, one
    workspace for all calls: eager calls without a wait between them, and captured ones,
    whose runs differ in their inputs only."""
    P, T, sets = 1040, 64, 4
    pre, own = tq.alloc_cache(1, 2, P, D, 8, 3), tq.alloc_cache(S, 2, T, D, 8, 3)
    q, lens, plens = torch.empty((S, 8, N, D), dtype=torch.bfloat16, device="cuda"), sc.ints([0] * S), sc.ints([0])
    data = []
    for i in range(sets):
        data.append((sc.cache(1, 2, P, D, 8, True, 3, 10 * i), sc.cache(S, 2, T, D, 8, True, 3, 10 * i + 3),
                     sc.normal(q.shape, 10 * i + 7), sc.ints([N + (5 * i + 11 * b) % (T - N) for b in range(S)]),
                     sc.ints([P - 300 * i])))

    def put(x):
        for a, b in ((pre, x[0]), (own, x[1])):
            for name in a:
                a[name].copy_(b[name])
        plens.copy_(x[4])
        lens.copy_(x[3])
        q.copy_(x[2])

    ws = torch.empty(tq.tq_prefix_attention_workspace_size(1, S, 8, 2, N, D), dtype=torch.uint8, device="cuda")

    def call():
        return tq.tq_prefix_attention(q, pre, P, own, T, 8, True, 3, prefix_lens=plens, lens=lens, workspace=ws)

    want = []
    for x in data:
        torch.cuda.synchronize()
        put(x)
        torch.cuda.synchronize()
        want.append([t.clone() for t in call()])
        ref = sc.reference(x[2], x[1], T, 8, True, 3, x[3].tolist(), prefix=x[0], P=P, prefix_lens=x[4].tolist(),
                           dtype=torch.bfloat16)
        sc.check(*want[-1], ref)
    got = []
    for i in range(40):
        put(data[i % sets])
        got.append(call())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = []
        for i in range(6):
            put(data[i % sets])
            kept.append(call())
    for i, g in enumerate(got):
        assert torch.equal(g[0], want[i % sets][0]) and torch.equal(g[1], want[i % sets][1])
    for turn in range(4):
        ws.fill_(0xFF if turn % 2 else 0)
        for x in kept:
            x[0].fill_(7.0)
        graph.replay()
        graph.replay()
        for i, g in enumerate(kept):
            assert torch.equal(g[0], want[i % sets][0]) and torch.equal(g[1], want[i % sets][1])
