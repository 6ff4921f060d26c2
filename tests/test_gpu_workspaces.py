"""The attention calls' workspaces on the GPU: two threads on one stream, and two captured
graphs, share none.  Needs a GB300."""
import pytest
import torch

from causal_linear_attention_chunkwise_gb300 import api
from tests.test_gpu_ssm_limits import run_together

pytestmark = pytest.mark.gpu


def _inputs(seed, d=64):
    g = torch.Generator().manual_seed(seed)
    q, k, v = ((torch.randn(1, 4, 4096, d, generator=g) / 8).bfloat16().cuda() for _ in range(3))
    return q, k, v, -0.01 * torch.rand(1, 4, 4096, d, generator=g).cuda()


CALLS = {
    "la_chunk_fwd": lambda q, k, v, a, **kw: api.la_chunk_fwd(q, k, v, **kw),
    "la_normalised_fwd": lambda q, k, v, a, **kw: api.la_normalised_fwd(q, k, v, **kw),
    "la_channel_gate_fwd": lambda q, k, v, a, **kw: api.la_channel_gate_fwd(q, k, v, a, **kw),
    "la_noncausal_fwd": lambda q, k, v, a, **kw: api.la_noncausal_fwd(q, k, v, **kw),
}


@pytest.fixture(autouse=True)
def _elu1():
    api.la_set_feature_map("elu1")


@pytest.mark.parametrize("name", CALLS)
def test_two_threads_on_one_stream(name, monkeypatch):
    runs = [_inputs(s) for s in (0, 1)]
    want = [CALLS[name](*r) for r in runs]
    got = run_together(monkeypatch, name, -3, [lambda r=r: CALLS[name](*r) for r in runs])
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    api.la_device_status()


@pytest.mark.parametrize("name", CALLS)
def test_two_captured_calls_replay_side_by_side(name):
    """Captured on one stream, replayed on two, with a larger eager call in between."""
    runs = []
    for seed in (2, 3):
        r = _inputs(seed)
        want = CALLS[name](*r)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = CALLS[name](*r)
        runs.append((r, want, got, graph, torch.cuda.Stream()))
    big = [torch.cat([t, t, t]) for t in _inputs(4)]
    CALLS[name](*big)
    torch.cuda.synchronize()
    for _ in range(3):
        for *_, graph, stream in runs:
            with torch.cuda.stream(stream):
                graph.replay()
    CALLS[name](*big)
    torch.cuda.synchronize()
    for _, want, got, *_ in runs:
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    api.la_device_status()
