"""The library's calls in perf/operators.py: passes of one shape that are in flight together."""
import importlib.util
import os

import pytest
import torch

from free_sparse_attention_b200 import capi

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "operators.py")


def _operators():
    spec = importlib.util.spec_from_file_location("operators_under_test", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.own = True
    return m


def _cases(m):
    return [m._norm("norm", 1, 4, 2, 300, (16, 24, 24), 5, 8, 0, "bf16", train=True),
            m._window("few", 1, 8, 2, 1, 3000, 128, 1, 2000, 0, 4, "bf16"),
            m._window("train", 2, 4, 2, 1500, 1500, 64, 1, 300, 0, 4, "bf16", train=True),
            m._window("f32", 1, 2, 2, 700, 700, 64, 1, 200, 0, 4, "f32", train=True)]


@pytest.mark.parametrize("which", range(4))
def test_a_pass_has_a_workspace_of_its_own(monkeypatch, which):
    """Nothing that a call writes is shared by two passes of one shape (they may run on two streams or in two graphs)."""
    m, seen = _operators(), []
    case = _cases(m)[which]

    def call(n):
        def f(p, *args, ws=None, **kw):
            if ws is not None:
                seen[-1].append(ws)
            return tuple(torch.zeros(1) for _ in range(n)) if n else torch.zeros(1)
        return f

    for name, n in (("qk_norm_rope3d", 2), ("qk_norm_rope3d_backward", 4), ("window_attention_backward", 3),
                    ("window_attention", 2 if case.get("train") else 0)):
        monkeypatch.setattr(capi, name, call(n))
    for name in ("alloc_qk_norm_workspace", "alloc_window_workspace"):
        monkeypatch.setattr(capi, name, lambda p, device=None: torch.empty(4096, dtype=torch.uint8))
    state = {"case": case, **{n: torch.zeros(1) for n in ("q", "k", "v", "g", "wq", "wk", "gq", "gk", "first",
                                                          "q_first", "k_len")}}
    for _ in range(3):
        seen.append([])
        m.run(state)
    assert all(seen)
    places = [{w.data_ptr() for w in ws} for ws in seen]
    assert not (places[0] & places[1] or places[0] & places[2] or places[1] & places[2])
    assert all(w.numel() == 4096 and w.dtype == torch.uint8 for ws in seen for w in ws)


def _flat(out):
    return [t.clone() for t in out]


@pytest.mark.gpu
@pytest.mark.parametrize("which", range(4))
def test_passes_of_one_shape_on_two_streams(which):
    """Two streams with passes of one shape, not waited for between, and two graphs of them replayed at once."""
    m = _operators()
    case = _cases(m)[which]
    states = [m.prepare(case, seed) for seed in (1, 2)]
    want = [_flat(m.run(s)) for s in states]
    streams = [torch.cuda.Stream() for _ in states]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for s, stream, g in zip(states, streams, got):
            with torch.cuda.stream(stream):
                g.append(m.run(s))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(x, y) for out in g for x, y in zip(out, w))
    graphs = []
    for s in states:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphs.append((graph, m.run(s)))
    for _ in range(8):
        for (graph, _out), stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for w, (_graph, out) in zip(want, graphs):
        assert all(torch.equal(x, y) for x, y in zip(out, w))
