"""Refusals of the query/key norm and window attention entry points: no GPU, nothing launched."""
import ctypes

import pytest
import torch

from free_sparse_attention_b200 import capi
from free_sparse_attention_b200.build import build

FAKE = 1 << 20


@pytest.fixture(scope="module")
def L():
    build()
    return capi.lib()


def _norm(**over):
    kw = dict(B=2, H=4, Hkv=2, N=30, d=64, d_t=16, d_h=24, d_w=24, Hg=3, Wg=5, first=0, eps=1e-6, base=1e4, dtype=1)
    kw.update(over)
    return capi.QkNormParams(**kw)


def _window(**over):
    kw = dict(B=2, H=4, Hkv=2, Nq=30, Nk=40, d=64, frame=1, left=5, right=0, sinks=1, q_first=10, dtype=1)
    kw.update(over)
    return capi.WindowParams(**kw)


NORM_BAD = [(dict(B=0), 1), (dict(H=0), 1), (dict(Hkv=0), 1), (dict(N=0), 1), (dict(Hg=0), 1), (dict(Wg=-1), 1),
            (dict(d_t=17, d_h=23), 1), (dict(d_t=18), 1), (dict(d_t=-16, d_h=56), 1), (dict(eps=-1.0), 1),
            (dict(eps=float("nan")), 1), (dict(base=0.0), 1), (dict(base=float("inf")), 1), (dict(dtype=2), 1),
            (dict(first=-1), 1), (dict(d=96, d_t=32, d_h=32, d_w=32), 2), (dict(N=(1 << 24) + 1), 2),
            (dict(B=1 << 10, H=1 << 11), 2), (dict(B=16, N=1 << 24, H=8), 2), (dict(first=(1 << 30) + 1), 2)]


@pytest.mark.parametrize("over,code", NORM_BAD)
def test_norm_parameters_refused(L, over, code):
    p = _norm(**over)
    assert L.scope_qk_norm_workspace_bytes(ctypes.byref(p)) == 0
    assert L.scope_qk_norm_rope3d(ctypes.byref(p), None, FAKE, FAKE, None, None, None, FAKE, FAKE, None) == code
    assert L.scope_qk_norm_rope3d_backward(ctypes.byref(p), None, FAKE, FAKE, None, None, FAKE, FAKE, None, FAKE, FAKE,
                                           FAKE, FAKE, FAKE, 1 << 30, None) == code


def test_norm_pointers_refused(L):
    p = ctypes.byref(_norm())
    f = L.scope_qk_norm_rope3d
    assert f(None, None, FAKE, FAKE, None, None, None, FAKE, FAKE, None) == 1
    assert f(p, None, None, FAKE, None, None, None, FAKE, FAKE, None) == 1
    assert f(p, None, FAKE, None, None, None, None, FAKE, FAKE, None) == 1        # keys out without keys in
    assert f(p, None, FAKE, FAKE, None, None, None, FAKE, None, None) == 1
    assert f(p, None, FAKE + 2, FAKE, None, None, None, FAKE, FAKE, None) == 1
    assert f(p, None, FAKE, FAKE, FAKE + 4, None, None, FAKE, FAKE, None) == 1
    assert f(p, None, FAKE, FAKE, None, None, FAKE + 4, FAKE, FAKE, None) == 1
    g, need = L.scope_qk_norm_rope3d_backward, L.scope_qk_norm_workspace_bytes(p)
    ok = [p, None, FAKE, FAKE, None, None, FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE, FAKE, need, None]
    for i, v, code in ((13, None, 1), (13, FAKE + 16, 1), (14, need - 1, 3), (6, None, 1), (7, None, 1), (10, None, 1),
                       (9, None, 1), (3, None, 1), (11, FAKE + 8, 1)):
        bad = list(ok)
        bad[i] = v
        assert g(*bad) == code, (i, v)


WINDOW_BAD = [(dict(B=0), 1), (dict(H=0), 1), (dict(Hkv=0), 1), (dict(Hkv=3), 1), (dict(Nq=0), 1), (dict(Nk=0), 1),
              (dict(frame=0), 1), (dict(left=-2), 1), (dict(right=-2), 1), (dict(sinks=-1), 1), (dict(q_first=-1), 1),
              (dict(dtype=5), 1), (dict(d=96), 2), (dict(Nq=(1 << 24) + 1), 2), (dict(Nk=(1 << 24) + 1), 2),
              (dict(frame=(1 << 24) + 1), 2), (dict(left=(1 << 30) + 1), 2), (dict(sinks=(1 << 30) + 1), 2),
              (dict(q_first=(1 << 30) + 1), 2), (dict(B=1 << 11, H=1 << 10), 2), (dict(Nq=1 << 24, H=128, Hkv=128), 2)]


@pytest.mark.parametrize("over,code", WINDOW_BAD)
def test_window_parameters_refused(L, over, code):
    p = _window(**over)
    assert L.scope_window_workspace_bytes(ctypes.byref(p)) == 0
    assert L.scope_window_attention(ctypes.byref(p), None, FAKE, FAKE, FAKE, None, None, FAKE, None, FAKE, 1 << 40,
                                    None) == code
    assert L.scope_window_attention_backward(ctypes.byref(p), None, *[FAKE] * 6, None, None, *[FAKE] * 4, 1 << 40,
                                             None) == code


def test_window_pointers_refused(L):
    p = ctypes.byref(_window())
    need = L.scope_window_workspace_bytes(p)
    ok = [p, None, FAKE, FAKE, FAKE, None, None, FAKE, None, FAKE, need, None]
    for i, v, code in ((0, None, 1), (2, None, 1), (3, None, 1), (4, None, 1), (7, None, 1), (9, None, 1),
                       (9, FAKE + 128, 1), (10, need - 1, 3), (3, FAKE + 8, 1), (5, FAKE + 4, 1), (6, FAKE + 4, 1),
                       (8, FAKE + 4, 1)):
        bad = list(ok)
        bad[i] = v
        assert L.scope_window_attention(*bad) == code, (i, v)
    ok = [p, None] + [FAKE] * 6 + [None, None] + [FAKE] * 4 + [need, None]
    for i, v, code in ((0, None, 1), (5, None, 1), (6, None, 1), (7, None, 1), (10, None, 1), (11, None, 1),
                       (12, None, 1), (13, None, 1), (14, need - 1, 3), (12, FAKE + 2, 1)):
        bad = list(ok)
        bad[i] = v
        assert L.scope_window_attention_backward(*bad) == code, (i, v)


@pytest.mark.parametrize("strides", [(0, 0, 64), (7680, 1920, 60), (7680, 1920, 68), (-7680, 1920, 64), (7680, 1856, 64),
                                     (100, 1920, 64), (7680, 0, 64), (7680, 64, 64), (1 << 50, 1920, 64)])
def test_layouts_refused(L, strides):
    """Zero or negative strides of a dimension longer than one, strides that are no multiple of
    16 bytes, and layouts in which two elements share a place."""
    p, lay = _window(), capi.WindowLayouts()
    lay.q = capi.Strides(*strides)
    need = L.scope_window_workspace_bytes(ctypes.byref(p))
    assert L.scope_window_attention(ctypes.byref(p), ctypes.byref(lay), FAKE, FAKE, FAKE, None, None, FAKE, None, FAKE,
                                    need, None) == 1
    q, lay = _norm(), capi.QkNormLayouts()
    lay.yk = capi.Strides(*strides)
    assert L.scope_qk_norm_rope3d(ctypes.byref(q), ctypes.byref(lay), FAKE, FAKE, None, None, None, FAKE, FAKE, None) == 1


def test_workspace_sizes(L):
    size = lambda **o: L.scope_window_workspace_bytes(ctypes.byref(_window(**o)))  # noqa: E731
    assert size() % 256 == 0 and size() > 0
    # few rows over a long cache: room for the shares of every row
    assert size(Nq=1, Nk=1 << 20, left=-1) >= 2 * 4 * 2 * 64 * 4
    assert L.scope_qk_norm_workspace_bytes(ctypes.byref(_norm())) % 256 == 0
    with pytest.raises(capi.ScopeError):
        capi.alloc_window_workspace(_window(d=96))
    with pytest.raises(capi.ScopeError):
        capi.alloc_qk_norm_workspace(_norm(N=0))


def test_binding_refuses_tensors_that_do_not_fit():
    """Shapes, types, devices and channel strides are checked before the library is called."""
    p = _window()
    Q, K = torch.zeros((2, 4, 30, 64)), torch.zeros((2, 2, 40, 64))
    for args in ((Q, K, K), (Q.bfloat16(), K.bfloat16(), K.bfloat16())):      # float32; not on a GPU
        with pytest.raises(ValueError):
            capi._tensors("f", p, -1, capi.WindowLayouts, (("q", args[0], (2, 4, 30, 64)), ("k", args[1], (2, 2, 40, 64))))
    with pytest.raises(ValueError):
        capi._vector("f", "k_len", torch.zeros(3, dtype=torch.int32), 2, torch.int32, -1)
    with pytest.raises(ValueError):
        capi._vector("f", "k_len", torch.zeros(2, dtype=torch.int64), 2, torch.int32, -1)
    with pytest.raises(ValueError):
        capi._workspace("f", torch.zeros(4, dtype=torch.float32), -1)


def test_binding_refuses_calls_off_the_gpu():
    p, q = _window(dtype=0), _norm(dtype=0)
    Q, K = torch.zeros((2, 4, 30, 64)), torch.zeros((2, 2, 40, 64))
    ws = torch.empty(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError):
        capi.window_attention(p, Q, K, K, ws=ws)
    with pytest.raises(ValueError):
        capi.window_attention_backward(p, Q, K, K, Q, Q, torch.zeros((2, 4, 30)), ws=ws)
    with pytest.raises(ValueError):
        capi.qk_norm_rope3d(q, Q, K[:, :, :30])
    with pytest.raises(ValueError):
        capi.qk_norm_rope3d_backward(q, Q, None, None, None, Q, Q, ws=ws)


class _OnGpu(torch.Tensor):
    """A host tensor that the binding takes for one on GPU 0."""

    def get_device(self):
        return 0


def _on_gpu(shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(_OnGpu)


_Q, _K = (2, 4, 30, 64), (2, 2, 40, 64)
_CALLS = {      # the tensors of each call that may have strides, in the order of its arguments
    "norm": (lambda t: capi.qk_norm_rope3d(_norm(), t["Q"], t["K"], out_q=t["out_q"], out_k=t["out_k"]),
             {"Q": _Q, "K": (2, 2, 30, 64), "out_q": _Q, "out_k": (2, 2, 30, 64)}),
    "norm_backward": (lambda t: capi.qk_norm_rope3d_backward(_norm(), t["Q"], t["K"], None, None, t["dYq"], t["dYk"],
                                                             ws=_on_gpu(1 << 20, torch.uint8), out_q=t["out_q"],
                                                             out_k=t["out_k"]),
                      {"Q": _Q, "K": (2, 2, 30, 64), "dYq": _Q, "dYk": (2, 2, 30, 64), "out_q": _Q,
                       "out_k": (2, 2, 30, 64)}),
    "window": (lambda t: capi.window_attention(_window(), t["Q"], t["K"], t["V"], ws=_on_gpu(1 << 20, torch.uint8),
                                               out=t["out"]),
               {"Q": _Q, "K": _K, "V": _K, "out": _Q}),
    "window_backward": (lambda t: capi.window_attention_backward(
        _window(), t["Q"], t["K"], t["V"], t["O"], t["dO"], _on_gpu(_Q[:3], torch.float32),
        ws=_on_gpu(1 << 20, torch.uint8), out=(t["dQ"], t["dK"], t["dV"])),
        {"Q": _Q, "K": _K, "V": _K, "O": _Q, "dO": _Q, "dQ": _Q, "dK": _K, "dV": _K}),
}


@pytest.mark.parametrize("call,name", [(c, n) for c, (_, names) in _CALLS.items() for n in names])
def test_broadcast_tensors_are_refused(L, call, name):
    """One row expanded to a whole tensor, as the gradient of a sum is: its strides of zero are not the layout of
    zeros that means a dense tensor.  Tensors repeated along one dimension are refused too."""
    run, shapes = _CALLS[call]
    shape = shapes[name]
    for part in ((1, 1, 1, shape[3]), (1, *shape[1:]), (shape[0], 1, *shape[2:]), (*shape[:2], 1, shape[3])):
        t = {n: _on_gpu(s) for n, s in shapes.items()}
        t[name] = _on_gpu(part).expand(shape)
        assert t[name].stride(3) == 1 and t[name].get_device() == 0
        with pytest.raises(ValueError, match="repeated"):
            run(t)


def test_dimensions_of_one_may_have_any_stride():
    """A stride of zero along a dimension of length one steps over nothing."""
    p = _window(B=1, H=1, Hkv=1)
    wide = _on_gpu((1, 30, 3, 64))[:, :, :1].transpose(1, 2)      # [1, 1, 30, 64], tokens 192 apart
    for t in (wide, wide.as_strided((1, 1, 30, 64), (0, 0, 192, 1))):
        lay = capi._tensors("f", p, 0, capi.WindowLayouts, (("q", t, (1, 1, 30, 64)),))._obj
        assert lay.q.token == 192


class _Log:
    """Stands for a stream of the caller's, and for the library: what is done to them, in order."""

    def __init__(self):
        self.done, self.cuda_stream = [], 7

    def wait_stream(self, other):
        self.done.append(("wait", other))

    def __getattr__(self, name):
        return lambda *args: self.done.append(name) or (1 << 20 if name.endswith("_bytes") else 0)


class _Kept(_OnGpu):
    def record_stream(self, stream):
        stream.done.append("kept")


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("call", ["norm", "norm_backward", "window", "window_backward"])
def test_memory_made_for_a_stream_of_the_callers(monkeypatch, call, given):
    """Outputs and workspaces that a call allocates come from the current stream, which may still read what lay
    there: the caller's stream waits for it before the launch.  With buffers of the caller's there is no wait."""
    log, t = _Log(), {n: _on_gpu(s).as_subclass(_Kept) for n, s in _CALLS[call][1].items()}
    monkeypatch.setattr(capi, "lib", lambda: log)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index=None: ("current", index))
    ws = torch.zeros(1 << 20, dtype=torch.uint8).as_subclass(_Kept)
    monkeypatch.setattr(capi, "alloc_window_workspace", lambda p, device: ws)
    monkeypatch.setattr(capi, "alloc_qk_norm_workspace", lambda p, device: ws)
    lse = _on_gpu(_Q[:3], torch.float32).as_subclass(_Kept)
    own = {"ws": ws} if given else {}
    if call == "norm":
        own = {"out_q": t["out_q"], "out_k": t["out_k"]} if given else {"out_k": t["out_k"]}
        capi.qk_norm_rope3d(_norm(), t["Q"], t["K"], stream=log, **own)
    elif call == "norm_backward":
        own = {"ws": ws, "out_q": t["out_q"], "out_k": t["out_k"]} if given else {}
        capi.qk_norm_rope3d_backward(_norm(), t["Q"], t["K"], None, None, t["dYq"], t["dYk"], stream=log, **own)
    elif call == "window":
        capi.window_attention(_window(), t["Q"], t["K"], t["V"], out=t["out"], stream=log, **own)
    else:
        out = (t["dQ"], t["dK"], t["dV"]) if given else None
        capi.window_attention_backward(_window(), t["Q"], t["K"], t["V"], t["O"], t["dO"], lse, out=out, stream=log, **own)
    launch = log.done[-1]
    assert launch.startswith("scope_") and "kept" in log.done
    # the weights' gradients are always the call's own
    assert (("wait", ("current", 0)) in log.done) == (not given or call == "norm_backward")


def _off(values, dtype):
    """A contiguous vector that starts 4 bytes behind a multiple of 16, as the rest of a longer one does."""
    whole = torch.zeros(len(values) + 4, dtype=dtype)
    skip = next(i for i in range(4) if (whole.data_ptr() + 4 * i) % 16 == 4)
    t = whole[skip:skip + len(values)]
    t.copy_(torch.tensor(values))
    return t.as_subclass(_OnGpu)


def test_vectors_may_start_anywhere(monkeypatch):
    """Positions, lengths, weights and lse that are slices of longer tensors reach the library at a multiple of 16 bytes."""
    places = {"scope_qk_norm_rope3d": {4: "w", 5: "w", 6: "first"}, "scope_window_attention": {5: "first", 6: "lens"},
              "scope_qk_norm_rope3d_backward": {4: "w", 5: "w", 8: "first"},
              "scope_window_attention_backward": {7: "lse", 8: "first", 9: "lens"}}
    vectors = {"first": _off([3, 5], torch.int32), "lens": _off([11, 13], torch.int32),
               "w": _off([0.5 * i for i in range(64)], torch.float32), "lse": _off([0.1 * i for i in range(240)], torch.float32)}
    called = []

    class Library:
        def __getattr__(self, name):
            def f(*args):
                for i, what in places.get(name, {}).items():
                    assert args[i] % 16 == 0, (name, what)
                    want = vectors[what]
                    got = (ctypes.c_uint8 * (4 * want.numel())).from_address(args[i])
                    assert bytes(got) == want.as_subclass(torch.Tensor).numpy().tobytes(), (name, what)
                called.append(name)
                return 0
            return f

    monkeypatch.setattr(capi, "lib", lambda: Library())
    monkeypatch.setattr(capi, "_raw_stream", lambda index: 0)
    first, lens, w, lse = (vectors[n] for n in ("first", "lens", "w", "lse"))
    ws = _on_gpu(1 << 20, torch.uint8)
    t = {call: {n: _on_gpu(s) for n, s in shapes.items()} for call, (_, shapes) in _CALLS.items()}
    x = t["norm"]
    capi.qk_norm_rope3d(_norm(), x["Q"], x["K"], w, w, first=first)
    x = t["norm_backward"]
    capi.qk_norm_rope3d_backward(_norm(), x["Q"], x["K"], w, w, x["dYq"], x["dYk"], first=first, ws=ws)
    x = t["window"]
    capi.window_attention(_window(), x["Q"], x["K"], x["V"], q_first=first, k_len=lens, ws=ws)
    x = t["window_backward"]
    capi.window_attention_backward(_window(), x["Q"], x["K"], x["V"], x["O"], x["dO"], lse.view(_Q[:3]), q_first=first,
                                   k_len=lens, ws=ws)
    assert sorted(called) == sorted(places)
