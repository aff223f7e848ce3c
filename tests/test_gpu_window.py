"""Window attention with sinks and the query/key norm with RoPE on the GPU, forward and
backward, against the binary64 forms and bounds of window_common."""
import math

import pytest
import torch

from free_sparse_attention_b200 import capi
from window_common import angles, attention, check, norm, visible

pytestmark = pytest.mark.gpu

DT = {"bf16": (torch.bfloat16, capi.SCOPE_BF16), "f32": (torch.float32, capi.SCOPE_F32)}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from free_sparse_attention_b200.build import build
    build()
    capi.lib()


def _randn(shape, dtype, seed, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * gain).to(dtype).cuda()


def _params(dtype, B=1, H=2, Hkv=None, Nq=100, Nk=None, d=64, frame=1, left=20, right=0, sinks=0, q_first=0):
    return capi.WindowParams(B=B, H=H, Hkv=Hkv or H, Nq=Nq, Nk=Nk or Nq, d=d, frame=frame, left=left, right=right,
                             sinks=sinks, q_first=q_first, dtype=DT[dtype][1])


def _inputs(p, dtype, seed=0):
    dt = DT[dtype][0]
    return (_randn((p.B, p.H, p.Nq, p.d), dt, seed, 1.5), _randn((p.B, p.Hkv, p.Nk, p.d), dt, seed + 1),
            _randn((p.B, p.Hkv, p.Nk, p.d), dt, seed + 2), _randn((p.B, p.H, p.Nq, p.d), dt, seed + 3))


def _run(p, dtype, q_first=None, k_len=None, seed=0, backward=True):
    Q, K, V, G = _inputs(p, dtype, seed)
    dev = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    at = {"q_first": dev(q_first), "k_len": dev(k_len)}
    vis = visible(p, q_first or [p.q_first] * p.B, k_len or [p.Nk] * p.B)
    ref = attention(Q, K, V, vis, G if backward else None)
    ws = capi.alloc_window_workspace(p)
    O, lse = capi.window_attention(p, Q, K, V, ws=ws, lse=True, **at)
    torch.cuda.synchronize()
    assert capi.get_device_status(ws) == 0
    check("O", O, *ref["O"])
    check("lse", lse, *ref["lse"])
    if backward:
        dQ, dK, dV = capi.window_attention_backward(p, Q, K, V, O, G, lse, ws=ws, **at)
        torch.cuda.synchronize()
        assert capi.get_device_status(ws) == 0
        for n, t in (("dQ", dQ), ("dK", dK), ("dV", dV)):
            check(n, t, *ref[n])
    return O


SHAPES = [
    dict(Nq=1), dict(Nq=2, left=0), dict(Nq=63), dict(Nq=64, right=3), dict(Nq=65, d=128, sinks=2),
    dict(Nq=127, left=200), dict(Nq=129, d=128, left=7, right=5), dict(Nq=257, H=1, left=40, sinks=5),
    dict(Nq=300, left=-1, right=0, d=128), dict(Nq=300, left=-1, right=-1),
    dict(Nq=390, frame=130, left=1, right=1, sinks=1), dict(Nq=513, frame=7, left=4, right=2, sinks=3, d=128),
    dict(Nq=400, left=3, sinks=400), dict(Nq=260, frame=1000, left=0, right=0), dict(Nq=700, left=-1, right=2, sinks=9),
    dict(B=2, H=6, Hkv=2, Nq=333, left=50, sinks=4, d=128), dict(B=1, H=8, Hkv=1, Nq=150, left=33, right=0),
    dict(Nq=100, Nk=500, left=90, q_first=400, sinks=2), dict(Nq=130, Nk=900, frame=64, left=3, q_first=770, d=128),
    dict(Nq=5, Nk=1000, left=600, q_first=995, sinks=1, H=4, Hkv=2), dict(Nq=200, Nk=90, left=30),
    dict(Nq=70, Nk=64, left=5, q_first=40),          # the last queries' windows lie past the keys
    dict(Nq=64, Nk=64, left=5, q_first=1 << 30),     # every window does
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(f"{k}{v}" for k, v in s.items()))
def test_window_attention_and_gradients(shape, dtype):
    _run(_params(dtype, **shape), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape,q_first,k_len", [
    (dict(B=3, Nq=200, left=30, sinks=2), None, [200, 77, 0]),
    (dict(B=3, Nq=200, left=30), None, [1, 130, 64]),
    (dict(B=4, H=8, Hkv=2, Nq=1, Nk=700, left=255, sinks=4, d=128), [699, 0, 511, 63], [700, 1, 512, 64]),
    (dict(B=2, H=4, Hkv=4, Nq=90, Nk=700, frame=30, left=2, right=0, sinks=1), [600, 210], [690, 300]),
    (dict(B=2, Nq=64, Nk=128, left=10, right=10), [1 << 20, -5], [1000, -3]),     # clamped
])
def test_window_attention_lengths_and_positions_per_entry(shape, q_first, k_len, dtype):
    p = _params(dtype, **shape)
    B = p.B
    # the reference takes the clamped values
    if q_first and min(q_first) < 0:
        Q, K, V, _ = _inputs(p, dtype)
        O = capi.window_attention(p, Q, K, V, q_first=torch.tensor(q_first, dtype=torch.int32, device="cuda"),
                                  k_len=torch.tensor(k_len, dtype=torch.int32, device="cuda"))
        vis = visible(p, [max(x, 0) for x in q_first], [min(max(n, 0), p.Nk) for n in k_len])
        check("O", O, *attention(Q, K, V, vis)["O"])
    else:
        _run(p, dtype, q_first or [0] * B, k_len)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Nq,H,Hkv", [(1, 1, 1), (1, 5, 5), (1, 32, 4), (1, 40, 1), (3, 8, 2), (16, 1, 1), (17, 2, 1), (40, 2, 2)])
def test_few_rows_over_a_long_cache(Nq, H, Hkv, dtype):
    """The split form: shares of a long key range joined, with sinks and without a window."""
    n = 9001
    for left, sinks, d in ((4095, 4, 128), (-1, 0, 64), (60, 70, 128)):
        p = _params(dtype, H=H, Hkv=Hkv, Nq=Nq, Nk=n, d=d, left=left, right=0, sinks=sinks, q_first=n - Nq)
        _run(p, dtype, backward=Nq == 3)


@pytest.mark.parametrize("H", [200, 148, 98, 74, 59, 49, 30, 2])
def test_few_rows_in_every_number_of_shares(H):
    """Heads that leave each a different number of shares of its keys, one to six joined as a cluster and more by a
    second kernel."""
    p = _params("bf16", H=H, Hkv=H, Nq=1, Nk=3001, d=64, frame=50, left=60, right=0, sinks=3, q_first=3000)
    _run(p, "bf16", backward=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape,k_len", [
    (dict(H=2, Hkv=1, Nq=1500, left=50, sinks=4), None),                              # only the sinks are cut
    (dict(H=1, Nq=1300, left=-1, right=0, d=128), None),                              # no sinks, every tile is
    (dict(B=2, H=4, Hkv=2, Nq=1111, frame=100, left=5, right=0, sinks=2, d=128), [1111, 150]),   # both
    (dict(H=3, Hkv=1, Nq=900, Nk=400, frame=300, left=0, right=-1, sinks=1), [399]),
])
def test_gradients_of_keys_that_many_queries_see(shape, k_len, dtype):
    """Key tiles whose walk over the queries is cut into shares: sinks, long windows, groups, short entries."""
    p = _params(dtype, **shape)
    _run(p, dtype, None, k_len)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_tensors(dtype):
    """Slices of one [B, N, 3, H, d] buffer in, slices of another out, forward and backward."""
    p = _params(dtype, B=2, H=3, Nq=150, d=64, left=40, right=4, sinks=3)
    dt = DT[dtype][0]
    qkv = _randn((p.B, p.Nq, 3, p.H, p.d), dt, 5)
    Q, K, V = (qkv[:, :, i].transpose(1, 2) for i in range(3))
    out = torch.zeros((p.B, p.Nq, p.H, p.d + 64), dtype=dt, device="cuda")
    O = out[..., :p.d].transpose(1, 2)
    _, lse = capi.window_attention(p, Q, K, V, out=O, lse=True)
    G = _randn((p.B, p.Nq, p.H, p.d), dt, 6).transpose(1, 2)
    ref = attention(Q, K, V, visible(p, [0] * p.B, [p.Nk] * p.B), G)
    check("O", O, *ref["O"])
    assert (out[..., p.d:] == 0).all()
    grad = torch.zeros_like(qkv)
    outs = tuple(grad[:, :, i].transpose(1, 2) for i in range(3))
    capi.window_attention_backward(p, Q, K, V, O, G, lse, out=outs)
    for n, t in zip(("dQ", "dK", "dV"), outs):
        check(n, t, *ref[n])
    # the same values as from dense copies
    dense = capi.window_attention(p, Q.contiguous(), K.contiguous(), V.contiguous())
    assert torch.equal(dense, O)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Nq", [300, 1])
def test_what_lies_behind_the_keys_is_not_used(dtype, Nq):
    """NaN and infinity at and beyond k_len, in the keys and in the values."""
    p = _params(dtype, B=2, H=2, Nq=Nq, Nk=300, d=128, left=70, right=70, sinks=2)
    Q, K, V, G = _inputs(p, dtype, 9)
    k_len = [171, 40]
    first = torch.tensor([max(n - Nq, 0) if Nq == 1 else 0 for n in k_len], dtype=torch.int32, device="cuda")
    lens = torch.tensor(k_len, dtype=torch.int32, device="cuda")
    O, lse = capi.window_attention(p, Q, K, V, q_first=first, k_len=lens, lse=True)
    grads = capi.window_attention_backward(p, Q, K, V, O, G, lse, q_first=first, k_len=lens)
    Kn, Vn = K.clone(), V.clone()
    for b, n in enumerate(k_len):
        Kn[b, :, n:] = float("nan")
        Vn[b, :, n:] = float("inf")
        Vn[b, :, n + 1:] = float("nan")
    O2, lse2 = capi.window_attention(p, Q, Kn, Vn, q_first=first, k_len=lens, lse=True)
    again = capi.window_attention_backward(p, Q, Kn, Vn, O2, G, lse2, q_first=first, k_len=lens)
    assert torch.equal(O, O2) and torch.equal(lse, lse2)
    for x, y in zip(grads, again):
        assert torch.equal(x, y)
    for b, n in enumerate(k_len):
        assert (again[1][b, :, n:] == 0).all() and (again[2][b, :, n:] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Nq", [200, 1])
def test_hidden_keys_that_are_not_finite_change_nothing_and_visible_ones_show(dtype, Nq):
    p = _params(dtype, Nq=Nq, Nk=200, d=64, left=20, right=0, q_first=200 - Nq)
    Q, K, V, _ = _inputs(p, dtype, 11)
    O = capi.window_attention(p, Q, K, V)
    Kn = K.clone()
    Kn[:, :, 30] = float("nan")
    On = capi.window_attention(p, Q, Kn, V)
    sees = visible(p, [p.q_first], [p.Nk])[0][:, 30]
    assert torch.equal(On[:, :, ~sees], O[:, :, ~sees])
    assert torch.isnan(On[:, :, sees]).all()
    if Nq == 1:
        Kn = K.clone()
        Kn[:, :, 190] = float("nan")
        assert torch.isnan(capi.window_attention(p, Q, Kn, V)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_logits(dtype):
    """Logits of hundreds, growing along the keys: the running maximum rescales every tile."""
    p = _params(dtype, Nq=140, Nk=600, d=64, left=-1, right=-1)
    Q, K, V, G = _inputs(p, dtype, 13)
    K = K + (torch.arange(600, device="cuda") / 25.0)[:, None].to(K.dtype) * Q[:, :, :1].sign()
    Q = Q.abs() * Q[:, :, :1].sign()
    ref = attention(Q, K, V, visible(p, [0], [600]), None)
    O = capi.window_attention(p, Q, K, V)
    check("O", O, *ref["O"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_gradients_of_large_logits(d, dtype):
    """The same logits of hundreds in the gradients, where P is 2^(c s - lse log2 e), the difference of two large numbers."""
    p = _params(dtype, Nq=140, Nk=600, d=d, left=-1, right=-1)
    Q, K, V, G = _inputs(p, dtype, 13)
    K = K + (torch.arange(600, device="cuda") / 25.0)[:, None].to(K.dtype) * Q[:, :, :1].sign()
    Q = Q.abs() * Q[:, :, :1].sign()
    ref = attention(Q, K, V, visible(p, [0], [600]), G)
    O, lse = capi.window_attention(p, Q, K, V, lse=True)
    assert 200 < lse.abs().max() < 2000
    check("O", O, *ref["O"])
    check("lse", lse, *ref["lse"])
    grads = capi.window_attention_backward(p, Q, K, V, O, G, lse)
    # The bounds above are relative.  Here most P are below 2^-126 (the logits span hundreds, 2^-126 is e^-87), the least
    # normal number, under which an exponential, a product or an operand may be flushed to 0: off by at most 2^-126 each.
    # P and dS = P (dP - D) are then off by 2^-126 and 2^-126 (|dP| + |D| + 1), the sums by that times the other factor,
    # and a result by 2^-126.
    tiny, sc = 2.0 ** -126, 1.0 / math.sqrt(d)
    q, k, v, g = (x.double() for x in (Q, K, V, G))
    ds = tiny * ((g @ v.mT).abs() + (g * ref["O"][0]).sum(-1, keepdim=True).abs() + 1)
    under = {"dQ": sc * ds @ k.abs() + tiny, "dK": sc * ds.mT @ q.abs() + tiny, "dV": tiny * (g.abs().sum(2, keepdim=True) + 1)}
    for n, t in zip(("dQ", "dK", "dV"), grads):
        check(n, t, ref[n][0], ref[n][1] + under[n])
    # sum_j P_ij = 1, so the keys' dV add up to the queries' dO whatever the logits.  A logit and lse meet in both
    # passes with the same bits: four roundings of up to |lse| and one each of 600 and 64 terms of the row sum, in
    # binary32; of the sums over 140 queries as many; half a step of bf16 on P and on every dV
    low = 2.0 ** -8 if dtype == "bf16" else 0.0
    u = low + 2.0 ** -24 * (4 * (1 + 2 * lse.double().abs()) + 664 + 204)
    bound = 1.02 * (G.double().abs() * u[..., None]).sum(2) + low * grads[2].double().abs().sum(2)
    assert ((grads[2].double().sum(2) - G.double().sum(2)).abs() <= bound).all()


@pytest.mark.parametrize("d", [64, 128])
def test_a_query_of_one_key_has_no_gradient_of_its_scores(d):
    """P = 1 whatever the score: dQ and dK are zeros, not what is left of two sums, and dV is dO."""
    p = _params("f32", H=2, Nq=131, left=0, d=d)
    Q, K, V, G = _inputs(p, "f32")
    O, lse = capi.window_attention(p, Q, K, V, lse=True)
    dQ, dK, dV = capi.window_attention_backward(p, Q, K, V, O, G, lse)
    assert not dQ.any() and not dK.any()
    # P = 2^(s c - lse log2 e): each rounding of a logit of up to |lse| is 2^-24 of it, four of them
    assert ((dV - G).abs() <= G.abs() * (4 * 2.0 ** -24 * (1 + 2 * lse.abs()))[..., None]).all()


def test_gradients_against_differences():
    """Central differences of the binary64 forward along random directions."""
    p = _params("f32", B=1, H=4, Hkv=2, Nq=96, d=64, left=30, right=2, sinks=2)
    Q, K, V, G = _inputs(p, "f32", 17)
    vis = visible(p, [0], [p.Nk])
    O, lse = capi.window_attention(p, Q, K, V, lse=True)
    grads = capi.window_attention_backward(p, Q, K, V, O, G, lse)
    loss = lambda *x: (attention(*x, vis)["O"][0] * G.double()).sum().item()  # noqa: E731
    xs = [Q.double(), K.double(), V.double()]
    h = 1e-5
    for i, g in enumerate(grads):
        for seed in range(3):
            e = _randn(xs[i].shape, torch.float32, 100 + seed).double()
            up, dn = list(xs), list(xs)
            up[i], dn[i] = xs[i] + h * e, xs[i] - h * e
            num = (loss(*up) - loss(*dn)) / (2 * h)
            got = (g.double() * e).sum().item()
            # difference error ~ h^2 third derivative and 1e-16 |L| / h; kernel error ~ 1e-6 per term
            assert abs(num - got) <= 1e-4 * (g.double().abs() * e.abs()).sum().item()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_same_bits_again_and_rows_do_not_mix(dtype):
    p = _params(dtype, B=2, H=4, Hkv=2, Nq=500, d=128, left=100, right=10, sinks=4)
    Q, K, V, G = _inputs(p, dtype, 19)
    O, lse = capi.window_attention(p, Q, K, V, lse=True)
    grads = capi.window_attention_backward(p, Q, K, V, O, G, lse)
    for _ in range(3):
        O2, lse2 = capi.window_attention(p, Q, K, V, lse=True)
        assert torch.equal(O, O2) and torch.equal(lse, lse2)
        for x, y in zip(grads, capi.window_attention_backward(p, Q, K, V, O2, G, lse2)):
            assert torch.equal(x, y)
    # batch entry 1 alone gives its own rows
    p1 = _params(dtype, B=1, H=4, Hkv=2, Nq=500, d=128, left=100, right=10, sinks=4)
    assert torch.equal(capi.window_attention(p1, Q[1:], K[1:], V[1:])[0], O[1])


@pytest.mark.parametrize("Nq", [1, 300])
def test_captured_and_replayed_on_another_stream(Nq):
    """Forward and backward in one graph, replayed with new inputs in the same buffers."""
    p = _params("bf16", H=4, Nq=Nq, Nk=1300, d=128, left=999, q_first=1300 - Nq, sinks=4)
    Q, K, V, G = _inputs(p, "bf16", 23)
    ws = capi.alloc_window_workspace(p)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        O, lse = capi.window_attention(p, Q, K, V, ws=ws, lse=True)
        capi.window_attention_backward(p, Q, K, V, O, G, lse, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        O, lse = capi.window_attention(p, Q, K, V, ws=ws, lse=True)
        dQ, dK, dV = capi.window_attention_backward(p, Q, K, V, O, G, lse, ws=ws)
    for seed in (30, 40):
        for t, x in zip((Q, K, V, G), _inputs(p, "bf16", seed)):
            t.copy_(x)
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
            graph.replay()
        torch.cuda.synchronize()
        O2, lse2 = capi.window_attention(p, Q, K, V, lse=True, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(O, O2)
        for x, y in zip((dQ, dK, dV), capi.window_attention_backward(p, Q, K, V, O2, G, lse2)):
            assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_training_step_captured_and_replayed_without_a_pause(dtype):
    """Norm, attention with cut key tiles, and both gradients in one graph, replayed three times over before the
    device is waited for; two graphs share the workspaces."""
    dt, code = DT[dtype]
    p = _params(dtype, H=4, Hkv=2, Nq=1200, d=64, left=60, sinks=4)
    n = capi.QkNormParams(B=1, H=4, Hkv=2, N=1200, d=64, d_t=16, d_h=24, d_w=24, Hg=5, Wg=8, first=0, eps=1e-6,
                          base=10000.0, dtype=code)
    Q, K, V, G = _inputs(p, dtype, 50)
    ws, nws = capi.alloc_window_workspace(p), capi.alloc_qk_norm_workspace(n)

    def step():
        Yq, Yk = capi.qk_norm_rope3d(n, Q, K)
        O, lse = capi.window_attention(p, Yq, Yk, V, ws=ws, lse=True)
        dYq, dYk, dV = capi.window_attention_backward(p, Yq, Yk, V, O, G, lse, ws=ws)
        return (O, lse, dV) + capi.qk_norm_rope3d_backward(n, Q, K, None, None, dYq, dYk, ws=nws)

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        graphs.append((graph, out))
    for seed in (60, 70):
        for t, x in zip((Q, K, V, G), _inputs(p, dtype, seed)):
            t.copy_(x)
        for _ in range(3):
            for graph, _out in graphs:
                graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        for _graph, out in graphs:
            for x, y in zip(out, want):
                assert torch.equal(x, y)


@pytest.mark.parametrize("d", [64, 128])
def test_captured_with_more_items_than_multiprocessors(d):
    """A forward of 200 items of 256 rows, whose counter is cleared by a node of its own in the graph."""
    p = _params("bf16", H=40, Hkv=8, Nq=1200, d=d, left=150, sinks=2)
    Q, K, V, G = _inputs(p, "bf16", 71)
    ws = capi.alloc_window_workspace(p)

    def step():
        O, lse = capi.window_attention(p, Q, K, V, ws=ws, lse=True)
        return (O, lse) + capi.window_attention_backward(p, Q, K, V, O, G, lse, ws=ws)

    want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert capi.get_device_status(ws) == 0
        assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("over", [dict(frame=1 << 24, left=1 << 30, right=1 << 30, sinks=1 << 30),
                                  dict(frame=1, left=0, right=1 << 30, sinks=1 << 30), dict(frame=1 << 24, left=0, right=0),
                                  dict(frame=3, left=1 << 30, right=0, q_first=(1 << 30) - 3),
                                  dict(frame=2, left=0, right=0, sinks=1, q_first=1 << 30)])
def test_windows_at_the_limits_of_their_numbers(over, dtype):
    """Limits of windows, frames and positions, whose products take 55 bits."""
    _run(_params(dtype, Nq=70, Nk=150, **{"left": 5, **over}), dtype)


def test_two_threads_at_once():
    """Two host threads, each on a stream of its own with default workspaces and outputs."""
    import threading
    ps = [_params("bf16", H=4, Hkv=2, Nq=700, d=128, left=200, sinks=4), _params("f32", H=2, Nq=400, left=90, sinks=1)]
    ins = [_inputs(p, t, 81) for p, t in zip(ps, ("bf16", "f32"))]

    def step(p, x):
        O, lse = capi.window_attention(p, *x[:3], lse=True)
        return (O, lse) + capi.window_attention_backward(p, *x[:3], O, x[3], lse)

    want = [step(p, x) for p, x in zip(ps, ins)]
    torch.cuda.synchronize()
    got, failed = [[], []], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got[i].append(step(ps[i], ins[i]))
                torch.cuda.current_stream().synchronize()
        except Exception as e:   # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for w, runs in zip(want, got):
        assert len(runs) == 20 and all(torch.equal(x, y) for out in runs for x, y in zip(out, w))


def test_whole_layer_sampled_rows():
    """17550 tokens in frames of 1350, 6 of 48 heads: rows of the first, a middle and the last
    frame against the binary64 form of those rows."""
    p = _params("bf16", H=6, Nq=17550, d=64, frame=1350, left=1, right=1, sinks=1)
    Q, K, V, _ = _inputs(p, "bf16", 29)
    ws = capi.alloc_window_workspace(p)
    O = capi.window_attention(p, Q, K, V, ws=ws)
    assert capi.get_device_status(ws) == 0
    for r0 in (0, 1349, 8000, 17500):
        r1 = min(r0 + 50, 17550)
        pr = _params("bf16", H=6, Nq=r1 - r0, Nk=17550, d=64, frame=1350, left=1, right=1, sinks=1, q_first=r0)
        ref = attention(Q[:, :, r0:r1], K, V, visible(pr, [r0], [17550]))
        check("O", O[:, :, r0:r1], *ref["O"])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("left", [0, 1])
def test_gaps_between_sinks_and_windows(left, d):
    """Row tiles across frame ends: one half sees many key tiles in a row that the other does
    not (more than the rings hold), behind the sinks and at the windows' ends."""
    p = _params("bf16", H=2, Nq=5200, d=d, frame=1300, left=left, right=0, sinks=1)
    Q, K, V, G = _inputs(p, "bf16", 41)
    ws = capi.alloc_window_workspace(p)
    O, lse = capi.window_attention(p, Q, K, V, ws=ws, lse=True)
    assert capi.get_device_status(ws) == 0
    grads = capi.window_attention_backward(p, Q, K, V, O, G, lse, ws=ws)
    assert capi.get_device_status(ws) == 0
    ref = attention(Q, K, V, visible(p, [0], [5200]), G)
    check("O", O, *ref["O"])
    for n, t in zip(("dQ", "dK", "dV"), grads):
        check(n, t, *ref[n])


def test_gradients_of_rows_that_see_few_keys():
    """With 1 to 8 visible keys the rounding of O to bf16 would move D = dO . O as much as the
    rounding of dS does: the bounds here count no error of D but binary32 sums'."""
    p = _params("bf16", B=2, H=3, Nq=700, d=128, left=3, right=0, sinks=4)
    Q, K, V, G = _inputs(p, "bf16", 43)
    k_len = torch.tensor([700, 220], dtype=torch.int32, device="cuda")     # entry 1: most rows see sinks only
    O, lse = capi.window_attention(p, Q, K, V, k_len=k_len, lse=True)
    dQ, dK, dV = capi.window_attention_backward(p, Q, K, V, O, G, lse, k_len=k_len)
    vis = visible(p, [0, 0], [700, 220]).cuda()[:, None]
    q, k, v, g = (x.double() for x in (Q, K, V, G))
    s = (q @ k.mT / math.sqrt(p.d)).masked_fill(~vis, -math.inf)
    P = torch.nan_to_num(torch.softmax(s, -1))
    dP = g @ v.mT
    dS = P * (dP - (P * dP).sum(-1, keepdim=True))
    # dS: one rounding to bf16; binary32 sums of 128 products in P (through the logits, at most
    # 2 * 132 units of about 40 |.|) and in dP and D
    bound = 2.0 ** -8 * dS.abs() + 2.0 ** -24 * P * (132 * (g.abs() @ v.abs().mT) * 2 + 600 * 8 * dP.abs().amax(-1, keepdim=True))
    want = dS @ k / math.sqrt(p.d)
    check("dQ", dQ, want, 2.0 ** -8 * want.abs() + 1.02 * (bound @ k.abs()) / math.sqrt(p.d))
    want = dS.mT @ q / math.sqrt(p.d)
    check("dK", dK, want, 2.0 ** -8 * want.abs() + 1.02 * (bound.mT @ q.abs()) / math.sqrt(p.d))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_beyond_32_bits(dtype):
    """Batch entries 2^31 elements apart: every kernel's address arithmetic."""
    dt, far = DT[dtype][0], 1 << 31
    big = torch.empty(far + 4096 * 64, dtype=dt, device="cuda")

    def place(x):
        """x [2, h, n, 64] into slices of `big`, entry 1 at 2^31 elements, packed one after another."""
        nonlocal used
        h, n = x.shape[1], x.shape[2]
        t = big.as_strided(x.shape, (far, n * 64, 64, 1), used)
        t.copy_(x)
        used += h * n * 64
        return t

    for Nq, Nk in ((150, 300), (1, 300)):
        used = 0
        p = _params(dtype, B=2, H=2, Nq=Nq, Nk=Nk, left=90, sinks=3, q_first=Nk - Nq)
        Q, K, V, G = _inputs(p, dtype, 47)
        dense, lse0 = capi.window_attention(p, Q, K, V, lse=True)
        want = capi.window_attention_backward(p, Q, K, V, dense, G, lse0)
        q, k, v, g = (place(x) for x in (Q, K, V, G))
        o = place(torch.zeros_like(Q))
        _, lse = capi.window_attention(p, q, k, v, out=o, lse=True)
        assert torch.equal(o, dense) and torch.equal(lse, lse0)
        outs = tuple(place(torch.zeros_like(x)) for x in (Q, K, V))
        capi.window_attention_backward(p, q, k, v, o, g, lse, out=outs)
        for x, y in zip(outs, want):
            assert torch.equal(x, y)
    used = 0
    np_ = _norm_params(dtype, B=2, H=3, N=50)
    X, G = _randn((2, 3, 50, 64), dt, 1), _randn((2, 3, 50, 64), dt, 2)
    y0, _ = capi.qk_norm_rope3d(np_, X, None)
    d0, _, w0, _ = capi.qk_norm_rope3d_backward(np_, X, None, None, None, G, None)
    x, g, y, dx = place(X), place(G), place(torch.zeros_like(X)), place(torch.zeros_like(X))
    capi.qk_norm_rope3d(np_, x, None, out_q=y)
    _, _, w, _ = capi.qk_norm_rope3d_backward(np_, x, None, None, None, g, None, out_q=dx)
    assert torch.equal(y, y0) and torch.equal(dx, d0) and torch.equal(w, w0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_calls_back_to_back_equal_calls_one_by_one(dtype):
    """Norm, attention and gradients in one stream without a pause, over shared buffers that the next call and torch
    overwrite, give the bits of the same calls with the device drained between them."""
    dt, code = DT[dtype]
    runs = [_params(dtype, H=4, Hkv=2, Nq=n, Nk=600, d=d, left=left, right=0, sinks=2, q_first=600 - n)
            for n, d, left in ((1, 128, 500), (300, 64, 40), (1, 64, 20), (600, 128, 200), (16, 128, 599))]

    def calls(pause):
        out = []

        def step(*tensors):
            if pause:
                torch.cuda.synchronize()
            out.extend(t.clone() for t in tensors)
            if pause:
                torch.cuda.synchronize()

        for p in runs:
            Q, K, V, G = _inputs(p, dtype, 3)
            ws = capi.alloc_window_workspace(p)
            n = capi.QkNormParams(B=1, H=4, Hkv=4, N=p.Nq, d=p.d, d_t=p.d // 2, d_h=p.d // 4, d_w=p.d // 4, Hg=4, Wg=5,
                                  first=0, eps=1e-6, base=10000.0, dtype=code)
            nws, O, Y = capi.alloc_qk_norm_workspace(n), torch.empty_like(Q), torch.empty_like(Q)
            for k in range(6):
                capi.qk_norm_rope3d(n, Q, None, out_q=Y)
                step()
                _, lse = capi.window_attention(p, Y, K, V, ws=ws, out=O, lse=True)
                step(O, lse)
                grads = capi.window_attention_backward(p, Y, K, V, O, G, lse, ws=ws)
                step(*grads)
                dx, _, dw, _ = capi.qk_norm_rope3d_backward(n, Q, None, None, None, grads[0], None, ws=nws, out_q=grads[0])
                step(dx, dw)
                Q.mul_(1.01 if k % 2 else 0.97)   # right behind the last reader
                K.copy_(K.flip(2))
        torch.cuda.synchronize()
        return out

    for x, y in zip(calls(False), calls(True)):
        assert torch.equal(x, y)


def test_two_streams_at_once():
    """Calls with workspaces of their own, enqueued on two streams without waiting between."""
    ps = [_params("bf16", H=4, Nq=900, d=128, left=300, sinks=4), _params("bf16", H=4, Nq=1, Nk=5000, d=128, left=-1, q_first=4999)]
    ins = [_inputs(p, "bf16", 51 + i) for i, p in enumerate(ps)]
    want = [capi.window_attention(p, *x[:3]) for p, x in zip(ps, ins)]
    ws = [capi.alloc_window_workspace(p) for p in ps]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[torch.empty_like(x[0]) for _ in range(20)] for x in ins]
    torch.cuda.synchronize()
    for r in range(20):
        for p, x, w, s, o in zip(ps, ins, ws, streams, outs):
            capi.window_attention(p, *x[:3], ws=w, out=o[r], stream=s)
    torch.cuda.synchronize()
    for o, y in zip(outs, want):
        assert all(torch.equal(t, y) for t in o)


def test_outputs_made_for_another_stream_wait_for_what_lay_there():
    """The output's memory was freed with a copy out of it still pending on the current stream."""
    p = _params("bf16", H=4, Nq=4096, d=128, left=100)
    Q, K, V, G = _inputs(p, "bf16", 57)
    want, lse = capi.window_attention(p, Q, K, V, lse=True)
    grads = capi.window_attention_backward(p, Q, K, V, want, G, lse)
    side = torch.cuda.Stream()
    for _ in range(3):
        old = [torch.full_like(x, 3.0) for x in (Q, Q, K, V)]
        kept = [torch.empty_like(x) for x in old]
        torch.cuda.synchronize()
        torch.cuda._sleep(10_000_000)
        for x, y in zip(kept, old):
            x.copy_(y)
        del old, x, y
        O, L = capi.window_attention(p, Q, K, V, lse=True, stream=side)
        got = capi.window_attention_backward(p, Q, K, V, O, G, L, stream=side)
        torch.cuda.synchronize()
        assert all((x == 3.0).all() for x in kept)
        assert torch.equal(O, want) and torch.equal(L, lse) and all(torch.equal(x, y) for x, y in zip(got, grads))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_entries_behind_the_first_of_a_longer_batch(dtype):
    """Entries 1 and 2 of a batch of three by slices of everything, positions, lengths and lse too (which then start
    4 bytes behind a multiple of 16), on the current stream and on another."""
    p = _params(dtype, B=3, H=3, Hkv=1, Nq=35, Nk=120, left=30, right=2, sinks=2)
    Q, K, V, G = _inputs(p, dtype, 61)
    first, lens = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([9, 60, 85], [44, 95, 120]))
    O, lse = capi.window_attention(p, Q, K, V, q_first=first, k_len=lens, lse=True)
    grads = capi.window_attention_backward(p, Q, K, V, O, G, lse, q_first=first, k_len=lens)
    rest = _params(dtype, B=2, H=3, Hkv=1, Nq=35, Nk=120, left=30, right=2, sinks=2)
    assert first[1:].data_ptr() % 16 == 4 and lse[1:].data_ptr() % 16 == 4
    n = capi.QkNormParams(B=3, H=3, Hkv=1, N=35, d=64, d_t=16, d_h=24, d_w=24, Hg=5, Wg=7, first=0, eps=1e-6, base=10000.0,
                          dtype=DT[dtype][1])
    n2 = capi.QkNormParams(B=2, H=3, Hkv=1, N=35, d=64, d_t=16, d_h=24, d_w=24, Hg=5, Wg=7, first=0, eps=1e-6, base=10000.0,
                           dtype=DT[dtype][1])
    w = 1 + 0.2 * _randn((65,), torch.float32, 62)
    Y, _ = capi.qk_norm_rope3d(n, Q, None, w[1:].clone(), first=first)
    dY, _, dw, _ = capi.qk_norm_rope3d_backward(n2, Q[1:], None, w[1:].clone(), None, G[1:], None, first=first[1:].clone())
    torch.cuda.synchronize()
    for stream in (None, torch.cuda.Stream()):
        at = {"q_first": first[1:], "k_len": lens[1:], "stream": stream}
        O2, lse2 = capi.window_attention(rest, Q[1:], K[1:], V[1:], lse=True, **at)
        got = capi.window_attention_backward(rest, Q[1:], K[1:], V[1:], O[1:], G[1:], lse[1:], **at)
        Y2, _ = capi.qk_norm_rope3d(n2, Q[1:], None, w[1:], first=first[1:], stream=stream)
        dY2, _, dw2, _ = capi.qk_norm_rope3d_backward(n2, Q[1:], None, w[1:], None, G[1:], None, first=first[1:], stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(Y2, Y[1:]) and torch.equal(dY2, dY) and torch.equal(dw2, dw)
        vis = visible(rest, [60, 85], [95, 120])
        ref = attention(Q[1:], K[1:], V[1:], vis, G[1:])
        check("O", O2, *ref["O"])
        check("lse", lse2, *ref["lse"])
        for name, x in zip(("dQ", "dK", "dV"), got):
            check(name, x, *ref[name])
        assert torch.equal(got[0], grads[0][1:])


# ------------------------------------------------------------------------------ norm + RoPE
def _norm_params(dtype, B=1, H=2, Hkv=None, N=50, split=(16, 24, 24), Hg=5, Wg=7, first=0, eps=1e-6, base=10000.0):
    return capi.QkNormParams(B=B, H=H, Hkv=Hkv or H, N=N, d=sum(split), d_t=split[0], d_h=split[1], d_w=split[2],
                             Hg=Hg, Wg=Wg, first=first, eps=eps, base=base, dtype=DT[dtype][1])


NORMS = [
    dict(N=1), dict(N=1, H=24, first=123456, Hg=45, Wg=80, split=(16, 56, 56)), dict(N=31), dict(N=33, H=5, Hkv=1),
    dict(B=3, N=257, H=7, Hkv=3, split=(44, 42, 42)), dict(N=1000, H=1, split=(128, 0, 0), Hg=1, Wg=1, first=1 << 20),
    dict(N=77, split=(0, 64, 0), Hg=40, Wg=1), dict(N=64, split=(0, 0, 128), Hg=1, Wg=1000, base=500.0),
    dict(N=130, split=(22, 20, 22), eps=0.0), dict(N=2000, H=48, Hkv=48, Hg=30, Wg=45),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", NORMS, ids=lambda s: "-".join(f"{k}{v}" for k, v in s.items()).replace(" ", ""))
def test_qk_norm_rope3d_and_gradients(shape, dtype):
    p = _norm_params(dtype, **shape)
    dt = DT[dtype][0]
    first = [p.first + 13 * b for b in range(p.B)]
    cs, sn = angles(p, first)
    at = torch.tensor(first, dtype=torch.int32, device="cuda") if p.B > 1 else None
    Q, K = _randn((p.B, p.H, p.N, p.d), dt, 1, 1.7), _randn((p.B, p.Hkv, p.N, p.d), dt, 2, 0.3)
    Gq, Gk = _randn(Q.shape, dt, 3), _randn(K.shape, dt, 4)
    wq, wk = 1 + 0.3 * _randn((p.d,), torch.float32, 5), 1 + 0.3 * _randn((p.d,), torch.float32, 6)
    Yq, Yk = capi.qk_norm_rope3d(p, Q, K, wq, wk, first=at)
    dQ, dK, dwq, dwk = capi.qk_norm_rope3d_backward(p, Q, K, wq, wk, Gq, Gk, first=at)
    torch.cuda.synchronize()
    for X, w, G, Y, dX, dw in ((Q, wq, Gq, Yq, dQ, dwq), (K, wk, Gk, Yk, dK, dwk)):
        ref = norm(X, w, cs, sn, p.eps, G)
        check("Y", Y, *ref["Y"])
        check("dX", dX, *ref["dX"])
        check("dw", dw, *ref["dw"])
    # queries only, no weights, in place
    Qi = Q.clone()
    Y1, none = capi.qk_norm_rope3d(p, Qi, None, first=at, out_q=Qi)
    assert none is None
    check("Y", Y1, *norm(Q, None, cs, sn, p.eps)["Y"])
    Gi = Gq.clone()
    d1, _, w1, _ = capi.qk_norm_rope3d_backward(p, Q, None, None, None, Gi, None, first=at, out_q=Gi)
    ref = norm(Q, None, cs, sn, p.eps, Gq)
    check("dX", d1, *ref["dX"])
    check("dw", w1, *ref["dw"])


@pytest.mark.parametrize("base", [10000.0, 100.0, 1.5, 0.5])
def test_qk_norm_rope3d_angles_of_the_farthest_positions(base):
    """Pairs (1, 0) turned by the angles of positions 2^30 and on, against angles of 40 digits.
    The frequency and its product with the position are each half a step of binary64 off, 2^-53 of at most 1.98 x 2^30
    radians (base 0.5, the last pair): 8 x 2^-24 in all, and 1 for the frequency's own arithmetic.  The rest is reduced to a turn, so its rounding to binary32
    is at most pi 2^-25, and cos and sin are within 2 units of 2^-24: 13 x 2^-24.  The mean of 128 squares of 0 and 1 is
    exact; eps, the root, and three products or sums take 5 steps of y = 2^(1/2) cos or sin."""
    import decimal
    D = decimal.Decimal
    p = _norm_params("f32", B=1, H=1, N=8, split=(128, 0, 0), Hg=1, Wg=1, first=1 << 30, base=base)
    Q = torch.zeros((1, 1, 8, 128), device="cuda")
    Q[..., 0::2] = 1
    Y, _ = capi.qk_norm_rope3d(p, Q, None)
    pi = D("3.1415926535897932384626433832795028841971693993751")
    want = torch.empty((8, 128), dtype=torch.float64)
    with decimal.localcontext() as c:
        c.prec = 40
        for i in range(64):
            f = (D(base).ln() * -2 * i / 128).exp()
            for n in range(8):
                a = float((((1 << 30) + n) * f) % (2 * pi))
                want[n, 2 * i], want[n, 2 * i + 1] = math.cos(a), math.sin(a)
    want *= 1 / math.sqrt(0.5 + 1e-6)
    assert (Y[0, 0].double().cpu() - want).abs().max() <= 18 * 2.0 ** -24 * math.sqrt(2)


def test_qk_norm_rope3d_rows_of_zeros():
    p = _norm_params("f32", N=9)
    Q = torch.zeros((1, 2, 9, 64), device="cuda")
    G = torch.ones_like(Q)
    Y, _ = capi.qk_norm_rope3d(p, Q, None)
    dQ, _, dw, _ = capi.qk_norm_rope3d_backward(p, Q, None, None, None, G, None)
    cs, sn = angles(p, [0])
    ref = norm(Q, None, cs, sn, p.eps, G)
    assert (Y == 0).all() and (dw == 0).all()
    check("dX", dQ, *ref["dX"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_qk_norm_rope3d_strided(dtype):
    """From slices of a [B, N, 3, H, d] projection to dense [B, H, N, d], and back into the
    slices of its gradient."""
    p = _norm_params(dtype, B=2, H=3, N=91, split=(44, 42, 42))
    dt = DT[dtype][0]
    qkv = _randn((2, 91, 3, 3, 128), dt, 7)
    Q, K = qkv[:, :, 0].transpose(1, 2), qkv[:, :, 1].transpose(1, 2)
    Yq, Yk = capi.qk_norm_rope3d(p, Q, K)
    Dq, Dk = capi.qk_norm_rope3d(p, Q.contiguous(), K.contiguous())
    assert torch.equal(Yq, Dq) and torch.equal(Yk, Dk) and Yq.is_contiguous()
    G = _randn(Yq.shape, dt, 8)
    grad = torch.zeros_like(qkv)
    out_q, out_k = grad[:, :, 0].transpose(1, 2), grad[:, :, 1].transpose(1, 2)
    capi.qk_norm_rope3d_backward(p, Q, K, None, None, G, G, out_q=out_q, out_k=out_k)
    dQ, dK, _, _ = capi.qk_norm_rope3d_backward(p, Q.contiguous(), K.contiguous(), None, None, G, G)
    assert torch.equal(out_q, dQ) and torch.equal(out_k, dK) and (grad[:, :, 2] == 0).all()


def test_qk_norm_rope3d_gradients_against_differences():
    p = _norm_params("f32", N=40, first=17)
    Q, G = _randn((1, 2, 40, 64), torch.float32, 9), _randn((1, 2, 40, 64), torch.float32, 10)
    w = 1 + 0.2 * _randn((64,), torch.float32, 11)
    cs, sn = angles(p, [17])
    dQ, _, dw, _ = capi.qk_norm_rope3d_backward(p, Q, None, w, None, G, None)
    f = lambda x, v: (norm(x, v, cs, sn, p.eps)["Y"][0] * G.double()).sum().item()  # noqa: E731
    x, v, h = Q.double(), w.double(), 1e-5
    e, ew = _randn(Q.shape, torch.float32, 12).double(), _randn((64,), torch.float32, 13).double()
    num = (f(x + h * e, v) - f(x - h * e, v)) / (2 * h)
    assert abs(num - (dQ.double() * e).sum().item()) <= 1e-5 * (dQ.double() * e).abs().sum().item()
    num = (f(x, v + h * ew) - f(x, v - h * ew)) / (2 * h)
    assert abs(num - (dw.double() * ew).sum().item()) <= 1e-5 * (dw.double() * ew).abs().sum().item()


# ------------------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_rope_window_attention_train_step(dtype):
    """One layer as a model runs it: projection slices -> norm + RoPE -> window attention, and
    the whole way back, against the chain of the binary64 forms' gradients (by autograd)."""
    B, T, Hg, Wg, H, d = 2, 4, 5, 9, 3, 64
    N = T * Hg * Wg
    np_ = _norm_params(dtype, B=B, H=H, N=N, Hg=Hg, Wg=Wg)
    wp = _params(dtype, B=B, H=H, Nq=N, d=d, frame=Hg * Wg, left=1, right=0, sinks=1)
    dt = DT[dtype][0]
    qkv = _randn((B, N, 3, H, d), dt, 21)
    wq, wk = 1 + 0.2 * _randn((d,), torch.float32, 22), 1 + 0.2 * _randn((d,), torch.float32, 23)
    G = _randn((B, H, N, d), dt, 24)
    Q, K, V = (qkv[:, :, i].transpose(1, 2) for i in range(3))
    Yq, Yk = capi.qk_norm_rope3d(np_, Q, K, wq, wk)
    O, lse = capi.window_attention(wp, Yq, Yk, V, lse=True)
    grad = torch.empty_like(qkv)
    gq, gk, gv = (grad[:, :, i].transpose(1, 2) for i in range(3))
    dYq, dYk = torch.empty_like(Yq), torch.empty_like(Yk)
    capi.window_attention_backward(wp, Yq, Yk, V, O, G, lse, out=(dYq, dYk, gv))
    _, _, dwq, dwk = capi.qk_norm_rope3d_backward(np_, Q, K, wq, wk, dYq, dYk, out_q=gq, out_k=gk)
    torch.cuda.synchronize()

    x = qkv.double().requires_grad_()
    a, b = wq.double().requires_grad_(), wk.double().requires_grad_()
    cs, sn = angles(np_, [0] * B)
    q, k, v = (x[:, :, i].transpose(1, 2) for i in range(3))
    yq, yk = norm(q, a, cs, sn, np_.eps)["Y"][0], norm(k, b, cs, sn, np_.eps)["Y"][0]
    vis = visible(wp, [0] * B, [N] * B).cuda()[:, None]
    s = (yq @ yk.mT / math.sqrt(d)).masked_fill(~vis, -math.inf)
    o = torch.softmax(s, -1) @ v
    (o * G.double()).sum().backward()
    # each stage rounds to the type once (the gradients twice more on the way): relative
    # 2-norm error of a few half steps
    tol = 6 * 2.0 ** -8 if dtype == "bf16" else 2e-5
    for n, got, want in (("O", O, o), ("dqkv", grad, x.grad), ("dwq", dwq, a.grad), ("dwk", dwk, b.grad)):
        rel = ((got.double() - want).norm() / want.norm()).item()
        assert rel <= tol, (n, rel)
