"""The gated feed-forward block and its gradients on the GPU against the formulas in 64 bits, every value within what
the roundings can do to it (experts_ref.ffn)."""
import numpy as np
import pytest
import torch

import experts_ref as ref
from quantized_routed_expert_softmax_gb300 import native

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_routed_expert_softmax_gb300 import build
    build.build()
    native.lib()


def _inputs(P, E, d, f, act, seed, weight=None):
    g = torch.Generator("cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    w = weight or 1.0 / d ** 0.5
    bf = torch.bfloat16
    nz = 2 * f if act == "swiglu" else f
    return (rand(P, d).to(bf), (w * rand(E, nz, d)).to(bf), (rand(E, d, f) / f ** 0.5).to(bf), (0.1 * rand(P, d)).to(bf))


def _offsets(counts, before=0):
    return torch.tensor(np.concatenate([[before], before + np.cumsum(counts)]), dtype=torch.int32, device="cuda")


def _close(name, got, want):
    v, b = want
    err = (got.double() - v).abs()
    assert torch.isfinite(got).all(), name
    assert (err <= b).all(), (name, (err - b).max().item(), err.max().item())


def _run(P, E, d, f, counts, act="swiglu", seed=0, before=0, weight=None, dtype=None):
    x, wgu, wd, dy = _inputs(P, E, d, f, act, seed, weight)
    off = None if counts is None else _offsets(counts, before)
    want = ref.ffn(x, wgu, wd, off, act, dy)
    ws = native.ffn_workspace(P, f, act, backward=True)
    y0 = native.ffn_forward(x, wgu, wd, off, act=act, workspace=ws, out=torch.zeros_like(x))
    y, (z, h) = native.ffn_forward(x, wgu, wd, off, act=act, save=True, out=torch.zeros_like(x), workspace=ws)
    mine = torch.zeros(P, dtype=torch.bool, device="cuda")
    for _, a, b in ref.spans(off, P, E):
        mine[a:b] = True
    for name, t in (("y", y), ("y", y0), ("z", z), ("h", h)):
        _close(name, torch.where(mine[:, None], t, 0), want[name])
    assert torch.equal(y, y0)
    dx, dgu, dd = native.ffn_backward(dy, x, wgu, wd, (z, h), off, act=act, workspace=ws, dtype=dtype)
    _close("dx", torch.where(mine[:, None], dx, 0), want["dx"])
    _close("dwgu", dgu, want["dwgu"])
    _close("dwd", dd, want["dwd"])
    assert native.device_status(ws) == 0
    return (x, wgu, wd, dy, off, ws), (y, z, h, dx, dgu, dd)


@pytest.mark.parametrize("act", ["swiglu", "relu2"])
@pytest.mark.parametrize("counts,d,f", [
    ([1], 16, 16), ([1], 64, 48), ([2, 0, 1], 48, 16), ([5, 7], 256, 144), ([63, 64, 65, 0, 1], 128, 80),
    ([128, 127, 129], 208, 256), ([31, 33, 300], 96, 400), ([513, 0, 255], 320, 208), ([1] * 30, 64, 64), ([257, 31], 528, 272)])
def test_block_and_gradients(counts, d, f, act):
    _run(sum(counts), len(counts), d, f, counts, act, seed=d + f)


@pytest.mark.parametrize("P", [1, 2, 5, 8, 9, 16, 17, 33, 64, 65, 200, 1000])
def test_dense_block(P):
    _run(P, 1, 176, 336, None, seed=P)


@pytest.mark.parametrize("P,d,f", [(2600, 272, 1040), (1500, 1040, 272), (700, 528, 528), (300, 1040, 1552), (4100, 1296, 640)])
def test_dense_block_in_tiles_of_every_height(P, d, f):
    _run(P, 1, d, f, None, seed=P, act="swiglu" if P % 200 else "relu2")


@pytest.mark.parametrize("counts", [[int(n) for n in np.random.default_rng(3).integers(0, 600, 48)], [3000] + [1] * 20 + [0, 900],
                                    [255, 256, 257, 512, 513, 511, 128, 129] * 6])
def test_many_row_tiles_an_expert(counts):
    _run(sum(counts), len(counts), 272, 144, counts, seed=len(counts))


def test_layer_shapes():
    _run(70, 4, 2816, 704, [9, 0, 60, 1], seed=1)
    _run(40, 3, 1024, 2688, [13, 1, 26], act="relu2", seed=2)


def test_many_experts():
    g = np.random.default_rng(3)
    counts = g.integers(0, 9, 1024) * (g.random(1024) < 0.3)
    _run(int(counts.sum()), 1024, 32, 16, counts, seed=3)


def test_gradients_in_fp32():
    # the same operands, unrounded: within the bound less one rounding
    (x, wgu, wd, dy, off, ws), (y, z, h, dx, dgu, dd) = _run(150, 3, 128, 96, [70, 0, 80], seed=4)
    _, g32, d32 = native.ffn_backward(dy, x, wgu, wd, (z, h), off, workspace=ws, dtype=torch.float32)
    assert g32.dtype == torch.float32 and torch.equal(g32.bfloat16(), dgu) and torch.equal(d32.bfloat16(), dd)
    for need in ((True, False, False), (False, True, False), (False, False, True), (False, False, False)):
        got = native.ffn_backward(dy, x, wgu, wd, (z, h), off, workspace=ws, need=need)
        for n, g, w in zip(need, got, (dx, dgu, dd)):
            assert (torch.equal(g, w) if n else g is None)


def test_large_gates():
    # gates of some hundreds: the sigmoid is 0 or 1, nothing overflows
    _run(90, 2, 64, 48, [40, 50], seed=5, weight=30.0)


def test_rows_no_expert_owns_and_bad_neighbours():
    """NaN and infinities in rows of another expert, or of none, reach no row and no gradient but their own."""
    P, d, f = 300, 128, 96
    counts, before = [70, 30, 0, 90], 11
    x, wgu, wd, dy = _inputs(P, 4, d, f, "swiglu", 6)
    off = _offsets(counts, before)
    clean = ref.ffn(x, wgu, wd, off, "swiglu", dy)
    bad = torch.zeros(P, dtype=torch.bool, device="cuda")
    bad[:11] = bad[81:111] = bad[201:] = True                  # before, the second expert's, behind
    xb, dyb = x.clone(), dy.clone()
    xb[bad], dyb[bad] = float("nan"), float("inf")
    ws = native.ffn_workspace(P, f, backward=True)
    out = torch.full((P, d), 7.0, dtype=torch.bfloat16, device="cuda")
    y, saved = native.ffn_forward(xb, wgu, wd, off, save=True, out=out, workspace=ws)
    for t in saved:                                            # what is behind them in memory may be anything
        t[:11], t[201:] = float("nan"), float("nan")
    dx, dgu, dd = native.ffn_backward(dyb, xb, wgu, wd, saved, off, workspace=ws)
    ok = ~bad
    for name, got in (("y", y), ("dx", dx)):
        _close(name, got[ok], tuple(t[ok] for t in clean[name]))
    assert (y[:11] == 7).all() and (y[201:] == 7).all() and torch.isnan(y[81:111]).all()
    for e in (0, 2, 3):
        _close("dwgu", dgu[e], tuple(t[e] for t in clean["dwgu"]))
        _close("dwd", dd[e], tuple(t[e] for t in clean["dwd"]))
    assert (dgu[2] == 0).all() and torch.isnan(dgu[1]).all()


def test_empty_batch():
    x, wgu, wd, dy = _inputs(0, 2, 64, 32, "swiglu", 7)
    off = _offsets([0, 0])
    y, saved = native.ffn_forward(x, wgu, wd, off, save=True)
    dx, dgu, dd = native.ffn_backward(dy, x, wgu, wd, saved, off, dtype=torch.float32)
    assert y.shape == dx.shape == (0, 64) and (dgu == 0).all() and (dd == 0).all()


def test_absurd_offsets_stay_in_the_buffers():
    P, E, d, f = 60, 4, 64, 48
    x, wgu, wd, dy = _inputs(P, E, d, f, "swiglu", 8)
    pad = torch.full((P + 64, d), 2.5, dtype=torch.bfloat16, device="cuda")
    for off in ([0, 2 ** 31 - 1, -5, 7, 3], [-2 ** 31, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, 0], [60, 55, 50, 70, 99]):
        o = torch.tensor(off, dtype=torch.int32, device="cuda")
        ws = native.ffn_workspace(P, f, backward=True)
        _, saved = native.ffn_forward(x, wgu, wd, o, save=True, out=pad[32 : 32 + P], workspace=ws)
        native.ffn_backward(dy, x, wgu, wd, saved, o, workspace=ws)
        assert native.device_status(ws) == 0
        assert (pad[:32] == 2.5).all() and (pad[32 + P :] == 2.5).all()


def test_same_bits_on_another_stream_and_in_a_graph():
    (x, wgu, wd, dy, off, ws), first = _run(500, 3, 192, 144, [260, 40, 200], seed=9)

    def step(w):
        y, saved = native.ffn_forward(x, wgu, wd, off, save=True, workspace=w)
        return (y, *saved, *native.ffn_backward(dy, x, wgu, wd, saved, off, workspace=w))

    s = torch.cuda.Stream()
    ws2 = native.ffn_workspace(500, 144, backward=True)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        other = step(ws2)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(ws)
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, got))
    assert native.device_status(ws) == 0


def test_a_training_step_of_routed_experts():
    """The parts as a routed layer's training step uses them: router, rows side by side, block, weighted sum, and
    back; the gradients against differences of the loss in 64 bits."""
    T, d, f, E, k = 50, 256, 64, 8, 2
    g = torch.Generator("cuda").manual_seed(10)
    bf = torch.bfloat16
    x = torch.randn(T, d, generator=g, device="cuda").to(bf)
    W = torch.randn(d, E, generator=g, device="cuda") * 0.05
    wgu = (torch.randn(E, 2 * f, d, generator=g, device="cuda") / 16).to(bf)
    wd = (torch.randn(E, d, f, generator=g, device="cuda") / 8).to(bf)
    target = torch.randn(T, d, generator=g, device="cuda")
    idx, w = native.router_topk(x, W, k)
    order = torch.argsort(idx.view(-1), stable=True)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = torch.bincount(idx.view(-1), minlength=E).cumsum(0)
    tok, pw = order // k, w.view(-1)[order]
    y, saved = native.ffn_forward(x[tok], wgu, wd, off, save=True)
    out = torch.zeros(T, d, device="cuda").index_add_(0, tok, y.float() * pw[:, None])
    dy = ((out - target)[tok] * pw[:, None]).to(bf)
    dx, dgu, dd = native.ffn_backward(dy, x[tok], wgu, wd, saved, off, dtype=torch.float32)
    dxt = torch.zeros(T, d, device="cuda").index_add_(0, tok, dx.float())

    def loss(x_, gu_, d_):
        yy = ref.ffn(x_[tok], gu_, d_, off)["y"][0]
        o = torch.zeros(T, d, dtype=torch.float64, device="cuda").index_add_(0, tok, yy * pw[:, None].double())
        return 0.5 * ((o - target.double()) ** 2).sum()

    for name, arg, grad in (("x", 0, dxt), ("w_gate_up", 1, dgu), ("w_down", 2, dd)):
        args = [x.double(), wgu.double(), wd.double()]
        v = torch.randn(args[arg].shape, generator=g, device="cuda", dtype=torch.float64)
        step = 1e-5
        args[arg] = args[arg] + step * v
        up = loss(*args)
        args[arg] = args[arg] - 2 * step * v
        diff = (up - loss(*args)) / (2 * step)
        # along v the gradient's roundings (three of bf16 at most in a row, of independent signs) add up like a
        # random walk: 12 times its size for an error of 3 U of every entry
        tol = 12 * 3 * ref.U * (grad.double() * v).norm()
        assert abs((grad.double() * v).sum() - diff) <= tol, (name, diff.item())
