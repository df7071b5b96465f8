"""The routed layer over per-channel int8 experts with int8 inputs (act_quant "int8"): routing and permutation as in every
format, h and the outputs against 64 bits on the same codes."""
import numpy as np
import pytest
import torch

import experts_ref as ref
from quantized_routed_expert_softmax_gb300 import layers, native, synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_routed_expert_softmax_gb300 import build
    build.build()
    native.lib()


W = {
    "swiglu": synth.Workload("i8_swiglu", d=512, f=96, E=16, k=3, act="swiglu", wfmt="int8pc", x_dtype="bf16", layers=1),
    "relu2": synth.Workload("i8_relu2", d=256, f=160, E=12, k=4, act="relu2", wfmt="int8pc", x_dtype="f32", layers=1),
    "deep": synth.Workload("i8_deep", d=1280, f=32, E=4, k=2, act="swiglu", wfmt="int8pc", x_dtype="bf16", layers=1),
}


def _layer(w):
    return layers.build_layer(w, source="numpy", act_quant="int8")


def _x(w, T):
    x = torch.from_numpy(synth.tokens(w, T, tag="i8")).cuda()
    return x.view(torch.bfloat16) if w.x_dtype == "bf16" else x


def _codes(a):
    q, s = ref.quantize(np.ascontiguousarray(a, dtype=np.float32))
    return q.astype(np.float64), s.astype(np.float64)


def _products(rows, mats, e):
    """z[r] = row r's product with matrix e[r]: the codes' sums, which fp64 holds exactly (0 where they cancel), scaled."""
    (qx, sx), out = rows, []
    for r, i in enumerate(e):
        qw, sw = mats[i]
        out.append((qw @ qx[r]) * sw * sx[r])
    return np.stack(out)


def _check_layer(w, x, out, tr):
    """h from the 64-bit product on the codes of x, and out from the codes of the h that the layer had.  The sums of codes
    are exact here (at most 1280 columns of random codes), so that z is off by the three roundings of its scaling; the combine adds k
    weighted terms in fp32, (k + 1) roundings of 2^-24 of sum w |y|.

    SiLU is g e / (1 + e) or g / (1 + e) with e = exp(-|g|) <= 1.  In steps of 2^-23, relative: e is off by 2 (expf), g e by
    half a step more, 1 + e by e / (1 + e) of e's 2, at most 1, and half, the division by 2: 6 together, 12 * 2^-24; the
    product with u is rounded once more."""
    T, P = x.shape[0], x.shape[0] * w.k
    idx, perm, pos = (tr[n].cpu().numpy() for n in ("idx", "perm", "pos"))
    wts = tr["w"].cpu().numpy().astype(np.float64)
    e = idx.reshape(-1)[perm]
    assert (np.diff(e) >= 0).all() and np.array_equal(pos[perm], np.arange(P))
    xq = tuple(a[perm // w.k] for a in _codes(x.float().cpu().numpy()))
    gu = [_codes(synth.expert_weights(w, 0, i)[0]) for i in range(w.E)]
    dn = [_codes(synth.expert_weights(w, 0, i)[1]) for i in range(w.E)]
    z = _products(xq, gu, e)
    ez = 3 * 2.0 ** -24 * np.abs(z)
    h = tr["h"].cpu().numpy()
    want = ref.activate(torch.from_numpy(z), w.act).numpy()
    if w.act == "swiglu":
        f = w.f
        g, u, eg, eu = z[:, :f], z[:, f:], ez[:, :f], ez[:, f:]
        err = 1.1 * eg * (np.abs(u) + eu) + np.abs(g) * eu + 13 * 2.0 ** -24 * np.abs(want)
    else:
        r = np.maximum(z, 0)
        err = 2 * r * ez + ez * ez + 2.0 ** -24 * r * r
    assert (np.abs(h - want) <= err + 1e-40).all()
    y = _products(_codes(h), dn, e)
    o, bound = np.zeros((T, w.d)), np.zeros((T, w.d))
    for t in range(T):
        for j in range(w.k):
            yy = y[pos[t * w.k + j]]
            o[t] += wts[t, j] * yy
            bound[t] += wts[t, j] * np.abs(yy) * (w.k + 1 + 3) * 2.0 ** -24
    assert (np.abs(out.cpu().numpy() - o) <= bound + 1e-40).all()


@pytest.mark.parametrize("T", [1, 2, 7, 33, 150, 700])
@pytest.mark.parametrize("name", list(W))
def test_layer(name, T):
    w = W[name]
    L, x, tr = _layer(w), _x(w, T), {}
    out = L.forward(x, trace=tr)
    assert L.device_status() == 0
    _check_layer(w, x, out, tr)
    # the same routing as without coded inputs
    plain = layers.build_layer(w, source="numpy")
    tp = {}
    plain.forward(x, trace=tp)
    assert torch.equal(tp["idx"], tr["idx"]) and torch.equal(tp["w"], tr["w"])
    # supplied routing: the same bits
    again = L.forward(x, idx_in=tr["idx"].clone(), w_in=tr["w"].clone())
    assert torch.equal(again, out)


def test_layer_is_its_operators():
    w = W["swiglu"]
    L, T = _layer(w), 40
    x, tr = _x(w, T), {}
    L.forward(x, trace=tr)
    rows = tr["perm"] // w.k
    q = native.quantize_int8(x, rows=rows.int())
    h = native.int8_matmul(q[0], L.gate_up, tr["offsets"], T * w.k, 2 * w.f, w.d, act="swiglu")
    assert torch.equal(h, tr["h"])


def test_layer_noalloc_stack_and_graph():
    w = W["swiglu"]
    L, x = _layer(w), _x(w, 5)
    out = L.forward(x)
    assert torch.equal(L.forward_noalloc(x), out) and L.noalloc_status() == 0
    one = L.forward(x[:1])
    st = native.MoEStack([L, L])
    outs = st.forward(x[:1])
    assert torch.equal(outs[:1], one) and torch.equal(outs[1:], L.forward(native.rmsnorm_bf16(one)))
    assert st.launches() == 2 * L.launches(1) + 1
    ws = torch.zeros(L.workspace_bytes(5), dtype=torch.uint8, device="cuda")
    again = torch.empty_like(out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.forward(x, out=again, workspace=ws)
    for _ in range(2):
        x.copy_(x.flip(0))
        again.zero_()
        g.replay()
        assert torch.equal(again, L.forward(x))


def test_layer_of_trained_experts():
    """Experts as the feed-forward block trains them (bf16), coded per channel: the layer's output is near the block's."""
    w = synth.Workload("i8_trained", d=512, f=128, E=8, k=2, act="swiglu", wfmt="int8pc", x_dtype="bf16", layers=1)
    g = torch.Generator("cuda").manual_seed(1)
    bf = torch.bfloat16
    wgu = (torch.randn(w.E, 2 * w.f, w.d, generator=g, device="cuda") / 22).to(bf)
    wd = (torch.randn(w.E, w.d, w.f, generator=g, device="cuda") / 11).to(bf)
    router = torch.randn(w.d, w.E, generator=g, device="cuda") * 0.05
    L = native.MoELayer(w.d, w.f, w.E, w.k, "swiglu", "int8pc", router, native.quantize_int8pc(wgu.float()), native.quantize_int8pc(wd.float()),
                        act_quant="int8")
    T = 64
    x, tr = torch.randn(T, w.d, generator=g, device="cuda").to(bf), {}
    out = L.forward(x, trace=tr)
    tok = (tr["perm"] // w.k).long()
    y = native.ffn_forward(x[tok], wgu, wd, tr["offsets"]).float()
    want = (y[tr["pos"].long()].view(T, w.k, w.d) * tr["w"].unsqueeze(-1)).sum(1)
    # codes of 127 steps at the row's largest: each of the four codings is off by amax / 254, uniformly, about
    # 3.2 / 254 / sqrt(3) = 0.8 % of rms for rows of some hundred normal values; together 1.5 %, three times that allowed
    assert (out - want).norm() <= 0.045 * want.norm()


def test_layer_refusals():
    w = W["swiglu"]
    L, x = _layer(w), _x(w, 4)
    for path in ("gemv", "gemm"):
        L.set_path(path)
        with pytest.raises(native.MoeError) as e:
            L.forward(x)
        assert e.value.status in (1, 5)
    q8 = synth.Workload("i8_q8", d=512, f=96, E=16, k=3, act="swiglu", wfmt="q8_0", x_dtype="bf16", layers=1)
    with pytest.raises(native.MoeError):
        layers.build_layer(q8, source="numpy", act_quant="int8").forward(_x(q8, 2))
