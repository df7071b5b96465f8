"""The routed layer over MXFP4 experts: routing and permutation as in every format, the coded inputs bit
for bit, h and the outputs against 64 bits on the same codes."""
import numpy as np
import pytest
import torch

import mxfp4_ref as ref
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
    "swiglu": synth.Workload("mx_swiglu", d=512, f=96, E=16, k=3, act="swiglu", wfmt="mxfp4", x_dtype="bf16", layers=1),
    "relu2": synth.Workload("mx_relu2", d=256, f=160, E=12, k=4, act="relu2", wfmt="mxfp4", x_dtype="f32", layers=1),
}


def _x(w, T):
    x = torch.from_numpy(synth.tokens(w, T, tag="mx")).cuda()
    return x.view(torch.bfloat16) if w.x_dtype == "bf16" else x


def _check_layer(w, L, x, out, tr):
    """h from the 64-bit product on the codes of x, and out from the codes of the h that the layer had.

    A sum of K / 64 partial sums loses at most 2^-23 of A = sum |x w| an addition; see the product's
    tests.  The combine adds k weighted terms in fp32, (k + 1) roundings of 2^-24 of sum w |y|."""
    T, P = x.shape[0], x.shape[0] * w.k
    idx, perm, pos = (tr[n].cpu().numpy() for n in ("idx", "perm", "pos"))
    wts = tr["w"].cpu().numpy().astype(np.float64)
    e = idx.reshape(-1)[perm]
    assert (np.diff(e) >= 0).all() and np.array_equal(pos[perm], np.arange(P))
    values = lambda a: ref.values(*ref.quantize(np.ascontiguousarray(a, dtype=np.float32)))  # noqa: E731
    xv = values(x.float().cpu().numpy())[perm // w.k]
    gu = [values(synth.expert_weights(w, 0, i)[0]) for i in range(w.E)]
    dn = [values(synth.expert_weights(w, 0, i)[1]) for i in range(w.E)]
    z = np.stack([gu[i] @ xv[r] for r, i in enumerate(e)])
    ez = (w.d / 64 + 2) * 2.0 ** -23 * np.stack([np.abs(gu[i]) @ np.abs(xv[r]) for r, i in enumerate(e)])
    h = tr["h"].cpu().numpy()
    want = ref.activate(z, w.act)
    if w.act == "swiglu":
        f = w.f
        g, u, eg, eu = z[:, :f], z[:, f:], ez[:, :f], ez[:, f:]
        err = 1.1 * eg * (np.abs(u) + eu) + np.abs(g) * eu + 8 * 2.0 ** -24 * np.abs(want)
    else:
        r = np.maximum(z, 0)
        err = 2 * r * ez + ez * ez + 2.0 ** -24 * r * r
    assert (np.abs(h - want) <= err + 1e-40).all()
    hv = values(h)
    y = np.stack([dn[i] @ hv[r] for r, i in enumerate(e)])
    ey = (w.f / 64 + 2) * 2.0 ** -23 * np.stack([np.abs(dn[i]) @ np.abs(hv[r]) for r, i in enumerate(e)])
    yt, eyt = y[pos].reshape(T, w.k, w.d), ey[pos].reshape(T, w.k, w.d)
    full = (wts[..., None] * yt).sum(1)
    bound = (wts[..., None] * (eyt + (w.k + 1) * 2.0 ** -24 * np.abs(yt))).sum(1)
    assert (np.abs(out.cpu().numpy() - full) <= bound + 1e-40).all()


@pytest.mark.parametrize("name", list(W))
@pytest.mark.parametrize("T", [1, 2, 17, 40, 333])
def test_layer_parity(name, T):
    w = W[name]
    L = layers.build_layer(w, source="numpy")
    x = _x(w, T)
    tr = {}
    out = torch.full((T, w.d), float("nan"), device="cuda")
    L.forward(x, out=out, trace=tr)
    assert L.device_status() == 0
    idx, wt = native.router_topk(x, L.router_w, w.k)
    assert torch.equal(tr["idx"], idx)
    _check_layer(w, L, x, out, tr)
    assert torch.equal(L.forward(x), out)                     # the same bits again
    sup = L.forward(x, idx_in=tr["idx"], w_in=tr["w"])        # and with the routing supplied
    assert torch.equal(sup, out)
    assert L.launches(T) > 1


def test_layer_supplied_routing_repeats_and_bad_indices():
    w = W["swiglu"]
    L = layers.build_layer(w, source="numpy")
    T = 21
    x = _x(w, T)
    g = torch.Generator("cuda").manual_seed(2)
    idx = torch.randint(0, w.E, (T, w.k), device="cuda", generator=g, dtype=torch.int32)
    idx[3] = 5                                                # one expert in all of a token's slots
    idx[4:] = torch.where(idx[4:] < 8, idx[4:], idx[4:] - 8)  # experts without tokens but few
    wt = torch.rand(T, w.k, device="cuda", generator=g)
    tr = {}
    out = L.forward(x, idx_in=idx, w_in=wt, trace=tr)
    assert torch.equal(tr["idx"], idx)
    _check_layer(w, L, x, out, tr)
    idx[0, 0] = 1000                                          # clamped and recorded
    L.forward(x, idx_in=idx, w_in=wt)
    assert L.device_status() == 1 and L.device_status() == 0


def test_layer_noalloc_stack_and_graph():
    w = W["swiglu"]
    L = layers.build_layer(w, source="numpy")
    x = _x(w, 5)
    out = L.forward(x)
    assert torch.equal(L.forward_noalloc(x), out) and L.noalloc_status() == 0
    one = L.forward(x[:1])
    st = native.MoEStack([L, L])
    outs = st.forward(x[:1])
    assert torch.equal(outs[:1], one)
    assert torch.equal(outs[1:], L.forward(native.rmsnorm_bf16(one)))
    assert st.launches() == 2 * L.launches(1) + 1
    ws = torch.zeros(L.workspace_bytes(5), dtype=torch.uint8, device="cuda")
    again = torch.empty_like(out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.forward(x, out=again, workspace=ws)
    for k in range(2):
        x.copy_(x.flip(0))
        again.zero_()
        g.replay()
        assert torch.equal(again, L.forward(x))


def test_layer_refusals():
    w = W["swiglu"]
    L = layers.build_layer(w, source="numpy")
    x = _x(w, 4)
    for path in ("gemv", "gemm"):
        L.set_path(path)
        with pytest.raises(native.MoeError) as e:
            L.forward(x)
        assert e.value.status in (1, 5)
    L.set_path("auto")
    L.desc.act_quant = native.ACT_QUANT["q8_0"]
    with pytest.raises(native.MoeError):
        L.forward(x)


def test_full_size_layer_on_a_sample():
    """The Gemma layer shape at 512 tokens: sampled rows of h and of the output."""
    w = synth.Workload("mx_gemma", d=2816, f=704, E=128, k=8, act="swiglu", wfmt="mxfp4", x_dtype="bf16", layers=1)
    L = layers.build_layer(w, keep_fp32=True)
    T = 512
    x = synth.tokens_cuda(w, T, tag="mxfull")
    tr = {}
    out = L.forward(x, trace=tr)
    assert L.device_status() == 0
    perm, idx = tr["perm"].long(), tr["idx"].reshape(-1).long()
    dq = lambda a, r, c: native.dequantize_mxfp4(native.quantize_mxfp4(a)[0], r, c).double()  # noqa: E731
    xv = dq(x, T, w.d)
    hv = dq(tr["h"], T * w.k, w.f)
    y = {}
    for t in (0, 1, 255, 511):
        full = torch.zeros(w.d, dtype=torch.float64, device="cuda")
        bound = torch.zeros_like(full)
        for j in range(w.k):
            e, r = int(idx[t * w.k + j]), int(tr["pos"][t * w.k + j])
            gu = dq(L.gate_up_f32[e], 2 * w.f, w.d)
            z, A = gu @ xv[t], gu.abs() @ xv[t].abs()
            ez = (w.d / 64 + 2) * 2.0 ** -23 * A
            g, u = z[: w.f], z[w.f :]
            want = g * torch.sigmoid(g) * u
            err = 1.1 * ez[: w.f] * (u.abs() + ez[w.f :]) + g.abs() * ez[w.f :] + 8 * 2.0 ** -24 * want.abs()
            assert ((tr["h"][r].double() - want).abs() <= err).all()
            dn = dq(L.down_f32[e], w.d, w.f)
            y, ey = dn @ hv[r], (w.f / 64 + 2) * 2.0 ** -23 * (dn.abs() @ hv[r].abs())
            wt = float(tr["w"].reshape(-1)[t * w.k + j])
            full += wt * y
            bound += wt * (ey + (w.k + 1) * 2.0 ** -24 * y.abs())
        assert ((out[t].double() - full).abs() <= bound).all()
