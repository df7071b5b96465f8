"""The MXFP4 and balance-loss entry points on the host: sizes and refusals, before anything is
launched.  No test here touches a GPU."""
import os
import shutil

import numpy as np
import pytest
import torch

import mxfp4_ref as ref
from quantized_routed_expert_softmax_gb300 import native

FAKE = 0x10000   # an aligned address that is never dereferenced: validation fails first


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(native.LIB_PATH):
        if not shutil.which("nvcc") and not os.path.exists("/usr/local/cuda/bin/nvcc"):
            pytest.skip("libmoe.so not built and no nvcc to build it")
        from quantized_routed_expert_softmax_gb300 import build
        build.build()
    return native.lib()


def test_sizes(L):
    for rows, cols in [(1, 32), (3, 96), (128, 128), (1408, 2816), (45013, 704), (2816, 704)]:
        assert L.moe_mxfp4_bytes(rows, cols) == ref.bytes_of(rows, cols)
    for rows, cols in [(0, 32), (-1, 32), (1, 0), (1, 33), (1, 65568), ((1 << 25) + 1, 32)]:
        assert L.moe_mxfp4_bytes(rows, cols) == 0
    assert L.moe_mxfp4_matmul_workspace_bytes() == 256
    assert L.moe_balance_workspace_bytes(4, 100, 128) > 0
    assert L.moe_balance_workspace_bytes(1, 16, 8) == 0          # one CTA's work: no workspace
    assert L.moe_balance_workspace_bytes(4, 0, 128) == 0 and L.moe_balance_workspace_bytes(1, 1, 1025) == 0


def test_quantiser_refusals(L):
    Q = lambda x=FAKE, xt=0, xr=4, src=None, n=1, r=4, c=64, d=FAKE: L.moe_quantize_mxfp4(x, xt, xr, src, n, r, c, d, None)  # noqa: E731
    assert Q(x=None) == 1 and Q(d=None) == 1 and Q(xt=2) == 1 and Q(n=-1) == 1
    assert Q(src=FAKE, n=2) == 1 and Q(src=FAKE, xr=-1) == 1
    assert Q(c=48) == 2 and Q(c=0) == 2 and Q(r=-1) == 2 and Q(n=65536) == 2 and Q(c=65568) == 2
    assert Q(x=FAKE + 4) == 3 and Q(d=FAKE + 8) == 3 and Q(src=FAKE + 2) == 3
    assert Q(r=0) == 0 and Q(n=0) == 0          # nothing to do, nothing launched
    D = lambda s=FAKE, n=1, r=4, c=64, o=FAKE, ot=0: L.moe_dequantize_mxfp4(s, n, r, c, o, ot, None)  # noqa: E731
    assert D(s=None) == 1 and D(o=None) == 1 and D(ot=7) == 1 and D(c=33) == 2 and D(s=FAKE + 1) == 3
    assert D(r=0) == 0


def test_matmul_refusals(L):
    def M(x=FAKE, P=4, w=FAKE, E=8, N=64, K=64, off=FAKE, act=0, out=FAKE, ot=0, ws=FAKE, nb=256):
        return L.moe_mxfp4_matmul(x, P, w, E, N, K, off, act, out, ot, ws, nb, None)
    assert M(x=None) == 1 and M(w=None) == 1 and M(out=None) == 1 and M(act=3) == 1 and M(ot=2) == 1
    assert M(off=None) == 1 and M(E=0) == 1     # offsets may be missing for one matrix only
    assert M(K=48) == 2 and M(P=-1) == 2 and M(N=0) == 2 and M(N=96) == 2 and M(E=1025) == 2
    assert M(P=(1 << 25) + 1) == 2 and M(N=131136) == 2
    assert M(x=FAKE + 8) == 3 and M(off=FAKE + 2) == 3 and M(out=FAKE + 4) == 3 and M(ws=FAKE + 4) == 3
    assert M(ws=None) == 4 and M(nb=255) == 4
    assert M(P=0, x=None, ws=None) == 0         # an empty batch touches nothing


def test_balance_refusals(L):
    def B(lg=FAKE, lt=0, ix=FAKE, S=2, T=4000, E=8, k=2, loss=FAKE, c=FAKE, p=FAKE, n=FAKE, ws=FAKE, nb=1 << 30):
        return L.moe_balance_loss(lg, lt, ix, None, S, T, E, k, loss, c, p, n, ws, nb, None)
    for kw in (dict(lg=None), dict(ix=None), dict(loss=None), dict(c=None), dict(p=None), dict(n=None), dict(lt=2),
               dict(k=0), dict(k=9), dict(E=64, k=33)):
        assert B(**kw) == 1, kw
    for kw in (dict(E=1025), dict(S=-1), dict(T=-1), dict(S=1 << 11, T=1 << 10), dict(T=1 << 40), dict(S=1 << 62, T=4)):
        assert B(**kw) == 2, kw
    assert B(lg=FAKE + 4) == 3 and B(ws=FAKE + 16) == 3
    assert B(ws=None) == 4 and B(nb=L.moe_balance_workspace_bytes(2, 4000, 8) - 1) == 4
    assert B(S=0) == 0 and B(T=0, lg=None) == 0

    def G(lg=FAKE, lt=0, c=FAKE, n=FAKE, g=FAKE, S=2, T=8, E=8, k=2, out=FAKE):
        return L.moe_balance_loss_backward(lg, lt, c, n, None, g, S, T, E, k, out, None)
    for kw in (dict(lg=None), dict(c=None), dict(n=None), dict(g=None), dict(out=None), dict(lt=3), dict(k=0)):
        assert G(**kw) == 1, kw
    assert G(E=0, k=1) == 1 and G(E=1025) == 2 and G(out=FAKE + 2) == 3 and G(T=0) == 0


def test_binding_refuses_what_it_cannot_pass_on(L):
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="GPU"):
        native.quantize_mxfp4(x, out=torch.zeros(1, 160, dtype=torch.uint8))
    with pytest.raises(TypeError):
        native.quantize_mxfp4(x.half())
    with pytest.raises(ValueError, match="one matrix"):
        native.quantize_mxfp4(x.view(2, 2, 64), rows=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="one length"):
        native.balance_loss(torch.zeros(7, 8), torch.zeros(7, 2, dtype=torch.int32), n_seq=2)


def test_reference_codec_on_the_format_s_own_values():
    # every E2M1 value times a power of two is its own code; halfway points go to the even code
    v = np.concatenate([ref.E2M1, -ref.E2M1, [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.9], np.full(8, 4.0)])
    x = np.stack([v * 2.0 ** k for k in (-60, 0, 60)]).astype(np.float32)
    c, s = ref.quantize(x)
    assert (c == c[0]).all() and (s[:, 0] == np.array([127 - 60, 127, 127 + 60])).all()
    assert c[0, :8].tolist() == list(range(8)) and c[0, 16:24].tolist() == [0, 2, 2, 4, 4, 6, 6, 7]
    assert c[0, 8] == 0                          # a zero magnitude is +0
    np.testing.assert_array_equal(ref.values(c, s)[:, :16], x[:, :16].astype(np.float64))


def test_layer_descriptor_with_mxfp4(L):
    import ctypes

    def desc(**kw):
        base = dict(d=256, f=96, E=8, k=2, act=0, wfmt=4, path=0, router_w=FAKE, w_gate_up=FAKE, w_down=FAKE)
        base.update(kw)
        return native.LayerDesc(**base)
    need = L.moe_layer_workspace_bytes(ctypes.byref(desc()), 16)
    assert need > 0
    F = lambda d, nb=need: L.moe_layer_forward(ctypes.byref(d), FAKE, 0, 16, None, None, FAKE, FAKE, nb, None, None)  # noqa: E731
    assert F(desc(f=80)) == 2 and F(desc(wfmt=3)) == 1 and F(desc(act=2)) == 1
    assert F(desc(path=1)) == 5 and F(desc(path=2)) == 5 and F(desc(act_quant=1)) == 5 and F(desc(flags=2)) == 5
    assert L.moe_layer_forward(ctypes.byref(desc()), FAKE, 0, 16, None, None, FAKE, FAKE, 1024, None, None) == 4
    # router, top-k, three of the permutation (or one kernel); coded x, gate.up, coded h, down, combine
    assert L.moe_layer_forward_launches(ctypes.byref(desc()), 4096, 0) == 10
    assert L.moe_layer_forward_launches(ctypes.byref(desc()), 4096, 1) == 8
