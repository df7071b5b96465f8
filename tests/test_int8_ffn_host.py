"""int8 operators and the feed-forward block on the host: sizes, refusals with their status, and the restatement's
gradients against differences.  No test here touches a GPU."""
import os
import shutil

import numpy as np
import pytest
import torch

import experts_ref as ref
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
    for rows, cols in ((1, 32), (3, 64), (4, 96), (128, 2816)):
        assert L.moe_int8_bytes(rows, cols) == ref.bytes_of(rows, cols)
    assert L.moe_int8_bytes(64, 160) == L.moe_int8pc_bytes(64, 160)
    for rows, cols in ((0, 32), (1, 33), (1, 0), (-1, 32), (1, 65568), (2 ** 25 + 1, 32)):
        assert L.moe_int8_bytes(rows, cols) == 0
    assert L.moe_int8_matmul_workspace_bytes() == 256
    assert L.moe_ffn_workspace_bytes(0, 16, 0, 1) == 256
    assert L.moe_ffn_workspace_bytes(10, 48, 0, 0) == 256 + 1024
    assert L.moe_ffn_workspace_bytes(10, 48, 0, 1) == 256 + 2048 and L.moe_ffn_workspace_bytes(10, 48, 1, 1) == 256 + 1024
    assert L.moe_ffn_workspace_bytes(10, 40, 0, 0) == 0 and L.moe_ffn_workspace_bytes(-1, 48, 0, 0) == 0
    assert L.moe_ffn_workspace_bytes(10, 48, 2, 0) == 0


def test_codec_refusals(L):
    Q, D = L.moe_quantize_int8, L.moe_dequantize_int8
    assert Q(None, 0, 0, None, 1, 4, 32, FAKE, None) == 1 and Q(FAKE, 0, 0, None, 1, 4, 32, None, None) == 1
    assert Q(FAKE, 2, 0, None, 1, 4, 32, FAKE, None) == 1
    assert Q(FAKE, 0, 4, FAKE, 2, 4, 32, FAKE, None) == 1 and Q(FAKE, 0, -1, FAKE, 1, 4, 32, FAKE, None) == 1
    assert Q(FAKE, 0, 0, None, 1, 4, 33, FAKE, None) == 2 and Q(FAKE, 0, 0, None, 65536, 4, 32, FAKE, None) == 2
    assert Q(FAKE, 0, 0, None, 1, 2 ** 25 + 1, 32, FAKE, None) == 2
    assert Q(FAKE + 4, 0, 0, None, 1, 4, 32, FAKE, None) == 3 and Q(FAKE, 0, 0, None, 1, 4, 32, FAKE + 8, None) == 3
    assert Q(None, 0, 0, None, 1, 0, 32, None, None) == 0 and Q(None, 0, 0, None, 0, 4, 32, None, None) == 0
    assert D(None, 1, 4, 32, FAKE, 0, None) == 1 and D(FAKE, 1, 4, 32, FAKE, 2, None) == 1
    assert D(FAKE, 1, 4, 48, FAKE, 0, None) == 2 and D(FAKE, 1, 4, 32, FAKE + 4, 0, None) == 3
    assert D(None, 1, 0, 32, None, 0, None) == 0


def test_product_refusals(L):
    def M(xq=FAKE, P=4, wq=FAKE, E=2, N=64, K=32, off=FAKE, act=2, out=FAKE, ot=0, ws=FAKE, n=256):
        return L.moe_int8_matmul(xq, P, wq, E, N, K, off, act, out, ot, ws, n, None)
    assert M(xq=None) == 1 and M(wq=None) == 1 and M(out=None) == 1 and M(off=None) == 1
    assert M(act=3) == 1 and M(ot=2) == 1 and M(E=0) == 1
    assert M(K=48) == 2 and M(K=0) == 2 and M(P=-1) == 2 and M(E=1025) == 2 and M(N=0) == 2 and M(N=131073) == 2
    assert M(act=0, N=96) == 2
    assert M(xq=FAKE + 8) == 3 and M(wq=FAKE + 8) == 3 and M(out=FAKE + 8) == 3 and M(off=FAKE + 2) == 3 and M(ws=FAKE + 8) == 3
    assert M(ws=None) == 4 and M(n=255) == 4
    assert M(P=0, xq=None, out=None) == 0


def test_block_refusals(L):
    def F(x=FAKE, P=4, gu=FAKE, dn=FAKE, E=2, d=32, f=48, off=FAKE, act=0, y=FAKE, z=FAKE, h=FAKE, ws=FAKE, n=256):
        return L.moe_ffn_forward(x, P, gu, dn, E, d, f, off, act, y, z, h, ws, n, None)
    assert F(x=None) == 1 and F(gu=None) == 1 and F(dn=None) == 1 and F(y=None) == 1 and F(off=None) == 1 and F(act=2) == 1
    for bad in (dict(d=24), dict(d=0), dict(f=40), dict(f=0), dict(E=0), dict(E=1025), dict(P=-1), dict(P=2 ** 25 + 1), dict(d=65552), dict(f=32784)):
        assert F(**bad) == 2, bad
    for bad in (dict(x=FAKE + 8), dict(gu=FAKE + 8), dict(dn=FAKE + 8), dict(y=FAKE + 8), dict(z=FAKE + 8), dict(h=FAKE + 8), dict(off=FAKE + 2), dict(ws=FAKE + 16)):
        assert F(**bad) == 3, bad
    assert F(ws=None) == 4 and F(n=255) == 4 and F(h=None) == 4 and F(P=0, x=None, y=None) == 0

    def B(dy=FAKE, x=FAKE, P=4, gu=FAKE, dn=FAKE, E=2, d=32, f=48, off=FAKE, act=0, z=FAKE, h=FAKE, dx=FAKE, dgu=FAKE, dd=FAKE, gt=0, ws=FAKE, n=1 << 20):
        return L.moe_ffn_backward(dy, x, P, gu, dn, E, d, f, off, act, z, h, dx, dgu, dd, gt, ws, n, None)
    for bad in (dict(dy=None), dict(x=None), dict(gu=None), dict(dn=None), dict(z=None), dict(h=None), dict(off=None), dict(act=2), dict(gt=2)):
        assert B(**bad) == 1, bad
    assert B(d=24) == 2 and B(f=40) == 2
    for bad in (dict(dy=FAKE + 8), dict(z=FAKE + 8), dict(dx=FAKE + 8), dict(dgu=FAKE + 8), dict(dd=FAKE + 8), dict(ws=FAKE + 16)):
        assert B(**bad) == 3, bad
    assert B(ws=None) == 4 and B(n=256 + 4 * 96 * 2 - 1) == 4


def test_binding_refusals():
    bf = torch.bfloat16
    x = torch.zeros(4, 32, dtype=bf)
    with pytest.raises(ValueError):
        native.ffn_forward(x, torch.zeros(2, 96, 32, dtype=bf), torch.zeros(2, 32, 32, dtype=bf))        # 2 f rows
    with pytest.raises(ValueError):
        native.ffn_forward(x, torch.zeros(2, 64, 32, dtype=bf), torch.zeros(32, 32, dtype=bf))           # one and many matrices
    with pytest.raises(ValueError):
        native.ffn_forward(x, torch.zeros(64, 32, dtype=bf), torch.zeros(32, 32, dtype=bf))              # not on the GPU
    with pytest.raises(TypeError):
        native.quantize_int8(torch.zeros(4, 32, dtype=torch.float16))
    with pytest.raises(ValueError):
        native.quantize_int8(torch.zeros(2, 4, 32), rows=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        native.int8_matmul(torch.zeros(10, dtype=torch.uint8), torch.zeros(1, 10, dtype=torch.uint8), None, 4, 32, 32, workspace=torch.zeros(256, dtype=torch.uint8))


@pytest.mark.parametrize("act", ["swiglu", "relu2"])
def test_the_restatements_gradients_against_differences(act):
    g = torch.Generator().manual_seed(1)
    P, E, d, f = 9, 3, 16, 16
    nz = 2 * f if act == "swiglu" else f
    ops = [torch.randn(s, generator=g, dtype=torch.float64) for s in ((P, d), (E, nz, d), (E, d, f))]
    dy = torch.randn(P, d, generator=g, dtype=torch.float64)
    off = [0, 4, 4, 9]
    want = ref.ffn(*ops, off, act, dy)
    for i, name in ((0, "dx"), (1, "dwgu"), (2, "dwd")):
        v = torch.randn(ops[i].shape, generator=g, dtype=torch.float64)
        hi, lo = list(ops), list(ops)
        hi[i], lo[i] = ops[i] + 1e-6 * v, ops[i] - 1e-6 * v
        diff = ((ref.ffn(*hi, off, act)["y"][0] - ref.ffn(*lo, off, act)["y"][0]) * dy).sum() / 2e-6
        got = (want[name][0] * v).sum()
        assert abs(got - diff) <= 1e-6 * (want[name][0] * v).abs().sum()


def test_the_restated_codec():
    x = np.array([[127.0, 0.5, -0.5, 126.5] + [0.0] * 28, [0.0] * 32, [np.inf] + [1.0] * 31], np.float32)
    q, s = ref.quantize(x)
    assert q[0, :4].tolist() == [127, 1, -1, 127] and s[0] == 1.0 and s[1] == 0.0 and np.isnan(s[2])
    assert not q[1:].any()


def test_layer_descriptor_refusals(L):
    import ctypes

    def ws(**kw):
        d = dict(d=512, f=96, E=16, k=3, act=0, wfmt=2, path=0, router_w=FAKE, w_gate_up=FAKE, w_down=FAKE, act_quant=3)
        d.update(kw)
        return L.moe_layer_workspace_bytes(ctypes.byref(native.LayerDesc(**d)), 64)

    plain = ws(act_quant=0)
    assert ws() >= plain + ref.bytes_of(192, 512) + ref.bytes_of(192, 96) - 2 * 256
    for bad in (dict(wfmt=0), dict(wfmt=4), dict(path=1), dict(path=2), dict(flags=2), dict(act_quant=2), dict(act_quant=4)):
        assert ws(**bad) == 0, bad
    F = lambda **kw: L.moe_layer_forward(ctypes.byref(native.LayerDesc(**{**dict(  # noqa: E731
        d=512, f=96, E=16, k=3, act=0, wfmt=2, path=0, router_w=FAKE, w_gate_up=FAKE, w_down=FAKE, act_quant=3), **kw})), FAKE, 1, 4, None, None, FAKE,
        FAKE, 1 << 30, None, None)
    assert F(wfmt=0) == 5 and F(path=1) == 5 and F(flags=2) == 5 and F(act_quant=4) == 1


class OnDevice:
    """What the binding asks of a tensor, with a device number of its own: no GPU here."""
    is_cuda = True

    def __init__(self, shape, dtype, device):
        self.shape, self.dtype, self.number, self.device = torch.Size(shape), dtype, device, f"cuda:{device}"

    def is_contiguous(self):
        return True

    def numel(self):
        return self.shape.numel()

    def get_device(self):
        return self.number

    def data_ptr(self):
        return 0x10000


def _calls(dev):
    """Every call with its operands on the devices of `dev` (0 for the rest)."""
    u8, i32, f32, bf = torch.uint8, torch.int32, torch.float32, torch.bfloat16
    t = lambda name, shape, dtype: OnDevice(shape, dtype, dev.get(name, 0))  # noqa: E731
    xq, wq = ref.bytes_of(4, 64), ref.bytes_of(64, 64)
    ws = t("workspace", (4096,), u8)
    block = lambda: (t("x", (4, 32), bf), t("w_gate_up", (2, 96, 32), bf), t("w_down", (2, 32, 48), bf))  # noqa: E731
    return {
        "quantize": lambda: native.quantize_int8(t("x", (4, 64), f32), rows=t("rows", (4,), i32), out=t("out", (1, xq), u8)),
        "dequantize": lambda: native.dequantize_int8(t("q", (xq,), u8), 4, 64, out=t("out", (4, 64), f32)),
        "matmul": lambda: native.int8_matmul(t("xq", (xq,), u8), t("wq", (2, wq), u8), t("offsets", (3,), i32), 4, 64, 64,
                                             out=t("out", (4, 64), f32), workspace=ws),
        "forward": lambda: native.ffn_forward(*block(), t("offsets", (3,), i32), out=t("out", (4, 32), bf), workspace=ws),
        "backward": lambda: native.ffn_backward(t("grad", (4, 32), bf), *block(), (t("z", (4, 96), f32), t("h", (4, 48), bf)),
                                                t("offsets", (3,), i32), workspace=ws),
    }


OPERANDS = {"quantize": ["x", "rows", "out"], "dequantize": ["q", "out"], "matmul": ["xq", "wq", "offsets", "out", "workspace"],
            "forward": ["x", "w_gate_up", "w_down", "offsets", "out", "workspace"],
            "backward": ["grad", "x", "w_gate_up", "w_down", "z", "h", "offsets", "workspace"]}


@pytest.mark.parametrize("call,operand", [(c, o) for c, names in OPERANDS.items() for o in names] + [(c, None) for c in OPERANDS])
def test_operands_of_another_device_are_refused(monkeypatch, call, operand):
    monkeypatch.setattr(native, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    monkeypatch.setattr(torch, "empty", lambda shape, dtype=torch.float32, device="cuda:0": OnDevice(
        (shape,) if isinstance(shape, int) else shape, dtype, int(str(device).split(":")[1])))

    class Lib:
        def __getattr__(self, name):
            return lambda *a: 256 if name.endswith("bytes") else 0
    monkeypatch.setattr(native, "lib", lambda: Lib())
    if operand is None:
        _calls({})[call]()                                             # all on the current device
        everything = {name: 1 for name in OPERANDS[call]}
        with pytest.raises(ValueError, match="current device"):
            _calls(everything)[call]()
    else:
        with pytest.raises(ValueError, match="device"):
            _calls({operand: 1})[call]()
