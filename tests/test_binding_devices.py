"""Operands of the MXFP4 and balance calls on a device that the call does not run on: refused on the host, before a
kernel of the current device gets another device's pointer.  Stand-ins for the tensors: no GPU here."""
import pytest
import torch

from quantized_routed_expert_softmax_gb300 import native


class OnDevice:
    """What the binding asks of a tensor, with a device number of its own."""
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

    def __getitem__(self, i):
        return self


@pytest.fixture(autouse=True)
def _no_launch(monkeypatch):
    monkeypatch.setattr(native, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(native, "_stream", lambda stream=None: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    made = lambda shape, dtype=torch.float32, device="cuda:0", **kw: OnDevice(  # noqa: E731
        (shape,) if isinstance(shape, int) else shape, dtype, int(str(device).split(":")[1]))
    monkeypatch.setattr(torch, "empty", made)

    class Lib:
        def __getattr__(self, name):
            return lambda *a: 256 if name.endswith("bytes") else 0
    monkeypatch.setattr(native, "lib", lambda: Lib())


U8, I32, F32 = torch.uint8, torch.int32, torch.float32


def _calls(dev):
    """Every call with its operands on the devices of `dev` (0 for the rest)."""
    t = lambda name, shape, dtype: OnDevice(shape, dtype, dev.get(name, 0))  # noqa: E731
    xq, wq = native._mxfp4_size(4, 64), native._mxfp4_size(64, 64)
    return {
        "quantize": lambda: native.quantize_mxfp4(t("x", (4, 64), F32), rows=t("rows", (4,), I32),
                                                  out=t("out", (1, xq), U8)),
        "dequantize": lambda: native.dequantize_mxfp4(t("q", (xq,), U8), 4, 64, out=t("out", (4, 64), F32)),
        "matmul": lambda: native.mxfp4_matmul(t("xq", (xq,), U8), t("wq", (2, wq), U8), t("offsets", (3,), I32), 4, 64, 64,
                                              out=t("out", (4, 64), F32), workspace=t("workspace", (256,), U8)),
        "balance": lambda: native.balance_loss(t("logits", (8, 8), F32), t("idx", (8, 2), I32), mask=t("mask", (8,), U8),
                                               workspace=t("workspace", (256,), U8)),
        "backward": lambda: native.balance_loss_backward(
            t("logits", (8, 8), F32), t("counts", (1, 8), I32), t("tokens", (1,), I32), t("grad_loss", (1,), F32), 2,
            mask=t("mask", (8,), U8), out=t("out", (8, 8), F32)),
    }


OPERANDS = [("quantize", n) for n in ("x", "rows", "out")] + [("dequantize", n) for n in ("q", "out")] + \
    [("matmul", n) for n in ("xq", "wq", "offsets", "out", "workspace")] + \
    [("balance", n) for n in ("logits", "idx", "mask", "workspace")] + \
    [("backward", n) for n in ("logits", "counts", "tokens", "grad_loss", "mask", "out")]


@pytest.mark.parametrize("call,operand", OPERANDS)
def test_operand_of_another_device_is_refused(call, operand):
    _calls({})[call]()
    with pytest.raises(ValueError, match="on device 1"):
        _calls({operand: 1})[call]()


def test_all_operands_of_a_device_that_is_not_the_current_one():
    names = {n for _, n in OPERANDS}
    for call in _calls({}).values():
        call()
    for call in _calls(dict.fromkeys(names, 1)).values():
        with pytest.raises(ValueError, match="on device 1"):
            call()
