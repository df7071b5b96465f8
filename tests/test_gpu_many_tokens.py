"""More tokens than a grid's second dimension holds blocks: the same rows as in calls of fewer."""
import pytest
import torch

from quantized_routed_expert_softmax_gb300 import layers, native, synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_routed_expert_softmax_gb300 import build
    build.build()
    native.lib()


def _layer(wfmt, x_dtype="bf16"):
    w = synth.Workload("many_" + wfmt, d=256, f=64, E=8, k=2, act="swiglu", wfmt=wfmt, x_dtype=x_dtype, layers=1)
    return w, layers.build_layer(w, source="numpy")


def _check(w, L, T, step):
    x = synth.tokens_cuda(w, T, tag="many")
    out = torch.full((T, w.d), float("nan"), device="cuda")
    L.forward(x, out=out)
    assert L.device_status() == 0
    for a in range(0, T, step):
        a = min(a, T - step)      # (a few tokens would take another path, with other roundings)
        assert torch.equal(out[a : a + step], L.forward(x[a : a + step])), a


@pytest.mark.parametrize("wfmt", ["mxfp4", "q8_0"])
@pytest.mark.parametrize("T", [65535, 65536, 2 * 65535 + 7])
def test_layer_past_65535_tokens(wfmt, T):
    w, L = _layer(wfmt)
    _check(w, L, T, 32769)
