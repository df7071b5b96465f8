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


@pytest.mark.parametrize("x_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E", [8, 12])      # eight experts a block, and four
def test_router_past_524280_tokens(E, x_dtype):
    T, d, k, step = 524288 + 9, 256, 2, 262149
    g = torch.Generator("cuda").manual_seed(E)
    x = torch.randn(T, d, device="cuda", generator=g).to(x_dtype)
    W = torch.randn(d, E, device="cuda", generator=g)
    idx, w, logits = native.router_topk(x, W, k, return_logits=True)
    for a in range(0, T, step):
        a = min(a, T - step)
        part = native.router_topk(x[a : a + step].contiguous(), W, k, return_logits=True)
        assert all(torch.equal(whole[a : a + step], p) for whole, p in zip((idx, w, logits), part)), a


def test_layer_of_the_largest_batch():
    w, L = _layer("mxfp4")
    _check(w, L, 1 << 20, 1 << 19)
