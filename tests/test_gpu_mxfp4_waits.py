"""A wait of the MXFP4 product that runs out: recorded as device error 2, without a fault, within the limit, and with
nothing left behind for the next call.

A product's waits are on its own copies and MMAs, and last a second at most.  The workspace's limit word (the int64 at
byte 32, as in a layer's workspace) shortens that: with -1 a wait gives up at its first look.  With K = 65536 the first
results are 256 K steps away, tens of microseconds, so the epilogue's wait gives up while loads and MMAs are on their way;
the kernel has to bring those to an end before it returns its shared and tensor memory."""
import time

import pytest
import torch

from quantized_routed_expert_softmax_gb300 import layers, native, synth

pytestmark = pytest.mark.gpu

LIMIT_QWORD = 4


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_routed_expert_softmax_gb300 import build
    build.build()
    native.lib()


@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("P,N", [(2, 64), (100, 512), (300, 64), (600, 4096)])      # row tiles of 32, 128, 192; several items a CTA
def test_product_gives_up_and_recovers(P, N, act):
    K = 65536
    g = torch.Generator("cuda").manual_seed(P)
    xq = native.quantize_mxfp4(torch.randn(P, K, device="cuda", generator=g))[0]
    wq = native.quantize_mxfp4(torch.randn(N, K, device="cuda", generator=g))[0]
    ws = native.mxfp4_workspace()
    ref = native.mxfp4_matmul(xq, wq, None, P, N, K, act=act, workspace=ws)
    assert native.device_status(ws) == 0
    for _ in range(3):
        ws.view(torch.int64)[LIMIT_QWORD] = -1
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        native.mxfp4_matmul(xq, wq, None, P, N, K, act=act, workspace=ws)
        torch.cuda.synchronize()
        took = time.perf_counter() - t0
        assert native.device_status(ws) == 2 and native.device_status(ws) == 0      # reading clears the word
        assert took < 0.5, took
        ws.view(torch.int64)[LIMIT_QWORD] = 0
        assert torch.equal(native.mxfp4_matmul(xq, wq, None, P, N, K, act=act, workspace=ws), ref)
        assert native.device_status(ws) == 0


def test_layer_reports_a_wait_that_ran_out():
    w = synth.Workload("mx_waits", d=65536, f=32, E=4, k=1, act="swiglu", wfmt="mxfp4", x_dtype="bf16", layers=1)
    L = layers.build_layer(w)
    x = synth.tokens_cuda(w, 5, tag="waits")
    ws = torch.zeros(L.workspace_bytes(5), dtype=torch.uint8, device="cuda")
    ref = L.forward(x, workspace=ws).clone()
    assert native.device_status(ws) == 0
    ws.view(torch.int64)[LIMIT_QWORD] = -1
    L.forward(x, workspace=ws)
    assert native.device_status(ws) == 2
    ws.view(torch.int64)[LIMIT_QWORD] = 0
    assert torch.equal(L.forward(x, workspace=ws), ref)
    assert native.device_status(ws) == 0
