"""A wait of the feed-forward block's products, and of the int8 product, that runs out: recorded as device error 2, without a fault, within the
limit, and with nothing left behind for the next call.

The workspace's limit word (the int64 at byte 32) shortens the limit: with -1 a wait gives up at its first look.  With sums
over 65536 columns (or as many rows) the first results are a thousand K steps away, so the epilogue's wait gives up while
loads and MMAs are on their way; the pair has to bring those to an end before it returns its memories."""
import time

import pytest
import torch

from quantized_routed_expert_softmax_gb300 import native

pytestmark = pytest.mark.gpu

LIMIT_QWORD = 4


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_routed_expert_softmax_gb300 import build
    build.build()
    native.lib()


def _gives_up_and_recovers(call, ws, sure=True):
    want = call()
    assert native.device_status(ws) == 0
    for _ in range(3):
        ws[:256].view(torch.int64)[LIMIT_QWORD] = -1
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        got = call()
        torch.cuda.synchronize()
        took = time.perf_counter() - t0
        status = native.device_status(ws)
        assert native.device_status(ws) == 0      # reading clears the word
        assert took < 0.5, took
        if sure or status != 0:
            assert status == 2
        else:
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        ws[:256].view(torch.int64)[LIMIT_QWORD] = 0
        assert all(torch.equal(a, b) for a, b in zip(call(), want))
        assert native.device_status(ws) == 0


@pytest.mark.parametrize("act", ["swiglu", "relu2"])
@pytest.mark.parametrize("P", [100, 700])
def test_block_gives_up_and_recovers(P, act):
    d, f, bf = 65536, 64, torch.bfloat16
    g = torch.Generator("cuda").manual_seed(P)
    rand = lambda *s: torch.randn(s, device="cuda", generator=g).to(bf)  # noqa: E731
    x, dy = rand(P, d), rand(P, d)
    wgu, wd = rand(2 * f if act == "swiglu" else f, d) / 256, rand(d, f) / 8
    ws = native.ffn_workspace(P, f, act, backward=True)
    _gives_up_and_recovers(lambda: (native.ffn_forward(x, wgu, wd, act=act, workspace=ws),), ws)
    y, saved = native.ffn_forward(x, wgu, wd, act=act, save=True, workspace=ws)
    _gives_up_and_recovers(lambda: native.ffn_backward(dy, x, wgu, wd, saved, act=act, workspace=ws, need=(True, False, False))[:1], ws)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_weight_gradients_give_up_and_recover(dtype):
    P, d, f, bf = 131072 - 17, 256, 64, torch.bfloat16
    g = torch.Generator("cuda").manual_seed(1)
    rand = lambda *s: torch.randn(s, device="cuda", generator=g).to(bf)  # noqa: E731
    x, dy, wgu, wd = rand(P, d), rand(P, d), rand(2 * f, d) / 16, rand(d, f) / 8
    ws = native.ffn_workspace(P, f, backward=True)
    _, saved = native.ffn_forward(x, wgu, wd, save=True, workspace=ws)
    _gives_up_and_recovers(lambda: native.ffn_backward(dy, x, wgu, wd, saved, workspace=ws, dtype=dtype, need=(False, False, True))[2:], ws)


@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("P,N", [(300, 512), (600, 4096)])
def test_int8_product_gives_up_and_recovers(P, N, act):
    K = 65536
    g = torch.Generator("cuda").manual_seed(P)
    xq = native.quantize_int8(torch.randn(P, K, device="cuda", generator=g))[0]
    wq = native.quantize_int8(torch.randn(N, K, device="cuda", generator=g))[0]
    ws = native.int8_workspace()
    # (its first sums are 8 K steps away, some microseconds, which a wait's first look may last)
    _gives_up_and_recovers(lambda: (native.int8_matmul(xq, wq, None, P, N, K, act=act, workspace=ws),), ws, sure=False)
