"""The int8 product's way out of a wait that ran out, which is code of its own in each of its kernels: taken at these sizes,
reported as device error 2, within the limit, and with nothing left behind for the next call.

The workspace's limit word (the int64 at byte 32) of -1 makes a wait give up after its first look.  A look may last some
microseconds, so that not every product has a wait that outlasts it; here one call of a few does."""
import time

import pytest
import torch

from quantized_routed_expert_softmax_gb300 import native

pytestmark = pytest.mark.gpu

LIMIT_QWORD = 4
CALLS = 12


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_routed_expert_softmax_gb300 import build
    build.build()
    native.lib()


@pytest.mark.parametrize("act,dtype", [("none", torch.float32), ("none", torch.bfloat16), ("swiglu", torch.bfloat16),
                                       ("swiglu", torch.float32), ("relu2", torch.float32), ("relu2", torch.bfloat16)])
@pytest.mark.parametrize("P,N,K", [(300, 512, 65536), (600, 4096, 65536), (2000, 8192, 8192), (40000, 2816, 704), (20000, 2816, 1024)])
def test_product_gives_up_and_recovers(P, N, K, act, dtype):
    g = torch.Generator("cuda").manual_seed(P)
    xq = native.quantize_int8(torch.randn(P, K, device="cuda", generator=g))[0]
    wq = native.quantize_int8(torch.randn(N, K, device="cuda", generator=g))[0]
    ws = native.int8_workspace()
    call = lambda: native.int8_matmul(xq, wq, None, P, N, K, act=act, dtype=dtype, workspace=ws)  # noqa: E731
    want = call()
    assert native.device_status(ws) == 0
    seen = []
    for _ in range(CALLS):
        ws.view(torch.int64)[LIMIT_QWORD] = -1
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        got = call()
        torch.cuda.synchronize()
        assert time.perf_counter() - t0 < 0.5
        seen.append(native.device_status(ws))
        assert native.device_status(ws) == 0                  # reading clears the word
        if seen[-1] == 0:                                     # every wait was over at its first look: a whole result
            assert torch.equal(got, want)
        ws.view(torch.int64)[LIMIT_QWORD] = 0
        assert torch.equal(call(), want) and native.device_status(ws) == 0
    assert set(seen) <= {0, 2} and 2 in seen, seen
