"""Every output form and activation of the MXFP4 product in every row tile (32, 128 and 192 rows; the kernel chooses by
rows and rows an expert), with few and with many K steps.  The groups lie far from the choice's borders: 1 to 5 rows an
expert, 64 to 73, and 300 to 577."""
import pytest
import torch

import test_gpu_mxfp4 as product
from quantized_routed_expert_softmax_gb300 import native

pytestmark = pytest.mark.gpu

GROUPS = {"32": [5, 0, 11], "128": [130, 5, 71, 85], "192": [577], "192 uneven": [600, 30]}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_routed_expert_softmax_gb300 import build
    build.build()
    native.lib()


@pytest.mark.parametrize("N", [1, 7, 17, 127, 130, 257])      # bf16 rows that 16-byte stores do not fit
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tile", list(GROUPS))
def test_odd_widths(tile, dtype, N):
    for act in ("none", "relu2"):
        product._case(GROUPS[tile], 96, N, act, dtype, seed=N, first=1, behind=3)


@pytest.mark.parametrize("act", ["none", "swiglu", "relu2"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tile", list(GROUPS))
def test_many_k_steps(tile, dtype, act):
    product._case(GROUPS[tile], 2816, 1408, act, dtype, seed=3)          # 11 steps, more than any ring's stages
    product._case(GROUPS[tile], 2816 + 32, 192, act, dtype, seed=4, first=2)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tile", list(GROUPS))
def test_many_items_of_odd_width(tile, dtype):
    # more weight tiles than CTAs, so that both accumulators and the stages come round within a CTA
    product._case(GROUPS[tile], 704, 20001, "relu2", dtype, seed=5)
