"""The activations in the MXFP4 product's epilogue over their whole range: products that are exact in fp32, so that
what is measured is the activation alone."""
import numpy as np
import pytest
import torch

from quantized_routed_expert_softmax_gb300 import native

pytestmark = pytest.mark.gpu

U = 2.0 ** -24   # half a unit of fp32, relative
# SiLU, in units of U: exp(-|g|) 2 units in the last place, 4, its product with g 1; the divisor 1 + e, at least 1, is
# off by 4 e + 1, at most 3 of itself; the division 2 units in the last place, 4; the product with up 1.
SILU_UNITS = 4 + 1 + 3 + 4 + 1


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_routed_expert_softmax_gb300 import build
    build.build()
    native.lib()


def _exact_weights(v):
    """Weight rows [len(v), 32 * 8] whose product with rows of ones in every block's first column is v: one E2M1
    value times a power of two a block, the largest first."""
    w = np.zeros((len(v), 8, 32), np.float32)
    rest = np.abs(v.astype(np.float64))
    for b in range(8):
        with np.errstate(divide="ignore"):
            p = np.exp2(np.floor(np.log2(rest)))
        t = np.where(rest > 0, np.where(rest >= 1.5 * p, 1.5 * p, p), 0)
        w[:, b, 0] = np.sign(v) * t
        rest = rest - t
    assert (rest == 0).all()
    return w.reshape(len(v), 256)


def _product(v, scales, act, dtype, rows):
    """z = scales x v through the product, `rows` times over (the row tile goes by their number)."""
    x = np.zeros((len(scales), 8, 32), np.float32)
    x[:, :, 0] = np.asarray(scales, np.float32)[:, None]
    x = np.tile(x.reshape(len(scales), 256), (rows, 1))
    xq = native.quantize_mxfp4(torch.from_numpy(x).cuda())[0]
    wq = native.quantize_mxfp4(torch.from_numpy(_exact_weights(v)).cuda())[0]
    z = x[:, :1].astype(np.float64) * v.astype(np.float64)
    plain = native.mxfp4_matmul(xq, wq, None, len(x), len(v), 256)
    assert np.array_equal(plain.cpu().numpy().astype(np.float64), z)      # the product is exact
    return native.mxfp4_matmul(xq, wq, None, len(x), len(v), 256, act=act, dtype=dtype), torch.from_numpy(z).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows", [1, 13, 70])      # row tiles of 32, 128, 192
def test_silu_from_small_to_saturated_gates(rows, dtype):
    gates = np.concatenate([np.arange(-110, 110, 0.25), [-128, 127, 120, -90.125, -87.875, -0.125, 0, 0.125]])
    gates = np.concatenate([gates, np.zeros(-len(gates) % 32)])
    up = np.resize([1.5, -0.75, 96.0, 1 / 64], len(gates))
    out, z = _product(np.concatenate([gates, up]).astype(np.float32), [1.0, 2.0 ** -7, -0.5], "swiglu", dtype, rows)
    g, u = z[:, : len(gates)], z[:, len(gates) :]
    want = g * torch.sigmoid(g) * u
    # subnormals: exp(-|g|) 2 units of 2^-149 (of which g and up make |g u| times as much), then three roundings to 2^-149
    err = SILU_UNITS * U * want.abs() + 2.0 ** -149 * (2 * g.abs() + 3) * (1 + u.abs())
    if dtype == torch.bfloat16:
        err = err + 2.0 ** -8 * (want.abs() + err) + 2.0 ** -133
    over = (out.double() - want).abs() - err
    assert (over <= 0).all(), (float(over.max()), float(g.flatten()[over.argmax()]))
    assert float(want.abs()[want != 0].min()) < 2.0 ** -126


@pytest.mark.parametrize("rows", [1, 13, 70])
def test_silu_and_relu2_of_huge_infinite_and_nan_products(rows):
    big = np.float32(2.0 ** 100)
    gates = np.resize(np.array([-big, big, -200.0, 200.0], np.float32), 32)
    up = np.full(32, 1.0, np.float32)
    out, z = _product(np.concatenate([gates, up]), [1.0, 2.0, -1.0], "swiglu", torch.float32, rows)
    g, u = z[:, :32], z[:, 32:]
    want = torch.where(g > 0, g, torch.zeros_like(g)) * u
    assert ((out.double() - want).abs() <= SILU_UNITS * U * want.abs()).all()      # (up is negative in a third of the rows)
    # 2^120 * 2^120 is an infinity; a block with a NaN is NaN
    x = np.zeros((4, 32), np.float32)
    x[:, 0] = [2.0 ** 120, -(2.0 ** 120), np.nan, 1.0]
    x = np.tile(x, (rows, 1))
    w = np.zeros((64, 32), np.float32)
    w[:32, 0] = 2.0 ** 120
    w[32:, 0] = 2.0 ** -120
    xq, wq = (native.quantize_mxfp4(torch.from_numpy(a).cuda())[0] for a in (x, w))
    r = native.mxfp4_matmul(xq, wq, None, len(x), 64, 32, act="relu2").view(rows, 4, 64)
    assert (r[:, 0, :32] == float("inf")).all() and (r[:, 0, 32:] == 1).all()
    assert (r[:, 1] == 0).all() and torch.isnan(r[:, 2]).all() and (r[:, 3, :32] == float("inf")).all()
    s = native.mxfp4_matmul(xq, wq, None, len(x), 64, 32, act="swiglu").view(rows, 4, 32)
    assert (s[:, 0] == float("inf")).all() and torch.isnan(s[:, 2]).all()
    assert ((s[:, 3] - 1).abs() <= SILU_UNITS * U).all()
