"""The int8 product over scales of every size that fp32 has: whatever the product of a row's and a channel's scale alone
would be, the results that fp32 can hold are right, and a sum of codes that is 0 gives 0."""
import numpy as np
import pytest
import torch

import experts_ref as ref
from quantized_routed_expert_softmax_gb300 import native

pytestmark = pytest.mark.gpu

MAX = float(np.finfo(np.float32).max)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_routed_expert_softmax_gb300 import build
    build.build()
    native.lib()


def _codes(g, P, N, K):
    """Rows and channels of codes; the sums of every third row with every fifth channel are 0."""
    x, w = g.integers(64, 128, (P, K)), g.integers(64, 128, (N, K))
    x[::3] = 127
    w[::5] = np.resize([127, -127], K)
    return x.astype(np.int8), w.astype(np.int8)


def _product(x, sx, w, sw):
    (P, K), N = x.shape, w.shape[0]
    xq, wq = (torch.from_numpy(ref.pack(c, s)[0]).cuda() for c, s in ((x, sx), (w, sw)))
    work = native.int8_workspace()
    out = native.int8_matmul(xq, wq, None, P, N, K, workspace=work).cpu().numpy()
    assert native.device_status(work) == 0
    total = x.astype(np.float64) @ w.astype(np.float64).T                     # (integers below 2^31: exact)
    each = np.abs(x.astype(np.float64)) @ np.abs(w.astype(np.float64)).T
    scale = sx.astype(np.float64)[:, None] * sw.astype(np.float64)
    # the joins of 1024 columns (one less than there are) and the conversion, then a rounding for each scale; one that ends among
    # the subnormal numbers is off by half of their step, 2^-150, and only the last one can round there (a whole number times a
    # subnormal scale is a whole number of their steps)
    n = (K + 1023) // 1024 + 3
    return out, total * scale, n * 2.0 ** -24 * each * scale + 2.0 ** -149


def _check(out, z, tol):
    fits = np.abs(z) + tol < MAX
    assert (np.abs(out[fits] - z[fits]) <= tol[fits]).all(), np.max((np.abs(out - z) - tol)[fits])
    over = np.abs(z) - tol > MAX * (1 + 2.0 ** -24)
    assert (out[over] == np.sign(z[over]) * np.inf).all()
    assert (out[z == 0] == 0).all()


SHAPES = [(4, 70, 96), (16, 64, 2816), (40, 70, 96), (300, 320, 704), (100, 64, 2816), (33, 261, 4128)]


@pytest.mark.parametrize("sx,sw", [(1e-25, 1e-18), (1e-18, 1e-25), (1e-40, 1e36), (1e36, 1e-40), (1e30, 1e30), (1e-38, 2.0 ** 97),
                                   (2.0 ** 121, 2.0 ** -120), (2.0 ** -120, 2.0 ** 121), (3e-45, 1e-3), (1e-20, 1e-25)])
@pytest.mark.parametrize("P,N,K", SHAPES)
def test_product_of_small_and_large_scales(P, N, K, sx, sw):
    g = np.random.default_rng(P + K)
    x, w = _codes(g, P, N, K)
    _check(*_product(x, (sx * g.uniform(0.7, 1.4, P)).astype(np.float32), w, (sw * g.uniform(0.7, 1.4, N)).astype(np.float32)))


@pytest.mark.parametrize("P,N,K", SHAPES)
def test_product_of_scales_of_every_size_at_once(P, N, K):
    g = np.random.default_rng(P * K)
    x, w = _codes(g, P, N, K)
    sx, sw = (np.exp2(g.uniform(-148, 121, n)).astype(np.float32) for n in (P, N))
    sx[1], sw[1] = 0, 0
    out, z, tol = _product(x, sx, w, sw)
    _check(out, z, tol)
    sx[0], sw[2] = np.nan, np.nan
    out, _, _ = _product(x, sx, w, sw)
    assert np.isnan(out[0]).all() and np.isnan(out[:, 2]).all()
    rest = np.delete(np.delete(out, 0, 0), 2, 1)
    assert not np.isnan(rest).any()


def test_rows_and_weights_of_extreme_size():
    """Through the codec: rows about 1e-23 by weights about 1e-16 and back from large rows, in relative terms as at ordinary sizes."""
    P, N, K = 50, 96, 320
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(P, K, device="cuda", generator=g)
    w = torch.randn(N, K, device="cuda", generator=g)
    for ex, ew in ((-76, -53), (-53, -76), (120, -110), (-110, 120)):
        xs, ws = x * 2.0 ** ex, w * 2.0 ** ew
        q, r = native.quantize_int8(xs)[0], native.quantize_int8(ws)[0]
        for rows in (16, 50):
            y = native.int8_matmul(native.quantize_int8(xs[:rows])[0], r, None, rows, N, K)
            want = (native.dequantize_int8(q, P, K).double()[:rows] @ native.dequantize_int8(r, N, K).double().T)
            # a rounding of each value, 2^-24, and of the product, three: of the sum of the products' magnitudes
            each = native.dequantize_int8(q, P, K).double()[:rows].abs() @ native.dequantize_int8(r, N, K).double().abs().T
            assert ((y.double() - want).abs() <= 5 * 2.0 ** -24 * each + 2.0 ** -149).all()
