"""The int8 codec's every byte at row counts where its blocks make several passes, and the product's sums where fp32
additions would round."""
import numpy as np
import pytest
import torch

import experts_ref as ref
from quantized_routed_expert_softmax_gb300 import native

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_routed_expert_softmax_gb300 import build
    build.build()
    native.lib()


def _coded(x):
    """x [rows, cols] on the GPU -> (codes int8, scales fp32) by the definition, 64-bit quotients rounded to 32."""
    bad = ~torch.isfinite(x).all(-1)
    v = torch.where(bad[:, None], torch.zeros((), dtype=x.dtype, device="cuda"), x).double()
    s = (v.abs().amax(-1) / 127).float()
    t = torch.where((s > 0)[:, None], v / s.double()[:, None], 0.0).float().double()
    q = (torch.sign(t) * torch.floor(t.abs() + 0.5)).clamp(-127, 127).to(torch.int8)
    return q, torch.where(bad, float("nan"), s)


def _check(got, q, s):
    rows, cols = q.shape
    assert got.numel() == ref.bytes_of(rows, cols)
    gs = got[: 4 * rows].view(torch.float32)
    nan = torch.isnan(s)
    assert torch.equal(torch.isnan(gs), nan) and torch.equal(gs[~nan].view(torch.int32), s[~nan].view(torch.int32))
    codes = got[-rows * cols :].view(torch.int8).view(cols // 32, rows, 32)
    wrong = (codes != q.view(rows, cols // 32, 32).transpose(0, 1)).any(-1).any(0).nonzero()
    assert wrong.numel() == 0, wrong[:8].flatten().tolist()


def _rows(rows, cols, dtype, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(rows, cols, device="cuda", generator=g) * torch.exp(torch.randn(rows, 1, device="cuda", generator=g))
    at = torch.randperm(rows, device="cuda", generator=g)
    x[at[:5], 3], x[at[5:9], cols - 1], x[at[9:14]], x[at[14:18]] = float("nan"), float("inf"), 0.0, 1e-40
    x[at[18:40]] = torch.linspace(-127, 127, cols, device="cuda").round() / 2     # middles between two codes
    x[at[18:40], 0] = 127.0
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(32764, 2816), (20001, 704), (20006, 704), (99999, 96), (100000, 160), (31111, 1312),
                                       (6001, 6176), (6006, 6176), (3002, 12320), (2003, 24576), (2005, 65536)])
def test_codec_of_many_rows(rows, cols, dtype):
    """(rows % 8 in 1 .. 4: the panels start 16 bytes off a sector; the columns: each number of steps a lane takes, 1, 2, 4 and 8
    warps a row, rows that are read again.)"""
    x = _rows(rows, cols, dtype, rows + cols)
    _check(native.quantize_int8(x)[0], *_coded(x))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(9, 96), (14, 96), (20001, 704), (20007, 704), (32764, 2816), (2050, 12320), (2055, 12320)])
def test_codec_of_gathered_rows_with_indices_out_of_range(rows, cols, dtype):
    n = 513
    x = _rows(n, cols, dtype, rows)
    idx = torch.randint(-n // 8, n + n // 8, (rows,), device="cuda", generator=torch.Generator("cuda").manual_seed(rows))
    idx[:4] = torch.tensor([-1, n, 2 ** 31 - 1, -2 ** 31], device="cuda")
    inside = (idx >= 0) & (idx < n)
    q, s = _coded(x)
    at = idx.clamp(0, n - 1)
    zero = torch.zeros((), device="cuda")
    _check(native.quantize_int8(x, rows=idx.int())[0], torch.where(inside[:, None], q[at], zero.to(torch.int8)), torch.where(inside, s[at], zero))


def test_codec_of_a_stack_of_many_matrices():
    x = _rows(300 * 45, 736, torch.float32, 5)
    for dtype in (torch.float32, torch.bfloat16):
        got = native.quantize_int8(x.to(dtype).view(300, 45, 736))
        for m in range(300):
            _check(got[m], *_coded(x[45 * m : 45 * m + 45].to(dtype)))


def _product(x, w, sx, sw, dtype=torch.float32):
    xq, wq = (torch.from_numpy(ref.pack(c, np.full(len(c), s, np.float32))[0]).cuda() for c, s in ((x, sx), (w, sw)))
    return native.int8_matmul(xq, wq, None, len(x), len(w), x.shape[1], dtype=dtype).cpu().numpy()


@pytest.mark.parametrize("N", [40, 64])
@pytest.mark.parametrize("P,K", [(1, 65536), (7, 65536), (16, 40992), (9, 8224), (1, 3104), (17, 1024), (200, 1024), (500, 992)])
def test_product_sums_codes_exactly(P, K, N):
    """Up to 16 rows all of K, otherwise up to 1024 columns: the exact sum, rounded once.  Its parts need more than 24 bits, and
    the scales are powers of two, so that a join in fp32 (or a tensor core's shorter sum) would be seen."""
    g = np.random.default_rng(P + K)
    x, w = (g.integers(126, 128, (n, K)).astype(np.int8) for n in (P, N))
    x[:, ::7], w[::2, 3::11] = -125, 1
    total = x.astype(np.int64) @ w.astype(np.int64).T
    if K > 1024:   # (joined in fp32, a thousand columns at a time, some of them would differ)
        joined = np.zeros((P, N), np.float32)
        for c in range(0, K, 1024):
            joined = joined + (x[:, c : c + 1024].astype(np.int64) @ w[:, c : c + 1024].astype(np.int64).T).astype(np.float32)
        assert (joined != total.astype(np.float32)).any()
    got = _product(x, w, 2.0 ** -9, 4.0)
    assert np.array_equal(got, np.ldexp(total.astype(np.float32), -7))
