"""MXFP4 on the GPU against its restatement in 64 bits: the codec bit for bit, the expert product at
the sizes and groupings where it can go wrong, and both behind the router as a layer uses them."""
import numpy as np
import pytest
import torch

import mxfp4_ref as ref
from quantized_routed_expert_softmax_gb300 import native

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_routed_expert_softmax_gb300 import build
    build.build()
    native.lib()


def _codec_rows(rows, cols, seed, dtype):
    """Random rows, and blocks with the values where a codec goes wrong."""
    g = np.random.default_rng(seed)
    x = (g.standard_normal((rows, cols)) * np.exp(g.standard_normal((rows, 1)))).astype(np.float32)
    edge = np.zeros((12, 32), np.float32)
    edge[1, 0] = np.float32(2.0 ** -149)                       # the smallest subnormal
    edge[2] = np.linspace(-1, 1, 32) * np.float32(1e-38)       # around the smallest scale
    edge[3] = np.linspace(-1, 1, 32) * np.float32(3.3e38)      # the largest binades
    edge[4, :16] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 6.5, 7.9, -0.25, -0.75, -5.0, -7.0, 4.0, -4.0]
    edge[5, :3] = [np.nan, 1.0, -2.0]
    edge[6, :3] = [np.inf, 1.0, -2.0]
    edge[7, 31] = -np.inf
    edge[8] = -0.0
    edge[9] = np.nextafter(np.float32(5.0), np.float32(6.0))
    edge[10, :2] = [4.0, np.nextafter(np.float32(0.25), np.float32(1))]
    edge[11] = np.float32(2.0) ** np.arange(-16, 16)
    n = min(12, rows * cols // 32)
    x.reshape(-1, 32)[:n] = edge[g.permutation(12)[:n]] if n < 12 else edge
    t = torch.from_numpy(x).cuda()
    if dtype == torch.bfloat16:
        t = t.to(torch.bfloat16)
    return t


def _host(t):
    return t.float().cpu().numpy()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 2816), (3, 96), (7, 160), (129, 128), (37, 704), (50, 1024)])
def test_codec_bit_for_bit(rows, cols, dtype):
    x = _codec_rows(rows, cols, rows * 7 + cols, dtype)
    c, s = ref.quantize(_host(x))
    want, end = ref.pack(c, s)
    q = native.quantize_mxfp4(x)
    assert q.shape == (1, want.size)
    assert np.array_equal(q[0].cpu().numpy()[:end], want[:end])
    v = ref.values(c, s)
    for out in (torch.float32, torch.bfloat16):
        got = native.dequantize_mxfp4(q[0], rows, cols, dtype=out)
        assert got.dtype == out and np.array_equal(_host(got), v.astype(np.float32), equal_nan=True)


def test_codec_of_a_stack_and_of_gathered_rows():
    x = _codec_rows(6, 5 * 96, 3, torch.float32).view(6, 5, 96)
    q = native.quantize_mxfp4(x)
    got = native.dequantize_mxfp4(q, 5, 96).cpu().numpy()
    for m in range(6):
        assert np.array_equal(got[m], ref.values(*ref.quantize(_host(x[m]))).astype(np.float32), equal_nan=True)
    # rows in any order, repeated, and indices that name no row
    rows = torch.tensor([4, 0, 0, -1, 3, 5, 2 ** 31 - 1, -2 ** 31, 1], dtype=torch.int32, device="cuda")
    got = native.dequantize_mxfp4(native.quantize_mxfp4(x[0], rows=rows)[0], 9, 96).cpu().numpy()
    plain = ref.values(*ref.quantize(_host(x[0]))).astype(np.float32)
    for i, r in enumerate(rows.tolist()):
        assert np.array_equal(got[i], plain[r] if 0 <= r < 5 else np.zeros(96, np.float32), equal_nan=True), i
    # nothing to do
    assert native.quantize_mxfp4(torch.empty(0, 96, device="cuda")).numel() == 0


def test_codec_on_16_byte_aligned_operands():
    # rows and results that start 16 bytes into their buffers (the 32-byte accesses do not apply)
    rows, cols = 37, 288
    for dtype in (torch.float32, torch.bfloat16):
        x = _codec_rows(rows, cols, 5, dtype)
        shift = 16 // x.element_size()
        buf = torch.zeros(rows * cols + shift, dtype=dtype, device="cuda")
        xs = buf[shift:].view(rows, cols)
        xs.copy_(x)
        assert xs.data_ptr() % 32 == 16
        q = native.quantize_mxfp4(xs)
        end = ref.pack(*ref.quantize(_host(x)))[1]
        assert torch.equal(q[:, :end], native.quantize_mxfp4(x)[:, :end])
        o = torch.full((rows * cols + 2 * shift,), 3.0, dtype=dtype, device="cuda")
        native.dequantize_mxfp4(q[0], rows, cols, out=o[shift : shift + rows * cols].view(rows, cols))
        v = ref.values(*ref.quantize(_host(x))).astype(np.float32)
        assert np.array_equal(_host(o[shift : shift + rows * cols]).reshape(rows, cols), v, equal_nan=True)
        assert (o[:shift] == 3).all() and (o[shift + rows * cols :] == 3).all()


def test_codec_past_32_bit_offsets():
    rows, cols = 1_050_000, 2112        # 2.2e9 values
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    q = native.quantize_mxfp4(x)
    got = native.dequantize_mxfp4(q[0], rows, cols, dtype=torch.bfloat16)
    for r in (0, 1, rows // 2, rows - 2, rows - 1):
        assert np.array_equal(_host(got[r]), ref.values(*ref.quantize(_host(x[r : r + 1])))[0].astype(np.float32)), r
    del x, q, got
    torch.cuda.empty_cache()


# ------------------------------------------------------------------------------------- the product


def _coded(rows, cols, seed, scale=1.0):
    x = scale * torch.randn(rows, cols, generator=torch.Generator().manual_seed(seed))
    q = native.quantize_mxfp4(x.cuda())[0]
    return q, native.dequantize_mxfp4(q, rows, cols).double()


def _stack(E, N, K, seed, scale):
    q, v = zip(*[_coded(N, K, seed + e, scale) for e in range(E)])
    return torch.stack(q), torch.stack(v)


def _want(xv, wv, offsets, act):
    """The product in 64 bits and the error its 32-bit sums may make.

    A 32-bit sum of K/64 partial sums that each hold 64 exact products loses at most one unit of its
    last place, 2^-23 of a magnitude of at most A = sum |x w|, an addition (a truncating adder; a
    rounding one half of it); two more for the partial sum itself.  SwiGLU: silu' is below 1.1 and the
    fp32 steps of silu(g) u are a few 2^-24 of it, 8 taken; ReLU^2: the square's derivative is 2 z."""
    P, K = xv.shape
    E, N, _ = wv.shape
    z = torch.zeros(P, N, dtype=torch.float64, device="cuda")
    A = torch.zeros(P, N, dtype=torch.float64, device="cuda")
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        z[a:b] = xv[a:b] @ wv[e].T
        A[a:b] = xv[a:b].abs() @ wv[e].abs().T
    ez = (K / 64 + 2) * 2.0 ** -23 * A
    if act == "swiglu":
        g, u, eg, eu = z[:, : N // 2], z[:, N // 2 :], ez[:, : N // 2], ez[:, N // 2 :]
        sg = g * torch.sigmoid(g)
        return sg * u, 1.1 * eg * (u.abs() + eu) + sg.abs() * eu + 8 * 2.0 ** -24 * (sg * u).abs()
    if act == "relu2":
        r = z.clamp(min=0)
        return r * r, 2 * r * ez + ez * ez + 2.0 ** -24 * r * r
    return z, ez


def _check(out, want, err):
    half = 0.0 if out.dtype == torch.float32 else 2.0 ** -8       # one rounding to bf16
    diff = (out.double() - want).abs()
    bound = err + half * (want.abs() + err) + 1e-40
    assert torch.isfinite(out).all()
    assert (diff <= bound).all(), float((diff / bound).max())


def _case(counts, K, N, act, dtype, seed=0, first=0, behind=0):
    """Groups of `counts` rows, `first` rows before them and `behind` rows after them."""
    E = len(counts)
    off = np.concatenate([[0], np.cumsum(counts)]) + first
    P = int(off[-1]) + behind
    xq, xv = _coded(P, K, seed, 1.0)
    wq, wv = _stack(E, N, K, seed + 100, K ** -0.5)
    width = N // 2 if act == "swiglu" else N
    out = torch.full((P, width), -77.0, dtype=dtype, device="cuda")
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    ws = native.mxfp4_workspace()
    native.mxfp4_matmul(xq, wq, offsets, P, N, K, act=act, out=out, workspace=ws)
    assert native.device_status(ws) == 0
    want, err = _want(xv, wv, off.tolist(), act)
    a, b = int(off[0]), int(off[-1])
    _check(out[a:b], want[a:b], err[a:b])
    assert (out[:a] == -77).all() and (out[b:] == -77).all()      # rows of no expert are left as they were
    return xq, wq, offsets, P, out


SHAPES = [  # K, N
    (32, 64), (64, 128), (96, 192), (160, 64), (256, 320), (288, 128), (512, 256), (704, 2816), (2816, 1408),
]
GROUPS = [[1], [0, 1, 0], [3, 0, 0, 17, 1], [16, 33, 64, 0, 7], [128, 129], [200, 0, 5, 300], [193, 0, 400], [577], [33, 64, 1, 0, 31, 32, 2, 0, 0, 70, 16, 15, 17, 4, 4, 4] + [2] * 20]


@pytest.mark.parametrize("act", ["none", "swiglu", "relu2"])
@pytest.mark.parametrize("K,N", SHAPES)
@pytest.mark.parametrize("groups", [[1], [3, 0, 0, 17, 1], [130, 5]])
def test_product_shapes(K, N, act, groups):
    _case(groups, K, N, act, torch.float32, seed=K + N)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("groups", GROUPS)
def test_product_groups(groups, act, dtype):
    _case(groups, 288, 192, act, dtype, seed=len(groups), first=3, behind=2)


@pytest.mark.parametrize("N", [1, 7, 17, 127, 130, 257])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_product_odd_widths(N, dtype):
    for act in ("none", "relu2"):
        _case([5, 0, 40], 96, N, act, dtype, seed=N)


def test_product_many_experts():
    g = np.random.default_rng(5)
    _case(g.integers(0, 4, 512).tolist(), 64, 64, "relu2", torch.bfloat16)
    _case((g.random(1024) < 0.1).astype(int).tolist(), 32, 128, "none", torch.float32)


@pytest.mark.parametrize("P,N,K", [(2, 8, 65536), (3, 131072, 32), (20, 64, 8192 + 96)])
def test_product_largest_dimensions(P, N, K):
    xq, xv = _coded(P, K, P)
    wq, wv = _coded(N, K, 9, K ** -0.5)
    out = native.mxfp4_matmul(xq, wq, None, P, N, K)
    want, err = _want(xv, wv[None], [0, P], "none")
    _check(out, want, err)


def test_product_from_two_streams_at_once():
    # overlapping calls with one error word, their outputs offset by 16 bytes in their buffers
    groups, K, N = [40, 0, 300, 7], 704, 256
    cases = [_case(groups, K, N, "none", torch.bfloat16, seed=s) for s in (1, 2)]
    ws = native.mxfp4_workspace()
    streams = [torch.cuda.Stream() for _ in cases]
    P = cases[0][3]
    outs = [[torch.zeros(P * N + 8, dtype=torch.bfloat16, device="cuda")[8:].view(P, N) for _ in range(6)] for _ in cases]
    torch.cuda.synchronize()
    for k in range(6):
        for c, s, o in zip(cases, streams, outs):
            native.mxfp4_matmul(c[0], c[1], c[2], P, N, K, out=o[k], workspace=ws, stream=s)
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        assert all(torch.equal(x, c[4]) for x in o)
    assert native.device_status(ws) == 0


def test_product_one_matrix_without_offsets():
    for P in (1, 31, 300):
        xq, xv = _coded(P, 224, P)
        wq, wv = _coded(200, 224, 9)
        out = native.mxfp4_matmul(xq, wq, None, P, 200, 224)
        want, err = _want(xv, wv[None], [0, P], "none")
        _check(out, want, err)


def test_product_scales_far_apart_and_nan():
    # products of large and small scales: 2^60 * 2^-60, and a block of NaN poisons its own row only
    K, N, P = 128, 64, 20
    x = torch.randn(P, K, generator=torch.Generator().manual_seed(1))
    w = torch.randn(N, K, generator=torch.Generator().manual_seed(2))
    for up in (0, 60, 110):
        xq = native.quantize_mxfp4((x * 2.0 ** up).cuda())[0]
        wq = native.quantize_mxfp4((w * 2.0 ** -up).cuda())[0]
        xv, wv = native.dequantize_mxfp4(xq, P, K).double(), native.dequantize_mxfp4(wq, N, K).double()
        want, err = _want(xv, wv[None], [0, P], "none")
        _check(native.mxfp4_matmul(xq, wq, None, P, N, K), want, err)
    x[3, 40] = float("nan")
    x[7, 100] = float("inf")
    out = native.mxfp4_matmul(native.quantize_mxfp4(x.cuda())[0], native.quantize_mxfp4(w.cuda())[0], None, P, N, K)
    bad = torch.isnan(out).all(1).cpu()
    assert bad.nonzero().flatten().tolist() == [3, 7] and torch.isfinite(out[~bad.cuda()]).all()


def test_product_offsets_are_clamped():
    # reversed ranges are empty, and no offset reaches outside the rows
    P, N, K = 40, 64, 64
    xq, xv = _coded(P, K, 1)
    wq, wv = _stack(4, N, K, 50, 0.1)
    off = torch.tensor([-5, 10, 4, 20, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    out = torch.full((P, N), -77.0, device="cuda")
    native.mxfp4_matmul(xq, wq, off, P, N, K, out=out)
    # expert 0: [0, 10); 1: [10, 4) empty; 2: [4, 20); 3: [20, 40) -- rows 4 .. 9 have two experts
    for e, a, b in ((0, 0, 4), (2, 10, 20), (3, 20, 40)):
        want, err = _want(xv[a:b], wv[e : e + 1], [0, b - a], "none")
        _check(out[a:b], want, err)
    off = torch.zeros(5, dtype=torch.int32, device="cuda")        # no rows at all
    out.fill_(-77.0)
    native.mxfp4_matmul(xq, wq, off, P, N, K, out=out)
    assert (out == -77).all()


def test_product_past_32_bit_offsets():
    P, N, K = 1_600_000, 1408, 32          # 2.25e9 outputs
    xq, _ = _coded(4096, K, 3)
    x = torch.randn(P, K, device="cuda", generator=torch.Generator("cuda").manual_seed(4))
    xq = native.quantize_mxfp4(x)[0]
    wq, wv = _stack(2, N, K, 7, 0.2)
    off = [0, 900_001, P]
    out = native.mxfp4_matmul(xq, wq, torch.tensor(off, dtype=torch.int32, device="cuda"), P, N, K, dtype=torch.bfloat16)
    xv = native.dequantize_mxfp4(xq, P, K)
    for e, a, b in ((0, 0, 50), (0, 899_970, 900_001), (1, 900_001, 900_040), (1, P - 33, P)):
        want, err = _want(xv[a:b].double(), wv[e : e + 1], [0, b - a], "none")
        _check(out[a:b], want, err)
    del x, xv, out
    torch.cuda.empty_cache()


def test_product_same_bits_on_another_stream_and_in_a_graph():
    xq, wq, offsets, P, out = _case([5, 0, 70, 1], 704, 256, "swiglu", torch.float32)
    ws = native.mxfp4_workspace()
    again = torch.empty_like(out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    native.mxfp4_matmul(xq, wq, offsets, P, 256, 704, act="swiglu", out=again, workspace=ws, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, again)
    # captured once, replayed on new rows: the quantiser and the product together
    x = torch.randn(P, 704, device="cuda", generator=torch.Generator("cuda").manual_seed(8))
    q = torch.empty_like(xq)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        native.quantize_mxfp4(x, out=q.view(1, -1))
        native.mxfp4_matmul(q, wq, offsets, P, 256, 704, act="swiglu", out=again, workspace=ws)
    for k in range(3):
        x.copy_(torch.randn(P, 704, device="cuda", generator=torch.Generator("cuda").manual_seed(20 + k)))
        again.zero_()
        g.replay()
        eager = native.mxfp4_matmul(native.quantize_mxfp4(x)[0], wq, offsets, P, 256, 704, act="swiglu")
        assert torch.equal(again, eager)
    assert native.device_status(ws) == 0


def test_binding_checks_its_operands():
    xq, wq, offsets, P, out = _case([4, 4], 64, 64, "none", torch.float32)
    with pytest.raises(ValueError):
        native.mxfp4_matmul(xq[:-16], wq, offsets, P, 64, 64)
    with pytest.raises(TypeError):
        native.mxfp4_matmul(xq, wq, offsets.long(), P, 64, 64)
    with pytest.raises(ValueError):
        native.mxfp4_matmul(xq, wq, offsets[:-1], P, 64, 64)
    with pytest.raises(ValueError):
        native.mxfp4_matmul(xq, wq, offsets, P, 64, 64, out=out.t())
    with pytest.raises(native.MoeError):
        native.mxfp4_matmul(xq, wq, offsets, P, 64, 64, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        native.quantize_mxfp4(torch.zeros(64, 64, device="cuda").t())


def test_router_to_experts_run():
    """Router, balance loss, rows sorted by expert, gate.up, down and the weighted sum, as a layer."""
    T, d, f, E, k = 45, 256, 96, 16, 4
    g = torch.Generator("cuda").manual_seed(11)
    x = torch.randn(T, d, device="cuda", generator=g)
    W = 0.1 * torch.randn(d, E, device="cuda", generator=g)
    idx, w, logits = native.router_topk(x, W, k, return_logits=True)
    loss, counts, prob, tokens = native.balance_loss(logits, idx)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts[0].cumsum(0)
    order = torch.sort(idx.reshape(-1), stable=True).indices
    rows = (order // k).int()
    wgu, vgu = _stack(E, 2 * f, d, 300, d ** -0.5)
    wdn, vdn = _stack(E, d, f, 500, f ** -0.5)
    P = T * k
    xq = native.quantize_mxfp4(x, rows=rows)[0]
    h = native.mxfp4_matmul(xq, wgu, offsets, P, 2 * f, d, act="swiglu")
    want, err = _want(native.dequantize_mxfp4(xq, P, d).double(), vgu, offsets.tolist(), "swiglu")
    _check(h, want, err)
    hq = native.quantize_mxfp4(h)[0]
    y = native.mxfp4_matmul(hq, wdn, offsets, P, d, f)
    want, err = _want(native.dequantize_mxfp4(hq, P, f).double(), vdn, offsets.tolist(), "none")
    _check(y, want, err)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(P, device="cuda")
    out = (y[pos].view(T, k, d) * w.unsqueeze(-1)).sum(1)
    full = (want[pos].view(T, k, d) * w.double().unsqueeze(-1)).sum(1)
    assert (out.double() - full).abs().max() <= 1e-5 * full.abs().max()   # k = 4 terms, each within err and 2^-22
    lref = ref.balance(logits.cpu().numpy(), idx.cpu().numpy(), None, 1)
    assert np.array_equal(counts.cpu().numpy(), lref[1]) and abs(float(loss) - lref[0]) <= 1e-6 * lref[0]
