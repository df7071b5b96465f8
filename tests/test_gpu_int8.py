"""int8 rows with one scale each on the GPU: the codec bit for bit, and the expert product against sums in 64 bits
at the sizes, groupings and values where it can go wrong."""
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


def _host(t):
    return t.float().cpu().numpy()


def _codec_rows(rows, cols, seed, dtype):
    """Random rows, and rows with the values where a codec goes wrong."""
    g = np.random.default_rng(seed)
    x = (g.standard_normal((rows, cols)) * np.exp(g.standard_normal((rows, 1)))).astype(np.float32)
    edge = [np.zeros(cols), np.full(cols, -0.0), np.full(cols, 2.0 ** -149), np.linspace(-1, 1, cols) * 1e-38,
            np.linspace(-1, 1, cols) * 3.3e38, np.resize([127.0, 0.5, -0.5, 1.5, -126.5, 63.5, 0.49999997], cols),
            np.where(np.arange(cols) == cols - 1, np.nan, 1.0), np.where(np.arange(cols) == 0, -np.inf, 1.0),
            np.resize([1.0, -1.0], cols)]
    for i, r in enumerate(g.permutation(rows)[: len(edge)]):
        x[r] = np.asarray(edge[(i + seed) % len(edge)], np.float64).astype(np.float32)
    t = torch.from_numpy(x).cuda()
    return t.to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 2816), (3, 96), (7, 160), (129, 128), (37, 704), (61, 1024), (5, 6176), (2, 65536)])
def test_codec_bit_for_bit(rows, cols, dtype):
    x = _codec_rows(rows, cols, rows * 7 + cols, dtype)
    q, s = ref.quantize(_host(x))
    want, known = ref.pack(q, s)
    got = native.quantize_int8(x)
    assert got.shape == (1, want.size) and native.int8_bytes(rows, cols) == want.size
    gb = got[0].cpu().numpy()
    nan = np.isnan(s)
    assert np.array_equal(np.isnan(gb[: 4 * rows].view("<f4")), nan)       # (which NaN is not said)
    sel = known.copy()
    sel[: 4 * rows] &= ~np.repeat(nan, 4)
    assert np.array_equal(gb[sel], want[sel])
    v = q.astype(np.float32) * s[:, None]
    for out in (torch.float32, torch.bfloat16):
        back = native.dequantize_int8(got[0], rows, cols, dtype=out)
        assert back.dtype == out and np.array_equal(_host(back), _host(torch.from_numpy(v).to(out)), equal_nan=True)


@pytest.mark.parametrize("exponent", [-130, -90, -83, -20, 0, 100, 127])
def test_codec_of_every_bf16_maximum(exponent):
    """A row for each mantissa of its maximum, with all bf16 numbers of both signs in the eleven octaves below it."""
    top = (min(max(exponent + 127, 0), 254) << 7) + np.arange(128, dtype=np.int64)
    bits = np.maximum(top[:, None] - np.arange(11 * 128), 0)
    bits = np.concatenate([bits, bits | 0x8000], 1)
    g = np.random.default_rng(exponent + 200)
    x = torch.from_numpy(g.permuted(bits, axis=1).astype(np.uint16).view(np.int16)).cuda().view(torch.bfloat16)
    want, known = ref.pack(*ref.quantize(_host(x)))
    assert np.array_equal(native.quantize_int8(x)[0].cpu().numpy()[known], want[known])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_codec_finds_what_is_not_finite_wherever_it_is(dtype):
    x = torch.randn(96, 544, device="cuda", generator=torch.Generator("cuda").manual_seed(2)).to(dtype)
    for i, v in enumerate([float("nan"), float("inf"), -float("inf")] * 32):
        x[i, 17 * i % 544 if i % 2 else 543 - i] = v
    x[::6] = -x[::6]        # NaNs of the other sign
    q = native.quantize_int8(x)[0].cpu().numpy()
    assert np.isnan(q[: 4 * 96].view("<f4")).all() and (q[4 * 96 :] == 0).all()


def test_codec_of_a_stack_and_of_gathered_rows():
    x = _codec_rows(30, 96, 3, torch.float32).view(6, 5, 96)
    q = native.quantize_int8(x)
    got = native.dequantize_int8(q, 5, 96).cpu().numpy()
    for m in range(6):
        c, s = ref.quantize(_host(x[m]))
        assert np.array_equal(got[m], c * s[:, None], equal_nan=True)
    rows = torch.tensor([4, 0, 0, -1, 3, 5, 2 ** 31 - 1, -2 ** 31, 1], dtype=torch.int32, device="cuda")
    got = native.dequantize_int8(native.quantize_int8(x[0], rows=rows)[0], 9, 96).cpu().numpy()
    c, s = ref.quantize(_host(x[0]))
    for i, r in enumerate(rows.tolist()):
        assert np.array_equal(got[i], c[r] * s[r] if 0 <= r < 5 else np.zeros(96, np.float32), equal_nan=True), i
    assert native.quantize_int8(torch.empty(0, 96, device="cuda")).numel() == 0


def test_codec_is_the_per_channel_packers():
    w = torch.randn(3, 64, 160, device="cuda", generator=torch.Generator("cuda").manual_seed(4))
    assert torch.equal(native.quantize_int8(w), native.quantize_int8pc(w, "device"))


def test_codec_on_16_byte_aligned_operands():
    rows, cols = 37, 288
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.randn(rows, cols, device="cuda").to(dtype)
        shift = 16 // x.element_size()
        buf = torch.zeros(rows * cols + shift, dtype=dtype, device="cuda")
        xs = buf[shift:].view(rows, cols)
        xs.copy_(x)
        q = native.quantize_int8(xs)
        n = ref.bytes_of(rows, cols)
        ob = torch.full((n + 32,), 7, dtype=torch.uint8, device="cuda")
        native.quantize_int8(xs, out=ob[16 : 16 + n])
        known = torch.from_numpy(ref.pack(*ref.quantize(_host(x)))[1]).cuda()
        assert torch.equal(ob[16 : 16 + n][known], native.quantize_int8(x)[0][known]) and torch.equal(q[0][known], ob[16 : 16 + n][known])
        assert (ob[:16] == 7).all() and (ob[16 + n :] == 7).all()
        o = torch.full((rows * cols + 2 * shift,), 3.0, dtype=dtype, device="cuda")
        native.dequantize_int8(q[0], rows, cols, out=o[shift : shift + rows * cols].view(rows, cols))
        assert torch.equal(o[shift : shift + rows * cols].view(rows, cols), native.dequantize_int8(q[0], rows, cols, dtype=dtype))
        assert (o[:shift] == 3).all() and (o[shift + rows * cols :] == 3).all()


def test_codec_past_32_bit_offsets():
    rows, cols = 1_050_000, 2112        # 2.2e9 values
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    q = native.quantize_int8(x)
    got = native.dequantize_int8(q[0], rows, cols, dtype=torch.bfloat16)
    for r in (0, 1, rows // 2, rows - 2, rows - 1):
        c, s = ref.quantize(_host(x[r : r + 1]))
        assert np.array_equal(_host(got[r]), _host(torch.from_numpy(c[0] * s).bfloat16())), r
    del x, q, got
    torch.cuda.empty_cache()


# ---------------------------------------------------------------------------------------- product
def _matrix(g, n, rows, cols, full=False):
    """n random int8 matrices: (bytes uint8 [n, ...], codes int8 [n, rows, cols], scales fp32 [n, rows])."""
    c = g.integers(-127, 128, (n, rows, cols)).astype(np.int8)
    if full:
        c[:] = 127
    s = (np.exp(g.standard_normal((n, rows))) * 0.01).astype(np.float32)
    b = np.stack([ref.pack(c[i], s[i])[0] for i in range(n)])
    return torch.from_numpy(b).cuda(), torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda()


def _check(P, E, N, K, counts, act, dtype, seed=0, full=False, before=0):
    g = np.random.default_rng(seed)
    xq, xc, xs = _matrix(g, 1, P, K, full)
    wq, wc, ws = _matrix(g, E, N, K, full)
    off = None
    if counts is not None:
        off = torch.tensor(np.concatenate([[before], before + np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    width = N // 2 if act == "swiglu" else N
    out = torch.full((P, width), 5.5, dtype=dtype, device="cuda")
    work = native.int8_workspace()
    native.int8_matmul(xq[0], wq, off, P, N, K, act=act, out=out, workspace=work)
    assert native.device_status(work) == 0
    want = torch.full((P, width), 5.5, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(want)
    for e, a, b in ref.spans(off, P, E):
        z = (xc[0, a:b].double() @ wc[e].double().T) * xs[0, a:b, None].double() * ws[e].double()
        y = ref.activate(z, act)
        # z: the sums of 1024 columns are exact, joining c of them rounds c - 1 times, the conversion and the two
        # scales (multiplied with one another first) three times, all within the sum of the codes' magnitudes
        c = (K + 1023) // 1024
        bz = (c + 3) * 2.0 ** -24 * (xc[0, a:b].double().abs() @ wc[e].double().abs().T) * xs[0, a:b, None].double() * ws[e].double()
        if c == 1:
            bz = 3 * 2.0 ** -24 * z.abs()
        if act == "swiglu":
            f = N // 2
            zg, zu, bg, bu = z[:, :f], z[:, f:], bz[:, :f], bz[:, f:]
            silu = zg * torch.sigmoid(zg)
            t = (1.1 * bg + (2.0 ** -20 + zg.abs().clamp(max=128) * 2.0 ** -22) * silu.abs() + 2.0 ** -120) * (zu.abs() + bu) + silu.abs() * bu
        elif act == "relu2":
            t = (2 * torch.relu(z) + bz) * bz + 2.0 ** -23 * y
        else:
            t = bz
        t = t + (torch.finfo(dtype).eps / 2) * (y.abs() + t)
        want[a:b], tol[a:b] = y, t
    err = (out.double() - want).abs()
    assert torch.isfinite(out).all()
    assert (err <= tol).all(), (err - tol).max().item()
    return out


@pytest.mark.parametrize("act,dtype", [("none", torch.float32), ("none", torch.bfloat16), ("swiglu", torch.bfloat16),
                                       ("swiglu", torch.float32), ("relu2", torch.float32), ("relu2", torch.bfloat16)])
@pytest.mark.parametrize("counts,N,K", [
    ([1], 64, 32), ([1, 0, 0, 2], 128, 64), ([5, 0, 1, 9], 192, 96), ([0, 16], 64, 2848), ([11, 5], 128, 4128), ([9, 0, 7, 1], 128, 96), ([0, 0, 3], 64, 704), ([17, 33, 0, 64, 130], 320, 160),
    ([128, 127, 129, 1], 256, 1024), ([300, 0, 70], 192, 1056), ([257, 256, 255], 64, 2816), ([1] * 40, 128, 2816), ([8] * 20, 64, 2080),
    ([400, 150, 0, 290], 320, 1024), ([193], 64, 96), ([389, 0, 160, 2], 128, 704), ([161, 224], 576, 32)])
def test_product(counts, N, K, act, dtype):
    _check(sum(counts), len(counts), N, K, counts, act, dtype, seed=N + K)


@pytest.mark.parametrize("N", [1, 7, 31, 33, 127, 129, 261])
@pytest.mark.parametrize("P", [1, 3, 16, 17, 40, 300])
def test_product_odd_widths(P, N):
    _check(P, 1, N, 224, None, "none", torch.float32, seed=P + N)
    _check(P, 1, N, 224, None, "relu2", torch.bfloat16, seed=P + N + 1)


@pytest.mark.parametrize("act,dtype", [("none", torch.bfloat16), ("none", torch.float32), ("swiglu", torch.bfloat16),
                                       ("swiglu", torch.float32), ("relu2", torch.bfloat16), ("relu2", torch.float32)])
@pytest.mark.parametrize("most,E,K", [(700, 24, 704), (700, 24, 1056), (160, 40, 96), (60, 60, 224)])
def test_product_of_more_tiles_than_pairs(most, E, K, act, dtype):
    """(Fewer are cut lower: these take tiles of 192, 128, 128 and 64 rows at most.)"""
    counts = [int(n) for n in np.random.default_rng(most + K).integers(0, most, E)]
    _check(sum(counts), E, 1088, K, counts, act, dtype, seed=K)


@pytest.mark.parametrize("P", [64, 96, 129, 700, 4097])
def test_product_of_one_matrix_in_low_tiles(P):
    _check(P, 1, 584, 736, None, "none", torch.float32, seed=P)
    _check(P, 1, 320, 1088, None, "swiglu", torch.bfloat16, seed=P + 1)


@pytest.mark.parametrize("P", [2, 100])
def test_product_of_the_largest_codes_is_exact_by_integers(P):
    # every product 127 * 127 at K = 65536: 1.06e9, far past 24 bits
    _check(P, 1, 64, 65536, None, "none", torch.float32, full=True)


def test_rows_no_expert_owns_are_left():
    out = _check(200, 3, 64, 96, [20, 0, 31], "none", torch.float32, before=9)
    assert (out[:9] == 5.5).all() and (out[60:] == 5.5).all()


def test_absurd_offsets_stay_in_the_buffers():
    P, E, N, K = 50, 4, 64, 64
    g = np.random.default_rng(1)
    xq, wq = _matrix(g, 1, P, K)[0], _matrix(g, E, N, K)[0]
    pad = torch.full((P + 64, N), 2.5, device="cuda")
    for off in ([0, 2 ** 31 - 1, -5, 7, 3], [-2 ** 31, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, 0], [60, 55, 50, 70, 99]):
        o = torch.tensor(off, dtype=torch.int32, device="cuda")
        work = native.int8_workspace()
        native.int8_matmul(xq[0], wq, o, P, N, K, out=pad[32 : 32 + P], workspace=work)
        assert native.device_status(work) == 0
        assert (pad[:32] == 2.5).all() and (pad[32 + P :] == 2.5).all()


def test_nan_rows_stay_their_own():
    x = torch.randn(70, 320, device="cuda")
    x[5, 3], x[40] = float("nan"), float("inf")
    q = native.quantize_int8(x)[0]
    w = native.quantize_int8(torch.randn(2, 64, 320, device="cuda"))
    off = torch.tensor([0, 33, 70], dtype=torch.int32, device="cuda")
    for act in ("none", "swiglu", "relu2"):
        y = native.int8_matmul(q, w, off, 70, 64, 320, act=act)
        bad = torch.zeros(70, dtype=torch.bool, device="cuda")
        bad[5] = bad[40] = True
        assert torch.isnan(y[bad]).all() and torch.isfinite(y[~bad]).all()


def test_same_bits_on_two_streams_and_in_a_graph():
    g = np.random.default_rng(2)
    counts = [3, 0, 50, 200]
    P, N, K = sum(counts), 192, 1056
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    xq, wq = _matrix(g, 1, P, K)[0], _matrix(g, 4, N, K)[0]
    work = native.int8_workspace()
    ref_out = native.int8_matmul(xq[0], wq, off, P, N, K, act="swiglu", workspace=work)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [native.int8_matmul(xq[0], wq, off, P, N, K, act="swiglu", workspace=work, stream=s) for s in streams for _ in range(5)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref_out) for o in outs)
    out = torch.empty_like(ref_out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q = native.quantize_int8(native.dequantize_int8(xq[0], P, K))
        native.int8_matmul(xq[0], wq, off, P, N, K, act="swiglu", out=out, workspace=work)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref_out)
    assert q.numel() == native.int8_bytes(P, K)
    assert native.device_status(work) == 0
