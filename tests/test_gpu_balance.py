"""The router balance loss, its counts and its gradient on the GPU against the definition in 64 bits."""
import numpy as np
import pytest
import torch

import mxfp4_ref as ref
from quantized_routed_expert_softmax_gb300 import native

pytestmark = pytest.mark.gpu

# p = exp(x - m) / sum: the difference, exp, the sum over at most 32 values a lane and 5 levels, the
# division and the product make at most about 48 roundings of 2^-24 (exp's own included) of p, which
# cancel in part; a mean over tokens adds fp32 sums of at most 2^8 terms, half an ulp each in the
# worst case.  Taken: 2^-18 relative for p-like values.  |x - m| <= 30 here: the subtraction's
# rounding, 2^-24 * 30, is inside it.
REL = 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_routed_expert_softmax_gb300 import build
    build.build()
    native.lib()


def _inputs(S, L, E, k, dtype, seed, pad=0.5):
    g = np.random.default_rng(seed)
    logits = torch.from_numpy((1.5 * g.standard_normal((S * L, E)) + g.standard_normal((1, E))).astype(np.float32))
    logits = logits.cuda().to(dtype)
    idx = logits.float().topk(k, dim=1).indices.int()
    mask = torch.from_numpy(g.random(S * L) >= pad).cuda() if pad else None
    return logits, idx, mask


def _check(logits, idx, mask, S, g=0.7):
    loss, counts, prob, tokens = native.balance_loss(logits, idx, mask=mask, n_seq=S)
    grad = native.balance_loss_backward(logits, counts, tokens, torch.full((1,), g, device="cuda"), idx.shape[1], mask=mask)
    want = ref.balance(logits.float().cpu().numpy(), idx.cpu().numpy(),
                       None if mask is None else mask.cpu().numpy(), S)
    assert np.array_equal(counts.cpu().numpy(), want[1])
    assert np.array_equal(tokens.cpu().numpy(), want[3])
    assert abs(float(loss) - want[0]) <= REL * abs(want[0])
    np.testing.assert_allclose(prob.cpu().numpy(), want[2], rtol=REL, atol=1e-37)
    d = g * want[4]
    # the bracket f_e - sum f p is a sum of |f - 1/E| p terms: its error is relative to the largest
    # of the row's |f_e - sum f p|, not to the one it lands on
    T, E = logits.shape
    k, n = idx.shape[1], np.maximum(want[3], 1)
    f = want[1] / (k * n[:, None])
    live = max(1, int((want[3] > 0).sum()))
    p = np.zeros((T, E))
    x = logits.float().cpu().numpy().astype(np.float64)
    with np.errstate(invalid="ignore"):
        m = x.max(1, keepdims=True)
        e = np.exp(x - np.where(np.isfinite(m), m, 0))
        p = e / np.maximum(e.sum(1, keepdims=True), 1e-300)
    spread = np.repeat((np.abs(f - 1 / E).max(1) * 2 * g * E / (live * n)), T // S)[:, None]
    tol = REL * 2 * p * spread + 1e-37
    # the 64-bit reference takes f - sum f p as it stands: E products and additions of at most max f, half a
    # unit of 2^-52 each, which is all there is to it where every f is the same (k = E)
    tol = tol + np.repeat((E + 4) * 2.0 ** -53 * f.max(1) * g * E / (live * n), T // S)[:, None] * p
    if logits.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(d) + tol)
    got = grad.float().cpu().numpy().astype(np.float64)
    assert grad.dtype == logits.dtype
    bad = np.abs(got - d) > tol
    assert not bad.any(), (np.abs(got - d) / tol).max()
    if mask is not None:
        assert (grad[~mask] == 0).all()
    return loss, counts, prob, tokens, grad


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("S,L,E,k", [(1, 1, 1, 1), (1, 1, 8, 2), (1, 16, 8, 2), (3, 7, 33, 5), (2, 65, 60, 4), (1, 129, 128, 8),
                                     (5, 40, 257, 6), (2, 33, 512, 22), (2, 20, 1024, 32), (70, 1, 16, 2), (1, 300, 64, 1), (3, 21, 16, 16), (2, 17, 32, 4), (2, 40, 200, 8),
                                     (2, 30, 321, 6), (1, 20, 513, 9), (2, 50, 256, 8), (9, 11, 4, 4)])
def test_against_definition(S, L, E, k, dtype):
    _check(*_inputs(S, L, E, k, dtype, S * L + E), S)
    _check(*_inputs(S, L, E, k, dtype, S * L + E + 1, pad=0), S)


def test_masks_that_leave_nothing():
    logits, idx, mask = _inputs(4, 30, 32, 4, torch.float32, 1)
    m = mask.view(4, 30).clone()
    m[1] = False                                  # a sequence of padding only
    m[2] = False
    m[2, 17] = True                               # and one of a single token
    out = _check(logits, idx, m.view(-1), 4)
    assert out[3].tolist()[1:3] == [0, 1] and (out[2][1] == 0).all()
    # what masked tokens hold is not looked at
    dirty, didx = logits.clone(), idx.clone()
    dirty[~m.view(-1)] = float("nan")
    didx[~m.view(-1)] = 12345678
    loss, counts, prob, tokens = native.balance_loss(dirty, didx, mask=m.view(-1), n_seq=4)
    assert torch.equal(loss, out[0]) and torch.equal(counts, out[1]) and torch.equal(prob, out[2])
    grad = native.balance_loss_backward(dirty, counts, tokens, torch.full((1,), 0.7, device="cuda"), 4, mask=m.view(-1))
    assert torch.equal(grad, out[4])
    none = torch.zeros(120, dtype=torch.uint8, device="cuda")
    loss, counts, prob, tokens = native.balance_loss(logits, idx, mask=none, n_seq=4)
    assert float(loss) == 0 and int(counts.sum()) == 0 and float(prob.sum()) == 0 and int(tokens.sum()) == 0
    assert (native.balance_loss_backward(logits, counts, tokens, torch.ones(1, device="cuda"), 4, mask=none) == 0).all()


def test_dropped_slots_repeats_and_masked_experts():
    logits, idx, mask = _inputs(2, 50, 24, 6, torch.float32, 3)
    idx[::3, 2:] = -1                             # dropped by a capacity limit
    idx[1::5, :3] = 7                             # the same expert more than once
    idx[2, 0] = 24                                # the first index past the experts
    logits[:, 5] = -float("inf")                  # an expert that no token may take
    logits[4] = torch.finfo(torch.float32).min    # a row of the lowest value: uniform
    _check(logits, idx, mask, 2)
    # a row of -inf has no probability and no gradient
    full = torch.ones(100, dtype=torch.bool, device="cuda")
    logits[6] = -float("inf")
    out = _check(logits, idx, full, 2)
    assert (out[4][6] == 0).all() and torch.isfinite(out[0]).all()
    # a NaN that counts is not hidden
    logits[8, 3] = float("nan")
    loss, counts, prob, tokens = native.balance_loss(logits, idx, mask=full, n_seq=2)
    assert torch.isnan(loss).all() and torch.isnan(prob[0]).all() and torch.isfinite(prob[1]).all()
    grad = native.balance_loss_backward(logits, counts, tokens, torch.ones(1, device="cuda"), 6, mask=full)
    assert torch.isnan(grad[8]).all() and torch.isfinite(grad[:8]).all() and torch.isfinite(grad[9:]).all()


def test_gradient_against_differences():
    logits, idx, mask = _inputs(2, 6, 12, 3, torch.float32, 9, pad=0.3)
    loss, counts, prob, tokens = native.balance_loss(logits, idx, mask=mask, n_seq=2)
    grad = native.balance_loss_backward(logits, counts, tokens, torch.ones(1, device="cuda"), 3, mask=mask).cpu().numpy()
    x, i, m = logits.cpu().numpy().astype(np.float64), idx.cpu().numpy(), mask.cpu().numpy()
    h = 1e-4   # central differences: h^2 times a third derivative below 1, and 1e-16 / h of rounding
    for t in range(12):
        for e in range(12):
            d = np.zeros_like(x)
            d[t, e] = h
            diff = (ref.balance(x + d, i, m, 2)[0] - ref.balance(x - d, i, m, 2)[0]) / (2 * h)
            assert abs(grad[t, e] - diff) <= 1e-7 + 1e-4 * abs(diff)


@pytest.mark.parametrize("S,L,E,k,dtype", [(3, 20011, 128, 8, torch.bfloat16), (16, 4096, 512, 22, torch.float32),
                                           (1, 1 << 20, 8, 2, torch.float32), (40000, 3, 12, 5, torch.float32)])
def test_long_batches(S, L, E, k, dtype):
    g = torch.Generator("cuda").manual_seed(E)
    logits = torch.randn(S * L, E, device="cuda", generator=g).to(dtype)
    idx = logits.float().topk(k, dim=1).indices.int()
    mask = torch.rand(S * L, device="cuda", generator=g) < 0.8
    loss, counts, prob, tokens = native.balance_loss(logits, idx, mask=mask, n_seq=S)
    again = native.balance_loss(logits, idx, mask=mask, n_seq=S)
    assert all(torch.equal(a, b) for a, b in zip((loss, counts, prob, tokens), again))
    p = torch.softmax(logits.double(), 1) * mask.unsqueeze(1)
    n = mask.view(S, L).sum(1)
    assert torch.equal(tokens, n.int())
    live, n = int((n > 0).sum()), n.clamp(min=1)
    for s in range(0, S, max(1, S // 50)):
        sel = idx[s * L : (s + 1) * L][mask[s * L : (s + 1) * L]].reshape(-1).long()
        assert torch.equal(counts[s], torch.bincount(sel, minlength=E).int())
    P = p.view(S, L, E).sum(1) / n.unsqueeze(1)
    assert ((prob.double() - P).abs() <= REL * P).all()
    f = counts.double() / (k * n).unsqueeze(1)
    want = (E * (f * P).sum(1)).sum() / live
    assert abs(float(loss) - float(want)) <= REL * float(want)
    grad = native.balance_loss_backward(logits, counts, tokens, torch.ones(1, device="cuda"), k, mask=mask)
    pv, fe = p.view(S, L, E), f.unsqueeze(1)
    d = E / (live * n.view(S, 1, 1)) * pv * (fe - (pv * fe).sum(-1, keepdim=True))
    spread = 2 * E / (live * n.view(S, 1, 1)) * (fe - 1 / E).abs().amax(-1, keepdim=True)
    tol = 2 * REL * pv * spread
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (d.abs() + tol)
    assert ((grad.double().view(S, L, E) - d).abs() <= tol + 1e-37).all()


def test_captured_and_on_another_stream():
    logits, idx, mask = _inputs(3, 100, 128, 8, torch.float32, 21)
    one = torch.ones(1, device="cuda")
    ws = torch.empty(int(native.lib().moe_balance_workspace_bytes(3, 100, 128)), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = native.balance_loss(logits, idx, mask=mask, n_seq=3, workspace=ws)
        ga = native.balance_loss_backward(logits, a[1], a[3], one, 8, mask=mask)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b = native.balance_loss(logits, idx, mask=mask, n_seq=3, workspace=ws)
        gb = native.balance_loss_backward(logits, b[1], b[3], one, 8, mask=mask)
    for _ in range(2):
        g.replay()
    assert all(torch.equal(u, v) for u, v in zip(a, b)) and torch.equal(ga, gb)
    # stream= with everything made by the call: results and workspace belong to that stream
    torch.cuda.synchronize()
    d = native.balance_loss(logits, idx, mask=mask, n_seq=3, stream=s)
    gd = native.balance_loss_backward(logits, d[1], d[3], one, 8, mask=mask, stream=s)
    noise = [torch.full((4 << 20,), 7.0, device="cuda") for _ in range(4)]      # on the current stream meanwhile
    s.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(a, d)) and torch.equal(ga, gd) and float(noise[0][0]) == 7
    logits.copy_(logits.flip(0))
    idx.copy_(idx.flip(0))
    g.replay()
    c = native.balance_loss(logits, idx, mask=mask, n_seq=3)
    assert all(torch.equal(u, v) for u, v in zip(b, c))


def test_empty_batch_and_refused_calls():
    out = native.balance_loss(torch.empty(0, 8, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda"))
    assert float(out[0]) == 0 and int(out[3][0]) == 0
    logits, idx, _ = _inputs(1, 8, 8, 2, torch.float32, 0, pad=0)
    with pytest.raises(TypeError):
        native.balance_loss(logits, idx.long())
    with pytest.raises(ValueError):
        native.balance_loss(logits, idx, mask=torch.ones(7, dtype=torch.bool, device="cuda"))
    with pytest.raises(ValueError):
        native.balance_loss(logits.t(), idx)
    with pytest.raises(native.MoeError):
        native.balance_loss(logits, torch.zeros(8, 9, dtype=torch.int32, device="cuda"))
