"""The balance loss's probabilities far below the row's largest: their error is relative to themselves."""
import numpy as np
import pytest
import torch

from quantized_routed_expert_softmax_gb300 import native

pytestmark = pytest.mark.gpu

U = 2.0 ** -24   # half a unit of fp32, relative


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_routed_expert_softmax_gb300 import build
    build.build()
    native.lib()


def _rows(S, E, dtype, seed):
    """Logits m - j / 8: the difference to the row's largest is exact in fp32, j up to 760 (e^-95 is below 2^-126)."""
    g = np.random.default_rng(seed)
    top = 64.0 if dtype == torch.float32 else 0.0
    steps = g.integers(0, 761, (S, E))
    if dtype == torch.bfloat16:      # 8 bits: steps of 1/8 below 32, of a half above
        steps = np.where(steps > 255, steps // 4 * 4, steps)
    steps[:, g.integers(0, E)] = 0
    x = torch.from_numpy((top - steps / 8).astype(np.float32)).cuda().to(dtype)
    assert torch.equal(x.double().cpu(), torch.from_numpy(top - steps / 8))
    return x


# In units of U: the exponential 2^-22, its remainder's product and addition 2: 6; the sum's terms 6, its additions at most
# 32 in a lane and 5 levels (each half a unit of the sum: 37), 1 / sum and its product 2; the mean of one token 1.
P_UNITS = 6 + 6 + 37 + 2 + 1
# Exponentials below 2^-126 are 0, and what is left of a product there is a multiple of 2^-149.
FLOOR = 2.0 ** -126 * (1 + 2.0 ** -20)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("S,E,k", [(40, 8, 2), (33, 60, 4), (700, 128, 8), (17, 257, 6), (20, 512, 22), (9, 1024, 32)])
def test_small_probabilities(S, E, k, dtype):
    x = _rows(S, E, dtype, S + E)
    idx = x.float().topk(k, 1).indices.int()
    loss, counts, prob, tokens = native.balance_loss(x, idx, n_seq=S)
    p = torch.softmax(x.double(), 1)
    assert float(p.min()) < 2.0 ** -126        # such ones are among them
    over = (prob.double() - p).abs() - FLOOR
    assert (over <= P_UNITS * U * p).all(), float((over / p).max() / U)
    grad = native.balance_loss_backward(x, counts, tokens, torch.ones(1, device="cuda"), k)
    f = counts.double() / k
    mean = (p * f).sum(1, keepdim=True)
    want = E / S * p * (f - mean)
    # f - 1/E from integers, its factor 4; sum f p: every term as p, 4 and E additions; the difference and the
    # product 2: relative to the largest |f - 1/E| times the row's probability
    spread = E / S * (f - 1 / E).abs().amax(1, keepdim=True) * 2
    err = (P_UNITS + 4) * U * want.abs() + (P_UNITS + 4 + 37 + 2) * U * p * spread + FLOOR * (1 + E / S)
    if dtype == torch.bfloat16:
        err = err + 2.0 ** -8 * (want.abs() + err) + 2.0 ** -133
    bad = (grad.double() - want).abs() - err
    assert (bad <= 0).all(), float(bad.max())
    torch.testing.assert_close(loss.double(), ((E * (f * p)).sum(1).mean()).view(1), rtol=(P_UNITS + 30) * U, atol=0)


def test_logits_of_the_lowest_value_and_infinities():
    low = torch.finfo(torch.float32).min
    inf = float("inf")
    rows = torch.tensor([[0, low, low, -inf], [1e30, -1e30, 0, -inf], [low, low, -inf, -inf], [-low, low, 0, 1],
                         [5, 5, -inf, low], [-inf, -inf, -inf, low], [2.5e38, -1e37, -2.4e38, 2.5e38]])
    for E in (4, 60, 257):
        x = torch.full((len(rows), E), -inf)
        x[:, :4] = rows
        want = torch.softmax(x.double(), 1).cuda()
        for dtype in (torch.float32, torch.bfloat16):
            y = x.cuda().to(dtype)
            if dtype == torch.bfloat16:
                want = torch.softmax(y.double().nan_to_num(posinf=inf, neginf=-inf), 1)
                keep = (y < inf).all(1)                   # the largest fp32 value rounds to an infinity
            else:
                keep = torch.ones(len(rows), dtype=torch.bool, device="cuda")
            idx = torch.zeros(len(rows), 1, dtype=torch.int32, device="cuda")
            keep &= (y > -inf).any(1)
            loss, counts, prob, tokens = native.balance_loss(y, idx, n_seq=len(rows))
            assert ((prob.double() - want).abs()[keep] <= P_UNITS * U * want[keep]).all()
            grad = native.balance_loss_backward(y, counts, tokens, torch.ones(1, device="cuda"), 1)
            assert torch.isfinite(grad[keep]).all()
    x = torch.zeros(3, 12, device="cuda")
    x[0, 3] = float("nan")
    x[1, 3] = inf
    prob = native.balance_loss(x, torch.zeros(3, 1, dtype=torch.int32, device="cuda"), n_seq=3)[2]
    assert torch.isnan(prob[0]).all() and torch.isnan(prob[1]).any() and torch.isfinite(prob[2]).all()
