"""The balance loss where many nearly equal terms are added: what a running fp32 sum rounds off is then
systematic.  Equal logits have exact answers: every probability is 1/E, and with m of every token's k slots
counted every sequence's loss is m / k."""
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


# In units of U, relative.  A probability: exp(0) = 1 and the sum E are exact, 1 / E rounds once: 1.
# Its mean over tokens: at most 65 equal terms (64 passes of a run, whose ends are rounded to 8 tokens) added in turn,
# sum_i i/65 = 33; groups of lanes 4 levels; eight warps in pairs 3; the runs' records without loss 1, and again
# eight warps 3; 1 / n and its product 2: with the term itself 47.
# The loss: P, the product with the count 1, 32 experts in a tree 5 levels, E / k, 1 / n_s, their product and the
# product with it 4: P + 10; over sequences without loss 1, the threads of a CTA 5 + 8, the division 1: P + 25.
P_LONG = 47


@pytest.mark.parametrize("S,L,E,k,dtype", [
    (1 << 20, 1, 12, 3, torch.float32),          # 4096 blocks a thread
    ((1 << 20) - 7, 1, 31, 2, torch.bfloat16),   # one expert a lane
    (1 << 20, 1, 1000, 31, torch.bfloat16),      # 131072 blocks a thread, offsets past 32 bits
    (1 << 18, 4, 12, 5, torch.float32),
    (1, 1 << 20, 1000, 2, torch.bfloat16),       # waves of runs, a row at a time
    (3, 349525, 520, 4, torch.float32),
    (1, 1 << 20, 6, 1, torch.float32),
    (1 << 20, 1, 12, 7, torch.float32),
    (300000, 3, 200, 3, torch.float32),
    (2, 1 << 19, 12, 12, torch.float32),
    (1, 16 * 32 * 3 + 5, 8, 2, torch.float32),   # few tokens: one CTA's run, or a few
    (511, 1, 8, 2, torch.float32),               # one CTA for every sequence
    (1, 257, 1023, 3, torch.float32),
])
def test_equal_logits(S, L, E, k, dtype):
    T = S * L
    logits = torch.full((T, E), 0.375, dtype=dtype, device="cuda")
    # slots spread over the experts, the first of several dropped
    idx = (torch.arange(T, device="cuda").view(-1, 1) + torch.arange(k, device="cuda") * (E // k)) % E
    m = k
    if k > 1:
        idx[:, 0] = -1
        m = k - 1
    loss, counts, prob, tokens = native.balance_loss(logits, idx.int(), n_seq=S)
    assert (tokens == L).all()
    assert torch.equal(counts.sum(1), torch.full((S,), L * m, device="cuda"))
    p_units = 3 if L == 1 else P_LONG        # one token: 1 / E, 1 / n (exact) and its product
    worst = max(float((c.double() * E - 1).abs().max()) for c in prob.split(1 << 16))
    assert worst <= p_units * U, worst / U
    assert abs(float(loss) * k / m - 1) <= (p_units + 25) * U, (float(loss) * k / m - 1) / U
