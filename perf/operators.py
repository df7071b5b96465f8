"""Measured cases of the MXFP4 operators and the router balance loss.

Three kinds of case, each one pass through public entry points of native.py:
  quantise  rows of activations or weights to MXFP4 (optionally gathered by a row index) and the
            values that the codes stand for;
  product   the expert-indexed product of MXFP4 rows, sorted by expert, with MXFP4 weights, with the
            layer's activation applied to it;
  balance   the router balance loss of a (padded) batch of sequences with its per-expert counts, and
            the gradient of the logits.

MXFP4 stores a matrix [rows, cols] as its E2M1 codes, row-major, two per byte (even column in the low
nibble), then the E8M0 scales in panels of 128 columns: 4 bytes of every row per panel (columns past
the end: byte 127), the whole rounded up to 16 bytes.
"""
import math

import torch

own = False

# ---------------------------------------------------------------------------------------- the cases


def listed():
    return [
        # one decoded token of the Gemma-shaped layer, as its expert input
        dict(name="quantise one token", op="quantise", rows=1, cols=2816, dtype="bf16", gather=0),
        # the (token, expert) rows of a 512-token prefill, gathered in the order of the experts
        dict(name="quantise gathered prefill", op="quantise", rows=4096, cols=2816, dtype="bf16", gather=512),
        # hidden activations in fp32, an odd number of rows
        dict(name="quantise fp32 hidden", op="quantise", rows=45013, cols=704, dtype="f32", gather=0),
        # the gate/up matrices of 32 experts, as a checkpoint is converted
        dict(name="quantise weights", op="quantise", rows=32 * 1408, cols=2816, dtype="f32", gather=0),
        # gate.up of one decoded token: 8 experts of 128
        dict(name="gate.up one token", op="product", T=1, k=8, E=128, K=2816, N=1408, act="swiglu", out="bf16"),
        # down of a few decoded tokens
        dict(name="down 4 tokens", op="product", T=4, k=8, E=128, K=704, N=2816, act="none", out="f32"),
        # latent experts, ReLU^2, a decode batch that touches most of 512 experts
        dict(name="latent up 32 tokens", op="product", T=32, k=22, E=512, K=1024, N=2688, act="relu2", out="bf16"),
        # gate.up of a short prefill
        dict(name="gate.up prefill 512", op="product", T=512, k=8, E=128, K=2816, N=1408, act="swiglu", out="bf16"),
        # down of a long prefill of ragged length
        dict(name="down prefill 8191", op="product", T=8191, k=8, E=128, K=704, N=2816, act="none", out="bf16"),
        # the smallest batch: a unit-test-sized router
        dict(name="balance tiny", op="balance", S=1, L=16, E=8, k=2, dtype="f32", pad=0.0),
        # a micro-batch of ragged sequences in bf16, padded to an odd length
        dict(name="balance ragged bf16", op="balance", S=7, L=1021, E=128, k=8, dtype="bf16", pad=0.4),
        # a training batch over 512 experts
        dict(name="balance batch", op="balance", S=16, L=4096, E=512, k=22, dtype="f32", pad=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantise", "product", "product", "balance"])
    if op == "quantise":
        cols = 32 * _log(rng, 4, 192)
        rows = max(1, min(_log(rng, 1, 100000), 120_000_000 // cols))
        return dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["f32", "bf16"]),
                    gather=rng.choice([0, max(1, rows // 8)]))
    if op == "product":
        E, k = rng.choice([(8, 2), (32, 4), (128, 8), (512, 22)])
        act = rng.choice(["none", "swiglu", "relu2"])
        K = 32 * _log(rng, 8, 88 if E < 512 else 32)
        f = 32 * _log(rng, 4, 44)
        N = 2 * f if act == "swiglu" else 2 * f + rng.choice([0, 0, 8, 17])
        T = min(_log(rng, 1, 8000), 100_000_000_000 // (k * K * N))
        out = "f32" if T * k <= 256 else "bf16"
        return dict(op=op, T=T, k=k, E=E, K=K, N=N, act=act, out=out)
    E, k = rng.choice([(8, 2), (60, 4), (128, 8), (257, 6), (512, 22)])
    S = _log(rng, 1, 32)
    L = _log(rng, 1, 60000 // S)
    return dict(op=op, S=S, L=L, E=E, k=k, dtype=rng.choice(["f32", "bf16"]), pad=round(rng.uniform(0.0, 0.6), 3))


# ------------------------------------------------------------------------------- the format, in torch


def _panels(cols):
    return (cols + 127) // 128


def _bytes(rows, cols):
    return (rows * cols // 2 + 4 * rows * _panels(cols) + 15) // 16 * 16


def _code(x):
    """x [n, rows, cols] -> (codes uint8 0..15, scale bytes uint8 [n, rows, cols/32])."""
    n, rows, cols = x.shape
    v = x.float().view(n, rows, cols // 32, 32)
    amax = v.abs().amax(-1)
    bad = ~(amax < math.inf)
    # floor(log2 amax): the exponent field of the fp32 value (subnormals are far below the clamp)
    X = ((amax.view(torch.int32) >> 23) - 127 - 2).clamp(min=-127)
    X = torch.where(bad, torch.zeros_like(X), X)
    # the scaling by 2^-X in two exact steps, as 2^127 is the largest fp32 power of two
    h = -X // 2
    two = lambda e: ((e + 127) << 23).view(torch.float32)  # noqa: E731
    v = v * two(h).unsqueeze(-1) * two(-X - h).unsqueeze(-1)
    a = v.abs()
    # E2M1 magnitudes 0 .5 1 1.5 2 3 4 6; ties go to the even code
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    c = torch.where((v < 0) & (c > 0), c + 8, c)
    c = torch.where(bad.unsqueeze(-1), torch.zeros_like(c), c)
    s = torch.where(bad, torch.full_like(X, 255), X + 127).to(torch.uint8)
    return c.view(n, rows, cols), s


def _pack(x):
    """x [n, rows, cols] -> uint8 [n, _bytes(rows, cols)]."""
    n, rows, cols = x.shape
    c, s = _code(x)
    out = torch.zeros((n, _bytes(rows, cols)), dtype=torch.uint8, device=x.device)
    out[:, : rows * cols // 2] = (c[..., 0::2] | (c[..., 1::2] << 4)).view(n, -1)
    p = torch.full((n, rows, 4 * _panels(cols)), 127, dtype=torch.uint8, device=x.device)
    p[..., : cols // 32] = s
    p = p.view(n, rows, _panels(cols), 4).transpose(1, 2)
    out[:, rows * cols // 2 : rows * cols // 2 + 4 * rows * _panels(cols)] = p.reshape(n, -1)
    return out


def _unpack(q, rows, cols):
    """The inverse of _pack's layout: (codes [n, rows, cols], scale bytes [n, rows, cols/32])."""
    n = q.shape[0]
    b = q[:, : rows * cols // 2].view(n, rows, cols // 2)
    c = torch.stack([b & 15, b >> 4], -1).view(n, rows, cols)
    s = q[:, rows * cols // 2 : rows * cols // 2 + 4 * rows * _panels(cols)]
    s = s.reshape(n, _panels(cols), rows, 4).transpose(1, 2).reshape(n, rows, -1)[..., : cols // 32]
    return c, s


def _values(c, s, dtype=torch.float32):
    """What codes and scale bytes stand for."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=dtype, device=c.device)
    table = torch.cat([table, -table])
    scale = ((s.long() - 127 + 1023) << 52).view(torch.float64)
    scale = torch.where(s == 255, torch.full_like(scale, math.nan), scale).to(dtype)
    n, rows, cols = c.shape
    return (table[c.int()].view(n, rows, cols // 32, 32) * scale.unsqueeze(-1)).view(n, rows, cols)


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


# ------------------------------------------------------------------------------------------- inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    if case["op"] == "quantise":
        rows, cols, T = case["rows"], case["cols"], case["gather"]
        # rows of differing size, some channels much larger than the others, as activations have them
        x = rand(T or rows, cols) * torch.exp(0.5 * rand(T or rows, 1)) * torch.exp(0.7 * rand(1, cols))
        src = torch.randint(0, T, (rows,), generator=g, device="cuda", dtype=torch.int32) if T else None
        return dict(case, x=x.to(_dtype(case["dtype"])), src=src)
    if case["op"] == "product":
        T, k, E, K, N = (case[n] for n in ("T", "k", "E", "K", "N"))
        # k distinct experts a token, some experts more popular than others
        score = rand(T, E) + 0.3 * rand(1, E)
        e = score.topk(k, dim=1).indices.reshape(-1)
        count = torch.bincount(e, minlength=E)
        offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        offsets[1:] = count.cumsum(0)
        xq = _pack(rand(1, T * k, K))
        wq = torch.cat([_pack(0.02 * rand(min(16, E - e0), N, K)) for e0 in range(0, E, 16)])
        st = dict(case, xq=xq, wq=wq, offsets=offsets, cap=int(count.max()))
        f = N // 2 if case["act"] == "swiglu" else N
        st["y"] = torch.empty((T * k, f), dtype=_dtype(case["out"]), device="cuda")
        st["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")  # the product's error word
        return st
    S, L, E, k = (case[n] for n in ("S", "L", "E", "k"))
    logits = (1.3 * rand(S * L, E) + 0.5 * rand(1, E)).to(_dtype(case["dtype"]))
    idx = logits.float().topk(k, dim=1).indices.int()
    keep = 1.0 - case["pad"] * torch.rand((S, 1), generator=g, device="cuda")
    mask = (torch.arange(L, device="cuda") < torch.ceil(keep * L)).view(-1)
    st = dict(case, logits=logits, idx=idx, mask=mask, grad=torch.full((1,), 0.01, device="cuda"))
    return st


# -------------------------------------------------------------------------------------- plain forms


def _plain_quantise(s):
    x = s["x"] if s["src"] is None else s["x"][s["src"].long()]
    return _values(*_code(x.unsqueeze(0)))[0].to(s["x"].dtype)


def _plain_product(s):
    P, E, K, N, cap = s["T"] * s["k"], s["E"], s["K"], s["N"], s["cap"]
    w = _values(*_unpack(s["wq"], N, K))
    x = _values(*_unpack(s["xq"], P, K))[0]
    off = s["offsets"].long()
    # the rows of every expert side by side, padded to the largest group
    at = (off[:-1, None] + torch.arange(cap, device=x.device)).clamp(max=P - 1)
    y = torch.bmm(x[at], w.transpose(1, 2))
    r = torch.arange(P, device=x.device)
    e = (r[:, None] >= off[None, 1:]).sum(1)
    y = y[e, r - off[e]]
    if s["act"] == "swiglu":
        gate, up = y[:, : N // 2], y[:, N // 2 :]
        y = gate / (1 + torch.exp(-gate)) * up
    elif s["act"] == "relu2":
        y = y.clamp(min=0).square()
    return y.to(_dtype(s["out"]))


def _plain_balance(s):
    S, L, E, k = (s[n] for n in ("S", "L", "E", "k"))
    x, valid = s["logits"].float().view(S, L, E), s["mask"].view(S, L)
    m = x.amax(-1, keepdim=True)
    ex = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    p = ex / ex.sum(-1, keepdim=True).clamp(min=1e-30)
    p = torch.where(valid.unsqueeze(-1), p, torch.zeros_like(p))
    tokens = valid.sum(1)
    n = tokens.clamp(min=1)
    prob = p.sum(1, dtype=torch.float64) / n.unsqueeze(-1)
    counted = (valid.view(-1, 1) & (s["idx"] >= 0) & (s["idx"] < E)).view(-1)
    seq = torch.arange(S, device=x.device).repeat_interleave(L * k)
    flat = torch.where(counted, seq * E + s["idx"].view(-1).clamp(0, E - 1), S * E)
    counts = torch.zeros(S * E + 1, dtype=torch.int32, device=x.device)
    counts.index_add_(0, flat, torch.ones_like(flat, dtype=torch.int32))
    counts = counts[: S * E].view(S, E)
    f = counts.double() / (k * n).unsqueeze(-1)
    live = (tokens > 0).sum().clamp(min=1)
    loss = (E * (f * prob).sum(-1)).sum() / live
    fe = f.unsqueeze(1)
    d = p * (fe - (p * fe).sum(-1, keepdim=True))
    d = d * (s["grad"].double() * E / (live * n)).view(S, 1, 1)
    return dict(loss=loss.float().view(1), counts=counts, prob=prob.float(), tokens=tokens.int(),
                grad=d.view(S * L, E).to(s["logits"].dtype))


# ---------------------------------------------------------------------------------------------- run


def run(s):
    if not own:
        return {"quantise": _plain_quantise, "product": _plain_product, "balance": _plain_balance}[s["op"]](s)
    from quantized_routed_expert_softmax_gb300 import native
    if s["op"] == "quantise":
        q = native.quantize_mxfp4(s["x"], rows=s["src"])
        return native.dequantize_mxfp4(q[0], s["rows"], s["cols"], dtype=s["x"].dtype)
    if s["op"] == "product":
        return native.mxfp4_matmul(s["xq"], s["wq"], s["offsets"], s["T"] * s["k"], s["N"], s["K"], act=s["act"],
                                   out=s["y"], workspace=s["ws"])
    loss, counts, prob, tokens = native.balance_loss(s["logits"], s["idx"], mask=s["mask"], n_seq=s["S"])
    grad = native.balance_loss_backward(s["logits"], counts, tokens, s["grad"], s["k"], mask=s["mask"])
    return dict(loss=loss, counts=counts, prob=prob, tokens=tokens, grad=grad)


def work(case):
    if case["op"] == "quantise":
        n, b = case["rows"] * case["cols"], 4 if case["dtype"] == "f32" else 2
        read = n if not case["gather"] else min(case["gather"], case["rows"]) * case["cols"]
        return dict(bytes=b * read + 2 * n * 17 / 32 + b * n, flops=2 * n)
    if case["op"] == "product":
        T, k, E, K, N = (case[n] for n in ("T", "k", "E", "K", "N"))
        P, f = T * k, N // 2 if case["act"] == "swiglu" else N
        live = E * (1 - (1 - k / E) ** T)
        return dict(bytes=live * N * K * 17 / 32 + P * K * 17 / 32 + P * f * (4 if case["out"] == "f32" else 2),
                    flops=2 * P * N * K)
    n, b = case["S"] * case["L"] * case["E"], 4 if case["dtype"] == "f32" else 2
    return dict(bytes=3 * b * n + 4 * case["S"] * case["L"] * case["k"], flops=12 * n)


# ------------------------------------------------------------------------------------------ 64 bits


def _nearest(v):
    """E2M1 value nearest to v (fp64), ties to the even code, from the distance to every value."""
    grid = torch.tensor([0.0, 1.0, 2.0, 4.0, 0.5, 1.5, 3.0, 6.0], dtype=torch.float64, device=v.device)
    best, dist = torch.zeros_like(v), v.abs()
    for c in grid[1:]:  # the even codes come first, so that an equal distance stays with them
        d = (v.abs() - c).abs()
        best = torch.where(d < dist, c, best)
        dist = torch.minimum(d, dist)
    return torch.copysign(best, v)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantise":
        x = s["x"] if s["src"] is None else s["x"].index_select(0, s["src"])
        out = torch.empty(x.shape, dtype=torch.float64, device="cuda")
        for r in range(0, x.shape[0], 4096):
            v = x[r : r + 4096].double().unflatten(1, (-1, 32))
            # frexp: |v| = m * 2^e with m in [0.5, 1), so floor(log2) is e - 1
            e = torch.frexp(v.abs().amax(-1, keepdim=True)).exponent.double() - 3
            scale = ((e.clamp(min=-127).long() + 1023) << 52).view(torch.float64)  # 2^e, exactly
            out[r : r + 4096] = (_nearest(v / scale) * scale).flatten(1)
        return out
    if case["op"] == "product":
        P, K, N = s["T"] * s["k"], s["K"], s["N"]
        off = s["offsets"].tolist()
        f = N // 2 if case["act"] == "swiglu" else N
        xv = _values(*_unpack(s["xq"], P, K), dtype=torch.float64)[0]
        y = torch.zeros((P, f), dtype=torch.float64, device="cuda")
        for e in range(case["E"]):
            a, b = off[e], off[e + 1]
            if a == b:
                continue
            wv = _values(*_unpack(s["wq"][e : e + 1], N, K), dtype=torch.float64)[0]
            z = xv[a:b] @ wv.T
            if case["act"] == "swiglu":
                z = torch.special.expit(z[:, :f]) * z[:, :f] * z[:, f:]
            elif case["act"] == "relu2":
                z = torch.relu(z) ** 2
            y[a:b] = z
        return y
    S, L, E, k = (s[n] for n in ("S", "L", "E", "k"))
    loss, grads, probs = 0.0, [], []
    seqs = [(s["logits"].view(S, L, E)[i], s["idx"].view(S, L, k)[i], s["mask"].view(S, L)[i]) for i in range(S)]
    live = max(1, sum(int(m.any()) for _, _, m in seqs))
    for lg, ix, m in seqs:
        lg = lg.double()
        n = max(1, int(m.sum()))
        p = torch.softmax(lg, -1) * m.unsqueeze(-1)
        f = torch.bincount(ix[m].long().reshape(-1), minlength=E).double() / (k * n)
        probs.append(p.sum(0) / n)
        loss = loss + E * torch.dot(f, probs[-1]) / live
        grads.append(float(s["grad"][0].double()) * E / (live * n) * p * (f - (p @ f).unsqueeze(-1)))
    return dict(loss=loss.view(1), counts=None, prob=torch.stack(probs), tokens=None, grad=torch.cat(grads))
