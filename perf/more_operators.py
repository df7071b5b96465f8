"""Measured cases of the 8-bit integer operators and of the feed-forward block with its gradients.

Four kinds of case, each one pass through public entry points of native.py:
  quantise  rows of activations or weights to 8-bit integers with one scale a row (optionally gathered
            by a row index) and the values that the codes stand for;
  product   the expert-indexed product of int8 rows, sorted by expert, with per-channel int8 weights,
            with the layer's activation applied to it;
  ffn       the gated feed-forward block in bf16, rows sorted by expert (one expert: a dense block);
  train     the same block forward and backward: gradients of its rows and of both weight stacks.

An int8 matrix [rows, cols] is the fp32 scale of every row (4 rows bytes, rounded up to 16), then panels
of 32 columns: the 32 codes of every row.
"""
import math

import torch

own = False

# ---------------------------------------------------------------------------------------- the cases


def listed():
    return [
        # one decoded token of the Gemma-shaped layer, as its expert input
        dict(name="quantise one token", op="quantise", rows=1, cols=2816, dtype="bf16", gather=0),
        # the (token, expert) rows of a ragged prefill, gathered in the order of the experts
        dict(name="quantise gathered prefill", op="quantise", rows=32764, cols=2816, dtype="bf16", gather=4097),
        # gate.up of one decoded token: 8 experts of 128
        dict(name="int8 gate.up one token", op="product", T=1, k=8, E=128, K=2816, N=1408, act="swiglu", out="bf16"),
        # latent experts, ReLU^2, a decode batch that touches most of 512 experts
        dict(name="int8 latent up 32 tokens", op="product", T=32, k=22, E=512, K=1024, N=2688, act="relu2", out="f32"),
        # gate.up of a short prefill
        dict(name="int8 gate.up prefill 512", op="product", T=512, k=8, E=128, K=2816, N=1408, act="swiglu", out="bf16"),
        # down of a long prefill of ragged length
        dict(name="int8 down prefill 8191", op="product", T=8191, k=8, E=128, K=704, N=2816, act="none", out="bf16"),
        # a shared (dense) expert at one decoded token
        dict(name="ffn dense one token", op="ffn", T=1, k=1, E=1, d=2816, f=2112),
        # trained experts answering a short prompt
        dict(name="ffn experts 512", op="ffn", T=512, k=8, E=128, d=2816, f=704),
        # a unit-test-sized layer with more experts than some of them have rows
        dict(name="train tiny", op="train", T=67, k=2, E=8, d=256, f=512),
        # a micro-batch over the Gemma-shaped experts
        dict(name="train experts 4096", op="train", T=4096, k=8, E=128, d=2816, f=704),
        # a dense block over a batch of odd length
        dict(name="train dense 8191", op="train", T=8191, k=1, E=1, d=2816, f=5632),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantise", "product", "product", "ffn", "train", "train"])
    if op == "quantise":
        cols = 32 * _log(rng, 4, 192)
        rows = max(1, min(_log(rng, 1, 100000), 90_000_000 // cols))
        return dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["f32", "bf16"]),
                    gather=rng.choice([0, max(1, rows // 8)]))
    if op == "product":
        E, k = rng.choice([(1, 1), (8, 2), (32, 4), (128, 8), (512, 22)])
        act = rng.choice(["none", "swiglu", "relu2"])
        K = 32 * _log(rng, 8, 88 if E < 512 else 32)
        f = 32 * _log(rng, 4, 44)
        N = 2 * f if act == "swiglu" else 2 * f + rng.choice([0, 0, 8, 17])
        T = min(_log(rng, 1, 8000), 100_000_000_000 // (k * K * N))
        out = "f32" if T * k <= 1024 else "bf16"
        return dict(op=op, T=T, k=k, E=E, K=K, N=N, act=act, out=out)
    E, k = rng.choice([(1, 1), (1, 1), (8, 2), (32, 4), (128, 8)])
    d = 16 * _log(rng, 16, 176)
    f = 16 * _log(rng, 8, 352 if E == 1 else 64)
    T = max(1, min(_log(rng, 1, 16000), 100_000_000_000 // (k * d * f)))
    return dict(op=op, T=T, k=k, E=E, d=d, f=f)


# ------------------------------------------------------------------------------- the format, in torch


def _bytes(rows, cols):
    return (4 * rows + 15) // 16 * 16 + rows * cols


def _away(v):
    """Round half away from zero (fp64)."""
    return torch.sign(v) * torch.floor(v.abs() + 0.5)


def _code(x):
    """x [n, rows, cols] -> (codes int8 [n, rows, cols], scales fp32 [n, rows])."""
    x = x.float()
    amax = x.abs().amax(-1)
    bad = ~(amax < math.inf)
    # the division by 127 in a tensor: a division by a number may become a product with its reciprocal
    s = amax / torch.full_like(amax, 127.0)
    q = x / torch.where(s > 0, s, torch.ones_like(s)).unsqueeze(-1)
    q = torch.where((bad | ~(s > 0)).unsqueeze(-1), torch.zeros_like(q), q)
    q = _away(q.double()).clamp(-127, 127).to(torch.int8)
    return q, torch.where(bad, torch.full_like(s, math.nan), s)


def _pack(x):
    """x [n, rows, cols] -> uint8 [n, _bytes(rows, cols)]."""
    n, rows, cols = x.shape
    q, s = _code(x)
    out = torch.zeros((n, _bytes(rows, cols)), dtype=torch.uint8, device=x.device)
    out[:, : 4 * rows] = s.contiguous().view(torch.uint8).view(n, -1)
    out[:, -rows * cols :] = q.view(n, rows, cols // 32, 32).transpose(1, 2).reshape(n, -1).view(torch.uint8)
    return out


def _unpack(q, rows, cols):
    """The inverse of _pack's layout: (codes int8 [n, rows, cols], scales fp32 [n, rows])."""
    n = q.shape[0]
    s = q[:, : 4 * rows].contiguous().view(torch.float32).view(n, rows)
    c = q[:, -rows * cols :].view(torch.int8).view(n, cols // 32, rows, 32).transpose(1, 2)
    return c.reshape(n, rows, cols), s


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


# ------------------------------------------------------------------------------------------- inputs


def _route(rand, T, k, E):
    """Offsets of T tokens' k distinct experts each, some experts more popular than others."""
    e = (rand(T, E) + 0.3 * rand(1, E)).topk(k, dim=1).indices.reshape(-1)
    count = torch.bincount(e, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = count.cumsum(0)
    return offsets, int(count.max())


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    if case["op"] == "quantise":
        rows, cols, T = case["rows"], case["cols"], case["gather"]
        # rows of differing size, some channels much larger than the others, as activations have them
        x = rand(T or rows, cols) * torch.exp(0.5 * rand(T or rows, 1)) * torch.exp(0.7 * rand(1, cols))
        src = torch.randint(0, T, (rows,), generator=g, device="cuda", dtype=torch.int32) if T else None
        return dict(case, x=x.to(_dtype(case["dtype"])), src=src)
    T, k, E = case["T"], case["k"], case["E"]
    P = T * k
    offsets, cap = _route(rand, T, k, E)
    if case["op"] == "product":
        K, N = case["K"], case["N"]
        xq = _pack(rand(1, P, K) * torch.exp(0.5 * rand(1, P, 1)))
        wq = torch.cat([_pack(0.02 * rand(min(16, E - e0), N, K)) for e0 in range(0, E, 16)])
        width = N // 2 if case["act"] == "swiglu" else N
        st = dict(case, xq=xq, wq=wq, offsets=offsets, cap=cap)
        st["y"] = torch.empty((P, width), dtype=_dtype(case["out"]), device="cuda")
        if own:
            from quantized_routed_expert_softmax_gb300 import native
            st["ws"] = native.int8_workspace()
        return st
    d, f = case["d"], case["f"]
    bf = torch.bfloat16
    stack = lambda rows, cols: torch.cat([(0.02 * rand(min(16, E - e0), rows, cols)).to(bf)  # noqa: E731
                                          for e0 in range(0, E, 16)])
    # rows as an RMS norm leaves them; the block's gradient is small beside its rows
    st = dict(case, x=rand(P, d).to(bf), wgu=stack(2 * f, d), wd=stack(d, f), offsets=offsets, cap=cap)
    if case["op"] == "train":
        st["dy"] = (0.05 * rand(P, d)).to(bf)
    if own:
        from quantized_routed_expert_softmax_gb300 import native
        st["ws"] = native.ffn_workspace(P, f, backward=case["op"] == "train")
    return st


# -------------------------------------------------------------------------------------- plain forms


def _plain_quantise(s):
    x = s["x"] if s["src"] is None else s["x"][s["src"].long()]
    q, scale = _code(x.unsqueeze(0))
    return (q[0].float() * scale[0].unsqueeze(-1)).to(s["x"].dtype)


def _groups(off, cap, P):
    """The rows of every expert side by side, padded to the largest group: (row of each place, whether it
    is one of the expert's)."""
    at = off[:-1, None] + torch.arange(cap, device=off.device)
    return at.clamp(max=P - 1), at < off[1:, None]


def _ungroup(y, off, P):
    r = torch.arange(P, device=y.device)
    e = (r[:, None] >= off[None, 1:]).sum(1)
    return y[e, r - off[e]]


def _plain_product(s):
    P, K, N = s["T"] * s["k"], s["K"], s["N"]
    w, sw = _unpack(s["wq"], N, K)
    x, sx = _unpack(s["xq"], P, K)
    off = s["offsets"].long()
    at, _ = _groups(off, s["cap"], P)
    y = torch.bmm(x[0].float()[at], w.float().transpose(1, 2)) * sw.unsqueeze(1)
    y = _ungroup(y, off, P) * sx[0].unsqueeze(-1)
    if s["act"] == "swiglu":
        gate, up = y[:, : N // 2], y[:, N // 2 :]
        y = gate / (1 + torch.exp(-gate)) * up
    elif s["act"] == "relu2":
        y = y.clamp(min=0).square()
    return y.to(_dtype(s["out"]))


def _plain_ffn(s):
    P, f, bf = s["T"] * s["k"], s["f"], torch.bfloat16
    off = s["offsets"].long()
    at, mine = _groups(off, s["cap"], P)
    wgu, wd = s["wgu"].float(), s["wd"].float()
    x = s["x"].float()[at]
    z = torch.bmm(x, wgu.transpose(1, 2))
    gate, up = z[..., :f], z[..., f:]
    sig = 1 / (1 + torch.exp(-gate))
    h = gate * sig * up
    y = _ungroup(torch.bmm(h, wd.transpose(1, 2)), off, P).to(bf)
    if s["op"] == "ffn":
        return y
    # places past an expert's rows hold other experts' rows: their gradients are nought
    dy = torch.where(mine.unsqueeze(-1), s["dy"].float()[at], torch.zeros((), device=x.device))
    dwd = torch.bmm(dy.transpose(1, 2), h).to(bf)
    dh = torch.bmm(dy, wd)
    dz = torch.cat([dh * up * sig * (1 + gate * (1 - sig)), dh * gate * sig], -1)
    dwgu = torch.bmm(dz.transpose(1, 2), x).to(bf)
    dx = _ungroup(torch.bmm(dz, wgu), off, P).to(bf)
    return dict(y=y, dx=dx, dwgu=dwgu, dwd=dwd)


# ---------------------------------------------------------------------------------------------- run


def run(s):
    if not own:
        return {"quantise": _plain_quantise, "product": _plain_product, "ffn": _plain_ffn, "train": _plain_ffn}[s["op"]](s)
    from quantized_routed_expert_softmax_gb300 import native
    if s["op"] == "quantise":
        q = native.quantize_int8(s["x"], rows=s["src"])
        return native.dequantize_int8(q[0], s["rows"], s["cols"], dtype=s["x"].dtype)
    if s["op"] == "product":
        return native.int8_matmul(s["xq"], s["wq"], s["offsets"], s["T"] * s["k"], s["N"], s["K"], act=s["act"],
                                  out=s["y"], workspace=s.get("ws"))
    if s["op"] == "ffn":
        return native.ffn_forward(s["x"], s["wgu"], s["wd"], s["offsets"], workspace=s.get("ws"))
    y, saved = native.ffn_forward(s["x"], s["wgu"], s["wd"], s["offsets"], save=True, workspace=s.get("ws"))
    dx, dwgu, dwd = native.ffn_backward(s["dy"], s["x"], s["wgu"], s["wd"], saved, s["offsets"], workspace=s.get("ws"))
    return dict(y=y, dx=dx, dwgu=dwgu, dwd=dwd)


def work(case):
    if case["op"] == "quantise":
        n, b = case["rows"] * case["cols"], 4 if case["dtype"] == "f32" else 2
        read = n if not case["gather"] else min(case["gather"], case["rows"]) * case["cols"]
        return dict(bytes=b * read + 2 * (n + 4 * case["rows"]) + b * n, flops=2 * n)
    T, k, E = case["T"], case["k"], case["E"]
    P, live = T * k, E * (1 - (1 - k / E) ** T)
    if case["op"] == "product":
        K, N = case["K"], case["N"]
        width = N // 2 if case["act"] == "swiglu" else N
        return dict(bytes=live * N * (K + 4) + P * (K + 4) + P * width * (4 if case["out"] == "f32" else 2),
                    flops=2 * P * N * K)
    d, f = case["d"], case["f"]
    if case["op"] == "ffn":
        return dict(bytes=2 * (3 * live * d * f + 2 * P * d), flops=6 * P * d * f)
    # x, dy, y and dx; the weights once and their gradients once
    return dict(bytes=2 * (4 * P * d + 3 * live * d * f + 3 * E * d * f), flops=18 * P * d * f)


# ------------------------------------------------------------------------------------------ 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantise":
        x = s["x"] if s["src"] is None else s["x"].index_select(0, s["src"])
        out = torch.empty(x.shape, dtype=torch.float64, device="cuda")
        for r in range(0, x.shape[0], 4096):
            v = x[r : r + 4096].double()
            # a quotient of two fp32 numbers in 64 bits, rounded to 32, is the correctly rounded one
            scale = (torch.linalg.vector_norm(v, math.inf, -1, keepdim=True) / 127.0).float().double()
            ratio = torch.nan_to_num(v / scale, nan=0.0).float().double()
            whole = torch.trunc(ratio)
            out[r : r + 4096] = scale * (whole + torch.where((ratio - whole).abs() >= 0.5, torch.sign(ratio), 0.0))
        return out
    off = s["offsets"].tolist()
    spans = [(e, off[e], off[e + 1]) for e in range(case["E"]) if off[e + 1] > off[e]]
    f64 = dict(dtype=torch.float64, device="cuda")
    if case["op"] == "product":
        P, K, N = s["T"] * s["k"], s["K"], s["N"]
        f = N // 2 if case["act"] == "swiglu" else N
        y = torch.zeros((P, f), **f64)
        xc, xs = _unpack(s["xq"], P, K)
        for e, a, b in spans:
            wc, ws = _unpack(s["wq"][e : e + 1], N, K)
            z = torch.einsum("rk,nk->rn", xc[0, a:b].double() * xs[0, a:b, None].double(), wc[0].double() * ws[0, :, None].double())
            if case["act"] == "swiglu":
                z = torch.special.expit(z[:, :f]) * z[:, :f] * z[:, f:]
            elif case["act"] == "relu2":
                z = torch.relu(z) ** 2
            y[a:b] = z
        return y
    P, d, f = s["T"] * s["k"], s["d"], s["f"]
    y = torch.zeros((P, d), **f64)
    if case["op"] == "ffn":
        for e, a, b in spans:
            z = s["x"][a:b].double() @ s["wgu"][e].double().T
            y[a:b] = (torch.special.expit(z[:, :f]) * z[:, :f] * z[:, f:]) @ s["wd"][e].double().T
        return y
    dx, dwgu, dwd = torch.zeros((P, d), **f64), torch.zeros((s["E"], 2 * f, d), **f64), torch.zeros((s["E"], d, f), **f64)
    for e, a, b in spans:
        x, dy = s["x"][a:b].double(), s["dy"][a:b].double()
        wg, wu, w2 = s["wgu"][e, :f].double(), s["wgu"][e, f:].double(), s["wd"][e].double()
        gate, up = x @ wg.T, x @ wu.T
        p = torch.special.expit(gate)
        act = gate * p
        y[a:b] = (act * up) @ w2.T
        dwd[e] = dy.T @ (act * up)
        dh = dy @ w2
        dgate = dh * up * (p + act * (1 - p))
        dup = dh * act
        dx[a:b] = dgate @ wg + dup @ wu
        dwgu[e, :f], dwgu[e, f:] = dgate.T @ x, dup.T @ x
    return dict(y=y, dx=dx, dwgu=dwgu, dwd=dwd)
