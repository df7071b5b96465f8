"""The int8 rows and their product, and the gated feed-forward block with its gradients, restated for the tests
from their definitions in 64 bits: the codec in numpy, value by value; the products in torch, expert by expert.

ffn() also bounds what the kernels' roundings can do to each result: U is half a step of bf16, and a sum of n
products in fp32, in any order and with each addition off by a step at most, is off by n * 2^-23 of the sum of the
products' magnitudes (the tensor cores may cut bits off where fp32 additions round)."""
import numpy as np
import torch

U = torch.finfo(torch.bfloat16).eps / 2


# ------------------------------------------------------------------------------------------- int8
def bytes_of(rows, cols):
    return (4 * rows + 15) // 16 * 16 + rows * cols


def quantize(x):
    """x [rows, cols] float32 -> (codes int8 [rows, cols], scales float32 [rows])."""
    finite = np.isfinite(x).all(-1)
    x = np.where(finite[:, None], x, np.float32(0))
    s = (np.abs(x).max(-1) / np.float32(127)).astype(np.float32)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        v = np.where(s[:, None] > 0, x / s[:, None], np.float32(0)).astype(np.float64)
    q = np.clip(np.sign(v) * np.floor(np.abs(v) + 0.5), -127, 127).astype(np.int8)
    return q, np.where(finite, s, np.float32(np.nan))


def pack(q, s):
    """(the bytes of one matrix, which of them are defined)."""
    rows, cols = q.shape
    out, known = np.zeros(bytes_of(rows, cols), np.uint8), np.ones(bytes_of(rows, cols), bool)
    out[: 4 * rows] = s.astype("<f4").view(np.uint8)
    at = (4 * rows + 15) // 16 * 16
    known[4 * rows : at] = False
    for b in range(cols // 32):
        out[at : at + 32 * rows] = np.ascontiguousarray(q[:, 32 * b : 32 * b + 32]).view(np.uint8).reshape(-1)
        at += 32 * rows
    return out, known


def activate(z, act):
    if act == "swiglu":
        g, u = z.chunk(2, -1)
        return g * torch.sigmoid(g) * u
    return torch.relu(z) ** 2 if act == "relu2" else z


# ------------------------------------------------------------------------------- feed-forward block
def spans(offsets, P, E):
    """Expert, first row, last row + 1 of the experts that have rows."""
    if offsets is None:
        return [(0, 0, P)] if P else []
    o = [min(max(int(v), 0), P) for v in offsets]
    return [(e, o[e], o[e + 1]) for e in range(E) if o[e + 1] > o[e]]


def ffn(x, wgu, wd, offsets, act="swiglu", dy=None):
    """name -> (values, bounds) of y, and with dy of z, h, dx, dwgu, dwd too; fp64, rows that no expert owns are 0."""
    x, wgu, wd = (t.double() for t in (x, wgu, wd))
    E, nz, d = wgu.shape
    f, P = wd.shape[2], x.shape[0]
    shapes = dict(y=(P, d), z=(P, nz), h=(P, f), dx=(P, d), dwgu=(E, nz, d), dwd=(E, d, f))
    if dy is None:
        shapes = {n: shapes[n] for n in ("y", "z", "h")}
    else:
        dy = dy.double()
    out = {n: (x.new_zeros(s), x.new_zeros(s)) for n, s in shapes.items()}
    acc = lambda n: n * 2.0 ** -23  # noqa: E731

    def put(name, at, v, b):
        u = 2.0 ** -24 if name == "z" else U       # (z is fp32)
        out[name][0][at], out[name][1][at] = v, b + u * (v.abs() + b)

    for e, r0, r1 in spans(offsets, P, E):
        X, W, D, r = x[r0:r1], wgu[e], wd[e], slice(r0, r1)
        z = X @ W.T
        bz = acc(d) * (X.abs() @ W.abs().T)
        put("z", r, z, bz)
        if act == "swiglu":
            g, u = z[:, :f], z[:, f:]
            bg, bu = bz[:, :f], bz[:, f:]
            sg = torch.sigmoid(g)
            h = g * sg * u
            # |silu'| <= 1.1; the sigmoid by a fast exponential and division: off by 2^-20 and 2^-22 per unit of |g|
            # (up to where it underflows, below -87)
            bs = 2.0 ** -20 + g.abs().clamp(max=128) * 2.0 ** -22
            bh = (1.1 * bg + bs * (g * sg).abs() + 2.0 ** -120) * (u.abs() + bu) + (g * sg).abs() * bu
        else:
            h = torch.relu(z) ** 2
            bh = (2 * torch.relu(z) + bz) * bz + 2.0 ** -23 * h
        put("h", r, h, bh)
        h16 = h.abs() + out["h"][1][r]             # at most, as the products read it
        put("y", r, h @ D.T, out["h"][1][r] @ D.abs().T + acc(f) * (h16 @ D.abs().T))
        if dy is None:
            continue
        Y = dy[r0:r1]
        dh = Y @ D
        bdh = acc(d) * (Y.abs() @ D.abs())
        zs, bzs = z, out["z"][1][r]                # the stored z
        if act == "swiglu":
            bg, bu = bzs[:, :f], bzs[:, f:]
            slope = sg * (1 + g * (1 - sg))        # |slope'| <= 0.5
            bslope = 0.5 * bg + 4 * bs
            dg, du = dh * u * slope, dh * g * sg
            bdg = bdh * (u.abs() + bu) * (slope.abs() + bslope) + dh.abs() * (bu * (slope.abs() + bslope) + u.abs() * bslope)
            bsilu = 1.1 * bg + 2 * bs * (g * sg).abs()
            bdu = bdh * ((g * sg).abs() + bsilu) + dh.abs() * bsilu
            dz, bdz = torch.cat([dg, du], 1), torch.cat([bdg, bdu], 1)
        else:
            dz = dh * 2 * torch.relu(z)
            bdz = bdh * 2 * (torch.relu(z) + bzs) + dh.abs() * 2 * bzs
        bdz = bdz + U * (dz.abs() + bdz) + 2.0 ** -22 * dz.abs() + 2.0 ** -120
        dz16 = dz.abs() + bdz
        put("dx", r, dz @ W, bdz @ W.abs() + acc(nz) * (dz16 @ W.abs()))
        n = r1 - r0
        put("dwgu", e, dz.T @ X, bdz.T @ X.abs() + acc(n) * (dz16.T @ X.abs()))
        put("dwd", e, Y.T @ h, Y.abs().T @ out["h"][1][r] + acc(n) * (Y.abs().T @ h16))
    return out
