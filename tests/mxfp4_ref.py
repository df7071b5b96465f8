"""MXFP4 and the router balance loss restated in numpy (64 bits) for the tests: the block codec from
the distances to the E2M1 values, the byte layout by explicit placement, the product row by row."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def bytes_of(rows, cols):
    return (rows * cols // 2 + 4 * rows * ((cols + 127) // 128) + 15) // 16 * 16


def quantize(x):
    """x [rows, cols] float32 -> (codes uint8 [rows, cols], scale bytes uint8 [rows, cols/32])."""
    rows, cols = x.shape
    v = x.astype(np.float64).reshape(rows, cols // 32, 32)
    bad = ~np.isfinite(v).all(-1)
    amax = np.abs(np.where(np.isfinite(v), v, 0.0)).max(-1)
    X = np.where(amax > 0, np.frexp(amax)[1] - 1 - 2, -127).clip(-127, None)
    X = np.where(bad, 0, X)
    a = np.where(bad[..., None], 0.0, np.abs(v) * np.exp2(-X.astype(np.float64))[..., None])
    # nearest value, an equal distance to the even code
    d = np.abs(a[..., None] - E2M1)
    order = np.array([0, 2, 4, 6, 1, 3, 5, 7])
    code = order[np.argmin(d[..., order], -1)].astype(np.uint8)
    code = np.where((v < 0) & (code > 0), code + 8, code).astype(np.uint8)
    return code.reshape(rows, cols), np.where(bad, 255, X + 127).astype(np.uint8)


def pack(codes, scales):
    """The bytes of one matrix; the tail up to a multiple of 16 is zero here and undefined on the device."""
    rows, cols = codes.shape
    out = np.zeros(bytes_of(rows, cols), np.uint8)
    out[: rows * cols // 2] = (codes[:, 0::2] | (codes[:, 1::2] << 4)).reshape(-1)
    at = rows * cols // 2
    for q in range((cols + 127) // 128):
        p = np.full((rows, 4), 127, np.uint8)
        s = scales[:, 4 * q : 4 * q + 4]
        p[:, : s.shape[1]] = s
        out[at : at + 4 * rows] = p.reshape(-1)
        at += 4 * rows
    return out, at


def values(codes, scales):
    rows, cols = codes.shape
    v = np.where(codes & 8, -1.0, 1.0) * E2M1[codes & 7]
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return (v.reshape(rows, cols // 32, 32) * s[..., None]).reshape(rows, cols)


def activate(z, act):
    if act == "swiglu":
        f = z.shape[1] // 2
        with np.errstate(over="ignore"):
            return z[:, :f] / (1 + np.exp(-z[:, :f])) * z[:, f:]
    return np.maximum(z, 0) ** 2 if act == "relu2" else z


def balance(logits, idx, mask, n_seq):
    """(loss, counts, prob, tokens, gradient for an incoming 1), all from the definition in 64 bits."""
    T, E = logits.shape
    L, k = T // n_seq, idx.shape[1]
    mask = np.ones(T, bool) if mask is None else mask.astype(bool)
    counts, prob = np.zeros((n_seq, E), np.int64), np.zeros((n_seq, E))
    tokens = mask.reshape(n_seq, L).sum(1)
    p = np.zeros((T, E))
    for t in np.flatnonzero(mask):
        x = logits[t].astype(np.float64)
        if np.all(x == -np.inf):
            continue
        e = np.exp(x - x.max())
        p[t] = e / e.sum()
    live = max(1, int((tokens > 0).sum()))
    loss, grad = 0.0, np.zeros((T, E))
    for s in range(n_seq):
        n = tokens[s]
        if n == 0:
            continue
        for t in range(s * L, (s + 1) * L):
            if mask[t]:
                for e in idx[t]:
                    if 0 <= e < E:
                        counts[s, e] += 1
        prob[s] = p[s * L : (s + 1) * L].sum(0) / n
        f = counts[s] / (k * n)
        loss += E * (f * prob[s]).sum() / live
        ps = p[s * L : (s + 1) * L]
        grad[s * L : (s + 1) * L] = E / (live * n) * ps * (f - (ps * f).sum(1, keepdims=True))
    return loss, counts, prob, tokens, grad
