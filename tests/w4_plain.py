"""Plain 64-bit forms of the 4-bit weight operators (numpy, no code shared with the library), with
the rounding bounds that the GPU tests compare against.

Bounds.  A sum in which no term passes through more than d additions, each rounding by at most u of
its result, is off by at most d u (1 + d u) sum|terms|.  The tensor cores' binary32 adder may cut
instead of round, so u = 2^-23 there; the products of bf16 numbers are exact.  A term of a product
with packed weights goes through at most 128 additions of its group, then one for each group of its
row, and 8 + 8 + 8 for the warps, the cluster and the parts of a binary32 x: depth(K, group)."""
import numpy as np

U = 2.0 ** -23
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def row_bytes(K):
    return -(-K // 128) * 64


def place(K):
    """(byte, shift) of the code of each k within its row."""
    k = np.arange(K)
    b, w, t, i = k // 128, k % 128 // 32, k % 32 // 8, k % 8
    nib = i // 2 + 4 * (i % 2)
    return 64 * b + 16 * t + 4 * w + nib // 2, 4 * (nib % 2)


def pack(codes):
    """Codes [N, K] -> packed rows [N, row_bytes(K)]."""
    N, K = codes.shape
    out = np.zeros((N, row_bytes(K)), np.uint8)
    byte, shift = place(K)
    for k in range(K):
        out[:, byte[k]] |= (codes[:, k].astype(np.uint8) << shift[k]).astype(np.uint8)
    return out


def unpack(wq, K):
    byte, shift = place(K)
    return (wq[:, byte] >> shift.astype(np.uint8)) & 15


def bf16(a):
    """binary32 rounded to bf16 (nearest, ties to even), as binary32."""
    u = np.ascontiguousarray(a, np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7fff + ((u >> 16) & 1)) & 0xffff0000
    return u.astype(np.uint32).view(np.float32)


def quantise(W, s, group, asym):
    """The definition in binary32, one rounding per operation: codes [N, K], scales [G, N], zeros [G, N] or None."""
    f = np.float32
    K, N = W.shape
    w = W.astype(f) if s is None else (s.astype(f)[:, None] * W.astype(f))
    codes = np.zeros((N, K), np.uint8)
    scales, zeros = [], []
    for k0 in range(0, K, group):
        v = w[k0:k0 + group]
        if asym:
            lo, hi = np.minimum(v.min(0), f(0)), np.maximum(v.max(0), f(0))
            sc = bf16((hi - lo) * (f(1) / f(15)))
        else:
            sc = bf16(np.abs(v).max(0) * (f(1) / f(7)))
        d = np.where(sc == 0, f(1), sc)
        q = np.where(sc == 0, f(0), np.rint(v / d))
        if asym:
            z = np.where(sc == 0, f(0), np.clip(np.rint(-lo / d), 0, 15))
            zeros.append(z.astype(np.uint8))
            c = np.clip(q + z, 0, 15)
        else:
            c = np.clip(q, -7, 7) + 8
        codes[:, k0:k0 + group] = c.T.astype(np.uint8)
        scales.append(sc)
    return codes, np.stack(scales), np.stack(zeros) if asym else None


def values(wq, sg, zp, K, group):
    """What packed weights stand for, [N, K] in binary64."""
    at = np.arange(K) // group
    zero = 8.0 if zp is None else zp.astype(np.float64).T[:, at]
    return (unpack(wq, K).astype(np.float64) - zero) * sg.astype(np.float64).T[:, at]


def depth(K, group):
    return 128 + -(-K // group) + 24


def product(x, w, group):
    """x [M, K] times w [N, K]^T in binary64, and the bound on a binary32 evaluation's error."""
    x = x.astype(np.float64)
    return x @ w.T, depth(x.shape[1], group) * U * 1.01 * (np.abs(x) @ np.abs(w).T)


def choose(x, wr, top_k, renorm):
    logits = x.astype(np.float64) @ wr.astype(np.float64).T
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :top_k]
    p = np.exp(logits - logits.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    w = np.take_along_axis(p, ids, 1)
    if renorm:
        w = w / w.sum(1, keepdims=True)
    return ids, w


def experts(x, ids, wts, w13, w2, group, h_part, w_off):
    """The experts' sum for choices ids, wts [T, k]; w13(e), w2(e): values.  Returns y and the bound on a
    binary32 evaluation whose h enters the last product with relative error h_part and whose weights are off by
    w_off of themselves.  exp and the division are within 4 + 1 units of 2^-24."""
    T, D = x.shape
    y, off = np.zeros((T, D)), np.zeros((T, D))
    for e in np.unique(ids[ids >= 0]):
        a, b = w13(int(e)), w2(int(e))
        F = b.shape[1]
        for t in range(T):
            w = wts[t][ids[t] == e].astype(np.float64).sum()
            if not (ids[t] == e).any():
                continue
            gu, dgu = product(x[t:t + 1], a, group)
            g, u, dg, du = gu[0, :F], gu[0, F:], dgu[0, :F], dgu[0, F:]
            silu = g / (1 + np.exp(-g))
            h = silu * u
            # |silu'| <= 1.1
            dh = 1.1 * dg * (np.abs(u) + du) + np.abs(silu) * du + np.abs(h) * (16 * 2.0 ** -24 + h_part)
            out, dout = product(h[None], b, group)
            dout = dout[0] + np.abs(b) @ dh * (1 + depth(F, group) * U * 1.01)
            y[t] += w * out[0]
            # the sum over the chosen experts: their number of additions, and one product each
            off[t] += abs(w) * (dout + np.abs(out[0]) * (w_off + 2.0 ** -20))
    return y, off
