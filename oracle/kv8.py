"""64-bit reference of the 8-bit key/value cache, the attention over it, and
4-bit weights with group scales (numpy).

A quotient that the format rounds to fp32 is formed in fp64 and rounded once,
which is the correctly rounded fp32 quotient (53 >= 2 * 24 + 2 bits).
"""
import numpy as np


def f32(x):
    return np.asarray(x, dtype=np.float64).astype(np.float32).astype(np.float64)


def bf16(x):
    """fp64 holding fp32 values -> fp64 holding the nearest bf16 (ties to even)."""
    w = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    w = (w + 0x7FFF + ((w >> 16) & 1)) >> 16 << 16
    return w.astype(np.uint32).view(np.float32).astype(np.float64)


def rows_of(q_start, lengths, n_tok):
    """(sequence, row, position) of every new row, in order."""
    out = []
    for b in range(len(lengths)):
        lo, hi = (min(max(int(q_start[i]), 0), n_tok) for i in (b, b + 1))
        for r in range(lo, hi):
            out.append((b, r, int(lengths[b]) - (hi - r)))
    return out


def block_of(table, b, pos, T, n_blocks):
    """The block that holds position pos of sequence b, or None."""
    if pos < 0 or pos // T >= table.shape[1]:
        return None
    i = int(table[b][pos // T])
    return i if 0 <= i < n_blocks else None


def append(x, codes, scale, q_start, lengths, table):
    """x fp64 [n_tok, KVH, D] into codes int8 [n_blocks, KVH, T, D] (V: pass it
    transposed) and scale fp32 [n_blocks, KVH], in place."""
    T = codes.shape[2]
    blocks = {}
    for b, r, pos in rows_of(q_start, lengths, len(x)):
        i = block_of(table, b, pos, T, len(codes))
        if i is not None:
            blocks.setdefault(i, []).append((pos % T, r))
    for i, new in blocks.items():
        slots, rows = [s for s, _ in new], [r for _, r in new]
        d = f32(np.abs(x[rows]).max(axis=(0, 2)) / 127)
        if min(slots) > 0:
            s = scale[i].astype(np.float64)
            for h in np.nonzero(d > s)[0]:
                fit = f32(s[h] / d[h])
                codes[i, h] = np.rint(f32(codes[i, h].astype(np.float64) * fit)).astype(np.int8)
            d = np.maximum(d, s)
        scale[i] = d
        safe = np.where(d > 0, d, 1)[None, :, None]
        q = np.clip(np.rint(f32(x[rows] / safe)), -127, 127) * (d > 0)[None, :, None]
        codes[i][:, slots] = q.transpose(1, 0, 2).astype(np.int8)


def attention(q, K, V, sk, sv, q_start, lengths, table, scale):
    """(out, wide, reach, far) fp64 for q fp64 [n_tok, QH, D]: the result, sum_j
    p_j |v_j| (what its rounding errors scale with), max_j scale sum |q k_j| and
    max_j scale max |q| sum |k_j|; rows of no sequence are NaN."""
    n_tok, QH, D = q.shape
    nb, KVH, T, _ = K.shape
    g = QH // KVH
    out = np.full(q.shape, np.nan)
    wide, reach, far = np.zeros(q.shape), np.zeros((n_tok, QH)), np.zeros((n_tok, QH))
    cached = {}
    for b, r, pos in rows_of(q_start, lengths, n_tok):
        if b not in cached:
            at = [(p, block_of(table, b, p, T, nb))
                  for p in range(min(int(lengths[b]), table.shape[1] * T))]
            at = [(p, i) for p, i in at if i is not None]
            p = np.array([p for p, _ in at], dtype=int)
            i = np.array([i for _, i in at], dtype=int)
            k = K[i, :, p % T].astype(np.float64) * sk[i].astype(np.float64)[..., None]
            v = V[i, :, :, p % T].astype(np.float64) * sv[i].astype(np.float64)[..., None]
            cached[b] = p, k, v
        p, k, v = cached[b]
        seen = p <= pos
        for h in range(QH):
            if not seen.any():
                out[r, h] = 0
                continue
            kk, vv = k[seen, h // g], v[seen, h // g]
            s = kk @ q[r, h] * scale
            w = np.exp(s - s.max())
            w /= w.sum()
            out[r, h], wide[r, h] = w @ vv, w @ np.abs(vv)
            reach[r, h] = abs(scale) * (np.abs(kk) @ np.abs(q[r, h])).max()
            far[r, h] = abs(scale) * np.abs(kk).sum(-1).max() * np.abs(q[r, h]).max()
    return out, wide, reach, far


def quant_w4(W, group):
    """W fp64 [N, K] -> codes int [N, K], scales fp64 [N, K / group]."""
    N, K = W.shape
    x = W.reshape(N, K // group, group)
    s = bf16(f32(np.abs(x).max(-1) / 7))
    safe = np.where(s > 0, s, 1)[..., None]
    q = np.clip(np.rint(f32(x / safe)), -7, 7) * (s > 0)[..., None]
    return q.reshape(N, K).astype(int), s


def unpack_w4(Wq4):
    """uint8 [N, K / 2] -> codes int [N, K]."""
    lo, hi = Wq4.astype(int) & 15, Wq4.astype(int) >> 4
    q = np.stack([lo, hi], -1).reshape(len(Wq4), -1)
    return np.where(q > 7, q - 16, q)
