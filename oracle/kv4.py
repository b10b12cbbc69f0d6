"""64-bit reference of the rotation, the 4-bit key/value cache, the attention
over it, and the reads of both caches (numpy).

What the format rounds to fp32 or fp16 is formed in fp64 and rounded once.
"""
import numpy as np

from .kv8 import block_of, f32, rows_of


def f16(x):
    return np.asarray(x, dtype=np.float64).astype(np.float16).astype(np.float64)


def f16_below(x):
    """The largest fp16 that is at most x: x's steps are 2^(e - 10), at least 2^-24."""
    x = np.asarray(x, dtype=np.float64)
    e = np.frexp(np.where(x == 0, 1, x))[1] - 1
    step = np.exp2(np.maximum(e, -14) - 10.0)
    return np.floor(x / step) * step


def rotate(x, pos, cos_sin, interleaved, room):
    """Rows x fp64 [n, heads, D], each turned for its position, rounded to fp32; rows
    at positions outside 0 .. room - 1 as they are."""
    out, rot = x.copy(), cos_sin.shape[1]
    half = rot // 2
    for r, p in enumerate(pos):
        if not 0 <= p < room:
            continue
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            c, s = (cos_sin[p, j].astype(np.float64) for j in (i, half + i))
            out[r, :, a] = f32(x[r, :, a] * c - x[r, :, b] * s)
            out[r, :, b] = f32(x[r, :, b] * c + x[r, :, a] * s)
    return out


def positions(q_start, lengths, n_tok, missing=-1):
    """Position of each row; `missing` for rows of no sequence."""
    pos = np.full(n_tok, missing, dtype=np.int64)
    for _, r, p in rows_of(q_start, lengths, n_tok):
        pos[r] = p
    return pos


def codes(x):
    """x fp64 [..., D] -> z, s fp64 [...] and codes int [..., D]."""
    x = np.clip(np.where(np.isnan(x), -65504, x), -65504, 65504)
    z = f16_below(x.min(-1))
    s = f16(f32(f32(x.max(-1) - z) / 15))
    safe = np.where(s > 0, s, 1)[..., None]
    u = np.clip(np.rint(f32(f32(x - z[..., None]) / safe)), 0, 15) * (s > 0)[..., None]
    return z, s, u.astype(int)


def unpack(K, V):
    """The cache's bytes -> codes int [n_blocks, KVH, T, D] of K and of V."""
    k = np.stack([K & 15, K >> 4], -1).reshape(*K.shape[:3], -1)
    v = np.stack([V & 15, V >> 4], -1).reshape(*V.shape[:4], 16)          # [..., T / 16, D, 16]
    v = v.transpose(0, 1, 2, 4, 3).reshape(k.shape)
    return k.astype(int), v.astype(int)


def pack(k, v):
    """unpack's inverse."""
    K = (k[..., 0::2] | k[..., 1::2] << 4).astype(np.uint8)
    nb, KVH, T, D = v.shape
    v = v.reshape(nb, KVH, T // 16, 16, D).transpose(0, 1, 2, 4, 3)
    return K, (v[..., 0::2] | v[..., 1::2] << 4).astype(np.uint8)


def append(x, u, zs, q_start, lengths, table):
    """Rows x fp64 [n_tok, KVH, D] into codes u int [n_blocks, KVH, T, D] and zs
    fp16 [n_blocks, KVH, T, 2], in place."""
    T = u.shape[2]
    for b, r, p in rows_of(q_start, lengths, len(x)):
        i = block_of(table, b, p, T, len(u))
        if i is not None:
            z, s, u[i, :, p % T] = codes(x[r])
            zs[i, :, p % T] = np.stack([z, s], -1)


def slots4(u, zs):
    """Every slot's values, fp64 [n_blocks, KVH, T, D], not rounded."""
    zs = zs.astype(np.float64)
    return zs[..., :1] + zs[..., 1:] * u


def read(slots, q_start, lengths, table, n_tok):
    """Rows [n_tok, KVH, D] of slots [n_blocks, KVH, T, D]; zeros where there is no
    token, NaN in rows of no sequence."""
    out = np.full((n_tok,) + slots.shape[1:2] + slots.shape[3:], np.nan)
    for b, r, p in rows_of(q_start, lengths, n_tok):
        i = block_of(table, b, p, slots.shape[2], len(slots))
        out[r] = 0 if i is None else slots[i, :, p % slots.shape[2]]
    return out


def attention(q, ku, kzs, vu, vzs, q_start, lengths, table, scale):
    """(out, wide, reach, far, near) fp64 for q fp64 [n_tok, QH, D] over codes and
    zs: the result, sum_j p_j (|z| + s u) of the values, max_j scale sum |q| (|z| + s u),
    max_j scale max |q| sum s u, and max_j scale sum |q k_j|; rows of no sequence
    are NaN."""
    n_tok, QH, D = q.shape
    nb, KVH, T, _ = ku.shape
    g = QH // KVH
    out = np.full(q.shape, np.nan)
    wide, reach, far, near = np.zeros(q.shape), *(np.zeros((n_tok, QH)) for _ in range(3))
    kzs, vzs = kzs.astype(np.float64), vzs.astype(np.float64)
    cached = {}
    for b, r, pos in rows_of(q_start, lengths, n_tok):
        if b not in cached:
            at = [(p, block_of(table, b, p, T, nb)) for p in range(min(int(lengths[b]), table.shape[1] * T))]
            at = [(p, i) for p, i in at if i is not None]
            p = np.array([p for p, _ in at], dtype=int)
            i = np.array([i for _, i in at], dtype=int)
            parts = []
            for u, zs in ((ku, kzs), (vu, vzs)):
                uu, z = u[i, :, p % T], zs[i, :, p % T]
                parts += [z[..., :1] + z[..., 1:] * uu, np.abs(z[..., :1]) + z[..., 1:] * uu]
            parts.append(kzs[i, :, p % T][..., 1:] * ku[i, :, p % T])
            cached[b] = p, parts
        p, parts = cached[b]
        seen = p <= pos
        for h in range(QH):
            if not seen.any():
                out[r, h] = 0
                continue
            k, ka, v, va, kc = (x[seen, h // g] for x in parts)
            s = k @ q[r, h] * scale
            w = np.exp(s - s.max())
            w /= w.sum()
            out[r, h], wide[r, h] = w @ v, w @ va
            reach[r, h] = abs(scale) * (ka @ np.abs(q[r, h])).max()
            far[r, h] = abs(scale) * kc.sum(-1).max() * np.abs(q[r, h]).max()
            near[r, h] = abs(scale) * (np.abs(k) @ np.abs(q[r, h])).max()
    return out, wide, reach, far, near
