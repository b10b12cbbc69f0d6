"""Host-side checks of the cache, attention and 4-bit weight calls, and of
their oracle (CPU only: every call below is refused or empty)."""
import ctypes

import numpy as np
import pytest

import ternary_weight_linear_absmean_amd as bl
from oracle import kv8 as ref
from ternary_weight_linear_absmean_amd._native import Kv8

OK, NULL, SHAPE, DTYPE, ALIGN, WS = 0, 1, 2, 3, 4, 5
A16, A4, A1 = 0x10000, 0x10004, 0x10001
INT_MAX = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    return bl.load()


def cache(**kw):
    d = dict(K=A16, V=A16, sk=A4, sv=A4, n_blocks=8, KVH=2, T=64, D=128)
    d.update(kw)
    return Kv8(*d.values())


def rows(n=3, q=A16, o=A16, dt=0, qs=A4, ln=A4, tb=A4, B=2, nb=4, c=None):
    return q, o, dt, n, qs, ln, tb, B, nb, cache() if c is None else c


def both(lib, **kw):
    """Status of the append and of the attention (8 query heads)."""
    q, o, dt, n, qs, ln, tb, B, nb, c = rows(**kw)
    a = lib.bitlinear_kv8_append(q, o, dt, n, qs, ln, tb, B, nb, c, None)
    t = lib.bitlinear_kv8_attention(q, dt, n, 8, qs, ln, tb, B, nb, c, 1.0, o, A16, 1 << 40, None)
    return a, t


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(n=2 ** 31), dict(B=-1), dict(B=1 << 24), dict(nb=-1), dict(nb=INT_MAX // 64 + 1),
    dict(c=cache(T=8)), dict(c=cache(T=48)), dict(c=cache(T=256)), dict(c=cache(D=32)), dict(c=cache(D=96)),
    dict(c=cache(D=0)), dict(c=cache(KVH=0)), dict(c=cache(KVH=65536)), dict(c=cache(n_blocks=-1)),
    dict(c=cache(n_blocks=2 ** 31))])
def test_cache_shapes(lib, bad):
    assert both(lib, **bad) == (SHAPE, SHAPE)


def test_cache_refusals(lib):
    assert both(lib, dt=7) == (DTYPE, DTYPE)
    for bad in (dict(q=None), dict(o=None), dict(qs=None), dict(ln=None), dict(tb=None), dict(c=cache(K=None)),
                dict(c=cache(V=None)), dict(c=cache(sk=None)), dict(c=cache(sv=None))):
        assert both(lib, **bad) == (NULL, NULL)
    for bad in (dict(q=A4), dict(o=A4), dict(qs=A1), dict(ln=A1), dict(tb=A1), dict(c=cache(K=A4)),
                dict(c=cache(V=A4)), dict(c=cache(sk=A1)), dict(c=cache(sv=A1))):
        assert both(lib, **bad) == (ALIGN, ALIGN)
    # no rows, no sequences
    assert both(lib, n=0, q=None, o=None) == (OK, OK)
    assert both(lib, B=0, qs=None, ln=None, tb=None) == (OK, OK)
    assert lib.bitlinear_kv8_append(*rows()[:9], ctypes.POINTER(Kv8)(), None) == NULL


def test_attention_refusals(lib):
    def att(QH=8, scale=1.0, ws=A16, ws_bytes=1 << 40, n=3, nb=4):
        q, o, dt, n, qs, ln, tb, B, nb, c = rows(n=n, nb=nb)
        return lib.bitlinear_kv8_attention(q, dt, n, QH, qs, ln, tb, B, nb, c, scale, o, ws, ws_bytes, None)
    assert [att(QH=h) for h in (0, -2, 3, 65536)] == [SHAPE] * 4
    assert att(QH=8, n=2 ** 28) == SHAPE
    assert [att(scale=x) for x in (float("nan"), float("inf"), -float("inf"))] == [SHAPE] * 3
    need = lib.bitlinear_kv8_attention_ws_bytes(3, 8, 2, 4000, 2, 64, 128)
    assert att(nb=4000, ws=A4) == ALIGN
    if need:
        assert att(nb=4000, ws=None) == WS
        assert att(nb=4000, ws_bytes=need - 1) == WS
    f = lib.bitlinear_kv8_attention_ws_bytes
    assert f(0, 8, 2, 4, 2, 64, 128) == 0 and f(3, 7, 2, 4, 2, 64, 128) == 0
    assert f(3, 8, 2, 4, 2, 63, 128) == 0 and f(3, 8, 2, -4, 2, 64, 128) == 0
    # the largest sizes: answered at once, and a workspace that a card can hold where a call may
    big = 2 ** 31 - 1
    for n, QH, B, nb, KVH, T in ((20000, 65535, 20000, 1000, 65535, 64), (32768, 65535, 2 ** 24 - 1, big // 16, 65535, 16),
                                 (big, 1, 256, big // 128, 1, 128), (32768, 65535, 256, big // 64, 65535, 64),
                                 (256, 65535, 256, big // 64, 65535, 64), (1, 65535, 1, big // 64, 1, 64),
                                 (1, 1, 2 ** 24 - 1, 0, 1, 64), (big, 1, 1, big // 64, 1, 64)):
        assert f(n, QH, B, nb, KVH, T, 128) < 2 ** 50, (n, QH, B)


def test_w4_refusals(lib):
    qt, dq, gv = lib.quant_weight_absmax_i4, lib.dequant_weight_i4, lib.bitlinear_gemv_w4

    def each(W=A16, dt=0, M=1, N=8, K=128, g=32, w=A16, s=A4, Y=A4):
        return (qt(W, dt, N, K, g, w, s, None), dq(w, s, N, K, g, W, dt, None),
                gv(W, dt, M, w, s, N, K, g, Y, None))
    for bad in (dict(N=-1), dict(N=2 ** 31), dict(K=-32), dict(K=2 * bl.BL_MAX_K), dict(K=96, g=64), dict(g=16),
                dict(g=0), dict(g=-32), dict(g=256), dict(N=INT_MAX, K=1024)):
        assert each(**bad) == (SHAPE,) * 3, bad
    assert each(dt=2) == (DTYPE,) * 3
    for bad in (dict(W=None), dict(w=None), dict(s=None)):
        assert each(**bad) == (NULL,) * 3
    for bad in (dict(W=A4), dict(w=A4), dict(s=A1)):
        assert each(**bad) == (ALIGN,) * 3
    assert gv(A16, 0, 1, A16, A4, 8, 128, 32, None, None) == NULL
    assert gv(A16, 0, 1, A16, A4, 8, 128, 32, A1, None) == ALIGN
    assert [gv(A16, 0, m, A16, A4, 8, 128, 32, A4, None) for m in (-1, 17)] == [SHAPE] * 2
    assert each(N=0, W=None, w=None, s=None) == (OK,) * 3
    assert each(K=0, W=None, w=None, s=None)[:2] == (OK,) * 2
    assert gv(None, 0, 0, None, None, 8, 128, 32, None, None) == OK


# ------------------------------------------------------------- the oracle

def test_oracle_append_by_hand():
    """One head, T = 4: a fresh block, a token below its scale, one above."""
    codes, scale = np.full((2, 1, 4, 2), 99, np.int8), np.full((2, 1), 9.0, np.float32)
    table = np.array([[1]])

    def put(x, n, length):
        ref.append(np.array(x, dtype=np.float64).reshape(n, 1, 2), codes, scale, [0, n], [length], table)
    put([[127, -64], [0.5, 1.5]], 2, 2)
    assert scale[1, 0] == 1 and codes[1, 0, :2].tolist() == [[127, -64], [0, 2]]
    put([[3, -126.6]], 1, 3)
    assert scale[1, 0] == 1 and codes[1, 0, 2].tolist() == [3, -127]
    put([[254, 1]], 1, 4)
    assert scale[1, 0] == 2
    assert codes[1, 0].tolist() == [[64, -32], [0, 1], [2, -64], [127, 0]]
    assert (codes[0] == 99).all() and scale[0, 0] == 9


def test_oracle_attention_by_hand():
    """Two keys with weights 1/4 and 3/4; causal; a row before them is zero."""
    K = np.zeros((1, 1, 16, 2), np.int8)
    K[0, 0, 1, 0] = 1
    V = np.zeros((1, 1, 2, 16), np.int8)
    V[0, 0, :, 0], V[0, 0, :, 1] = [4, 8], [8, -8]
    q = np.array([[[np.log(3.0), 5.0]]] * 3)
    one = np.ones((1, 1), np.float32)
    out, wide, _, _ = ref.attention(q, K, V, one, one, [0, 3], [2], np.array([[0]]), 1.0)
    assert np.allclose(out[:, 0], [[0, 0], [4, 8], [7, -4]])
    assert np.allclose(wide[2, 0], [7, 8])


def test_oracle_w4_by_hand():
    W = np.zeros((1, 64))
    W[0, :4] = [7, -3.5, 0.5, 1.5]
    W[0, 33] = 14
    q, s = ref.quant_w4(W, 32)
    assert q[0, :4].tolist() == [7, -4, 0, 2] and q[0, 33] == 7 and s.tolist() == [[1, 2]]
    assert ref.unpack_w4(np.array([[0xF8, 0x71]], np.uint8)).tolist() == [[-8, -1, 1, 7]]
    assert ref.bf16(np.array([1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8])).tolist() == [1, 1 + 2.0 ** -6]


def test_stack_kv_refusals(lib):
    from ternary_weight_linear_absmean_amd._native import Layer, StackDims
    f, need = lib.bitlinear_decode_stack_kv, lib.bitlinear_decode_stack_kv_ws_bytes

    def dims(H=512, KV=128, F=640, D=64, eps=1e-5, path=0):
        return StackDims(H, KV, F, D, eps, path, 0, 0)

    def call(d=None, L=None, n=1, c=None, x=A16, ws=A16, size=1 << 40, nb=4, qs=A4, ln=A4, tb=A4, scale=1.0):
        L = L or Layer(*[A16] * 14, None)
        c = cache(D=64) if c is None else c
        return f(L, c, n, d or dims(), qs, ln, tb, nb, scale, x, None, ws, size, None)
    for d in (dims(H=500), dims(D=32), dims(D=256), dims(path=2), dims(path=-1), dims(eps=-1.0), dims(KV=192)):
        assert call(d) == SHAPE
        assert need(d, 64, 4) == 0
    for c in (cache(D=128), cache(D=64, KVH=1), cache(D=64, T=8), cache(D=64, n_blocks=-1)):
        assert call(c=c) == SHAPE
    assert call(nb=-1) == SHAPE and call(nb=2 ** 31) == SHAPE and call(n=-1) == SHAPE
    assert call(scale=float("nan")) == SHAPE
    assert call(n=0, x=None, ws=None) == OK
    for kw in (dict(x=None), dict(qs=None), dict(ln=None), dict(tb=None), dict(c=cache(D=64, K=None)),
               dict(L=Layer(*[A16] * 13, None, None))):
        assert call(**kw) == NULL
    for kw in (dict(x=A4), dict(ws=A4), dict(qs=A1), dict(c=cache(D=64, V=A4))):
        assert call(**kw) == ALIGN
    size = need(dims(), 64, 4)
    assert size >= lib.bl_workspace_bytes(bl.BL_OP_DECODE_STACK, 1, 512, 128, 640)
    assert call(ws=None) == WS and call(size=size - 1) == WS


def test_scales_past_the_kernels_range(lib):
    """scale * log2(e) is an fp32 in the kernels: refused where it would be infinite."""
    from ternary_weight_linear_absmean_amd._native import Layer, StackDims
    q, o, dt, n, qs, ln, tb, B, nb, c = rows()
    for scale in (2.0 ** 127, 2.4e38, -2.4e38, 3.4e38, -3.4e38):
        assert lib.bitlinear_kv8_attention(q, dt, n, 8, qs, ln, tb, B, nb, c, scale, o, A16, 1 << 40, None) == SHAPE
        assert lib.bitlinear_decode_stack_kv(Layer(*[A16] * 14, None), cache(D=64), 1,
                                             StackDims(512, 128, 640, 64, 1e-5, 0, 0, 0), A4, A4, A4, 4, scale, A16,
                                             None, A16, 1 << 40, None) == SHAPE


def test_attention_refuses_out_over_q(lib):
    """3 rows of 8 heads of 128 values, in each type."""
    for dt, size in ((0, 3 * 8 * 128 * 4), (1, 3 * 8 * 128 * 2)):
        for by in (0, 16, -16, size - 16, 16 - size):
            q, o, _, n, qs, ln, tb, B, nb, c = rows(q=A16 << 4, o=(A16 << 4) + by)
            assert lib.bitlinear_kv8_attention(q, dt, n, 8, qs, ln, tb, B, nb, c, 1.0, o, A16, 1 << 40, None) == ALIGN
            assert b"overlaps" in lib.bl_last_error()


def test_attention_workspace_is_asked_for_and_checked(lib):
    """Sizes that are cut or read in parts: a size above 0, and one byte less refused."""
    f = lib.bitlinear_kv8_attention_ws_bytes
    for n, QH, B, nb, KVH in ((3, 8, 2, 4000, 2), (1, 8, 1, 63, 2), (64, 8, 64, 4000, 2), (200, 8, 2, 1000, 2),
                              (300, 8, 1, 1000, 2), (256, 8, 256, 4000, 2)):
        need = f(n, QH, B, nb, KVH, 64, 128)
        # a line of 128 values and its two sums for each row of two pieces at least
        assert need >= 2 * 4 * 130 * min(16, n * QH // KVH), (n, B, nb)
        q, o, dt, _, qs, ln, tb, _, _, c = rows(q=A16, o=1 << 40)
        for ws, size in ((None, need), (A16, need - 1), (A16, 0)):
            assert lib.bitlinear_kv8_attention(q, dt, n, QH, qs, ln, tb, B, nb, c, 1.0, o, ws, size, None) == WS
    # nothing is cut: short tables, and more than 256 sequences of few rows
    assert f(3, 8, 2, 4, 2, 64, 128) == 0 and f(257, 8, 257, 4000, 2, 64, 128) == 0
