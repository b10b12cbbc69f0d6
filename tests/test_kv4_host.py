"""Host-side checks of the rotated appends, the 4-bit cache and the reads, and of
their oracle (CPU only: every call below is refused or empty)."""
import ctypes

import numpy as np
import pytest

import ternary_weight_linear_absmean_amd as bl
from oracle import kv4 as ref
from ternary_weight_linear_absmean_amd._native import BlRope, Kv4, Kv8

OK, NULL, SHAPE, DTYPE, ALIGN, WS = 0, 1, 2, 3, 4, 5
A16, B16, A4, A1 = 0x10000, 0x10000000, 0x10004, 0x10001
INT_MAX = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    return bl.load()


def kind(bits, **kw):
    d = dict(K=A16, V=A16, s1=A16, s2=A16, n_blocks=8, KVH=2, T=64, D=128)
    d.update(kw)
    return (Kv8 if bits == 8 else Kv4)(*d.values())


def rope(**kw):
    d = dict(cos_sin=A16, rows=1 << 40, rot=64, interleaved=0, reserved=0)
    d.update(kw)
    return BlRope(*d.values())


def each(lib, k=A16, v=B16, q=A16, o=B16, dt=0, n=3, QH=8, qs=A4, ln=A4, tb=A4, B=2, nb=4, r=None, c=None):
    """Status of the two appends and the two reads."""
    c = c or {}
    r = rope() if r is None else r
    rows = qs, ln, tb, B, nb
    return (lib.bitlinear_kv8_append_rope(k, v, q, o, dt, n, QH, *rows, kind(8, **c), r, None),
            lib.bitlinear_kv4_append(k, v, q, o, dt, n, QH, *rows, kind(4, **c), r, None),
            lib.bitlinear_kv8_read(kind(8, **c), *rows, n, k, v, dt, None),
            lib.bitlinear_kv4_read(kind(4, **c), *rows, n, k, v, dt, None))


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(n=2 ** 31), dict(B=-1), dict(B=1 << 24), dict(nb=-1), dict(nb=INT_MAX // 64 + 1),
    dict(c=dict(T=8)), dict(c=dict(T=48)), dict(c=dict(T=256)), dict(c=dict(D=32)), dict(c=dict(D=96)),
    dict(c=dict(D=0)), dict(c=dict(KVH=0)), dict(c=dict(KVH=65536)), dict(c=dict(n_blocks=-1)),
    dict(c=dict(n_blocks=2 ** 31))])
def test_shapes(lib, bad):
    assert each(lib, **bad) == (SHAPE,) * 4


@pytest.mark.parametrize("bad", [
    dict(r=rope(rot=0)), dict(r=rope(rot=8)), dict(r=rope(rot=24)), dict(r=rope(rot=-16)), dict(r=rope(rot=144)),
    dict(r=rope(rot=80), c=dict(D=64)), dict(r=rope(rows=255)), dict(r=rope(rows=-1)), dict(QH=-1), dict(QH=65536),
    dict(QH=65535, n=32769), dict(n=0, r=rope(rot=8)), dict(n=0, r=rope(rows=3))])
def test_rotations(lib, bad):
    assert each(lib, **bad)[:2] == (SHAPE,) * 2


def test_refusals(lib):
    assert each(lib, dt=7) == (DTYPE,) * 4
    for bad in (dict(k=None), dict(v=None), dict(qs=None), dict(ln=None), dict(tb=None), dict(c=dict(K=None)),
                dict(c=dict(V=None)), dict(c=dict(s1=None)), dict(c=dict(s2=None))):
        assert each(lib, **bad) == (NULL,) * 4, bad
    for bad in (dict(k=A4), dict(v=A4), dict(qs=A1), dict(ln=A1), dict(tb=A1), dict(c=dict(K=A4)),
                dict(c=dict(V=A4)), dict(c=dict(s1=A1)), dict(c=dict(s2=A1))):
        assert each(lib, **bad) == (ALIGN,) * 4, bad
    # 4-bit scales are read 16 bytes at a time
    assert each(lib, c=dict(s1=A4))[1::2] == (ALIGN,) * 2 and each(lib, c=dict(s2=A4))[1::2] == (ALIGN,) * 2
    for bad in (dict(q=None), dict(o=None), dict(r=rope(cos_sin=None))):
        assert each(lib, **bad)[:2] == (NULL,) * 2, bad
    for bad in (dict(q=A4), dict(o=A4), dict(r=rope(cos_sin=A4))):
        assert each(lib, **bad)[:2] == (ALIGN,) * 2, bad
    # no rows, no sequences, no room for a token
    assert each(lib, n=0, k=None, v=None, q=None, o=None) == (OK,) * 4
    assert each(lib, B=0, qs=None, ln=None, tb=None) == (OK,) * 4
    rows = A4, A4, A4, 2, 4
    assert lib.bitlinear_kv8_append_rope(A16, B16, None, None, 0, 3, 0, *rows, kind(8), None, None) == NULL
    for f, c, r in ((lib.bitlinear_kv8_append_rope, Kv8, rope()), (lib.bitlinear_kv4_append, Kv4, None)):
        assert f(A16, B16, None, None, 0, 3, 0, *rows, ctypes.POINTER(c)(), r, None) == NULL
    for f, c in ((lib.bitlinear_kv8_read, Kv8), (lib.bitlinear_kv4_read, Kv4)):
        assert f(ctypes.POINTER(c)(), *rows, 3, A16, B16, 0, None) == NULL


def test_overlaps(lib):
    """3 rows of 8 heads (q) or 2 (k, v) of 128 values, in each type."""
    for dt, es in ((0, 4), (1, 2)):
        size = 3 * 8 * 128 * es
        for by in (16, -16, size - 16, 16 - size):
            assert each(lib, dt=dt, q=B16, o=B16 + by)[:2] == (ALIGN,) * 2
        size = 3 * 2 * 128 * es
        for by in (0, 16, -16, size - 16, 16 - size):
            assert each(lib, dt=dt, k=B16, v=B16 + by)[2:] == (ALIGN,) * 2


def attend(lib, q=A16, o=1 << 40, dt=0, n=3, QH=8, qs=A4, ln=A4, tb=A4, B=2, nb=4, c=None, scale=1.0, ws=A16,
           size=1 << 40):
    c = kind(4, **(c or {}))
    return lib.bitlinear_kv4_attention(q, dt, n, QH, qs, ln, tb, B, nb, c, scale, o, ws, size, None)


def test_attention_refusals(lib):
    for bad in (dict(n=-1), dict(B=1 << 24), dict(nb=INT_MAX // 64 + 1), dict(c=dict(T=48)), dict(c=dict(D=96)),
                dict(c=dict(KVH=0)), dict(c=dict(n_blocks=-1)), dict(QH=0), dict(QH=-2), dict(QH=3), dict(QH=65536),
                dict(n=2 ** 28), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=2.0 ** 127)):
        assert attend(lib, **bad) == SHAPE, bad
    assert attend(lib, dt=2) == DTYPE
    for bad in (dict(q=None), dict(o=None), dict(qs=None), dict(ln=None), dict(tb=None), dict(c=dict(K=None)),
                dict(c=dict(s2=None))):
        assert attend(lib, **bad) == NULL, bad
    for bad in (dict(q=A4), dict(o=A4), dict(qs=A1), dict(c=dict(V=A4)), dict(c=dict(s1=A4)), dict(c=dict(s2=A4)),
                dict(ws=A4, nb=4000), dict(o=A16), dict(o=A16 + 3 * 8 * 128 * 4 - 16)):
        assert attend(lib, **bad) == ALIGN, bad
    assert attend(lib, n=0, q=None, o=None) == OK and attend(lib, B=0, qs=None, ln=None, tb=None) == OK


def test_attention_workspace(lib):
    """Sizes that are cut or read in parts ask for one; one byte less is refused.  The
    largest sizes are answered at once."""
    f = lib.bitlinear_kv4_attention_ws_bytes
    for n, QH, B, nb, KVH in ((3, 8, 2, 4000, 2), (64, 8, 64, 4000, 2), (300, 8, 1, 1000, 2), (256, 8, 256, 4000, 2)):
        need = f(n, QH, B, nb, KVH, 64, 128)
        assert need >= 2 * 4 * 130 * min(16, n * QH // KVH), (n, B, nb)
        for ws, size in ((None, need), (A16, need - 1), (A16, 0)):
            assert attend(lib, n=n, QH=QH, B=B, nb=nb, ws=ws, size=size) == WS
    assert f(3, 8, 2, 4, 2, 64, 128) == 0
    for bad in ((0, 8, 2, 4, 2, 64, 128), (3, 7, 2, 4, 2, 64, 128), (3, 8, 2, 4, 2, 63, 128), (3, 8, 2, -4, 2, 64, 128)):
        assert f(*bad) == 0
    big = 2 ** 31 - 1
    for n, QH, B, nb, KVH, T in ((20000, 65535, 20000, 1000, 65535, 64), (32768, 65535, 2 ** 24 - 1, big // 16, 65535, 16),
                                 (big, 1, 256, big // 128, 1, 128), (32768, 65535, 256, big // 64, 65535, 64),
                                 (1, 65535, 1, big // 64, 1, 64), (big, 1, 1, big // 64, 1, 64)):
        assert f(n, QH, B, nb, KVH, T, 128) < 2 ** 50, (n, QH, B)


def test_stack_refusals(lib):
    from ternary_weight_linear_absmean_amd._native import Layer, StackDims
    need8, need4 = lib.bitlinear_decode_stack_kv_ws_bytes, lib.bitlinear_decode_stack_kv4_ws_bytes

    def dims(H=512, KV=128, F=640, D=64, eps=1e-5, path=0):
        return StackDims(H, KV, F, D, eps, path, 0, 0)

    def call(d=None, L=None, n=1, c=None, x=A16, ws=A16, size=1 << 40, nb=4, qs=A4, ln=A4, tb=A4, scale=1.0, r=None):
        L = L or Layer(*[A16] * 14, None)
        c, r = dict(D=64) if c is None else c, rope() if r is None else r
        rest = n, d or dims(), qs, ln, tb, nb, r, scale, x, None, ws, size, None
        return (lib.bitlinear_decode_stack_kv_rope(L, kind(8, **c), *rest),
                lib.bitlinear_decode_stack_kv4(L, kind(4, **c), *rest))
    for d in (dims(H=500), dims(D=32), dims(path=2), dims(eps=-1.0), dims(KV=192)):
        assert call(d) == (SHAPE,) * 2 and need4(d, 64, 4) == 0
    for kw in (dict(c=dict(D=128)), dict(c=dict(D=64, KVH=1)), dict(c=dict(D=64, T=8)), dict(nb=-1), dict(n=-1),
               dict(scale=float("nan")), dict(r=rope(rot=24)), dict(r=rope(rot=128)), dict(r=rope(rows=255))):
        assert call(**kw) == (SHAPE,) * 2, kw
    assert call(n=0, x=None, ws=None) == (OK,) * 2
    for kw in (dict(x=None), dict(qs=None), dict(c=dict(D=64, s1=None)), dict(r=rope(cos_sin=None))):
        assert call(**kw) == (NULL,) * 2, kw
    for kw in (dict(x=A4), dict(ws=A4), dict(c=dict(D=64, V=A4)), dict(r=rope(cos_sin=A4))):
        assert call(**kw) == (ALIGN,) * 2, kw
    assert lib.bitlinear_decode_stack_kv_rope(Layer(*[A16] * 14, None), kind(8, D=64), 1, dims(), A4, A4, A4, 4, None, 1.0,
                                              A16, None, A16, 1 << 40, None) == NULL
    for need in (need8, need4):
        assert need(dims(), 64, 4) >= lib.bl_workspace_bytes(bl.BL_OP_DECODE_STACK, 1, 512, 128, 640)
    assert call(ws=None) == (WS,) * 2 and call(size=min(need8(dims(), 64, 4), need4(dims(), 64, 4)) - 1) == (WS,) * 2


# ------------------------------------------------------------- the oracle

def test_oracle_rotation_by_hand():
    """A quarter and an eighth of a turn, both pairings; the last two values stay."""
    h = np.float32(0.5) ** np.float32(0.5)
    table = np.array([[1, 1, 0, 0], [0, h, 1, h]], np.float32)
    x = np.array([[[1.0, 2, 3, 4, 5, 6]]] * 3)
    halves = ref.rotate(x, [0, 1, 7], table, False, 2)
    assert halves[0].tolist() == halves[2].tolist() == x[0].tolist()
    r = float(h)
    assert np.allclose(halves[1, 0], [-3, -2 * r, 1, 6 * r, 5, 6], rtol=1e-7)
    near = ref.rotate(x, [1], table, True, 2)
    assert np.allclose(near[0, 0], [-2, 1, -r, 7 * r, 5, 6], rtol=1e-7)


def test_oracle_codes_by_hand():
    z, s, u = ref.codes(np.array([[0.0, 15, 7.4, 7.5], [-2, -2, -2, -2], [1e6, -1e6, 0, 1]]))
    assert z.tolist() == [0, -2, -65504] and s.tolist() == [1, 0, 8736]
    assert u.tolist() == [[0, 15, 7, 8], [0, 0, 0, 0], [15, 0, 7, 7]]
    below = ref.f16_below(np.array([1.0, 1 + 2.0 ** -11, -1 - 2.0 ** -11, 0, -1e-9, 1e-9, 65504, -65504, 2.0 ** -24]))
    assert below.tolist() == [1, 1, -1 - 2.0 ** -10, 0, -2.0 ** -24, 0, 65504, -65504, 2.0 ** -24]


def test_oracle_f16_below_is_the_neighbour():
    x = np.random.default_rng(1).standard_normal(4000) * 10.0 ** np.random.default_rng(2).uniform(-8, 4, 4000)
    b = ref.f16_below(x)
    assert (b.astype(np.float16) == b).all() and (b <= x).all()
    up = np.nextafter(b.astype(np.float16), np.float16(np.inf)).astype(np.float64)
    assert (up > x).all()


def test_oracle_packing():
    u = np.random.default_rng(0).integers(0, 16, (2, 2, 3, 32, 64))
    K, V = ref.pack(*u)
    assert K.shape == (2, 3, 32, 32) and V.shape == (2, 3, 2, 64, 8)
    assert K[1, 2, 5, 3] == u[0, 1, 2, 5, 6] | u[0, 1, 2, 5, 7] << 4
    assert V[1, 2, 1, 9, 3] == u[1, 1, 2, 22, 9] | u[1, 1, 2, 23, 9] << 4
    k, v = ref.unpack(K, V)
    assert np.array_equal(k, u[0]) and np.array_equal(v, u[1])


def test_turned_queries_apart_from_the_new_rows(lib):
    """3 query rows of 8 heads beside key and value rows of 2, of 128 values each."""
    far = 1 << 40
    for dt, es in ((0, 4), (1, 2)):
        q_size, size = 3 * 8 * 128 * es, 3 * 2 * 128 * es
        for by in (0, 16 - q_size, size - 16):
            for q in (far, B16 + by):                       # from elsewhere and in place
                assert each(lib, dt=dt, k=B16, v=2 * far, q=q, o=B16 + by)[:2] == (ALIGN,) * 2
                assert each(lib, dt=dt, k=2 * far, v=B16, q=q, o=B16 + by)[:2] == (ALIGN,) * 2


def test_binding_has_no_thread_local_storage():
    """_calls.so has no PT_TLS (7) among its ELF program headers (see build.py)."""
    import struct

    from ternary_weight_linear_absmean_amd import build

    with open(build.CALLS, "rb") as f:
        elf = f.read()
    assert elf[:5] == b"\x7fELF\x02"
    offset, = struct.unpack_from("<Q", elf, 32)
    size, count = struct.unpack_from("<HH", elf, 54)
    assert 7 not in [struct.unpack_from("<I", elf, offset + i * size)[0] for i in range(count)]


def test_a_lone_sequence_may_bring_fewer_rows_than_its_call(lib):
    """A captured call holds rows for more tokens than a replay brings: one token on 4000
    keys in it is read in parts all the same, which shows in the workspace (5 heads of 4, blocks
    of 64)."""
    for f, most in ((lib.bitlinear_kv8_attention_ws_bytes, 128), (lib.bitlinear_kv4_attention_ws_bytes, 512)):
        for rows in (1, 32, 64, 100, 128, 206, 256, 400, 512):
            if rows <= most:
                assert f(rows, 20, 1, 63, 5, 64, 128) > 0, rows
    # on the 8-bit cache also where the keys are few; on the 4-bit one while a full call's units
    # do not fill the GPU
    for rows in (52, 128, 200, 224):
        assert lib.bitlinear_kv8_attention_ws_bytes(rows, 20, 1, 28, 5, 64, 128) > 0, rows
    for rows in (52, 128, 256, 400):
        assert lib.bitlinear_kv4_attention_ws_bytes(rows, 20, 1, 28, 5, 64, 128) > 0, rows


@pytest.fixture
def unloaded(lib):
    """The binding before its first load(); as it was afterwards."""
    native = bl._native
    was = native._lib, native._calls
    native._lib = native._calls = None
    yield native
    native._lib, native._calls = was
    if was[1] is not None:
        native._bind(was[0], was[1])


def test_the_short_way_is_built_here(lib):
    """Where the build has all it needs, the calls on the caches go through _calls.so."""
    assert bl._native._calls is not None


@pytest.mark.parametrize("error", [ImportError("No module named _calls"), ImportError("undefined symbol")])
def test_the_library_loads_without_the_short_way(unloaded, monkeypatch, error):
    """_calls.so saves host time and nothing else: where it cannot be imported, the calls
    are made through ctypes."""
    def fails(name, package=None):
        raise error
    monkeypatch.setattr(unloaded.importlib, "import_module", fails)
    with pytest.warns(RuntimeWarning, match="_calls"):
        loaded = unloaded.load()
    assert loaded.bl_abi_version() and unloaded._calls is None


def test_a_short_way_of_another_torch_is_not_taken(unloaded, monkeypatch):
    calls = unloaded.importlib.import_module("._calls", bl.__name__)
    monkeypatch.setattr(calls, "built_for", "torch 0.4.1, Python 3.6")
    with pytest.warns(RuntimeWarning, match="0.4.1"):
        unloaded.load()
    assert unloaded._calls is None
    with pytest.raises(TypeError):                     # refused by the long way
        bl.bitlinear_kv4_attention(None, None, None, None, None)


def test_the_library_builds_without_the_short_way(monkeypatch, tmp_path, capsys):
    """A compiler that is missing or fails: the build says so, and leaves no _calls.so of an
    earlier build behind."""
    from ternary_weight_linear_absmean_amd import build
    for compiler in ("false", str(tmp_path / "none")):
        old = tmp_path / "_calls.so"
        old.write_bytes(b"")
        monkeypatch.setattr(build, "CALLS", str(old))
        monkeypatch.setenv("CXX", compiler)
        assert build.build_calls(False) is None
        assert not old.exists() and "_calls.so" in capsys.readouterr().err


def test_oracle_codes_are_this_near():
    """|x - (z + s u)| <= max(s / 2, 15 2^-25).  Away from the last code a value is off by
    half a step; at the last one by 15 times what s lost, 2^-25 where s is subnormal and
    2^-11 of it (less than half a step) where not.  x - z and the quotient are rounded
    to 24 bits, so a border between codes may move by 2^-22 of the spread."""
    r = np.random.default_rng(5)
    worst = 0.0
    for spread in 10.0 ** np.arange(-10, 4.6, 0.25):
        for middle in (0.0, 1.0, -0.37):
            x = ((r.random((400, 64)) - 0.5 + middle) * spread).astype(np.float32).astype(np.float64)
            z, s, u = ref.codes(x)
            wide = x.max(-1) - z
            off = np.abs(x - z[:, None] - s[:, None] * u).max(-1)
            assert (off <= np.maximum(s / 2, 15 * 2.0 ** -25) + wide * 2.0 ** -22).all(), (spread, middle)
            # for subnormal steps the second bound is needed, and met within a factor of two
            if s.max() < 2.0 ** -14:
                worst = max(worst, (off / (15 * 2.0 ** -25))[off > s].max(initial=0.0))
    assert 0.5 < worst <= 1
