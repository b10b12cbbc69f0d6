"""The rotated appends, the 4-bit key/value cache and the reads of both caches
against the 64-bit oracle: bytes, scales and rotated values exactly."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import kv4 as ref
from oracle import kv8 as ref8

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def make(seed, n, lens, T, D, KVH, dtype, G=1, bits=4, rot=0, near=False, spare=3, behind=0, before=0, width=0):
    """A filled cache, the new rows, a rotation and the arrays of a call: sequence b
    has lens[b] tokens, n[b] of them new; `before` / `behind` rows of no
    sequence; a table of `width` entries a sequence at least."""
    g = torch.Generator().manual_seed(seed)
    need = [max(0, -(-x // T)) for x in lens]
    nb = sum(need) + spare
    order = torch.randperm(nb, generator=g).tolist()
    table = torch.full((len(n), max(need + [1, width - 1]) + 1), -1, dtype=torch.int32)
    for b, m in enumerate(need):
        for j in range(m):
            table[b, j] = order.pop()
    rows = before + sum(n) + behind
    q_start = torch.tensor([before] + [before + sum(n[:b + 1]) for b in range(len(n))], dtype=torch.int32)
    s = dict(table=table, q_start=q_start, lengths=torch.tensor(lens, dtype=torch.int32))
    if bits == 8:
        def codes(*shape):
            return torch.randint(-127, 128, shape, generator=g).to(torch.int8)

        def scales():
            return (0.5 + torch.rand(nb, KVH, generator=g)) / 40
        s["cache"] = [codes(nb, KVH, T, D), codes(nb, KVH, D, T), scales(), scales()]
    else:
        def codes(*shape):
            return torch.randint(0, 256, shape, generator=g).to(torch.uint8)

        def zs():
            r = torch.rand(nb, KVH, T, 2, generator=g)
            return torch.stack([-3 * r[..., 0], 0.1 + 0.3 * r[..., 1]], -1).half()
        s["cache"] = [codes(nb, KVH, T, D // 2), codes(nb, KVH, T // 16, D, 8), zs(), zs()]
    for x, heads in (("k", KVH), ("v", KVH), ("q", KVH * G)):
        s[x] = torch.randn(rows, heads, D, generator=g).to(dtype)
    if rot:
        at = torch.arange(table.shape[1] * T, dtype=torch.float64)[:, None]
        a = at * 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
        s["cos_sin"], s["near"] = torch.cat([a.cos(), a.sin()], 1).float(), near
    return s


def cuda(s):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else [x.cuda() for x in v] if isinstance(v, list) else v
            for k, v in s.items()}


def host(s):
    return {k: v.cpu() if isinstance(v, torch.Tensor) else [x.cpu() for x in v] if isinstance(v, list) else v
            for k, v in s.items()}


def copied(s):
    return {k: v.clone() if isinstance(v, torch.Tensor) else [x.clone() for x in v] if isinstance(v, list) else v
            for k, v in s.items()}


def meta(s):
    return s["q_start"], s["lengths"], s["table"]


def meta64(s):
    return [x.cpu().numpy() for x in meta(s)]


def n64(t):
    return t.double().cpu().numpy()


def bits_of(s):
    return 8 if s["cache"][0].dtype == torch.int8 else 4


def append(bl, s, q=True, **kw):
    rope = bl.Rope(s["cos_sin"], s["near"]) if "cos_sin" in s else None
    q = s["q"] if q and rope else None
    if bits_of(s) == 8:
        return bl.bitlinear_kv8_append_rope(s["k"], s["v"], *meta(s), s["cache"], rope, q=q, **kw)
    return bl.bitlinear_kv4_append(s["k"], s["v"], *meta(s), s["cache"], rope, q=q, **kw)


def rows64(s, dtype):
    """The oracle's rotated q (rounded to dtype) and k, and v."""
    q, k, v = (n64(s[x]) for x in "qkv")
    if "cos_sin" in s:
        pos = ref.positions(*meta64(s)[:2], len(k))
        room = s["table"].shape[1] * s["cache"][2 if bits_of(s) == 4 else 0].shape[2]
        q, k = (ref.rotate(x, pos, s["cos_sin"].cpu().numpy(), s["near"], room) for x in (q, k))
    if dtype == BF16:
        q = ref8.bf16(q)
    return q, k, v


def want_append(s):
    """The cache after the call, and q rotated, by the oracle."""
    q, k, v = rows64(s, s["k"].dtype)
    c = [x.cpu().numpy().copy() for x in s["cache"]]
    m = meta64(s)
    if bits_of(s) == 8:
        vt = np.ascontiguousarray(c[1].transpose(0, 1, 3, 2))
        ref8.append(k, c[0], c[2], *m)
        ref8.append(v, vt, c[3], *m)
        c[1] = vt.transpose(0, 1, 3, 2)
    else:
        ku, vu = ref.unpack(c[0], c[1])
        ref.append(k, ku, c[2], *m)
        ref.append(v, vu, c[3], *m)
        c[0], c[1] = ref.pack(ku, vu)
    return c, q


def check_append(bl, s):
    d = cuda(s)
    fill = torch.full_like(d["q"], 77.0)
    out = append(bl, d, q_out=fill) if "cos_sin" in s else append(bl, d)
    c, q = want_append(s)
    for got, want in zip(d["cache"], c):
        assert np.array_equal(got.cpu().numpy(), want, equal_nan=got.dtype in (F32, torch.float16))
    if "cos_sin" in s:
        assert out is fill
        of_none = ref.positions(*meta64(s)[:2], len(q), missing=-10 ** 12) == -10 ** 12
        q[of_none] = 77.0
        assert np.array_equal(n64(out), q)
    return d


CASES = [
    # n, lens, T, D, KVH, G
    ([1], [1], 64, 128, 5, 4),
    ([1], [2], 16, 64, 1, 1),
    ([1], [200], 64, 128, 5, 4),
    ([1, 1, 1], [64, 65, 63], 64, 128, 2, 4),
    ([1] * 7, [1, 17, 16, 15, 128, 129, 300], 16, 64, 3, 7),
    ([1] * 70, [3 + 5 * i for i in range(70)], 32, 128, 1, 2),
    ([5, 3, 1, 0, 2], [5, 130, 77, 20, 2], 32, 64, 2, 4),
    ([40, 1, 90], [100, 31, 90], 16, 128, 2, 3),
    ([130], [259], 128, 64, 2, 1),
    ([129, 7], [300, 7], 128, 128, 1, 8),
    ([0, 0, 1, 0], [0, 9, 33, 0], 64, 64, 2, 16),
    ([2], [50], 64, 128, 1, 40),
    ([300], [300], 64, 128, 1, 4),
    ([33], [600], 64, 64, 3, 4),
]
ROTS = [(128, False), (64, True), (16, False), (32, True), (16, True), (48, False)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_append4(gpu, case, dtype):
    n, lens, T, D, KVH, G = CASES[case]
    check_append(gpu, make(case, n, lens, T, D, KVH, dtype, before=case % 3, behind=(case + 1) % 3))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_append_rotated(gpu, case, dtype, bits):
    n, lens, T, D, KVH, G = CASES[case]
    rot, near = ROTS[(case + (dtype == BF16)) % len(ROTS)]
    check_append(gpu, make(20 + case, n, lens, T, D, KVH, dtype, G, bits, min(rot, D), near, before=case % 3,
                           behind=(case + 1) % 3))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D,rot,near", [(64, 64, False), (128, 128, True), (128, 16, False), (64, 48, True),
                                        (128, 112, False), (64, 32, False)])
def test_rotations(gpu, D, rot, near, bits):
    check_append(gpu, make(50, [3, 40, 1], [70, 41, 90], 32, D, 3, F32, 2, bits, rot, near))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("near", [False, True])
def test_queries_rotated_in_place(gpu, near, dtype, bits):
    """q_out may be q itself; a part of it is refused."""
    s = make(51, [5, 1, 30], [70, 41, 90], 32, 128, 2, dtype, 4, bits, 64, near)
    d = cuda(s)
    assert append(gpu, d, q_out=d["q"]) is d["q"]
    assert np.array_equal(n64(d["q"]), want_append(s)[1])
    n = len(s["q"])
    buf = torch.zeros((n + 1,) + s["q"].shape[1:], dtype=dtype, device="cuda")
    d["q"] = buf[:n]
    with pytest.raises(gpu.BitLinearError) as e:
        append(gpu, d, q_out=buf[1:])
    assert e.value.status == 4


@pytest.mark.parametrize("bits", [4, 8])
def test_keys_without_queries(gpu, bits):
    """The cache is the same with and without q."""
    s = make(52, [5, 1, 30], [70, 41, 90], 32, 128, 2, F32, 4, bits, 64)
    d = cuda(s)
    assert append(gpu, d, q=False) is None
    for got, want in zip(d["cache"], want_append(s)[0]):
        assert np.array_equal(got.cpu().numpy(), want)


def test_4_bit_values_at_their_limits(gpu):
    """Rows of one value, of zeros, of subnormal, large and too large values, and of a
    single value apart; every code's border."""
    s = make(53, [24], [24], 16, 64, 2, F32)
    k, v = s["k"], s["v"]
    k[0] = 0
    k[1] = 3.14159
    k[2] = -3.14159
    k[3] = -0.0
    k[4] = 1e-9
    k[5] = -1e-9
    k[6] = torch.linspace(-1e-6, 1e-6, 64)
    k[7] = torch.linspace(-3e-5, 9e-5, 64)
    k[8] = torch.linspace(-65504, 65504, 64)
    k[9] = torch.linspace(-3e38, 3e38, 64)
    k[10] = torch.linspace(65000, 70000, 64)
    k[11] = -65504
    k[12] = 0
    k[12, :, 5] = 100
    k[13] = torch.linspace(99.9, 100.1, 64)
    k[14] = torch.linspace(-100.1, -99.9, 64)
    k[15] = (torch.arange(64) % 31) / 2.0       # steps of 1 and the borders between them
    k[16] = (torch.arange(64) % 31) / 2.0 - 8
    k[17] = float("inf")
    k[18] = -float("inf")
    k[19] = torch.linspace(-6.2e-5, 6.0e-5, 64)
    v.copy_(k.flip(0))
    d = check_append(gpu, s)
    got = gpu.bitlinear_kv4_read(*meta(d), d["cache"], 24)[0].cpu()
    assert torch.equal(got[0], torch.zeros_like(got[0]))
    assert torch.equal(got[15], torch.round(k[15]))                # ties to even
    step = (k[20:].amax(-1) - k[20:].amin(-1)) / 15
    assert ((got[20:] - k[20:]).abs().amax(-1) < 0.52 * step).all()


def test_append_twice_is_append_once(gpu):
    for bits in (4, 8):
        s = cuda(make(15, [1] * 9 + [100], [5 * i + 1 for i in range(9)] + [150], 64, 128, 3, BF16, 2, bits, 128))
        append(gpu, s)
        once = copied(s)
        append(gpu, s)
        assert all(torch.equal(a, b) for a, b in zip(s["cache"], once["cache"]))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("n", [[1, 1, 1], [40, 2, 3]])
def test_blocks_out_of_range_hold_nothing(gpu, n, bits):
    lens = [200, 40, 90]
    s = make(11, n, lens, 16, 64, 2, F32, 2, bits, 64)
    s["table"][0, 2] = -5
    s["table"][0, 5] = len(s["cache"][0])
    s["table"][0, 12] = 2 ** 31 - 1            # the block of the newest tokens
    s["table"][2, :] = -2 ** 31                # a sequence without any token
    check_append(gpu, s)
    check_read(gpu, s)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("n", [[3, 1, 2], [50, 2, 30]])
def test_odd_lengths_and_starts(gpu, n, bits):
    """Lengths below the new tokens' number, zero, negative, beyond the table;
    starts beyond the rows: what has no place is not written, q there is copied."""
    s = make(12, n, [max(3, x - 2) for x in n], 16, 64, 1, F32, 2, bits, 32)
    room = s["table"].shape[1] * 16
    s["table"] = torch.randperm(len(s["cache"][0]) * 4)[:s["table"].numel()].int().view(s["table"].shape)
    for lengths in ([n[0] - 2, 0, 0], [n[0] - 2, 0, room + 1], [-7, -2 ** 31, 2 ** 31 - 1]):
        s["lengths"] = torch.tensor(lengths, dtype=torch.int32)
        check_append(gpu, s)
        check_read(gpu, s)
    s["q_start"][3] = 2 ** 31 - 1
    s["q_start"][0] = -9
    s["lengths"] = torch.tensor([n[0] - 2, 0, 17], dtype=torch.int32)
    check_append(gpu, s)
    check_read(gpu, s)


# ------------------------------------------------------------------ the reads

def read(bl, s, n_tok, **kw):
    f = bl.bitlinear_kv8_read if bits_of(s) == 8 else bl.bitlinear_kv4_read
    return f(*meta(s), s["cache"], n_tok, **kw)


def check_read(bl, s, dtype=F32):
    """Each value z + s code (or s code) is rounded to fp32 once, then to bf16."""
    d, n_tok = cuda(s), len(s["k"])
    D, KVH = s["k"].shape[2], s["k"].shape[1]
    k, v = (torch.full((n_tok, KVH, D), 77.0, dtype=dtype, device="cuda") for _ in range(2))
    got = read(bl, d, n_tok, dtype=dtype, k=k, v=v)
    assert got[0] is k and got[1] is v
    c = [x.cpu().numpy() for x in d["cache"]]
    if bits_of(s) == 8:
        slots = [c[0] * c[2].astype(np.float64)[:, :, None, None],
                 c[1].transpose(0, 1, 3, 2) * c[3].astype(np.float64)[:, :, None, None]]
    else:
        slots = [ref.slots4(u, zs) for u, zs in zip(ref.unpack(c[0], c[1]), c[2:])]
    for x, y in zip(slots, got):
        want = f32 = ref8.f32(ref.read(x, *meta64(s), n_tok))
        if dtype == BF16:
            want = ref8.bf16(f32)
        want[np.isnan(f32)] = 77.0
        assert np.array_equal(n64(y), want)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_read(gpu, case, dtype, bits):
    n, lens, T, D, KVH, G = CASES[case]
    check_read(gpu, make(60 + case, n, lens, T, D, KVH, F32, 1, bits, before=case % 3, behind=(case + 1) % 3), dtype)
    check_read(gpu, make(80 + case, lens, lens, T, D, KVH, F32, 1, bits, behind=case % 2), dtype)


@pytest.mark.parametrize("bits", [4, 8])
def test_read_outputs_apart(gpu, bits):
    s = cuda(make(90, [20], [20], 16, 64, 2, F32, 1, bits))
    buf = torch.zeros(39, 2, 64, device="cuda")
    with pytest.raises(gpu.BitLinearError) as e:
        read(gpu, s, 20, k=buf[:20], v=buf[19:])
    assert e.value.status == 4
    assert read(gpu, s, 0)[0].shape == (0, 2, 64)


def test_moved_from_8_to_4_bits(gpu):
    """read and append: a sequence's tokens from one cache into the other, its values
    within half a step of the 4-bit codes."""
    s = cuda(make(91, [100, 37], [100, 37], 32, 128, 3, F32, 1, 8))
    k, v = read(gpu, s, 137)
    t = cuda(make(92, [100, 37], [100, 37], 16, 128, 3, F32))
    t["k"], t["v"] = k, v
    append(gpu, t)
    for x, y in zip((k, v), read(gpu, t, 137)):
        step = (x.amax(-1) - x.amin(-1)) / 15
        # z lies up to a step of fp16 below the least value, the codes' step is rounded to 11 bits
        assert ((x - y).abs().amax(-1) <= (0.5 + 15 * 2.0 ** -11) * step + 1.1 * 2.0 ** -10 * x.abs().amax(-1)).all()


def test_offsets_past_32_bits(gpu):
    """Blocks whose bytes start behind 2^32."""
    T, D, KVH = 128, 128, 8
    nb = 2 ** 33 // (T * D * KVH) + 40
    s = make(16, [1, 20], [260, 300], T, D, KVH, F32, 4, 4, 128)
    small = copied(s)
    s = cuda(s)
    ids = torch.randperm(40, generator=torch.Generator().manual_seed(1))[:len(s["cache"][0])].cuda() + nb - 40
    for i, x in enumerate(s["cache"]):
        big = torch.empty((nb,) + x.shape[1:], dtype=x.dtype, device="cuda")
        big[ids] = x
        s["cache"][i] = big
    s["table"] = torch.where(s["table"] >= 0, ids[s["table"].clamp(min=0)].int(), s["table"])
    append(gpu, s)
    want = check_append(gpu, small)
    for got, x in zip(s["cache"], want["cache"]):
        assert torch.equal(got[ids], x)
    for a, b in zip(read(gpu, s, 21), read(gpu, want, 21)):
        assert torch.equal(a, b)


def test_refusals(gpu):
    bl = gpu
    for bits in (4, 8):
        s = cuda(make(18, [2, 1], [40, 30], 16, 64, 2, F32, 4, bits, 32))
        call = bl.bitlinear_kv8_append_rope if bits == 8 else bl.bitlinear_kv4_append
        rope, c = bl.Rope(s["cos_sin"]), s["cache"]
        for k, v, q, out in ((s["k"].half(), s["v"], None, None), (s["k"], s["v"].to(BF16), None, None),
                             (s["k"], s["v"][:1], None, None), (s["k"], s["v"], s["q"][:1], None),
                             (s["k"], s["v"], s["q"].to(BF16), None), (s["k"], s["v"], s["q"][0], None),
                             (s["k"], s["v"], s["q"], s["q"][:, :1]), (s["k"], s["v"], None, s["q"]),
                             (s["k"].transpose(0, 1), s["v"], None, None), (s["k"].cpu(), s["v"], None, None)):
            with pytest.raises((TypeError, ValueError)):
                call(k, v, *meta(s), c, rope, q=q, q_out=out)
        for bad in (s["cos_sin"].half(), s["cos_sin"][0], s["cos_sin"].cpu(), s["cos_sin"].t()):
            with pytest.raises((TypeError, ValueError)):
                call(s["k"], s["v"], *meta(s), c, bl.Rope(bad))
        # too few rows, a rotation of 24, of 80 values
        for bad in (s["cos_sin"][:-1], s["cos_sin"][:, :24].contiguous(), s["cos_sin"].repeat(1, 3)[:, :80].contiguous()):
            with pytest.raises(bl.BitLinearError) as e:
                call(s["k"], s["v"], *meta(s), c, bl.Rope(bad))
            assert e.value.status == 2
        for i in range(4):
            with pytest.raises((TypeError, ValueError)):
                call(s["k"], s["v"], *meta(s), c[:i] + [c[i][:1]] + c[i + 1:] if i else [c[0][0]] + c[1:], rope)
        with pytest.raises((TypeError, ValueError)):
            read(bl, s, 3, dtype=torch.float16)
        with pytest.raises((TypeError, ValueError)):
            read(bl, s, 3, k=s["k"][:1])
        with pytest.raises((TypeError, ValueError)):
            read(bl, s, -1)
        assert append(bl, dict(s, k=s["k"][:0], v=s["v"][:0], q=s["q"][:0])).shape == s["q"][:0].shape
    with pytest.raises(ValueError):                          # nothing to rotate q by
        bl.bitlinear_kv4_append(s["k"], s["v"], *meta(s), bl.kv4_cache(4, 2, 16, 64), None, q=s["q"])
    with pytest.raises(ValueError):
        bl.bitlinear_kv8_append_rope(s["k"], s["v"], *meta(s), s["cache"], None)
    with pytest.raises(bl.BitLinearError) as e:              # T = 48
        bl.bitlinear_kv4_append(s["k"], s["v"], *meta(s), bl.kv4_cache(4, 2, 48, 64))
    assert e.value.status == 2


def test_calls_from_python_and_from_c(gpu):
    """The same results whichever way the binding takes: its short one for plain
    arguments, and the long one that a stream of the caller's asks for."""
    bl = gpu
    calls = bl._native._calls
    for bits in (4, 8):
        s = make(19, [2, 40, 1], [40, 90, 300], 16, 64, 2, BF16, 4, bits, 32)
        one, two = cuda(s), cuda(s)
        c = one["cache"]
        q = append(bl, one)
        assert torch.equal(q, append(bl, two, stream=torch.cuda.current_stream()))
        assert all(torch.equal(a, b) for a, b in zip(c, two["cache"]))
        for a, b in zip(read(bl, one, 43, dtype=BF16), read(bl, two, 43, dtype=BF16, stream=torch.cuda.current_stream())):
            assert torch.equal(a, b)
        f = bl.bitlinear_kv8_attention if bits == 8 else bl.bitlinear_kv4_attention
        for kw in (dict(), dict(scale=0.3), dict(scale=1)):
            assert torch.equal(f(q, *meta(one), c, **kw), f(q, *meta(one), c, stream=torch.cuda.current_stream(), **kw))
        # the short way took them
        rope = bl.Rope(one["cos_sin"])
        assert calls.append(bits, one["k"], one["v"], *meta(one), c, rope, one["q"], None) is not NotImplemented
        assert calls.read(bits, *meta(one), tuple(c), 43, BF16, None, None) is not NotImplemented
        assert calls.attention(bits, q, *meta(one), c, None, None, None) is not NotImplemented
        # and leaves alone what is not as it should be
        for bad in (q.half(), q[:, :, :32], q.transpose(0, 1), q.cpu(), None, 3):
            assert calls.attention(bits, bad, *meta(one), c, None, None, None) is NotImplemented
        assert calls.attention(bits, q, *meta(one), c[:3], None, None, None) is NotImplemented
        assert calls.attention(bits, q, *meta(one), c, "x", None, None) is NotImplemented
        assert calls.attention(bits, q, *meta(one), c, None, q[1:], None) is NotImplemented
        assert calls.attention(12 - bits, q, *meta(one), c, None, None, None) is NotImplemented
        assert calls.read(bits, *meta(one), c, -1, BF16, None, None) is NotImplemented
        assert calls.read(bits, *meta(one), c, 43, torch.float16, None, None) is NotImplemented
        assert calls.read(bits, *meta(one), c, 43, None, None, None) is NotImplemented
        assert calls.append(bits, one["k"], one["v"], *meta(one), c, rope, None, q) is NotImplemented
        assert calls.append(bits, one["k"], one["v"]) is NotImplemented


def test_a_failed_launch_is_not_made_again(gpu):
    """A launch that is reported as failed may have been made (an earlier error of the
    runtime is reported too): queries rotated in place may not be rotated again."""
    bl, native = gpu, gpu._native
    entries = [ctypes.cast(getattr(native.load(), name), ctypes.c_void_p).value for name in native._ENTRIES]
    calls = []
    failing = ctypes.CFUNCTYPE(ctypes.c_int)(lambda: calls.append(1) or 7)
    address = ctypes.cast(failing, ctypes.c_void_p).value
    try:
        native._calls.bind(native._check, *([address] * 7 + entries[7:]))
        for bits in (4, 8):
            s = cuda(make(20, [2, 1], [40, 30], 16, 64, 2, F32, 4, bits, 32))
            was = copied(s)
            attend = bl.bitlinear_kv8_attention if bits == 8 else bl.bitlinear_kv4_attention
            out = [torch.full_like(s["q"], 7.0), torch.full_like(s["k"], 7.0), torch.full_like(s["k"], 7.0)]
            for call in (lambda: append(bl, s, q_out=s["q"]), lambda: attend(s["q"], *meta(s), s["cache"], out=out[0]),
                         lambda: read(bl, s, 3, k=out[1], v=out[2])) + \
                        ((lambda: bl.bitlinear_kv8_append(s["k"], s["v"], *meta(s), s["cache"]),) if bits == 8 else ()):
                del calls[:]
                with pytest.raises(bl.BitLinearError) as e:
                    call()
                assert e.value.status == 7 and len(calls) == 1
            torch.cuda.synchronize()
            assert torch.equal(s["q"], was["q"]) and all(bool((x == 7.0).all()) for x in out)
            for a, b in zip(s["cache"], was["cache"]):
                assert torch.equal(a, b)
    finally:
        native._calls.bind(native._check, *entries)


@pytest.mark.parametrize("bits", [4, 8])
def test_captured_append_and_read(gpu, bits):
    """An append with queries turned in place and the read of the new tokens, captured once and
    replayed as the sequences grow out of their table's room."""
    bl = gpu
    s = cuda(make(21, [1, 5, 1], [15, 40, 62], 16, 128, 2, BF16, 4, bits, 64))
    room = s["table"].shape[1] * 16
    start, eager = copied(s), copied(s)
    k, v = torch.zeros_like(s["k"]), torch.zeros_like(s["k"])

    def step(x, **kw):
        append(bl, x, q_out=x["q"])
        return read(bl, x, 7, dtype=BF16, **kw)
    step(s, k=k, v=v)
    for a, b in zip(s["cache"] + [s["q"]], start["cache"] + [start["q"]]):
        a.copy_(b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(s, k=k, v=v)
    for i in range(8):
        for x in ("q", "k", "v"):
            rows = torch.randn(s[x].shape, generator=torch.Generator().manual_seed(i)).to(BF16).cuda()
            s[x].copy_(rows), eager[x].copy_(rows)
        graph.replay()
        want = step(eager)
        torch.cuda.synchronize()
        for a, b in zip([s["q"], k, v] + s["cache"], [eager["q"], *want] + eager["cache"]):
            assert torch.equal(a, b)
        s["lengths"] += 7
        eager["lengths"] += 7
    assert int(s["lengths"].max()) > room


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("near", [False, True])
@pytest.mark.parametrize("n", [1, 700])
def test_no_room_at_all(gpu, n, near, bits):
    """A table of no blocks, and so a rotation of no rows (its address is null): queries are
    copied, nothing is appended, reads and attention give zeros."""
    bl = gpu
    s = cuda(make(22, [n], [n], 16, 64, 2, F32, 4, bits, 32, near))
    s["table"], s["cos_sin"] = s["table"][:, :0].contiguous(), s["cos_sin"][:0].contiguous()
    was = copied(s)
    out = append(bl, s, q_out=torch.full_like(s["q"], 77.0))
    assert torch.equal(out, s["q"])
    for a, b in zip(s["cache"], was["cache"]):
        assert torch.equal(a, b)
    assert append(bl, s, q_out=s["q"]) is s["q"] and torch.equal(s["q"], was["q"])
    assert all(not x.any() for x in read(bl, s, n))
    attend = bl.bitlinear_kv8_attention if bits == 8 else bl.bitlinear_kv4_attention
    assert not attend(s["q"], *meta(s), s["cache"]).any()


def test_fresh_tensors_under_torch_modes(gpu):
    """Tensors that a call makes: filled where torch is asked to fill them, seen by a
    dispatch mode, of another device's or inference mode's kind like torch.empty's."""
    from torch.utils._python_dispatch import TorchDispatchMode

    class Seen(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            seen.append(str(func))
            return func(*args, **(kwargs or {}))

    bl = gpu
    s = cuda(make(23, [2], [40], 16, 64, 2, F32, 4, rot=32, behind=1))
    plain = append(bl, s)
    was, fill = torch.are_deterministic_algorithms_enabled(), torch.utils.deterministic.fill_uninitialized_memory
    try:
        torch.use_deterministic_algorithms(True)
        torch.utils.deterministic.fill_uninitialized_memory = True
        q = append(bl, s)
        k, v = read(bl, s, 3)
        out = bl.bitlinear_kv4_attention(s["q"], *meta(s), s["cache"])
    finally:
        torch.use_deterministic_algorithms(was)
        torch.utils.deterministic.fill_uninitialized_memory = fill
    assert torch.equal(q[:2], plain[:2]) and all(bool(x[2:].isnan().all()) for x in (q, k, v, out))
    assert not any(bool(x[:2].isnan().any()) for x in (q, k, v, out))
    seen = []
    with Seen():
        assert torch.equal(append(bl, s)[:2], plain[:2])
    assert any("empty" in x for x in seen)
    with torch.inference_mode():
        q = append(bl, s)
        assert q.is_inference() and torch.equal(q[:2], plain[:2])
    assert not append(bl, s).is_inference()
    g = s["q"].clone().requires_grad_()
    assert not append(bl, dict(s, q=g)).requires_grad


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("KVH,G", [(17, 1), (1, 257), (300, 3), (4111, 3), (5, 1009), (65535, 1)])
def test_many_heads(gpu, KVH, G, bits):
    """Numbers of heads of every size that a call takes, key heads and query heads apart."""
    check_append(gpu, make(24, [1, 1], [1, 17], 16, 64, KVH, F32, G, bits, 16, True))


@pytest.mark.parametrize("D", [64, 128])
def test_small_rows_are_this_near(gpu, D):
    """Rows that span 1e-9 to 1e-2, through the cache and back: off by max(s / 2, 15 2^-25),
    a border between codes by 2^-22 of the spread, the value read by half a step of fp32."""
    s = make(25, [90], [90], 32, D, 2, F32)
    g = torch.Generator().manual_seed(25)
    span = 10.0 ** (-9 + 7 * torch.arange(90) / 89.0)[:, None, None]
    s["k"] = (torch.rand(90, 2, D, generator=g) - 0.5) * span
    s["v"] = (torch.rand(90, 2, D, generator=g) + 0.3) * span
    d = check_append(gpu, s)
    for x, y, zs in zip((s["k"], s["v"]), gpu.bitlinear_kv4_read(*meta(d), d["cache"], 90), d["cache"][2:]):
        zs = zs.cpu().double()[s["table"][0, torch.arange(90) // 32].long(), :, torch.arange(90) % 32]
        x, y = x.double(), y.cpu().double()
        wide = x.amax(-1) - zs[..., 0]
        tol = torch.clamp(zs[..., 1] / 2, min=15 * 2.0 ** -25) + wide * 2.0 ** -22 + y.abs().amax(-1) * 2.0 ** -24
        assert ((x - y).abs().amax(-1) <= tol).all()


# calls of more than kFewTurnedRows = 512 rows turn a row's heads by one wave, four times
# 512 / D of them at once; heads that fill that not at all, once, and several times with a rest
MANY_HEADS = [(128, 2, 10, 128, False), (128, 3, 2, 64, True), (128, 1, 33, 16, False), (64, 7, 10, 32, True),
              (64, 3, 3, 64, False), (64, 1, 32, 48, False)]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D,KVH,G,rot,near", MANY_HEADS)
def test_queries_of_many_rows(gpu, D, KVH, G, rot, near, dtype, bits):
    """Into another tensor and in place, rows of no sequence before and behind."""
    s = make(26, [30, 1, 12], [90, 1, 333], 32, D, KVH, dtype, G, bits, rot, near, before=5, behind=480)
    assert len(s["q"]) > 512
    want = n64(check_append(gpu, s)["q"])                    # q itself is left
    assert np.array_equal(want, n64(s["q"]))
    d = cuda(s)
    assert append(gpu, d, q_out=d["q"]) is d["q"]
    q = want_append(s)[1]
    of_none = ref.positions(*meta64(s)[:2], len(q), missing=-10 ** 12) == -10 ** 12
    q[of_none] = n64(s["q"])[of_none]
    assert np.array_equal(n64(d["q"]), q)


@pytest.mark.parametrize("bits", [4, 8])
def test_queries_of_a_prompt(gpu, bits):
    """600 rows of a sequence behind 50 tokens: every row's own position."""
    s = make(27, [600, 3], [650, 40], 64, 64, 2, BF16, 10, bits, 16, False)
    check_append(gpu, s)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D,KVH,T", [(128, 1, 64), (128, 5, 32), (64, 6, 16), (64, 9, 128), (128, 4, 128)])
def test_read_of_many_values(gpu, D, KVH, T, dtype, bits):
    """Reads above kAtOnce = 2^21 threads take four heads a workgroup: numbers of heads that
    are and are not their multiple, groups of 16 tokens that end early, blocks that hold nothing."""
    behind = (1 << 21) // (KVH * 2 * D) * 16 + 40
    s = make(28, [100, 37, 0, 1, 70], [100, 41, 9, 1, 333], T, D, KVH, F32, 1, bits, before=7, behind=behind)
    assert (len(s["k"]) // 16 + 10) * KVH * 2 * D > 1 << 21
    s["table"][0, 0] = -3
    s["table"][4, 333 // T] = len(s["cache"][0])
    check_read(gpu, s, dtype)
