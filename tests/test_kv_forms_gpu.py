"""The attentions over both caches by the form that a call's sizes lead to, which the
tests of the 4-bit one look up: 16-row units (few rows), 128-row tiles (many), or both in
one launch (mixed)."""
import ctypes
import functools

import numpy as np
import pytest
import torch

import test_kv4_attention_gpu as four
import test_kv8_gpu as eight
from test_kv4_gpu import BF16, CASES, F32, cuda, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,rows,length,T,D,KVH,G", [
    (1, 128, 4000, 64, 128, 5, 4), (3, 256, 1777, 32, 64, 8, 2), (1, 500, 1777, 32, 64, 8, 2),
    (17, 500, 2049, 16, 128, 2, 4), (0, 128, 4000, 64, 128, 5, 4), (1, 128, 700, 128, 64, 5, 4)])
def test_fewer_rows_than_the_call(gpu, n, rows, length, T, D, KVH, G, dtype, bits):
    """A lone sequence that brings a few of the rows that its call has room for: cut into
    parts, or not where its keys are few; the rows behind are left."""
    if bits == 4:
        four.check_filled(gpu, make(150, [n], [length], T, D, KVH, dtype, G, behind=rows - n))
        return
    s = eight.make(150, [n], [length], T, D, KVH, dtype, G, behind=rows - n)
    d = cuda(s)
    out = torch.full_like(d["q"], 77.0)
    used = eight.check_attention(s, eight.attend(gpu, d, out=out))
    assert (out.cpu().float().numpy()[~used] == 77.0).all()
    assert np.count_nonzero(used) == n * KVH * G * D


# ------------------------------------------- which kernels a call launches

class Dim3(ctypes.Structure):
    _fields_ = [("x", ctypes.c_uint32), ("y", ctypes.c_uint32), ("z", ctypes.c_uint32)]


class KernelNode(ctypes.Structure):
    """hipKernelNodeParams."""
    _fields_ = [("block", Dim3), ("extra", ctypes.c_void_p), ("func", ctypes.c_void_p), ("grid", Dim3),
                ("params", ctypes.c_void_p), ("lds", ctypes.c_uint)]


def launched(bl, call):
    """(function, grid's z) of each kernel that a call launches, from a graph that is
    captured of it and not run."""
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    hip, handle = bl.load(), ctypes.c_void_p(graph.raw_cuda_graph())
    n = ctypes.c_size_t(64)
    nodes = (ctypes.c_void_p * 64)()
    assert hip.hipGraphGetNodes(handle, nodes, ctypes.byref(n)) == 0
    out = []
    for node in nodes[:n.value]:
        p = KernelNode()
        assert hip.hipGraphKernelNodeGetParams(ctypes.c_void_p(node), ctypes.byref(p)) == 0
        out.append((p.func, p.grid.z))
    assert out
    return out


@functools.lru_cache(None)
def few_kernel(bl, dtype, D):
    d = cuda(make(1, [1], [20], 16, D, 1, dtype, 1))
    (func, _), = launched(bl, lambda: four.attend(bl, d))
    return func


def form(bl, d):
    """(few, many or mixed, number of launches, parts of the keys or 0 where not known)
    of the 4-bit attention's call."""
    kernels = launched(bl, lambda: four.attend(bl, d))
    if kernels[0][0] == few_kernel(bl, d["q"].dtype, d["q"].shape[2]):
        return "few", len(kernels), 0
    if len(d["lengths"]) == 1:
        return "many", len(kernels), kernels[0][1]
    return "mixed", len(kernels), 0


# ------------------------------------------------------ a bound for each form

def exact(s):
    """In 64 bits, by row and head: the result, sum p (|z| + s u), max_j scale sum |q| (|z|
    + s u), max_j scale max |q| sum s u, max_j scale sum |q k_j|, the keys seen, and by value
    the sums over keys of p^2 (s u)^2, p^2 v^2 and p^2 (v - out)^2 scale^2 sum q^2 k^2."""
    K, V, zk, zv = (x.cuda() for x in s["cache"])
    T, D = zk.shape[2], s["q"].shape[2]
    G = s["q"].shape[1] // K.shape[1]
    scale = D ** -0.5
    q = s["q"].cuda().double()
    r = {x: torch.full_like(q, float("nan")) for x in ("out", "wide", "su2", "v2", "moved2")}
    r.update({x: torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda") for x in ("reach", "far", "near", "keys")})
    starts, lens = s["q_start"].tolist(), s["lengths"].tolist()
    for b, (r0, r1, L) in enumerate(zip(starts, starts[1:], lens)):
        n = r1 - r0
        if n == 0:
            continue
        table = s["table"].cuda()[b]
        at = torch.arange(max(0, min(L, len(table) * T)), device="cuda")
        at = at[(table[at // T] >= 0) & (table[at // T] < len(K))]
        ids, slot = table[at // T].long(), at % T
        hidden = (at[None] > torch.arange(L - n, L, device="cuda")[:, None]).repeat_interleave(G, 0)
        for h in range(K.shape[1]):
            k_byte, v_byte = K[ids, h, slot], V[ids, h, slot // 16, :, slot % 16 // 2]
            ku = torch.stack((k_byte & 15, k_byte >> 4), -1).flatten(1).double()
            vu = torch.where((slot % 2 == 1)[:, None], v_byte >> 4, v_byte & 15).double()
            (kz, ks), (vz, vs) = (x[ids, h, slot].double().T[..., None] for x in (zk, zv))
            k, ka, kc = kz + ks * ku, kz.abs() + ks * ku, ks * ku
            v, va, vc = vz + vs * vu, vz.abs() + vs * vu, vs * vu
            heads = slice(h * G, h * G + G)
            x = q[r0:r1, heads].reshape(n * G, D)

            def largest(y):
                return torch.cat((y.masked_fill(hidden, 0.0), y.new_zeros(n * G, 1)), 1).amax(-1).view(n, G) * scale
            p = torch.softmax((x @ k.T * scale).masked_fill(hidden, float("-inf")), -1).nan_to_num(0.0)   # no key: zeros
            out = p @ v
            dx2 = scale ** 2 * (x ** 2 @ (k ** 2).T)
            m2 = p ** 2 * dx2
            moved2 = m2 @ v ** 2 - 2 * out * (m2 @ v) + out ** 2 * m2.sum(-1, keepdim=True)
            for name, y in (("out", out), ("wide", p @ va), ("su2", p ** 2 @ vc ** 2), ("v2", p ** 2 @ v ** 2),
                            ("moved2", moved2.clamp(min=0))):
                r[name][r0:r1, heads] = y.view(n, G, D)
            r["reach"][r0:r1, heads] = largest(x.abs() @ ka.T)
            r["near"][r0:r1, heads] = largest(x.abs() @ k.abs().T)
            r["far"][r0:r1, heads] = largest(x.abs().amax(-1, keepdim=True) * kc.sum(-1)[None])
            r["keys"][r0:r1, heads] = (~hidden).sum(-1).view(n, G).double()
    return r


def check_bf16(s, got, many):
    """Value by value.  A score is off by ds <= reach (2^-21 + (D + 16) 2^-24) + far 2^-38 (as
    four.check has it), where keys are rounded to fp16 (many) also by near 2^-11 and D max |q|
    scale 2^-25; that moves a weight by twice it.  Weights and sums add (keys + 64) 2^-24 of
    sum p (|z| + s u).  p s is rounded to 11 bits: 2^-11 of that, and by half of its smallest step, 2^-34 of a
    power of two up to twice the largest s (many: 2^-38 of the largest weight's), times a
    code of 15: keys 2^-30 max s; values to fp16 (many) 2^-11 and 2^-25 more.  The result to
    bf16: 2^-8.

    In the 2-norm, over rows that see 16 keys and more.  Rounding x to bf16, whose neighbours
    are g apart, leaves an error uniform in +-g / 2: its squares have the sum
    sum g^2 / 12, of variance sum g^4 / 180; five deviations are allowed.  Roundings to 11
    bits are independent and each at most 2^-11 of its value, so their squares' sum is
    below 2^-22 times sum p^2 (s u)^2 for the weights, for many rows sum p^2 v^2 for the
    weights and again for the values, and sum p^2 (v - out)^2 dx^2 for the keys, dx^2 = scale^2 sum
    q^2 k^2 (a uniform error's mean square is a third of its largest: what is left is for
    chance and for fp32's roundings, 2^-13 of these)."""
    e = exact(s)
    D = s["q"].shape[2]
    scale = D ** -0.5
    keys = float(e["keys"].max())
    sv = float(s["cache"][3][..., 1].float().max())
    ds = e["reach"] * (2.0 ** -21 + (D + 16) * 2.0 ** -24) + e["far"] * 2.0 ** -38
    if many:
        ds = ds + e["near"] * 2.0 ** -11 + D * n_max(s) * scale * 2.0 ** -25
    tol = e["wide"] * (torch.expm1(2 * ds)[..., None] + (keys + 64) * 2.0 ** -24) + keys * 2.0 ** -30 * sv
    tol = tol + e["wide"] * 2.0 ** -11
    if many:
        tol = tol + e["wide"] * 2.0 ** -11 + 2.0 ** -25
    out = e["out"]
    tol = tol + (out.abs() + tol) * 2.0 ** -8
    used = ~out.isnan()
    got = got.double().cuda()
    assert bool(got[used].isfinite().all())
    off = (got - out).abs()
    assert float((off - tol)[used].max()) <= 0
    rows = (e["keys"] >= 16) & used[..., 0]
    if int(rows.sum()) * D >= 2000:
        gap = torch.exp2(torch.floor(torch.log2(out[rows].abs())) - 7)
        rounding = (gap ** 2).sum() / 12 + 5 * ((gap ** 4).sum() / 180) ** 0.5
        parts = 2 * e["v2"] + e["moved2"] if many else e["su2"]
        bound = rounding ** 0.5 + (parts[rows].sum() * 2.0 ** -22) ** 0.5
        assert float((off[rows] ** 2).sum() ** 0.5) <= float(bound), (float((off[rows] ** 2).sum() ** 0.5), float(bound))
    return used


def n_max(s):
    return s["q"].cuda().double().abs().amax(-1)


def check_form(bl, s, want):
    """The form is what the case is for; the result is within its bound, twice the same, and
    rows of no sequence are left."""
    d = cuda(s)
    assert form(bl, d)[:len(want)] == want
    out = torch.full_like(d["q"], 77.0)
    four.attend(bl, d, out=out)
    used = check_bf16(s, out, want[0] != "few")
    assert bool((out[~used] == 77.0).all())
    assert torch.equal(four.attend(bl, d)[used], out[used])


@pytest.mark.parametrize("case", range(len(CASES)))
def test_few_bf16_rows(gpu, case):
    n, lens, T, D, KVH, G = CASES[case]
    check_form(gpu, make(case, n, lens, T, D, KVH, BF16, G, before=case % 3, behind=(case + 1) % 3), ("few",))


@pytest.mark.parametrize("width", [0, 9000])
@pytest.mark.parametrize("case", range(len(eight.LINES)))
def test_few_bf16_rows_in_pieces(gpu, case, width):
    n, lens, T, KVH, G = eight.LINES[case]
    D = (128, 64)[case // 2 % 2]
    check_form(gpu, make(160 + case, n, lens, T, D, KVH, BF16, G, before=case % 2, behind=2, width=-(-width // T)), ("few",))


MANY = [
    # n, lens, T, D, KVH, G, width in keys, form, launches, parts (of a lone sequence)
    ([200], [400], 16, 128, 2, 4, 70000, "many", 2, 40),
    ([300], [300], 32, 64, 4, 4, 30000, "many", 2, 13),
    ([1800], [2500], 64, 128, 4, 4, 0, "many", 2, 2),
    ([900], [4000], 128, 64, 2, 8, 9000, "many", 2, 4),
    # in one part: two workgroups a CU, whose second half of the order turns round, and more
    ([1500], [1500], 64, 128, 4, 8, 0, "many", 1, 1),
    ([1500], [1500], 16, 64, 4, 8, 0, "many", 1, 1),
    ([1100], [1100], 128, 64, 8, 8, 0, "many", 1, 1),
    ([1100], [1100], 32, 128, 8, 8, 0, "many", 1, 1),
    # beside others: in one part, in several
    ([600, 1, 500, 40], [700, 300, 900, 40], 16, 128, 8, 8, 0, "mixed", 1),
    ([600, 1, 500, 3, 40], [700, 300, 900, 40, 40], 64, 64, 8, 8, 0, "mixed", 1),
    ([500, 1, 300, 0, 7], [2000, 5000, 300, 0, 900], 32, 128, 2, 4, 30000, "mixed", 3),
    ([400, 350], [1000, 2100], 128, 64, 4, 4, 20000, "mixed", 3),
    ([5, 400, 9, 350], [700, 1000, 9, 2100], 16, 64, 4, 4, 20000, "mixed", 3),
    ([60, 1, 70, 2, 33], [70, 300, 70, 2500, 700], 64, 128, 1, 4, 800000, "mixed", 3),
]


@pytest.mark.parametrize("case", range(len(MANY)))
def test_many_bf16_rows(gpu, case):
    n, lens, T, D, KVH, G, width, *want = MANY[case]
    check_form(gpu, make(200 + case, n, lens, T, D, KVH, BF16, G, before=case % 3, behind=(case + 1) % 3, width=-(-width // T)),
               tuple(want))


WIDE = 2_000_000                # keys of room: calls of a few dozen rows take the 128-row form


@pytest.mark.parametrize("fill", [0, 255])
@pytest.mark.parametrize("case", range(len(MANY)))
def test_workspace_of_many_bf16_rows(gpu, case, fill):
    """On the first bytes of a buffer and whatever it held; the bytes behind them stay."""
    n, lens, T, D, KVH, G, width, *want = MANY[case]
    s = make(220 + case, n, lens, T, D, KVH, BF16, G, width=-(-width // T))
    d = cuda(s)
    need = gpu.load().bitlinear_kv4_attention_ws_bytes(len(s["q"]), KVH * G, len(n), s["table"].shape[1], KVH, T, D)
    assert want[1] == 1 or need > 0
    buf = torch.full((need + (1 << 20),), fill, dtype=torch.uint8, device="cuda")
    buf[need:] = 170
    out = four.attend(gpu, d, ws=buf[:need])
    assert bool((buf[need:] == 170).all())
    assert torch.equal(out, four.attend(gpu, d))


@pytest.mark.parametrize("n", [[60, 2, 3], [40]])
@pytest.mark.parametrize("D", [64, 128])
def test_blocks_out_of_range_hold_nothing(gpu, n, D):
    lens = [200, 40, 90][:len(n)]
    s = make(11, n, lens, 16, D, 2, BF16, 2, width=WIDE // 16)
    s["table"][0, 2] = -5
    s["table"][0, 5] = len(s["cache"][0])
    s["table"][0, 12] = 2 ** 31 - 1            # the block of the newest tokens
    if len(n) > 2:
        s["table"][2, :] = -2 ** 31            # a sequence without any token
    d = cuda(s)
    assert form(gpu, d)[0] == ("mixed" if len(n) > 1 else "many")
    out = four.attend(gpu, d)
    four.check(s, out)
    assert len(n) == 1 or bool((out[-n[2]:] == 0).all())


@pytest.mark.parametrize("D", [64, 128])
def test_odd_lengths_and_starts(gpu, D):
    """Lengths below the new tokens' number, zero, negative, beyond the table; starts beyond
    the rows."""
    n = [50, 2, 30]
    s = make(12, n, [max(3, x - 2) for x in n], 16, D, 1, BF16, 2, width=WIDE // 16)
    assert form(gpu, cuda(s))[0] == "mixed"
    for lengths in ([n[0] - 2, 0, 17], [n[0] - 2, 0, 90], [-7, -2 ** 31, 17], [0, 5, 2]):
        s["lengths"] = torch.tensor(lengths, dtype=torch.int32)
        for start in (0, -9):
            for end in (sum(n), 2 ** 31 - 1):
                s["q_start"][0], s["q_start"][3] = start, end
                four.check(s, four.attend(gpu, cuda(s)))


@pytest.mark.parametrize("n,lens,T,D,lengths", [
    ([1500], [1500], 64, 128, [2200]), ([1500], [1500], 128, 64, [1536]), ([1500], [1500], 16, 128, [2 ** 31 - 1]),
    ([1500], [1500], 32, 64, [1499]), ([1500], [1500], 64, 128, [700]),
    ([600, 1, 500, 400], [700, 300, 900, 400], 16, 128, [1400, 930, 2 ** 31 - 1, 41]),
    ([600, 1, 500, 400], [700, 300, 900, 400], 64, 64, [599, 0, 960, -5])])
def test_lengths_beyond_the_table(gpu, n, lens, T, D, lengths):
    """Rows at positions that the table has no room for see all that it holds, those below 0
    nothing."""
    s = make(14, n, lens, T, D, 6, BF16, 8)
    s["lengths"] = torch.tensor(lengths, dtype=torch.int32)
    check_form(gpu, s, ("many",) if len(n) == 1 else ("mixed",))


def test_extreme_steps(gpu):
    """Steps of zero, of fp16's least and of large values from token to token."""
    s = make(13, [1, 60], [400, 60], 16, 64, 2, BF16, 4, width=WIDE // 16)
    assert form(gpu, cuda(s))[0] == "mixed"
    k, v = s["cache"][2], s["cache"][3]
    v[:, :, ::3, 1] = 0
    v[:, :, 1::3] *= 1e-6
    k[:, :, ::4, 1] = 0
    k[:, :, 1::4] *= 30
    four.check(s, four.attend(gpu, cuda(s)))
    s["q"][0] *= 1e-30
    four.check(s, four.attend(gpu, cuda(s)))
    s["q"][0] = 0
    for scale in (-0.7, 0.0):
        four.check(s, four.attend(gpu, cuda(s), scale=scale), scale=scale)
    v[..., 1] = 0                              # values all of one level
    four.check(s, four.attend(gpu, cuda(s)))
    for z, step in ((-2.0 ** 13, 2.0 ** 10), (2.0 ** -24, 2.0 ** -24), (0.0, 2.0 ** -15), (-65504.0, 8704.0)):
        v[:] = torch.tensor([z, step]).half()
        four.check(s, four.attend(gpu, cuda(s)))


def test_steps_past_fp16(gpu):
    """z + 15 s above 65504, as the append writes it for values at the type's ends: the step
    counts as the largest that does not pass, at most 2^-10 smaller (of s u, which is
    at most twice sum p (|z| + s u) here)."""
    s = make(15, [60], [400], 16, 64, 2, BF16, 4, width=WIDE // 16)
    s["cache"][3][:] = torch.tensor([-65504.0, 8736.0]).half()
    d = cuda(s)
    assert form(gpu, d)[0] == "many"
    got = four.attend(gpu, d)
    assert bool(got.isfinite().all())
    e = exact(s)
    # weights and values to 11 bits, the step's 2^-10, scores by near 2^-11 twice, bf16
    tol = e["wide"] * (2 * 2.0 ** -11 + 2.0 ** -10 + torch.expm1(2 * e["near"] * 2.0 ** -11 + e["reach"] * 2.0 ** -15)[..., None])
    tol = tol + (e["out"].abs() + tol) * 2.0 ** -8
    assert bool(((got.double() - e["out"]).abs() <= tol).all())


@pytest.mark.parametrize("n,lens", [([1, 20], [260, 300]), ([20], [300])])
def test_offsets_past_32_bits(gpu, n, lens):
    T, D, KVH = 128, 128, 8
    nb = 2 ** 33 // (T * D * KVH) + 40
    s = cuda(make(16, n, lens, T, D, KVH, BF16, 4, width=WIDE // T))
    assert form(gpu, s)[0] != "few"
    want = four.attend(gpu, s)
    ids = torch.randperm(40, generator=torch.Generator().manual_seed(1))[:len(s["cache"][0])].cuda() + nb - 40
    for i, x in enumerate(s["cache"]):
        big = torch.empty((nb,) + x.shape[1:], dtype=x.dtype, device="cuda")
        big[ids] = x
        s["cache"][i] = big
    s["table"] = torch.where(s["table"] >= 0, ids[s["table"].clamp(min=0)].int(), s["table"])
    assert torch.equal(four.attend(gpu, s), want)


@pytest.mark.parametrize("bad", [[float("nan")] * 2, [float("inf")] * 2, [-float("inf"), -1.0], [65504.0, -65504.0]])
@pytest.mark.parametrize("n,lens", [([70, 20, 30], [300, 20, 31]), ([90], [333])])
def test_what_is_masked_never_shows(gpu, n, lens, bad):
    """NaN, infinite and negative steps and any codes behind a length, in spare blocks
    and in blocks that no valid entry names."""
    s = make(9, n, lens, 32, 64, 2, BF16, 4, spare=8, width=WIDE // 32)
    assert form(gpu, cuda(s))[0] == ("mixed" if len(n) > 1 else "many")
    want = four.attend(gpu, cuda(s))
    keep = torch.zeros(s["cache"][2].shape[:3], dtype=torch.bool)
    for b in range(len(n)):
        for p in range(lens[b]):
            keep[int(s["table"][b, p // 32]), :, p % 32] = True
    four.poison(s, bad, keep)
    free = [i for i in range(len(keep)) if not keep[i].any()]
    s["table"][s["table"] < 0] = free[0]
    assert torch.equal(want, four.attend(gpu, cuda(s)))


def test_graph_of_many_bf16_rows(gpu):
    """A captured call of prompts beside single tokens, replayed as the lengths and the rows
    of each sequence change, with eager work between."""
    s = cuda(make(17, [200, 1, 150, 3], [900, 3000, 1500, 40], 32, 64, 3, BF16, 4, width=120000 // 32))
    assert form(gpu, s)[0] == "mixed"
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(s["q"])
    four.attend(gpu, s, out=out, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        four.attend(gpu, s, out=out, ws=ws)
    for n, lens in (([200, 1, 150, 3], [900, 3000, 1500, 40]), ([354, 0, 0, 0], [354, 3000, 1500, 40]),
                    ([1, 1, 1, 1], [900, 1, 1500, 40]), ([10, 300, 5, 39], [10, 2000, 5, 40]), ([0, 9, 8, 7], [5, 9, 1508, 17])):
        s["q_start"].copy_(torch.tensor([0] + n).cumsum(0))
        s["lengths"].copy_(torch.tensor(lens))
        out.fill_(77.0)
        graph.replay()
        want = four.attend(gpu, s, out=torch.full_like(s["q"], 77.0))
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        check_bf16({k: v if isinstance(v, list) else v.cpu() for k, v in s.items()}, out, True)


@pytest.mark.parametrize("n,lens,width", [([1] * 8, [900] * 8, 0), ([300], [600], 70000), ([300, 1], [600, 40], 70000)])
def test_an_error_of_a_few_thousandths_is_seen(gpu, n, lens, width):
    """The bound of check_bf16 leaves no room for one: results off by 0.4% are outside it."""
    s = make(18, n, lens, 64, 128, 2, BF16, 4, width=width // 64)
    got = four.attend(gpu, cuda(s))
    check_bf16(s, got, bool(width))
    for off in (1.004, 0.996):
        with pytest.raises(AssertionError):
            check_bf16(s, got.double() * off, bool(width))
