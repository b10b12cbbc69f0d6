"""The attention over the 4-bit key/value cache against the 64-bit oracle, within a
bound from its arithmetic, and runs of the calls as a program makes them."""
import numpy as np
import pytest
import torch

from oracle import kv4 as ref
from oracle import kv8 as ref8
from test_kv4_gpu import BF16, CASES, F32, append, check_append, copied, cuda, host, make, meta, meta64, n64, rows64
from test_kv8_gpu import FAR, LINES, MANY

pytestmark = pytest.mark.gpu


def attend(bl, s, **kw):
    return bl.bitlinear_kv4_attention(s["q"], *meta(s), s["cache"], **kw)


def oracle(s, scale):
    c = [x.cpu().numpy() for x in s["cache"]]
    ku, vu = ref.unpack(c[0], c[1])
    with np.errstate(invalid="ignore"):
        return ref.attention(n64(s["q"]), ku, c[2], vu, c[3], *meta64(s), scale)


def check(s, got, scale=None):
    """A score is off by at most reach (2^-21 for the operands' 22 bits + (D + 16)
    2^-24 for the sums and what is multiplied and added after) + far 2^-38 (the
    smallest step of q in 16 bits), for bf16 rows also by near 2^-11 and D max |q| scale
    2^-25 (keys rounded to fp16, or its smallest half step); that moves a weight by
    twice it.  Weights and sums add (keys + 64) 2^-24 of sum p (|z| + s u), the smallest step of p s in 16
    bits 2^-38 of a power of two that is at most twice the largest s, each times
    a code of 15: keys 2^-33 max s.  bf16 rows: weights rounded to 11 bits (2^-11),
    values likewise or to half of fp16's smallest step, the result to bf16 (2^-8)."""
    D = s["q"].shape[2]
    scale = D ** -0.5 if scale is None else scale
    out, wide, reach, far, near = oracle(s, scale)
    keys = min(max(int(x) for x in s["lengths"]), s["table"].shape[1] * s["cache"][2].shape[2])
    keys = max(keys, 0)
    ds = reach * (2.0 ** -21 + (D + 16) * 2.0 ** -24) + far * 2.0 ** -38
    if s["q"].dtype == BF16:
        top = np.abs(n64(s["q"])).max(-1)
        ds = ds + near * 2.0 ** -11 + D * top * abs(scale) * 2.0 ** -25
    sv = s["cache"][3][..., 1].float().cpu()
    sv = float(sv[torch.isfinite(sv)].max())
    tol = wide * (np.expm1(2 * ds)[..., None] + (keys + 64) * 2.0 ** -24) + keys * 2.0 ** -33 * sv
    if s["q"].dtype == BF16:
        tol = tol + 2 * wide * 2.0 ** -11 + 2.0 ** -25
        tol = tol + (np.abs(out) + tol) * 2.0 ** -8
    got = n64(got)
    used = ~np.isnan(out)
    assert np.isfinite(got[used]).all()
    worst = np.max((np.abs(got - out) - tol)[used], initial=-1.0)
    assert worst <= 0, worst
    return used


def check_filled(bl, s, **kw):
    """Against the oracle, rows of no sequence left, twice the same."""
    d = cuda(s)
    out = torch.full_like(d["q"], 77.0)
    assert attend(bl, d, out=out, **kw) is out
    used = check(s, out)
    assert (out.cpu().float().numpy()[~used] == 77.0).all()
    again = attend(bl, d)
    assert np.array_equal(again.cpu().float().numpy()[used], out.cpu().float().numpy()[used])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(gpu, case, dtype):
    n, lens, T, D, KVH, G = CASES[case]
    check_filled(gpu, make(case, n, lens, T, D, KVH, dtype, G, before=case % 3, behind=(case + 1) % 3))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_row_counts_around_the_bounds(gpu, dtype):
    """Calls and sequences of 31 to 33 rows a head, and just below and above."""
    for G, n in ((4, [1] * 8), (1, [32]), (1, [16, 16]), (1, [31, 33]), (1, [33, 32, 1]), (2, [16]), (8, [4, 1]),
                 (8, [2, 2]), (32, [1, 2])):
        s = make(31, n, [40 + 3 * i + x for i, x in enumerate(n)], 16, 64, 1, dtype, G)
        check(s, attend(gpu, cuda(s)))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_long_sequence_in_parts(gpu, dtype):
    s = make(5, [1, 1, 6], [9000, 4097, 8191], 64, 128, 2, dtype, 4)
    check(s, attend(gpu, cuda(s)))


@pytest.mark.parametrize("width", [0, 9000, 60000])
@pytest.mark.parametrize("case", range(len(LINES)))
def test_cut_by_the_lengths(gpu, case, width):
    n, lens, T, KVH, G = LINES[case]
    dtype, D = (F32, BF16)[case % 2], (128, 64)[case // 2 % 2]
    check_filled(gpu, make(40 + case, n, lens, T, D, KVH, dtype, G, before=case % 2, behind=2, width=-(-width // T)))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", range(len(MANY)))
def test_many_rows(gpu, case, dtype):
    n, lens, T, D, KVH, G, width = MANY[case]
    check_filled(gpu, make(70 + case, n, lens, T, D, KVH, dtype, G, before=case % 3, behind=1, width=-(-width // T)))


def poison(s, bad, keep):
    """Every z and s and code that no kept slot holds."""
    for i in (2, 3):
        zs = s["cache"][i]
        zs[~keep] = torch.tensor(bad, dtype=torch.float16)
    K = s["cache"][0]
    K[~keep] = 255


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", [[float("nan")] * 2, [float("inf")] * 2, [-float("inf"), -1.0], [65504.0, -65504.0]])
@pytest.mark.parametrize("width", [0, 70000])
@pytest.mark.parametrize("n,lens", [([1] * 3, [500, 1, 90]), ([70, 20, 30], [300, 20, 31]), ([200, 1], [333, 17])])
def test_what_is_masked_never_shows(gpu, n, lens, width, bad, dtype):
    """NaN, infinite and negative steps and any codes behind a length, in spare blocks
    and in blocks that no valid entry names."""
    s = make(9, n, lens, 32, 64, 2, dtype, 4, spare=8, width=width // 32)
    want = attend(gpu, cuda(s))
    keep = torch.zeros(s["cache"][2].shape[:3], dtype=torch.bool)
    for b in range(len(n)):
        for p in range(lens[b]):
            keep[int(s["table"][b, p // 32]), :, p % 32] = True
    poison(s, bad, keep)
    free = [i for i in range(len(keep)) if not keep[i].any()]
    s["table"][s["table"] < 0] = free[0]
    assert torch.equal(want, attend(gpu, cuda(s)))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", [[float("nan")] * 2, [float("inf")] * 2, [65504.0, 65504.0]])
@pytest.mark.parametrize("n,length,T,D,KVH,G,width", [
    (60, 70, 16, 64, 2, 4, 0), (40, 1300, 32, 128, 1, 3, 9000), (200, 333, 32, 64, 2, 4, 70000),
    (200, 333, 16, 128, 2, 8, 70000), (301, 2500, 64, 128, 2, 4, 30000)])
def test_later_tokens_never_show(gpu, n, length, T, D, KVH, G, width, bad, dtype):
    """A token that overflowed: rows before it are as if it held ones; also beside
    rows that see it."""
    s = make(140, [n, 1], [length, 40], T, D, KVH, dtype, G, width=-(-width // T))
    at = length - n // 2 + 3                     # its position, the first row that sees it
    rows = at - (length - n)
    block = int(s["table"][0, at // T])
    for i in (2, 3):
        s["cache"][i][block, :, at % T] = torch.tensor(bad, dtype=torch.float16)
    got = attend(gpu, cuda(s))
    for i in (2, 3):
        s["cache"][i][block, :, at % T] = 0.25
    plain = attend(gpu, cuda(s)).cpu()
    keep = got.cpu()
    keep[rows:n] = plain[rows:n]
    check(s, keep)


@pytest.mark.parametrize("width", [0, 120000])
@pytest.mark.parametrize("n", [[1, 1, 1], [40, 2, 3], [60, 2, 3]])
def test_blocks_out_of_range_hold_nothing(gpu, n, width):
    lens = [200, 40, 90]
    s = make(11, n, lens, 16, 64, 2, F32, 2, width=width // 16)
    s["table"][0, 2] = -5
    s["table"][0, 5] = len(s["cache"][0])
    s["table"][0, 12] = 2 ** 31 - 1            # the block of the newest tokens
    s["table"][2, :] = -2 ** 31                # a sequence without any token
    out = attend(gpu, cuda(s))
    check(s, out)
    assert (out[-n[2]:] == 0).all()


@pytest.mark.parametrize("width", [0, 120000])
@pytest.mark.parametrize("n", [[3, 1, 2], [50, 2, 30]])
def test_odd_lengths_and_starts(gpu, n, width):
    """Lengths below the new tokens' number, zero, negative, beyond the table;
    starts beyond the rows."""
    s = make(12, n, [max(3, x - 2) for x in n], 16, 64, 1, F32, 2, width=width // 16)
    s["lengths"] = torch.tensor([n[0] - 2, 0, s["table"].shape[1] * 16 + 5], dtype=torch.int32)
    s["table"] = torch.arange(s["table"].numel(), dtype=torch.int32).view(s["table"].shape) % len(s["cache"][0])
    s["table"][2] = s["table"][0]
    check(s, attend(gpu, cuda(s)))
    s["lengths"] = torch.tensor([-7, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32)
    check(s, attend(gpu, cuda(s)))
    s["q_start"][3] = 2 ** 31 - 1
    s["q_start"][0] = -9
    s["lengths"] = torch.tensor([n[0] - 2, 0, 17], dtype=torch.int32)
    check(s, attend(gpu, cuda(s)))


@pytest.mark.parametrize("width", [0, 70000])
def test_extreme_steps_and_scores(gpu, width):
    """Steps of zero, of fp16's least and of large values from token to token, scores
    far apart."""
    s = make(13, [1, 60], [400, 60], 16, 64, 2, F32, 4, width=width // 16)
    k, v = s["cache"][2], s["cache"][3]
    v[:, :, ::3, 1] = 0
    v[:, :, 1::3] *= 1e-6
    k[:, :, ::4, 1] = 0
    k[:, :, 1::4] *= 30
    check(s, attend(gpu, cuda(s)))
    s["q"][0] *= 1e-30
    s["q"][1:] *= 1e3
    check(s, attend(gpu, cuda(s)))
    s["q"][0] = 0
    check(s, attend(gpu, cuda(s), scale=-0.7), scale=-0.7)
    check(s, attend(gpu, cuda(s), scale=0.0), scale=0.0)
    v[..., 1] = 0                              # values all of one level
    check(s, attend(gpu, cuda(s)))
    v[:] = torch.tensor([-2.0 ** 13, 2.0 ** 10]).half()
    check(s, attend(gpu, cuda(s)))
    v[:] = torch.tensor([2.0 ** -24, 2.0 ** -24]).half()
    check(s, attend(gpu, cuda(s)))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("far", [10, 17, 18, 19, 20, 22, 25, 28, 40, 100])
@pytest.mark.parametrize("case", range(len(FAR)))
def test_scores_far_from_zero(gpu, case, far, dtype):
    """Scores of 2^far and more, of both signs.  A score is off by ds at most (see
    check; a step of the rounded score is less), so each weight by e^ds either way:
    the result by (e^ds - 1) e^ds sum p |v - out|, and never by more than the seen
    values' reach, as it lies among them.  Where ds is 1 and more that sum is below
    64 bits' range; but a key whose score is 2 ds + 40 below the largest stays 40
    below it, with a weight under e^-40: the result is a mean of the other keys'
    values up to keys e^-40 of the reach."""
    n, lens, width = FAR[case]
    T, D, KVH, G = 16, 64, 2, 4
    s = make(100 + case, n, lens, T, D, KVH, dtype, G, width=width // T)
    s["q"] *= 2.0 ** far
    got = n64(attend(gpu, cuda(s)))
    assert np.isfinite(got).all()
    q = n64(s["q"])
    c = [x.numpy() for x in s["cache"]]
    ku, vu = ref.unpack(c[0], c[1])
    k_all, v_all = ref.slots4(ku, c[2]), ref.slots4(vu, c[3])
    ka_all, va_all = ref.slots4(ku, np.abs(c[2])), ref.slots4(vu, np.abs(c[3]))
    for b, r, pos in ref8.rows_of(s["q_start"].numpy(), lens, len(q)):
        p = np.arange(pos + 1)
        i = s["table"].numpy()[b, p // T]
        for h in range(KVH):
            k, v, ka, va = (x[i, h, p % T] for x in (k_all, v_all, ka_all, va_all))
            x = q[r, h * G:(h + 1) * G] @ k.T * D ** -0.5
            w = np.exp(x - x.max(-1, keepdims=True))
            w /= w.sum(-1, keepdims=True)
            out, wide = w @ v, w @ va
            dev = np.einsum("gj,gjd->gd", w, np.abs(v[None] - out[:, None]))
            top = np.abs(q[r, h * G:(h + 1) * G])
            ds = (top @ ka.T).max(-1) * D ** -0.5 * (2.0 ** -21 + (D + 16) * 2.0 ** -24)
            ds += top.max(-1) * ka.sum(-1).max() * D ** -0.5 * 2.0 ** -38
            if dtype == BF16:
                ds += (top @ np.abs(k).T).max(-1) * D ** -0.5 * 2.0 ** -11 + D ** 0.5 * top.max(-1) * 2.0 ** -25
            reach = np.maximum(v.max(0) - out, out - v.min(0))
            keys = len(p)
            moved = dev * (np.expm1(np.minimum(ds, 1)) * np.exp(np.minimum(ds, 1)))[:, None]
            for g in np.nonzero(ds >= 1)[0]:
                near = x[g] >= x[g].max() - 2 * ds[g] - 40
                moved[g] = np.abs(v[near] - out[g]).max(0) + keys * np.exp(-40.0) * reach[g]
            # the weights' roundings also move a result beyond the values
            tol = np.minimum(moved, reach) + np.maximum(wide, va.max(0)) * (keys + 64) * 2.0 ** -24
            tol = tol + keys * 2.0 ** -33 * c[3][..., 1].max().astype(float)
            if dtype == BF16:
                tol = tol + 2 * va.max(0) * 2.0 ** -11 + 2.0 ** -25
                tol = tol + (np.abs(out) + tol) * 2.0 ** -8
            off = np.abs(got[r, h * G:(h + 1) * G] - out)
            assert (off <= tol).all(), (b, r, h, (off - tol).max())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("far", [0, 17, 18, 20, 26, 60])
@pytest.mark.parametrize("case", range(len(FAR)))
def test_equal_scores_far_from_zero(gpu, case, far, dtype):
    """One key in every slot: equal scores, however large, and the mean of the values."""
    n, lens, width = FAR[case]
    s = make(110 + case, n, lens, 16, 64, 2, dtype, 4, width=width // 16)
    s["cache"][0][:] = s["cache"][0][0, :, :1]
    s["cache"][2][:] = torch.tensor([-1.3, 0.21]).half()
    s["q"] *= 2.0 ** far
    got = n64(attend(gpu, cuda(s)))
    s["q"][:] = 0                               # the same weights without a score's rounding
    check(s, torch.tensor(got))


def test_offsets_past_32_bits(gpu):
    T, D, KVH = 128, 128, 8
    nb = 2 ** 33 // (T * D * KVH) + 40
    for width in (0, 70000):
        s = cuda(make(16, [1, 20], [260, 300], T, D, KVH, F32, 4, width=width // T))
        want = attend(gpu, s)
        ids = torch.randperm(40, generator=torch.Generator().manual_seed(1))[:len(s["cache"][0])].cuda() + nb - 40
        for i, x in enumerate(s["cache"]):
            big = torch.empty((nb,) + x.shape[1:], dtype=x.dtype, device="cuda")
            big[ids] = x
            s["cache"][i] = big
        s["table"] = torch.where(s["table"] >= 0, ids[s["table"].clamp(min=0)].int(), s["table"])
        assert torch.equal(attend(gpu, s), want)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_step_after_another(gpu, dtype):
    """Prompt, then single tokens and drafts: keys and queries rotated on the way into
    the cache, the attention over it, the values read back, as a decode loop does."""
    bl, T, D, KVH, G = gpu, 16, 64, 2, 4
    g = torch.Generator().manual_seed(3)
    first = make(3, [1, 1], [96, 96], T, D, KVH, dtype, G, rot=32, spare=0)
    c = bl.kv4_cache(12, KVH, T, D)
    ku, vu = np.zeros((12, KVH, T, D), int), np.zeros((12, KVH, T, D), int)
    zk, zv = np.zeros((12, KVH, T, 2), np.float16), np.zeros((12, KVH, T, 2), np.float16)
    table = torch.randperm(12, generator=g).int().view(2, 6)
    lens = [0, 0]
    for n in [[21, 5]] + [[1, 1]] * 14 + [[3, 0], [0, 4]]:
        lens = [a + b for a, b in zip(lens, n)]
        s = dict(first, q_start=torch.tensor([0, n[0], sum(n)], dtype=torch.int32),
                 lengths=torch.tensor(lens, dtype=torch.int32), table=table, cache=list(c))
        for x, heads in (("q", KVH * G), ("k", KVH), ("v", KVH)):
            s[x] = (torch.randn(sum(n), heads, D, generator=g) * (1 + lens[0] / 20)).to(dtype)
        d = cuda(s)
        d["cache"] = list(c)
        q = append(bl, d)
        out = attend(bl, dict(d, q=q))
        want_q, want_k, want_v = rows64(s, dtype)
        assert np.array_equal(n64(q), want_q)
        m = meta64(s)
        ref.append(want_k, ku, zk, *m)
        ref.append(want_v, vu, zv, *m)
        K, V = ref.pack(ku, vu)
        for got, want in zip(c, (K, V, zk, zv)):
            assert np.array_equal(got.cpu().numpy(), want)
        check(host(dict(d, q=q)), out)
        starts = torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32, device="cuda")
        k, v = bl.bitlinear_kv4_read(starts, d["lengths"], d["table"], c, sum(lens))
        m[0] = starts.cpu().numpy()
        for got, u, zs in ((k, ku, zk), (v, vu, zv)):
            assert np.array_equal(n64(got), ref8.f32(ref.read(ref.slots4(u, zs), *m, sum(lens))))


def test_graph_follows_its_arrays(gpu):
    """One captured step, replayed as the sequences grow, with eager work
    between the replays."""
    bl = gpu
    s = cuda(make(17, [1, 1], [40, 700], 64, 128, 2, BF16, 4, rot=128))
    start = copied(s)
    eager = copied(s)
    out, q = torch.zeros_like(s["q"]), torch.zeros_like(s["q"])
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")

    def step(x, **kw):
        return attend(bl, dict(x, q=append(bl, x, q_out=kw.pop("q_out", None))), **kw)
    step(s, out=out, ws=ws, q_out=q)
    for a, b in zip(s["cache"], start["cache"]):
        a.copy_(b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(s, out=out, ws=ws, q_out=q)
    for i in range(5):
        for k in ("q", "k", "v"):
            x = torch.randn(s[k].shape, generator=torch.Generator().manual_seed(i)).to(BF16).cuda()
            s[k].copy_(x), eager[k].copy_(x)
        graph.replay()
        want = step(eager)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert all(torch.equal(a, b) for a, b in zip(s["cache"], eager["cache"]))
        s["lengths"] += 1
        eager["lengths"] += 1


def test_graphs_cut_by_new_lengths(gpu):
    """Two captured calls on one workspace, decode and mixed, replayed in turn as
    lengths change at random."""
    one = cuda(make(18, [1] * 5, [9000, 1, 700, 2500, 64], 64, 128, 2, BF16, 4, width=400))
    two = cuda(make(19, [1, 200, 3], [5000, 1500, 2300], 32, 64, 3, F32, 4, width=2000))
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    graphs, full = [], [s["lengths"].clone() for s in (one, two)]
    for s in (one, two):
        out = torch.zeros_like(s["q"])
        attend(gpu, s, out=out, ws=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            attend(gpu, s, out=out, ws=ws)
        graphs.append((g, out))
    r = torch.Generator().manual_seed(3)
    for step in range(6):
        for s, most in zip((one, two), full):
            share = torch.rand(len(most), generator=r).cuda() ** 3 if step else 1.0
            s["lengths"].copy_((most * share).int())
        for g, _ in graphs:
            g.replay()
        wants = [attend(gpu, s) for s in (one, two)]
        torch.cuda.synchronize()
        for s, want, (_, out) in zip((one, two), wants, graphs):
            assert torch.equal(out, want)
            check(host(s), out)


def test_two_streams(gpu):
    """Steps on streams of their own, outputs and workspaces allocated by the calls."""
    jobs = [cuda(make(20 + i, [1, 1], [3000 + i, 2500], 64, 128, 2, F32, 4, rot=64)) for i in range(2)]

    def step(s, **kw):
        q = append(gpu, s, **kw)
        return attend(gpu, dict(s, q=q), **kw), q
    want = [step(s) for s in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = []
    for _ in range(4):
        for s, st in zip(jobs, streams):
            got.append(step(s, stream=st))
    torch.cuda.synchronize()
    for i, pair in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(pair, want[i % 2]))


def test_refusals(gpu):
    bl = gpu
    s = cuda(make(18, [2, 1], [40, 30], 16, 64, 2, F32, 4))
    c, ok = bl.Kv4Cache(*s["cache"]), s["q"]
    for bad, err in ((ok.half(), TypeError), (ok.cpu(), TypeError), (ok[:, :, :32], ValueError),
                     (ok.transpose(0, 1), ValueError), (ok[0], ValueError)):
        with pytest.raises(err):
            bl.bitlinear_kv4_attention(bad, *meta(s), c)
    for i, bad in ((0, s["q_start"].long()), (0, s["q_start"][1:]), (1, s["lengths"].cpu()),
                   (1, s["lengths"][:1]), (2, s["table"][0]), (2, s["table"].t())):
        m = list(meta(s))
        m[i] = bad
        with pytest.raises((TypeError, ValueError)):
            bl.bitlinear_kv4_attention(ok, *m, c)
    for bad in (c._replace(V=c.V.transpose(3, 4).contiguous()), c._replace(zk=c.zk.float()), c._replace(zv=c.zv[..., 0]),
                c._replace(K=c.K.view(torch.int8))):
        with pytest.raises((TypeError, ValueError)):
            bl.bitlinear_kv4_attention(ok, *meta(s), bad)
    with pytest.raises(ValueError):
        bl.bitlinear_kv4_attention(ok, *meta(s), c, out=torch.empty_like(ok)[:1])
    for kw in (dict(scale=float("nan")), dict(scale=2.0 ** 127)):
        with pytest.raises(bl.BitLinearError) as e:
            attend(bl, s, **kw)
        assert e.value.status == 2
    with pytest.raises(bl.BitLinearError) as e:                       # QH not a multiple of KVH
        bl.bitlinear_kv4_attention(ok[:, :7].contiguous(), *meta(s), c)
    assert e.value.status == 2
    with pytest.raises(bl.BitLinearError) as e:
        attend(bl, s, out=s["q"])
    assert e.value.status == 4
    empty = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert bl.bitlinear_kv4_attention(ok[:0], empty, empty[:0], empty[:0].view(0, 3), c).shape == ok[:0].shape


GUARDED = [("LINES", i) for i in (0, 2, 4, 6, 9, 11, 12, 13, 14, 16)] + [("MANY", i) for i in (0, 3, 4, 5, 7, 8)]


@pytest.mark.parametrize("fill", [0, 255])
@pytest.mark.parametrize("name,case", GUARDED)
def test_workspace_of_the_asked_size(gpu, name, case, fill):
    """Cut few rows, prompts in parts, and both, on the first bytes of a buffer
    and whatever it held; the bytes behind them stay."""
    if name == "LINES":
        n, lens, T, KVH, G = LINES[case]
        D, width = 128, 60000
    else:
        n, lens, T, D, KVH, G, width = MANY[case]
    s = make(130 + case, n, lens, T, D, KVH, (F32, BF16)[case % 2], G, width=-(-width // T))
    d = cuda(s)
    need = gpu.load().bitlinear_kv4_attention_ws_bytes(len(s["q"]), KVH * G, len(n), s["table"].shape[1], KVH, T, D)
    buf = torch.full((need + (1 << 20),), fill, dtype=torch.uint8, device="cuda")
    buf[need:] = 170
    out = attend(gpu, d, ws=buf[:need])
    assert (buf[need:] == 170).all()
    check(s, out)
    assert torch.equal(out, attend(gpu, d))
