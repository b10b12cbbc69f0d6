"""The 8-bit key/value cache and the attention over it against the 64-bit
oracle: the cache's bytes and scales exactly, the attention within a bound
from its arithmetic."""
import numpy as np
import pytest
import torch

from oracle import kv8 as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def make(seed, n, lens, T, D, KVH, dtype, G=1, spare=3, behind=0, before=0, width=0):
    """A filled cache, the new rows and the arrays of a call: sequence b has
    lens[b] tokens, n[b] of them new; `before` / `behind` rows of no sequence; a
    table of `width` entries a sequence at least."""
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

    def codes(*shape):
        return torch.randint(-127, 128, shape, generator=g).to(torch.int8)

    def scales():
        return (0.5 + torch.rand(nb, KVH, generator=g)) / 40
    s = dict(K=codes(nb, KVH, T, D), V=codes(nb, KVH, D, T), sk=scales(), sv=scales(), table=table,
             q_start=q_start, lengths=torch.tensor(lens, dtype=torch.int32),
             k=torch.randn(rows, KVH, D, generator=g).to(dtype),
             v=torch.randn(rows, KVH, D, generator=g).to(dtype),
             q=torch.randn(rows, KVH * G, D, generator=g).to(dtype))
    return s


def cuda(s):
    return {k: v.cuda() for k, v in s.items()}


def cache(bl, s):
    return bl.Kv8Cache(s["K"], s["V"], s["sk"], s["sv"])


def append(bl, s, **kw):
    bl.bitlinear_kv8_append(s["k"], s["v"], s["q_start"], s["lengths"], s["table"], cache(bl, s), **kw)


def attend(bl, s, **kw):
    return bl.bitlinear_kv8_attention(s["q"], s["q_start"], s["lengths"], s["table"], cache(bl, s), **kw)


def n64(t):
    return t.double().cpu().numpy()


def check_append(bl, s):
    d = cuda(s)
    append(bl, d)
    K, V = s["K"].numpy().copy(), s["V"].numpy().transpose(0, 1, 3, 2).copy()
    sk, sv = s["sk"].numpy().copy(), s["sv"].numpy().copy()
    meta = s["q_start"].numpy(), s["lengths"].numpy(), s["table"].numpy()
    ref.append(n64(s["k"]), K, sk, *meta)
    ref.append(n64(s["v"]), V, sv, *meta)
    assert np.array_equal(d["sk"].cpu().numpy(), sk, equal_nan=True)
    assert np.array_equal(d["sv"].cpu().numpy(), sv, equal_nan=True)
    assert np.array_equal(d["K"].cpu().numpy(), K)
    assert np.array_equal(d["V"].cpu().numpy(), V.transpose(0, 1, 3, 2))
    return d


def check_attention(s, got, scale=None):
    """A score is off by at most reach * (2^-21 for the operands' 22 bits + (D +
    8) 2^-24 for the sum), which moves every weight by twice that; weights and
    sums add (keys + 64) 2^-24 of sum p |v|; bf16 rows' weights are rounded to
    11 bits (2^-11) and the result to bf16 (2^-8 of it).  What is held in 16
    bits has a smallest step too: 2^-38 of a row's largest |q| (a score moves
    by `far` of it), and 2^-38 of the largest weight times value scale, each
    code at most 128: keys 2^-31 max sv."""
    D = s["q"].shape[2]
    scale = D ** -0.5 if scale is None else scale
    out, wide, reach, far = ref.attention(n64(s["q"]), s["K"].cpu().numpy(), s["V"].cpu().numpy(),
                                     s["sk"].cpu().numpy(), s["sv"].cpu().numpy(),
                                     s["q_start"].cpu().numpy(), s["lengths"].cpu().numpy(),
                                     s["table"].cpu().numpy(), scale)
    keys = min(max(int(x) for x in s["lengths"]), s["table"].shape[1] * s["K"].shape[2])
    ds = reach * (2.0 ** -21 + (D + 8) * 2.0 ** -24) + far * 2.0 ** -38
    sv = s["sv"].cpu()
    sv = float(sv[torch.isfinite(sv)].max())
    tol = wide * (2 * ds[..., None] + (keys + 64) * 2.0 ** -24) + keys * 2.0 ** -31 * sv
    if s["q"].dtype == BF16:
        tol = tol + wide * 2.0 ** -11
        tol = tol + (np.abs(out) + tol) * 2.0 ** -8
    got = n64(got)
    used = ~np.isnan(out)
    assert np.isfinite(got[used]).all()
    worst = np.max((np.abs(got - out) - tol)[used], initial=-1.0)
    assert worst <= 0, worst
    return used


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


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_append_is_exact(gpu, case, dtype):
    n, lens, T, D, KVH, G = CASES[case]
    check_append(gpu, make(case, n, lens, T, D, KVH, dtype, before=case % 3, behind=(case + 1) % 3))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(gpu, case, dtype):
    n, lens, T, D, KVH, G = CASES[case]
    s = make(case, n, lens, T, D, KVH, dtype, G, before=case % 3, behind=(case + 1) % 3)
    d = cuda(s)
    out = torch.full_like(d["q"], 77.0)
    assert attend(gpu, d, out=out) is out
    used = check_attention(s, out)
    # rows of no sequence stay
    assert (out.cpu().float().numpy()[~used] == 77.0).all()
    again = attend(gpu, d)
    assert np.array_equal(again.cpu().float().numpy()[used], out.cpu().float().numpy()[used])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_row_counts_around_the_bounds(gpu, dtype):
    """Calls and sequences of 31 to 33 rows a head, and just below and above."""
    for G, n in ((4, [1] * 8), (1, [32]), (1, [16, 16]), (1, [31, 33]), (1, [33, 32, 1]), (2, [16]), (8, [4, 1]),
                 (8, [2, 2]), (32, [1, 2])):
        s = make(31, n, [40 + 3 * i + x for i, x in enumerate(n)], 16, 64, 1, dtype, G)
        check_attention(s, attend(gpu, cuda(s)))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_long_sequence_in_parts(gpu, dtype):
    s = make(5, [1, 1, 6], [9000, 4097, 8191], 64, 128, 2, dtype, 4)
    check_attention(s, attend(gpu, cuda(s)))


LINES = [
    # n, lens, T, KVH, G: few rows, cut by the lengths that stand in the table's width
    ([1], [3000], 64, 2, 4),
    ([1, 1, 1], [1200, 4100, 0], 64, 2, 4),
    ([1, 0, 3, 1], [1300, 9, 5000, 1], 32, 5, 4),
    ([1] * 5, [700, 20, 1500, 2, 1025], 16, 3, 7),
    ([1] * 64, [1 + 37 * i % 1000 for i in range(63)] + [9000], 128, 5, 1),
    ([1] * 65 + [2], [1 + 37 * i % 1000 for i in range(65)] + [9000], 128, 4, 2),
    ([i % 3 for i in range(256)], [2 + 37 * i % 500 for i in range(256)], 128, 1, 4),
    ([1] * 257, [1 + 37 * i % 500 for i in range(257)], 128, 1, 4),
    ([9] * 30, [9 + 37 * i % 500 for i in range(29)] + [6000], 64, 2, 3),
    ([1] * 32, [1500] * 30 + [1400, 1500], 64, 5, 4),
    ([1] * 7, [4000] * 7, 64, 3, 4),
    # with sequences of many rows
    ([1, 100, 2, 1], [5000, 300, 700, 2600], 64, 2, 4),
    ([0, 400, 1, 1], [0, 1000, 3000, 1], 64, 1, 8),
    ([1] * 20 + [300], [1 + 37 * i % 1000 for i in range(20)] + [4000], 64, 1, 4),
    ([70], [3000], 64, 2, 4),
    ([40, 50], [4000, 300], 32, 2, 4),
    ([3, 1] * 70 + [1500], [3 + 37 * i % 700 for i in range(140)] + [1500], 128, 1, 2),
]


@pytest.mark.parametrize("width", [0, 9000, 60000])
@pytest.mark.parametrize("case", range(len(LINES)))
def test_cut_by_the_lengths(gpu, case, width):
    n, lens, T, KVH, G = LINES[case]
    dtype, D = (F32, BF16)[case % 2], (128, 64)[case // 2 % 2]
    s = make(40 + case, n, lens, T, D, KVH, dtype, G, before=case % 2, behind=2, width=-(-width // T))
    d = cuda(s)
    out = torch.full_like(d["q"], 77.0)
    attend(gpu, d, out=out)
    used = check_attention(s, out)
    assert (out.cpu().float().numpy()[~used] == 77.0).all()


MANY = [
    # n, lens, T, D, KVH, G, width in keys: calls with much to do
    ([300], [500], 64, 64, 8, 8, 0),
    ([250, 70, 1], [450, 100, 33], 16, 128, 8, 8, 0),
    ([400, 0, 40], [400, 7, 590], 128, 64, 7, 7, 0),
    ([300], [300], 64, 128, 1, 4, 70000),
    ([40, 1, 90], [100, 31, 90], 16, 128, 2, 3, 70000),
    ([129, 7], [1500, 7], 128, 128, 1, 8, 70000),
    ([33], [600], 64, 64, 3, 4, 70000),
    ([70, 4, 50], [2000, 1500, 300], 32, 64, 2, 4, 30000),
    ([9, 300], [4000, 2500], 64, 128, 2, 4, 9000),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", range(len(MANY)))
def test_many_rows(gpu, case, dtype):
    n, lens, T, D, KVH, G, width = MANY[case]
    s = make(70 + case, n, lens, T, D, KVH, dtype, G, before=case % 3, behind=1, width=-(-width // T))
    d = cuda(s)
    out = torch.full_like(d["q"], 77.0)
    attend(gpu, d, out=out)
    used = check_attention(s, out)
    assert (out.cpu().float().numpy()[~used] == 77.0).all()


@pytest.mark.parametrize("width", [0, 70000])
@pytest.mark.parametrize("n,lens", [([1] * 3, [500, 1, 90]), ([70, 20, 30], [300, 20, 31])])
def test_what_is_masked_never_shows(gpu, n, lens, width):
    """NaN and infinite scales and any codes in blocks and slots behind a
    length, in spare blocks and in blocks that no valid entry names."""
    s = make(9, n, lens, 32, 64, 2, F32, 4, spare=8, width=width // 32)
    want = attend(gpu, cuda(s))
    used = {int(s["table"][b, j]) for b in range(len(n)) for j in range(-(-lens[b] // 32))}
    free = [i for i in range(len(s["sk"])) if i not in used]
    s["sk"][free] = float("nan")
    s["sv"][free] = float("inf")
    s["table"][s["table"] < 0] = free[0]
    for b in range(len(n)):
        if lens[b] % 32:
            i = int(s["table"][b, lens[b] // 32])
            s["K"][i, :, lens[b] % 32:] = -128
            s["V"][i, :, :, lens[b] % 32:] = -128
    got = attend(gpu, cuda(s))
    assert torch.equal(want, got)


@pytest.mark.parametrize("width", [0, 120000])
@pytest.mark.parametrize("n", [[1, 1, 1], [40, 2, 3], [60, 2, 3]])
def test_blocks_out_of_range_hold_nothing(gpu, n, width):
    lens = [200, 40, 90]
    s = make(11, n, lens, 16, 64, 2, F32, 2, width=width // 16)
    s["table"][0, 2] = -5
    s["table"][0, 5] = len(s["K"])
    s["table"][0, 12] = 2 ** 31 - 1            # the block of the newest tokens
    s["table"][2, :] = -2 ** 31                # a sequence without any token
    check_append(gpu, s)
    out = attend(gpu, cuda(s))
    check_attention(s, out)
    assert (out[-n[2]:] == 0).all()


@pytest.mark.parametrize("width", [0, 120000])
@pytest.mark.parametrize("n", [[3, 1, 2], [50, 2, 30]])
def test_odd_lengths_and_starts(gpu, n, width):
    """Lengths below the new tokens' number, zero, negative, beyond the table;
    starts beyond the rows."""
    s = make(12, n, [max(3, x - 2) for x in n], 16, 64, 1, F32, 2, width=width // 16)
    s["lengths"] = torch.tensor([n[0] - 2, 0, s["table"].shape[1] * 16 + 5], dtype=torch.int32)
    s["table"] = torch.arange(s["table"].numel(), dtype=torch.int32).view(s["table"].shape) % len(s["K"])
    s["table"][2] = s["table"][0]
    d = cuda(s)
    check_attention(s, attend(gpu, d))
    s["lengths"][2] = 0
    check_append(gpu, s)
    s["lengths"] = torch.tensor([-7, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32)
    check_attention(s, attend(gpu, cuda(s)))
    s["q_start"][3] = 2 ** 31 - 1
    s["q_start"][0] = -9
    s["lengths"] = torch.tensor([n[0] - 2, 0, 17], dtype=torch.int32)
    check_attention(s, attend(gpu, cuda(s)))


@pytest.mark.parametrize("width", [0, 70000])
def test_extreme_scales_and_scores(gpu, width):
    """Zero and very different scales from block to block, scores far apart."""
    s = make(13, [1, 60], [400, 60], 16, 64, 2, F32, 4, width=width // 16)
    s["sv"][::3] = 0
    s["sv"][1::3] *= 1e-7
    s["sk"][::4] = 0
    s["sk"][1::4] *= 30
    check_attention(s, attend(gpu, cuda(s)))
    s["q"][0] *= 1e-30
    s["q"][1:] *= 1e3
    check_attention(s, attend(gpu, cuda(s)))
    s["q"][0] = 0
    check_attention(s, attend(gpu, cuda(s), scale=-0.7), scale=-0.7)
    check_attention(s, attend(gpu, cuda(s), scale=0.0), scale=0.0)


def test_append_zero_tiny_and_growing(gpu):
    s = make(14, [3, 20], [9, 40], 16, 64, 2, F32)
    s["k"][:] = 0                              # nothing new above the old scale
    s["v"][:3] = 1e-42                         # a / 127 underflows
    d = check_append(gpu, s)
    s = {k: v.cpu() for k, v in d.items()}
    s["v"] *= 1e3
    s["k"][:] = torch.linspace(-200, 200, s["k"].numel()).view(s["k"].shape)
    check_append(gpu, s)


def test_append_twice_is_append_once(gpu):
    s = cuda(make(15, [1] * 9 + [100], [5 * i + 1 for i in range(9)] + [150], 64, 128, 3, BF16))
    append(gpu, s)
    once = {k: v.clone() for k, v in s.items()}
    append(gpu, s)
    assert all(torch.equal(s[k], once[k]) for k in ("K", "V", "sk", "sv"))


@pytest.mark.parametrize("width", [0, 70000])
def test_offsets_past_32_bits(gpu, width):
    """Blocks whose bytes start behind 2^32."""
    T, D, KVH = 128, 128, 8
    nb = 2 ** 32 // (T * D * KVH) + 40
    s = make(16, [1, 20], [260, 300], T, D, KVH, F32, 4, width=width // T)
    small = {k: v.clone() for k, v in s.items()}
    s = cuda(s)
    ids = torch.randperm(40, generator=torch.Generator().manual_seed(1))[:len(s["sk"])].cuda() + nb - 40
    for name in ("K", "V", "sk", "sv"):
        big = torch.empty((nb,) + s[name].shape[1:], dtype=s[name].dtype, device="cuda")
        big[ids] = s[name]
        s[name] = big
    s["table"] = torch.where(s["table"] >= 0, ids[s["table"].clamp(min=0)].int(), s["table"])
    append(gpu, s)
    want = check_append(gpu, small)
    for name in ("K", "V", "sk", "sv"):
        assert torch.equal(s[name][ids], want[name])
    assert torch.equal(attend(gpu, s), attend(gpu, want))


def test_a_step_after_another(gpu):
    """Prompt, then single tokens: append and attend, as a decode loop does,
    the cache against the oracle's after every step."""
    bl, T, D, KVH, G = gpu, 16, 64, 2, 4
    g = torch.Generator().manual_seed(3)
    c = bl.kv8_cache(12, KVH, T, D)
    K, V = np.zeros((12, KVH, T, D), np.int8), np.zeros((12, KVH, T, D), np.int8)
    sk, sv = np.zeros((12, KVH), np.float32), np.zeros((12, KVH), np.float32)
    table = torch.randperm(12, generator=g).int().view(2, 6)
    lens = [0, 0]
    for n in [[21, 5]] + [[1, 1]] * 14 + [[3, 0], [0, 4]]:
        lens = [a + b for a, b in zip(lens, n)]
        s = dict(q_start=torch.tensor([0, n[0], sum(n)], dtype=torch.int32),
                 lengths=torch.tensor(lens, dtype=torch.int32), table=table)
        for x, heads in (("q", KVH * G), ("k", KVH), ("v", KVH)):
            s[x] = torch.randn(sum(n), heads, D, generator=g) * (1 + lens[0] / 20)
        d = dict(cuda(s), K=c.K, V=c.V, sk=c.sk, sv=c.sv)
        append(bl, d)
        out = attend(bl, d)
        meta = s["q_start"].numpy(), s["lengths"].numpy(), s["table"].numpy()
        ref.append(n64(s["k"]), K, sk, *meta)
        ref.append(n64(s["v"]), V, sv, *meta)
        assert np.array_equal(c.K.cpu().numpy(), K)
        assert np.array_equal(c.V.cpu().numpy().transpose(0, 1, 3, 2), V)
        assert np.array_equal(c.sk.cpu().numpy(), sk) and np.array_equal(c.sv.cpu().numpy(), sv)
        check_attention({k: v.cpu() for k, v in d.items()}, out)


def test_graph_follows_its_arrays(gpu):
    """One captured step, replayed as the sequences grow, with eager work
    between the replays."""
    bl = gpu
    first = make(17, [1, 1], [40, 700], 64, 128, 2, BF16, 4)
    s = cuda(first)
    eager = {k: v.clone() for k, v in s.items()}
    out = torch.zeros_like(s["q"])
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    append(bl, s), attend(bl, s, out=out, ws=ws)
    for k in s:
        s[k].copy_(eager[k])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        append(bl, s)
        attend(bl, s, out=out, ws=ws)
    for step in range(5):
        for k in ("q", "k", "v"):
            x = torch.randn(s[k].shape, generator=torch.Generator().manual_seed(step)).to(BF16).cuda()
            s[k].copy_(x), eager[k].copy_(x)
        graph.replay()
        append(bl, eager)
        want = attend(bl, eager)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert all(torch.equal(s[k], eager[k]) for k in ("K", "V", "sk", "sv"))
        s["lengths"] += 1
        eager["lengths"] += 1


def test_graphs_cut_by_new_lengths(gpu):
    """Two captured calls on one workspace, decode and mixed, replayed in turn as
    lengths change at random."""
    one = cuda(make(18, [1] * 5, [9000, 1, 700, 2500, 64], 64, 128, 2, BF16, 4, width=400))
    two = cuda(make(19, [1, 200, 3], [5000, 1500, 2300], 32, 64, 3, F32, 4, width=2000))
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
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
            check_attention({k: v.cpu() for k, v in s.items()}, out)


def test_two_streams(gpu):
    """Calls on streams of their own, outputs and workspaces allocated by the calls."""
    jobs = [cuda(make(20 + i, [1, 1], [3000 + i, 2500], 64, 128, 2, F32, 4)) for i in range(2)]
    want = [attend(gpu, s) for s in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = []
    for _ in range(4):
        for s, st in zip(jobs, streams):
            got.append(attend(gpu, s, stream=st))
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 2])


def test_refusals(gpu):
    bl = gpu
    s = cuda(make(18, [2, 1], [40, 30], 16, 64, 2, F32, 4))
    c = cache(bl, s)
    meta = s["q_start"], s["lengths"], s["table"]
    ok = s["q"]
    for bad, err in ((ok.half(), TypeError), (ok.cpu(), TypeError), (ok[:, :, :32], ValueError),
                     (ok.transpose(0, 1), ValueError), (ok[0], ValueError)):
        with pytest.raises(err):
            bl.bitlinear_kv8_attention(bad, *meta, c)
    for i, bad in ((0, s["q_start"].long()), (0, s["q_start"][1:]), (1, s["lengths"].cpu()),
                   (1, s["lengths"][:1]), (2, s["table"][0]), (2, s["table"].t())):
        m = list(meta)
        m[i] = bad
        with pytest.raises((TypeError, ValueError)):
            bl.bitlinear_kv8_attention(ok, *m, c)
        with pytest.raises((TypeError, ValueError)):
            bl.bitlinear_kv8_append(s["k"], s["v"], *m, c)
    with pytest.raises(ValueError):                                   # V as K is laid out
        bl.bitlinear_kv8_attention(ok, *meta, c._replace(V=c.V.transpose(2, 3).contiguous()))
    with pytest.raises(TypeError):
        bl.bitlinear_kv8_append(s["k"], s["v"].to(BF16), *meta, c)
    with pytest.raises(ValueError):
        bl.bitlinear_kv8_attention(ok, *meta, c, out=torch.empty_like(ok)[:1])
    with pytest.raises(bl.BitLinearError) as e:                       # QH not a multiple of KVH
        bl.bitlinear_kv8_attention(ok[:, :7].contiguous(), *meta, c)
    assert e.value.status == 2
    with pytest.raises(bl.BitLinearError) as e:
        bl.bitlinear_kv8_attention(ok, *meta, c, scale=float("nan"))
    assert e.value.status == 2
    with pytest.raises(bl.BitLinearError) as e:                       # T = 8
        bl.bitlinear_kv8_append(s["k"], s["v"], *meta, bl.kv8_cache(4, 2, 8, 64))
    assert e.value.status == 2
    # nothing to do
    empty = torch.zeros(1, dtype=torch.int32, device="cuda")
    none = empty[:0]
    bl.bitlinear_kv8_append(s["k"][:0], s["v"][:0], s["q_start"], s["lengths"], s["table"], c)
    assert bl.bitlinear_kv8_attention(ok[:0], empty, none, none.view(0, 3), c).shape == ok[:0].shape


FAR = [
    # n, lens, width in keys: few rows, cut ones, many rows, both, many rows in parts
    ([1], [400], 0),
    ([1, 5, 3], [3000, 40, 3], 0),
    ([200], [400], 70000),
    ([1, 60], [400, 60], 70000),
    ([100, 1], [2000, 1000], 70000),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("far", [10, 17, 18, 19, 20, 22, 25, 28, 40, 100])
@pytest.mark.parametrize("case", range(len(FAR)))
def test_scores_far_from_zero(gpu, case, far, dtype):
    """Scores of 2^far and more, of both signs.  A score is off by ds at most (see
    check_attention; a step of the rounded score is less), so each weight by e^ds
    either way: the result by (e^ds - 1) e^ds sum p |v - out|, and never by more
    than the seen values' reach, as it lies among them."""
    n, lens, width = FAR[case]
    T, D, KVH, G = 16, 64, 2, 4
    s = make(100 + case, n, lens, T, D, KVH, dtype, G, width=width // T)
    s["q"] *= 2.0 ** far
    got = n64(attend(gpu, cuda(s)))
    assert np.isfinite(got).all()
    q, K, V, sk, sv = (n64(s[x]) for x in ("q", "K", "V", "sk", "sv"))
    for b, r, pos in ref.rows_of(s["q_start"].numpy(), lens, len(q)):
        p = np.arange(pos + 1)
        i = s["table"].numpy()[b, p // T]
        for h in range(KVH):
            k, v = K[i, h, p % T] * sk[i, h][:, None], V[i, h, :, p % T] * sv[i, h][:, None]
            x = q[r, h * G:(h + 1) * G] @ k.T * D ** -0.5
            w = np.exp(x - x.max(-1, keepdims=True))
            w /= w.sum(-1, keepdims=True)
            out, wide = w @ v, w @ np.abs(v)
            dev = np.einsum("gj,gjd->gd", w, np.abs(v[None] - out[:, None]))
            top = np.abs(q[r, h * G:(h + 1) * G])
            ds = (top @ np.abs(k).T).max(-1) * D ** -0.5 * (2.0 ** -21 + (D + 8) * 2.0 ** -24)
            ds += top.max(-1) * np.abs(k).sum(-1).max() * D ** -0.5 * 2.0 ** -38
            reach = np.maximum(v.max(0) - out, out - v.min(0))
            with np.errstate(divide="ignore", over="ignore"):
                moved = np.exp(np.minimum(np.log(dev) + np.where(ds < 1, np.log(np.expm1(ds)) + ds, 2 * ds)[:, None], 50))
            # the weights' roundings also move a result beyond the values
            keys = len(p)
            tol = np.minimum(moved, reach) + wide * (keys + 64) * 2.0 ** -24 + keys * 2.0 ** -31 * sv.max()
            if dtype == BF16:
                tol = tol + wide * 2.0 ** -11
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
    s["K"][:] = s["K"][0, :, :1]
    s["sk"][:] = 0.02
    s["q"] *= 2.0 ** far
    got = n64(attend(gpu, cuda(s)))
    s["q"][:] = 0                               # the same weights without a score's rounding
    check_attention(s, torch.tensor(got))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_out_beside_q(gpu, dtype):
    """out may begin where q ends and end where it begins; over q it is refused."""
    s = cuda(make(120, [1, 3], [300, 40], 16, 64, 2, dtype, 4))
    want, n = attend(gpu, s), len(s["q"])
    buf = torch.zeros((3 * n,) + s["q"].shape[1:], dtype=dtype, device="cuda")
    buf[n:2 * n] = s["q"]
    s["q"] = buf[n:2 * n]
    for out in (buf[:n], buf[2 * n:]):
        assert torch.equal(attend(gpu, s, out=out), want)
    for at in (1, n, 2 * n - 1):
        with pytest.raises(gpu.BitLinearError) as e:
            attend(gpu, s, out=buf[at:at + n])
        assert e.value.status == 4
    assert torch.equal(attend(gpu, s), want)


def test_a_call_past_the_runtimes_grid_writes_nothing(gpu):
    """512 rows of 65520 heads in 256 sequences with room for cuts: the join of
    their 33 million rows would be 2^33 threads."""
    B, n, KVH, G, T, D = 256, 512, 4095, 16, 16, 64
    c = gpu.kv8_cache(1, KVH, T, D)
    q = torch.empty(n, KVH * G, D, dtype=BF16, device="cuda")
    out = torch.full_like(q, 77.0)
    q_start = torch.arange(0, n + 1, n // B, dtype=torch.int32, device="cuda")
    lengths = torch.full((B,), 2, dtype=torch.int32, device="cuda")
    table = torch.full((B, 512), -1, dtype=torch.int32, device="cuda")
    with pytest.raises(gpu.BitLinearError) as e:
        gpu.bitlinear_kv8_attention(q, q_start, lengths, table, c, out=out)
    assert e.value.status == 7
    torch.cuda.synchronize()
    assert all(bool((x == 77.0).all()) for x in out.split(64))


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
    need = gpu.load().bitlinear_kv8_attention_ws_bytes(len(s["q"]), KVH * G, len(n), s["table"].shape[1], KVH, T, D)
    assert need > 0 or (name, case) == ("MANY", 0)
    buf = torch.full((need + (1 << 20),), fill, dtype=torch.uint8, device="cuda")
    buf[need:] = 170
    out = attend(gpu, d, ws=buf[:need])
    assert (buf[need:] == 170).all()
    check_attention(s, out)
    assert torch.equal(out, attend(gpu, d))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", [float("inf"), float("nan"), 3e38])
@pytest.mark.parametrize("n,length,T,D,KVH,G,width", [
    (60, 70, 16, 64, 2, 4, 0), (40, 1300, 32, 128, 1, 3, 9000), (200, 333, 32, 64, 2, 4, 70000),
    (200, 333, 16, 128, 2, 8, 70000), (301, 2500, 64, 128, 2, 4, 30000)])
def test_later_blocks_never_show(gpu, n, length, T, D, KVH, G, width, bad, dtype):
    """Scales of a block that overflowed: rows whose tokens all stand before it
    are as if it held ones; also beside rows that see it."""
    s = make(140, [n, 1], [length, 40], T, D, KVH, dtype, G, width=-(-width // T))
    at = (length - n // 2) // T                # the block, and where it begins among the rows
    rows = at * T - (length - n)
    assert 0 < rows < n
    block = int(s["table"][0, at])
    for name in ("sk", "sv"):
        s[name][block] = bad
    got = attend(gpu, cuda(s))
    for name in ("sk", "sv"):
        s[name][block] = 0.02
    keep = torch.cat([got[:rows], torch.zeros_like(got[rows:n]), got[n:]]).cpu()
    plain = attend(gpu, cuda(s)).cpu()
    keep[rows:n] = plain[rows:n]
    check_attention(s, keep)
