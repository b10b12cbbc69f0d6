"""The decode stacks with rotated queries and keys and over 4-bit caches: token by
token against the oracle's parts fed with the GPU's own trace, and captured."""
import numpy as np
import pytest
import torch

import workloads
from oracle import kv4 as ref4
from oracle import kv8 as ref
from test_stack_kv_gpu import SEGMENTS, bitlinear, build, scaled

pytestmark = pytest.mark.gpu

SIZES = [(512, 128, 640, 64, 16), (512, 256, 704, 128, 64), (640, 640, 512, 128, 32)]


def cos_sin(rows, rot):
    at = torch.arange(rows, dtype=torch.float64)[:, None]
    a = at * 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    return torch.cat([a.cos(), a.sin()], 1).float()


@pytest.mark.parametrize("kind", ["8 halves", "8 neighbours", "4", "4 halves", "4 neighbours"])
@pytest.mark.parametrize("H,KV,F,D,T", SIZES)
def test_token_by_token(gpu, H, KV, F, D, T, kind):
    """Each token: the cache is the oracle's of the traced k (rotated) and v to the
    bit; o is the BitLinear of the oracle's attention of the traced q (rotated;
    its last bits may move codes by one step); the sums are exact."""
    bl, n_layers, n_tok, nb = gpu, 2, 37, 5
    layers, plain = build(bl, 3, n_layers, H, KV, F)
    heads, rot = KV // D, 32 if "neighbours" in kind else D
    table = torch.tensor([[3, 0, 4, 1, 2]], dtype=torch.int32)
    q_start = torch.tensor([0, 1], dtype=torch.int32)
    turn = cos_sin(nb * T, rot)
    rope = None if kind == "4" else bl.Rope(turn.cuda(), "neighbours" in kind)
    eight = kind.startswith("8")
    call = bl.bitlinear_decode_stack_kv_rope if eight else bl.bitlinear_decode_stack_kv4
    caches = [(bl.kv8_cache if eight else bl.kv4_cache)(nb, heads, T, D) for _ in range(n_layers)]
    if eight:
        mine = [[np.zeros((nb, heads, T, D), np.int8), np.zeros((nb, heads, T, D), np.int8),
                 np.zeros((nb, heads), np.float32), np.zeros((nb, heads), np.float32)] for _ in range(n_layers)]
    else:
        mine = [[np.zeros((nb, heads, T, D), int), np.zeros((nb, heads, T, D), int),
                 np.zeros((nb, heads, T, 2), np.float16), np.zeros((nb, heads, T, 2), np.float16)]
                for _ in range(n_layers)]
    worst = 0.0
    for t in range(n_tok):
        x = workloads.stack_token(100 + t, H).cuda()
        x_in = x.cpu().numpy()
        length = torch.tensor([t + 1], dtype=torch.int32)
        tr = call(layers, caches, x, q_start.cuda(), length.cuda(), table.cuda(), H=H, KV=KV, F=F, D=D, rope=rope,
                  trace=True).cpu().numpy()
        cuts = np.cumsum([0, H, H, KV, KV, H, H, H])
        meta = q_start.numpy(), length.numpy(), table.numpy()
        for l in range(n_layers):
            s = {n: tr[l][cuts[i]:cuts[i + 1]] for i, n in enumerate(SEGMENTS)}
            assert np.array_equal(s["x_in"], x_in)
            for n, w, g in (("q", "Wq", "gq"), ("k", "Wk", "gk"), ("v", "Wv", "gv")):
                assert np.array_equal(s[n], bitlinear(x_in, plain[l], w, g)), (t, l, n)
            q, k, v = (s[n].astype(np.float64).reshape(1, -1, D) for n in "qkv")
            if rope is not None:
                q, k = (ref4.rotate(y, [t], turn.numpy(), rope.interleaved, nb * T) for y in (q, k))
            K, V, ak, av = mine[l]
            c = [y.cpu().numpy() for y in caches[l]]
            if eight:
                ref.append(k, K, ak, *meta)
                ref.append(v, V, av, *meta)
                assert np.array_equal(c[0], K) and np.array_equal(c[1].transpose(0, 1, 3, 2), V)
                a = ref.attention(q, K, V.transpose(0, 1, 3, 2), ak, av, *meta, D ** -0.5)[0].reshape(-1)
            else:
                ref4.append(k, K, ak, *meta)
                ref4.append(v, V, av, *meta)
                for got, want in zip(c, ref4.pack(K, V)):
                    assert np.array_equal(got, want)
                a = ref4.attention(q, K, ak, V, av, *meta, D ** -0.5)[0].reshape(-1)
            assert np.array_equal(c[2], ak) and np.array_equal(c[3], av)
            o = bitlinear(a, plain[l], "Wo", "go")
            # codes that sit within fp32's error of a tie may move by one step:
            # each moves o by a step times gamma, and few do
            step = scaled(a) * plain[l]["go"][0]
            worst = max(worst, np.abs(s["o"] - o).max() / step)
            assert np.array_equal(s["x_mid"], (s["x_in"] + s["o"]).astype(np.float32))
            x_in = (s["x_mid"] + s["y"]).astype(np.float32)
        assert np.array_equal(x.cpu().numpy(), x_in)
    assert worst <= 2.01, worst


@pytest.mark.parametrize("bits", [4, 8])
def test_without_a_turn_it_is_the_stack_without_rotation(gpu, bits):
    """A table of cosines 1 and sines 0 gives the unrotated stack's bits; with no trace
    the same as with one."""
    bl, (H, KV, F, D, T) = gpu, SIZES[0]
    layers, _ = build(bl, 5, 2, H, KV, F)
    still = torch.cat([torch.ones(3 * T, D // 2), torch.zeros(3 * T, D // 2)], 1).cuda()
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32).cuda()
    q_start = torch.tensor([0, 1], dtype=torch.int32).cuda()
    make = bl.kv8_cache if bits == 8 else bl.kv4_cache
    one, two, three = ([make(3, KV // D, T, D) for _ in range(2)] for _ in range(3))
    for t in range(20):
        x = workloads.stack_token(t, H).cuda()
        n = torch.tensor([t + 1], dtype=torch.int32).cuda()
        a, b, c = x.clone(), x.clone(), x.clone()
        args = q_start, n, table, H, KV, F, D
        if bits == 8:
            bl.bitlinear_decode_stack_kv(layers, one, a, *args)
            bl.bitlinear_decode_stack_kv_rope(layers, two, b, *args, bl.Rope(still))
            bl.bitlinear_decode_stack_kv_rope(layers, three, c, *args, bl.Rope(still, True), trace=True)
        else:
            bl.bitlinear_decode_stack_kv4(layers, one, a, *args)
            bl.bitlinear_decode_stack_kv4(layers, two, b, *args, bl.Rope(still))
            bl.bitlinear_decode_stack_kv4(layers, three, c, *args, bl.Rope(still, True), trace=True)
        assert torch.equal(a, b) and torch.equal(a, c)
    for p, q in zip(one, two):
        assert all(torch.equal(u, v) for u, v in zip(p, q))


def test_captured(gpu):
    """A step of the 4-bit stack with rotation, captured once and replayed token by
    token, against the call made anew."""
    bl, (H, KV, F, D, T) = gpu, SIZES[1]
    layers, _ = build(bl, 7, 2, H, KV, F)
    rope = bl.Rope(cos_sin(4 * T, D).cuda())
    table = torch.tensor([[2, 0, 3, 1]], dtype=torch.int32).cuda()
    q_start = torch.tensor([0, 1], dtype=torch.int32).cuda()
    length = torch.tensor([1], dtype=torch.int32).cuda()
    x = torch.zeros(H, device="cuda")
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    mine, eager = ([bl.kv4_cache(4, KV // D, T, D) for _ in range(2)] for _ in range(2))
    bl.bitlinear_decode_stack_kv4(layers, mine, x, q_start, length, table, H, KV, F, D, rope, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bl.bitlinear_decode_stack_kv4(layers, mine, x, q_start, length, table, H, KV, F, D, rope, ws=ws)
    for t in range(8):
        token = workloads.stack_token(t, H).cuda()
        x.copy_(token)
        length.fill_(t + 1)
        graph.replay()
        want = token.clone()
        bl.bitlinear_decode_stack_kv4(layers, eager, want, q_start, length, table, H, KV, F, D, rope)
        torch.cuda.synchronize()
        assert torch.equal(x, want)
    for p, q in zip(mine, eager):
        assert all(torch.equal(u, v) for u, v in zip(p, q))


def test_refusals(gpu):
    bl, (H, KV, F, D, T) = gpu, SIZES[0]
    layers, _ = build(bl, 9, 1, H, KV, F)
    meta = (torch.tensor([0, 1], dtype=torch.int32).cuda(), torch.tensor([1], dtype=torch.int32).cuda(),
            torch.zeros(1, 2, dtype=torch.int32).cuda())
    x, turn = workloads.stack_token(1, H).cuda(), cos_sin(2 * T, D).cuda()
    c8, c4 = [bl.kv8_cache(2, KV // D, T, D)], [bl.kv4_cache(2, KV // D, T, D)]
    for f, right, wrong in ((bl.bitlinear_decode_stack_kv_rope, c8, c4), (bl.bitlinear_decode_stack_kv4, c4, c8)):
        with pytest.raises((TypeError, ValueError)):
            f(layers, wrong, x, *meta, H, KV, F, D, bl.Rope(turn))
        with pytest.raises(ValueError):
            f(layers, right * 2, x, *meta, H, KV, F, D, bl.Rope(turn))
        with pytest.raises(bl.BitLinearError) as e:              # a table that is too short
            f(layers, right, x, *meta, H, KV, F, D, bl.Rope(turn[:-1]))
        assert e.value.status == 2
        with pytest.raises(bl.BitLinearError) as e:
            f(layers, right, x, *meta, H, KV, F, D, bl.Rope(turn), ws=torch.empty(64, dtype=torch.uint8).cuda())
        assert e.value.status == 5
    with pytest.raises(ValueError):
        bl.bitlinear_decode_stack_kv_rope(layers, c8, x, *meta, H, KV, F, D, None)
