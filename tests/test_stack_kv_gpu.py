"""The decode stack over 8-bit caches (bitlinear_decode_stack_kv): a run of the
calls as a decode loop makes them, against the oracle's parts fed with the
GPU's own trace, and the whole step from layers to output head."""
import numpy as np
import pytest
import torch

import oracle
import workloads
from oracle import kv8 as ref

pytestmark = pytest.mark.gpu

NAMES = workloads.STACK_NAMES
GAMMAS = ("gq", "gk", "gv", "go", "gg", "gu", "gd")
SEGMENTS = ("x_in", "q", "k", "v", "o", "x_mid", "y")


def build(bl, seed, n_layers, H, KV, F):
    out, plain = [], []
    for l in range(n_layers):
        W = workloads.stack_layer_weights(seed, l, H, KV, F)
        L = dict(ffn_norm=workloads.stack_norm_gain(seed, l, F).cuda())
        for name, g in zip(NAMES, GAMMAS):
            L[name], L[g] = bl.quant_weight_absmean_pack(W[name].cuda())
        out.append(L)
        plain.append({k: v.cpu().numpy() for k, v in L.items()})
    return out, plain


def bitlinear(x, L, w, g):
    Xq, d = oracle.quant_act(np.ascontiguousarray(x, dtype=np.float32)[None])
    acc, _ = oracle.bitlinear(Xq, d, L[w], L[g][0], len(x))
    return oracle.dequant_f32(acc, d, L[g][0])[0]


def scaled(x):
    """Absmax int8 codes move where their input does by a rounding; what one step
    of one code is worth, the largest value / 127."""
    return np.abs(x).max() / 127


@pytest.mark.parametrize("H,KV,F,D,T", [(512, 128, 640, 64, 16), (512, 256, 704, 128, 64), (640, 640, 512, 128, 32)])
def test_token_by_token(gpu, H, KV, F, D, T):
    """Each token: q, k, v are the BitLinears of the traced input to the bit; the
    cache is the oracle's of the traced k, v to the bit; o is the BitLinear of
    the oracle's attention (whose last bits may move codes by one step); the
    sums are exact."""
    bl, n_layers, n_tok, nb = gpu, 2, 37, 5
    layers, plain = build(bl, 3, n_layers, H, KV, F)
    heads = KV // D
    caches = [bl.kv8_cache(nb, heads, T, D) for _ in range(n_layers)]
    mine = [[np.zeros((nb, heads, T, D), np.int8), np.zeros((nb, heads, T, D), np.int8),
             np.zeros((nb, heads), np.float32), np.zeros((nb, heads), np.float32)] for _ in range(n_layers)]
    table = torch.tensor([[3, 0, 4, 1, 2]], dtype=torch.int32)
    q_start = torch.tensor([0, 1], dtype=torch.int32)
    dims = dict(H=H, KV=KV, F=F, D=D)
    worst = 0.0
    for t in range(n_tok):
        x = workloads.stack_token(100 + t, H).cuda()
        x0 = x.clone()
        length = torch.tensor([t + 1], dtype=torch.int32)
        tr = bl.bitlinear_decode_stack_kv(layers, caches, x, q_start.cuda(), length.cuda(), table.cuda(), **dims,
                                          trace=True)
        tr = tr.cpu().numpy()
        cuts = np.cumsum([0, H, H, KV, KV, H, H, H])
        x_in = x0.cpu().numpy()
        for l in range(n_layers):
            s = {n: tr[l][cuts[i]:cuts[i + 1]] for i, n in enumerate(SEGMENTS)}
            assert np.array_equal(s["x_in"], x_in)
            for n, w, g in (("q", "Wq", "gq"), ("k", "Wk", "gk"), ("v", "Wv", "gv")):
                assert np.array_equal(s[n], bitlinear(x_in, plain[l], w, g)), (t, l, n)
            K, V, sk, sv = mine[l]
            meta = q_start.numpy(), length.numpy(), table.numpy()
            for codes, scale, y in ((K, sk, s["k"]), (V, sv, s["v"])):
                ref.append(y.astype(np.float64).reshape(1, heads, D), codes, scale, *meta)
            c = caches[l]
            assert np.array_equal(c.K.cpu().numpy(), K) and np.array_equal(c.sk.cpu().numpy(), sk)
            assert np.array_equal(c.V.cpu().numpy().transpose(0, 1, 3, 2), V)
            assert np.array_equal(c.sv.cpu().numpy(), sv)
            a = ref.attention(s["q"].astype(np.float64).reshape(1, H // D, D), K, V.transpose(0, 1, 3, 2), sk, sv,
                              *meta, D ** -0.5)[0].reshape(-1)
            o = bitlinear(a, plain[l], "Wo", "go")
            # codes that sit within fp32's error of a tie may move by one step:
            # each moves o by a step times gamma, and few do
            step = scaled(a) * plain[l]["go"][0]
            worst = max(worst, np.abs(s["o"] - o).max() / step)
            assert np.array_equal(s["x_mid"], (s["x_in"] + s["o"]).astype(np.float32))
            x_in = (s["x_mid"] + s["y"]).astype(np.float32)
        assert np.array_equal(x.cpu().numpy(), x_in)
    assert worst <= 2.01, worst


def test_first_token_is_near_the_stand_in(gpu):
    """With one token the attention gives its value as the cache holds it: within
    half a step of v, so q, k, v of the first layer are the stand-in's."""
    H, KV, F, D = 512, 128, 640, 64
    layers, _ = build(gpu, 5, 1, H, KV, F)
    x = workloads.stack_token(9, H).cuda()
    a, b = x.clone(), x.clone()
    want = gpu.bitlinear_decode_stack(layers, a, H, KV, F, D, trace=True, path=gpu.BL_STACK_LAUNCHES)
    got = gpu.bitlinear_decode_stack_kv(layers, [gpu.kv8_cache(1, KV // D, 64, D)], b,
                                        torch.tensor([0, 1], dtype=torch.int32).cuda(),
                                        torch.tensor([1], dtype=torch.int32).cuda(),
                                        torch.zeros(1, 1, dtype=torch.int32).cuda(), H, KV, F, D, trace=True)
    n = 2 * H + 2 * KV
    assert torch.equal(want[:, :n], got[:, :n])


def test_step_to_the_head_in_a_graph(gpu):
    """Layers over caches, then 4-bit head: captured once, replayed token by
    token, against the same calls made one by one."""
    bl = gpu
    H, KV, F, D, T, nb, vocab = 512, 128, 640, 64, 16, 4, 1000
    layers, _ = build(bl, 7, 2, H, KV, F)
    Wh = torch.randn(vocab, H, generator=torch.Generator().manual_seed(1)).cuda()
    head = bl.quant_weight_absmax_i4(Wh, group=64)
    q_start = torch.tensor([0, 1], dtype=torch.int32).cuda()
    table = torch.tensor([[2, 0, 3, 1]], dtype=torch.int32).cuda()

    def state():
        return dict(caches=[bl.kv8_cache(nb, KV // D, T, D) for _ in range(2)], x=torch.zeros(H, device="cuda"),
                    length=torch.zeros(1, dtype=torch.int32, device="cuda"), Y=torch.zeros(1, vocab, device="cuda"))

    def step(s):
        bl.bitlinear_decode_stack_kv(layers, s["caches"], s["x"], q_start, s["length"], table, H, KV, F, D)
        bl.bitlinear_gemv_w4(s["x"].view(1, H), *head, Y=s["Y"])

    a, b = state(), state()
    step(state())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a)
    for t in range(40):
        x = workloads.stack_token(200 + t, H)
        for s in (a, b):
            s["x"].copy_(x)
            s["length"].fill_(t + 1)
        graph.replay()
        step(b)
        torch.cuda.synchronize()
        assert torch.equal(a["x"], b["x"]) and torch.equal(a["Y"], b["Y"]), t
        for c, d in zip(a["caches"], b["caches"]):
            assert all(torch.equal(u, v) for u, v in zip(c, d))
    W = ref.unpack_w4(head[0].cpu().numpy()) * np.repeat(head[1].double().cpu().numpy(), 64, 1)
    x = b["x"].double().cpu().numpy()
    tol = np.abs(W) @ np.abs(x) * (2.0 ** -22 + (H + 8) * 2.0 ** -24) + np.abs(x).max() * np.abs(W).sum(1) * 2.0 ** -22
    assert (np.abs(b["Y"].double().cpu().numpy()[0] - W @ x) <= tol).all()


def test_refusals(gpu):
    bl = gpu
    H, KV, F, D = 512, 128, 640, 64
    layers, _ = build(bl, 3, 1, H, KV, F)
    q_start = torch.tensor([0, 1], dtype=torch.int32).cuda()
    length = torch.tensor([1], dtype=torch.int32).cuda()
    table = torch.zeros(1, 1, dtype=torch.int32).cuda()
    x = torch.zeros(H).cuda()
    c = bl.kv8_cache(1, KV // D, 64, D)
    ok = (layers, [c], x, q_start, length, table, H, KV, F, D)

    def call(**kw):
        names = ("layers", "caches", "x", "q_start", "lengths", "table", "H", "KV", "F", "D")
        args = dict(zip(names, ok))
        args.update(kw)
        return bl.bitlinear_decode_stack_kv(**args)
    for kw in (dict(caches=[]), dict(x=x[:64]), dict(F=576), dict(table=table.view(1, 1, 1)),
               dict(q_start=torch.zeros(3, dtype=torch.int32).cuda(), lengths=torch.zeros(2, dtype=torch.int32).cuda(),
                    table=torch.zeros(2, 1, dtype=torch.int32).cuda())):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(caches=[bl.kv8_cache(1, 1, 64, D)]), dict(caches=[bl.kv8_cache(1, 1, 64, 128)]),
               dict(caches=[bl.kv8_cache(1, KV // D, 8, D)]), dict(scale=float("inf"))):
        with pytest.raises(bl.BitLinearError) as e:
            call(**kw)
        assert e.value.status == 2
    with pytest.raises(bl.BitLinearError) as e:
        call(ws=torch.zeros(64, dtype=torch.uint8).cuda())
    assert e.value.status == 5
    assert torch.equal(x, torch.zeros_like(x))
