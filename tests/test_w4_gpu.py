"""4-bit weights with group scales against the 64-bit oracle: codes, scales and
dequantised weights exactly, the product within a bound from its arithmetic."""
import numpy as np
import pytest
import torch

from oracle import kv8 as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def n64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,K,group", [(1, 32, 32), (3, 64, 32), (7, 64, 64), (5, 640, 128), (129, 96, 32),
                                       (33, 2560, 64), (2, 128, 128), (17, 8192, 128)])
def test_quantiser_is_exact(gpu, N, K, group, dtype):
    g = torch.Generator().manual_seed(N + K)
    W = (torch.randn(N, K, generator=g) * 0.02).to(dtype)
    W[0, :group] = 0                                        # an empty group
    W[-1, -group:] = torch.arange(group) % 15 - 7.0         # ties and the codes themselves
    W[-1, -1] = 7.5 if dtype == F32 else 7.0
    if N > 2:
        W[1, :group] *= 1e-36                               # tiny and large scales
        W[1, group:2 * group] *= 1e30
        W[2, :group] = 1e-44 if dtype == F32 else 1e-40
    Wq4, s = gpu.quant_weight_absmax_i4(W.cuda(), group=group)
    q, sc = ref.quant_w4(n64(W), group)
    assert np.array_equal(n64(s), sc)
    assert np.array_equal(ref.unpack_w4(Wq4.cpu().numpy()), q)
    v = q * np.repeat(sc, group, 1)
    assert np.array_equal(n64(gpu.dequant_weight_i4(Wq4, s)), v)
    assert np.array_equal(n64(gpu.dequant_weight_i4(Wq4, s, dtype=BF16)), ref.bf16(v))


def test_dequantiser_takes_every_code(gpu):
    Wq4 = torch.arange(256, dtype=torch.uint8).view(4, 64).cuda()
    s = torch.tensor([[1.0, 0.5], [-2.0, 0.0], [3.0, 1e-3], [1e30, 7.0]]).to(BF16).cuda()
    want = ref.unpack_w4(Wq4.cpu().numpy()) * np.repeat(n64(s), 64, 1)
    assert np.array_equal(n64(gpu.dequant_weight_i4(Wq4, s)), np.float32(want).astype(np.float64))


def check_product(bl, X, Wq4, s, group, **kw):
    """An fp32 x loses at most 2^-22 of the largest of 128 elements; bf16 loses
    nothing.  A sum of K products and K / group group sums, each of at most K
    additions, adds K 2^-24 of the terms' magnitude and two roundings a group.
    bf16 products from three tokens on run with the codes + 24 and take 24 sum x
    off again, 32 elements at a time: 64 additions of terms that come to (|code|
    + 48) |x| s at most, so another 64 2^-24 of those."""
    Y = bl.bitlinear_gemv_w4(X.cuda(), Wq4.cuda(), s.cuda(), **kw)
    W = ref.unpack_w4(Wq4.numpy()) * np.repeat(n64(s), group, 1)
    x, K = n64(X), X.shape[1]
    pad = np.zeros((len(x), -K % 128))
    top = np.abs(np.concatenate([x, pad], 1)).reshape(len(x), -1, 128).max(-1)
    top = np.repeat(top, 128, 1)[:, :K]
    tol = top @ np.abs(W).T * 2.0 ** -22 + np.abs(x) @ np.abs(W).T * (K + 8) * 2.0 ** -24
    if X.dtype == BF16 and len(x) > 2:
        tol += np.abs(x) @ (np.abs(W) + 48 * np.abs(np.repeat(n64(s), group, 1))).T * 64 * 2.0 ** -24
    got = n64(Y)
    assert np.isfinite(got).all()
    worst = np.max(np.abs(got - x @ W.T) - tol, initial=-1.0)
    assert worst <= 0, worst
    return Y


def weights(g, N, K, group):
    Wq4 = torch.randint(0, 256, (N, K // 2), generator=g).to(torch.uint8)
    s = (0.01 * (0.5 + torch.rand(N, K // group, generator=g))).to(BF16)
    return Wq4, s


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,N,K,group", [
    (1, 1, 32, 32), (1, 16, 128, 128), (1, 17, 64, 64), (2, 33, 96, 32), (3, 100, 160, 32), (16, 1, 128, 64),
    (1, 640, 2560, 128), (5, 257, 2560, 64), (16, 640, 2560, 32), (7, 48, 6912, 128), (1, 2000, 192, 64),
    (9, 31, 4096, 64), (13, 5000, 128, 32), (1, 20000, 256, 128), (16, 40, 20480, 128), (1, 3, 131072, 128),
])
def test_product(gpu, M, N, K, group, dtype):
    g = torch.Generator().manual_seed(M * N + K)
    Wq4, s = weights(g, N, K, group)
    X = torch.randn(M, K, generator=g)
    X[:, torch.randperm(K, generator=g)[:max(1, K // 100)]] *= 20
    X = X.to(dtype)
    Y = check_product(gpu, X, Wq4, s, group)
    assert torch.equal(Y, gpu.bitlinear_gemv_w4(X.cuda(), Wq4.cuda(), s.cuda()))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,N,K,group", [
    (1, 8191, 96, 32), (2, 8192, 96, 32), (2, 8199, 640, 64), (1, 16383, 128, 128), (1, 16384, 160, 32),
    (1, 32767, 64, 64), (1, 32769, 544, 32), (2, 32768, 512, 128), (2, 65535, 96, 32), (1, 65537, 64, 32),
    (2, 65536, 1056, 32), (1, 9000, 16384, 128), (2, 9000, 8192, 64), (2, 9000, 8320, 64),
    (3, 4096, 96, 32), (7, 4097, 256, 64), (16, 8192, 128, 128), (5, 8200, 96, 32), (16, 9001, 640, 64),
    (3, 24576, 64, 64), (9, 24577, 160, 32), (16, 33001, 128, 128)])
def test_product_at_the_bounds_of_the_forms(gpu, M, N, K, group, dtype):
    test_product(gpu, M, N, K, group, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_product_over_the_number_range(gpu, dtype):
    """Tokens that are zero, tiny, huge, and of mixed magnitude."""
    g = torch.Generator().manual_seed(4)
    Wq4, s = weights(g, 50, 512, 64)
    X = torch.randn(6, 512, generator=g)
    X[0] = 0
    X[1] *= 1e-36
    X[2] *= 1e34
    X[3] *= 10.0 ** torch.linspace(-30, 3, 512)
    X[4] = 0
    X[4, 130] = -3.0
    check_product(gpu, X.to(dtype), Wq4, s, 64)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M", [1, 2, 3, 16])
@pytest.mark.parametrize("group", [32, 128])
def test_product_at_the_largest_tokens(gpu, M, group, dtype):
    """Just below 2^116, of one sign and of both, with the codes' extremes."""
    g = torch.Generator().manual_seed(6)
    Wq4, s = weights(g, 40, 512, group)
    Wq4[:8], Wq4[8:16], Wq4[16:24] = 0x77, 0x88, 0x87      # 7 7, -8 -8, 7 -8
    X = torch.full((M, 512), 2.0 ** 116 * (1 - 2.0 ** -8))
    X[::2] *= torch.randint(0, 2, X[::2].shape, generator=g) * 2 - 1
    s *= 2.0 ** -6                                          # the result itself stays in range
    check_product(gpu, X.to(dtype), Wq4, s, group)


def test_product_of_the_quantisers_weights(gpu):
    """Quantise, multiply: as a head is used, against the dequantised weights."""
    g = torch.Generator().manual_seed(6)
    W = torch.randn(900, 640, generator=g) * 0.02
    Wq4, s = gpu.quant_weight_absmax_i4(W.cuda(), group=64)
    X = torch.randn(2, 640, generator=g)
    check_product(gpu, X, Wq4.cpu(), s.cpu(), 64)


def test_writes_its_rows_only(gpu):
    g = torch.Generator().manual_seed(8)
    for M, N, K in ((1, 37, 256), (11, 50, 96)):
        Wq4, s = weights(g, N, K, 32)
        X = torch.randn(M, K, generator=g).cuda()
        buf = torch.full((M + 2, N), 5.0, device="cuda")
        gpu.bitlinear_gemv_w4(X, Wq4.cuda(), s.cuda(), Y=buf[1:-1])
        assert (buf[0] == 5).all() and (buf[-1] == 5).all()
        assert not (buf[1:-1] == 5).any()
        w = torch.full((N * K + 64,), 9.0, dtype=BF16, device="cuda")
        gpu.dequant_weight_i4(Wq4.cuda(), s.cuda(), dtype=BF16, W=w[:N * K].view(N, K))
        assert (w[N * K:] == 9).all()


def test_graph_and_streams(gpu):
    g = torch.Generator().manual_seed(9)
    W = torch.randn(300, 512, generator=g).cuda()
    X = torch.randn(4, 512, generator=g).cuda()
    Wq4, s = gpu.quant_weight_absmax_i4(W, group=32)
    Y = torch.zeros(4, 300, device="cuda")
    gpu.bitlinear_gemv_w4(X, Wq4, s, Y=Y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu.quant_weight_absmax_i4(W, group=32, Wq4=Wq4, s=s)
        gpu.bitlinear_gemv_w4(X, Wq4, s, Y=Y)
    other = torch.cuda.Stream()
    for i in range(4):
        W.mul_(-1.5)
        X.add_(0.25)
        graph.replay()
        q, t = gpu.quant_weight_absmax_i4(W, group=32)
        torch.cuda.synchronize()
        want = gpu.bitlinear_gemv_w4(X, q, t, stream=other)
        torch.cuda.synchronize()
        assert torch.equal(Y, want) and torch.equal(q, Wq4) and torch.equal(s, t)


def test_refusals(gpu):
    W = torch.randn(8, 128).cuda()
    Wq4, s = gpu.quant_weight_absmax_i4(W, group=32)
    X = torch.randn(2, 128).cuda()
    for bad in (dict(group=16), dict(group=256), dict(group=96)):
        with pytest.raises(ValueError):
            gpu.quant_weight_absmax_i4(W, **bad)
    with pytest.raises(ValueError):
        gpu.quant_weight_absmax_i4(W.t())
    for bad, err in ((W.half(), TypeError), (W.cpu(), TypeError), (W[0], ValueError)):
        with pytest.raises(err):
            gpu.quant_weight_absmax_i4(bad)
    for X_, W_, s_ in ((X[:, :64], Wq4, s), (X.half(), Wq4, s), (X, Wq4.char(), s), (X, Wq4, s.float()),
                       (X, Wq4, s[:, :3]), (X, Wq4, s[:7]), (X, Wq4.t(), s), (X, Wq4.cpu(), s)):
        with pytest.raises((TypeError, ValueError)):
            gpu.bitlinear_gemv_w4(X_, W_, s_)
    with pytest.raises(gpu.BitLinearError) as e:
        gpu.bitlinear_gemv_w4(torch.zeros(17, 128).cuda(), Wq4, s)
    assert e.value.status == 2
    with pytest.raises(ValueError):
        gpu.bitlinear_gemv_w4(X, Wq4, s, Y=torch.zeros(2, 7).cuda())
    with pytest.raises(TypeError):
        gpu.dequant_weight_i4(Wq4, s, dtype=torch.float16)
    # nothing to do
    assert gpu.bitlinear_gemv_w4(X[:0], Wq4, s).shape == (0, 8)
    assert gpu.bitlinear_gemv_w4(X, Wq4[:0], s[:0]).shape == (2, 0)
    none, sn = gpu.quant_weight_absmax_i4(W[:, :0], group=32)
    assert (gpu.bitlinear_gemv_w4(X[:, :0].contiguous(), none, sn) == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,N", [(1, 16383), (1, 16384), (1, 32768), (1, 65536), (2, 8192), (2, 40000), (2, 70000),
                                 (3, 40000), (16, 70000)])
def test_product_over_nothing_is_zero(gpu, M, N, dtype):
    """K = 0 at row counts of every form; the empty operands' addresses are NULL."""
    for group in (32, 64, 128):
        X = torch.empty(M, 0, dtype=dtype, device="cuda")
        Wq4, s = gpu.quant_weight_absmax_i4(torch.empty(N, 0, device="cuda"), group=group)
        assert X.data_ptr() == Wq4.data_ptr() == s.data_ptr() == 0
        Y = torch.full((M + 1, N), 5.0, device="cuda")
        gpu.bitlinear_gemv_w4(X, Wq4, s, Y=Y[:M])
        assert (Y[:M] == 0).all() and (Y[M] == 5).all()


PRODUCTS = [
    (1, 1, 32, 32), (1, 17, 64, 64), (2, 33, 96, 32), (3, 100, 160, 32), (16, 1, 128, 64), (1, 640, 2560, 128),
    (5, 257, 2560, 64), (16, 640, 2560, 32), (7, 48, 6912, 128), (1, 2000, 192, 64), (9, 31, 4096, 64), (4, 70, 224, 32),
    (13, 5000, 192, 64), (1, 20000, 256, 128), (1, 20000, 544, 32), (2, 9000, 1056, 32), (2, 40000, 576, 64),
    (1, 66000, 1120, 32), (3, 4097, 2592, 32), (6, 9000, 320, 64), (16, 25000, 288, 32), (16, 40, 20480, 128),
    (1, 3, 131072, 128), (2, 20, 131008, 64), (3, 5, 131072, 32), (16, 20, 131040, 32), (8, 3, 130944, 64),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,N,K,group", PRODUCTS)
def test_product_of_small_integers_is_exact(gpu, M, N, K, group, dtype):
    """Tokens of -3 .. 3 and scales of 1, 2 and 4: every product and sum is an
    integer below 131072 * 3 * 8 * 4 < 2^24 (with the codes + 24 those of a group,
    128 * 3 * 48), so nothing is rounded; a value left out or taken twice shows."""
    g = torch.Generator().manual_seed(K + N)
    Wq4, s = weights(g, N, K, group)
    s = (2.0 ** torch.randint(0, 3, s.shape, generator=g)).to(BF16)
    X = torch.randint(-3, 4, (M, K), generator=g).to(dtype)
    Y = gpu.bitlinear_gemv_w4(X.cuda(), Wq4.cuda(), s.cuda())
    q = torch.stack(((Wq4 & 15 ^ 8).to(torch.int8) - 8, (Wq4 >> 4 ^ 8).to(torch.int8) - 8), -1).view(N, K)
    W = q.double().view(N, -1, group) * s.double()[..., None]
    assert torch.equal(Y.cpu().double(), X.double() @ W.view(N, K).T)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,N,K,group", PRODUCTS)
def test_product_by_its_additions(gpu, M, N, K, group, dtype):
    """A term is rounded once in each addition that it passes through, by 2^-24 of
    the sum.  One or two tokens: 16 of a lane's 32 values, the two halves, a slice
    of 512 values after another, 4 steps over the lanes, 8 waves.  More: the
    products of a group and as many of the other half of X or the -24 (each
    counted twice, as a matrix instruction may cut and not round), the groups, 16
    waves.  fp32 tokens from three on lose 2^-22 of the largest of 128 values
    besides; bf16 tokens' +24 and -24 times x pass through the 64 additions of two
    matrix instructions, counted twice, and are gone then."""
    g = torch.Generator().manual_seed(M * N + K + 1)
    Wq4, s = weights(g, N, K, group)
    X = torch.randn(M, K, generator=g)
    X[:, torch.randperm(K, generator=g)[:max(1, K // 100)]] *= 20
    X = X.to(dtype)
    got = gpu.bitlinear_gemv_w4(X.cuda(), Wq4.cuda(), s.cuda()).cpu().double()
    q = torch.stack(((Wq4 & 15 ^ 8).to(torch.int8) - 8, (Wq4 >> 4 ^ 8).to(torch.int8) - 8), -1).view(N, K).double()
    d = s.double().repeat_interleave(group, 1)
    x = X.double()
    want = x @ (q * d).T
    through = 17 + K / 512 + 1 + 4 + 8 if M <= 2 else 4 * group + K / group + 16
    tol = x.abs() @ (q.abs() * d).T * through * 1.001 * 2.0 ** -24
    if M > 2 and dtype == BF16:
        tol += x.abs() @ d.T * 48 * 128 * 1.001 * 2.0 ** -24
    if M > 2 and dtype == F32:
        top = torch.nn.functional.pad(x.abs(), (0, -K % 128)).view(M, -1, 128).amax(-1)
        tol += top.repeat_interleave(128, 1)[:, :K] @ (q.abs() * d).T * 2.0 ** -22
    assert ((got - want).abs() <= tol).all(), float(((got - want).abs() - tol).max())
