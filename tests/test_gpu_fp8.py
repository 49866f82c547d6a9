"""FP8 quantisers and the FP8 product on the GPU, against the FP64 oracle.

Tolerance of the product, from the number of roundings: a block's sum is four MMA steps
of 32 products added to an FP32 accumulator.  Aligning 33 terms to the largest and
cutting them loses at most 33 units of 2^-23 of the largest partial, which the sum of the
magnitudes S_b bounds; four steps: 132 * 2^-23 S_b.  Scaling and adding KB blocks rounds
at most 2 KB + 2 times by 2^-24 of S.  Hence |err| <= (132 + KB + 1) 2^-23 S, plus half a
BF16 step (2^-8 |y|) where y is BF16.
"""

import numpy as np
import pytest
import torch

from oracle import fp8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nb():
    import nvfp4_binary_rank_b200 as nb
    nb.load()
    return nb


def bits(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16).cuda()


def activation(rng, M, K):
    x = rng.standard_normal((M, K)).astype(np.float32)
    x[:, rng.choice(K, max(1, K // 100), replace=False)] *= 20
    return bf16(x)


def tolerance(y, S, K, dtype):
    KB = -(-K // 128)
    return (133 + KB) * 2.0 ** -23 * S + (2.0 ** -8 * np.abs(y) if dtype == torch.bfloat16 else 0.0) + 1e-300


def operands(nb, rng, M, N, K):
    x = activation(rng, M, K)
    w = torch.from_numpy((rng.standard_normal((N, K)) * 0.02).astype(np.float32)).cuda()
    return (*nb.fp8_quant_act(x), *nb.fp8_pack_weight(w))


def check(nb, xc, xs, wc, ws, y):
    want, S = fp8.gemm(bits(xc), xs.cpu().numpy(), bits(wc), ws.cpu().numpy())
    got = y.double().cpu().numpy()
    err = np.abs(got - want)
    bad = err > tolerance(want, S, xc.shape[1], y.dtype)
    assert not bad.any(), f"{bad.sum()} of {bad.size}, first {np.argwhere(bad)[:3].tolist()}, worst {err.max()}"
    assert nb.last_error() == 0


# ---- quantisers: bit-exact

@pytest.mark.parametrize("M,K", [(1, 16), (1, 128), (3, 144), (5, 512), (7, 528), (33, 2064), (1, 13824)])
def test_quant_act_bits(nb, M, K):
    x = activation(np.random.default_rng(M * K), M, K)
    c, s = nb.fp8_quant_act(x)
    wc, ws = fp8.quant_rows(x.float().cpu().numpy())
    assert s.shape == ws.shape and np.array_equal(s.cpu().numpy(), ws)
    assert np.array_equal(bits(c), wc)


def test_quant_act_special_values(nb):
    x = np.zeros((6, 256), np.float32)
    x[0, :] = 2.0 ** -126                       # below the smallest maximum the scale follows
    x[1, 5], x[1, 140] = np.nan, 3.0            # NaN stays in its block
    x[2, 7], x[2, 9] = np.inf, 1.0
    x[3, :] = 3.3e38
    x[4, :] = -0.0
    x[5, :] = np.float32(448) * 2.0 ** np.arange(-127, 129).clip(-100, 100)
    t = bf16(x)
    c, s = nb.fp8_quant_act(t)
    with np.errstate(invalid="ignore", over="ignore"):
        wc, ws = fp8.quant_rows(t.float().cpu().numpy())
    c, s = bits(c), s.cpu().numpy()
    assert np.array_equal(s, ws, equal_nan=True)
    nan = np.isnan(fp8.decode(wc))
    assert np.array_equal(nan, np.isnan(fp8.decode(c))) and np.array_equal(c[~nan], wc[~nan])
    assert nan[1, :128].all() and not nan[1, 128:].any() and nan[2, 7] and not nan[2, 128:].any()


def test_quant_act_strided_rows(nb):
    wide = activation(np.random.default_rng(5), 9, 400)
    x = wide[:, 64:64 + 272]
    c, s = nb.fp8_quant_act(x)
    c2, s2 = nb.fp8_quant_act(x.contiguous())
    assert torch.equal(c.view(torch.uint8), c2.view(torch.uint8)) and torch.equal(s, s2)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,K", [(1, 16), (128, 128), (100, 144), (257, 400)])
def test_pack_weight_bits(nb, N, K, dtype):
    rng = np.random.default_rng(N + K)
    w = torch.from_numpy(rng.standard_normal((2, N, K)).astype(np.float32)).to(dtype).cuda()
    c, s = nb.fp8_pack_weight(w)
    for e in range(2):
        wc, ws = fp8.quant_tiles(w[e].float().cpu().numpy())
        assert np.array_equal(s[e].cpu().numpy(), ws) and np.array_equal(bits(c[e]), wc)
    c1, s1 = nb.fp8_pack_weight(w[1].contiguous())
    assert torch.equal(c1.view(torch.uint8), c[1].view(torch.uint8)) and torch.equal(s1, s[1])


# ---- the product

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 16), (1, 128, 128), (2, 7, 48), (5, 130, 400), (16, 256, 1040), (17, 100, 256), (32, 384, 512),
    (33, 129, 2064), (64, 128, 640), (65, 250, 144), (100, 1000, 272), (128, 128, 1024), (129, 16, 16),
    (130, 255, 144), (200, 513, 528), (256, 256, 256), (333, 1000, 2064), (1, 1000, 5120), (16, 640, 13824)])
def test_gemm_parity(nb, M, N, K, dtype):
    xc, xs, wc, ws = operands(nb, np.random.default_rng(M + 7 * N + K), M, N, K)
    y = nb.fp8_gemm(xc, xs, wc, ws, out_dtype=dtype)
    assert y.shape == (M, N) and y.dtype == dtype
    check(nb, xc, xs, wc, ws, y)


@pytest.mark.parametrize("M,N,K", [(1, 5120, 5120), (16, 13824, 1024), (100, 5120, 1024), (700, 2600, 1040),
                                   (2048, 5120, 512)])
def test_gemm_parity_many_tiles(nb, M, N, K):
    """More tiles than SMs, several tiles per CTA: against an FP64 product on the GPU."""
    xc, xs, wc, ws = operands(nb, np.random.default_rng(11), M, N, K)
    y = nb.fp8_gemm(xc, xs, wc, ws, out_dtype=torch.float32).double()
    x = xc.double() * xs.t().repeat_interleave(128, 1)[:, :K].double()
    w = wc.double() * ws.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K].double()
    S = x.abs() @ w.abs().t()
    assert bool(((y - x @ w.t()).abs() <= (133 + -(-K // 128)) * 2.0 ** -23 * S).all())
    assert nb.last_error() == 0


@pytest.mark.parametrize("M", [1, 40, 300])
def test_gemm_one_hot_rows_are_exact(nb, M):
    """y[m, n] = one product: every code, scale and position has to be the right one."""
    N, K = 300, 656
    rng = np.random.default_rng(M)
    codes = rng.integers(0, 0x7F, (N, K)).astype(np.uint8) | (rng.integers(0, 2, (N, K)).astype(np.uint8) << 7)
    wc = torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn)
    ws = torch.from_numpy(2.0 ** rng.integers(-8, 8, (3, 6)).astype(np.float32)).cuda()
    at = rng.integers(0, K, M)
    xc = np.zeros((M, K), np.uint8)
    xc[np.arange(M), at] = 0x38                                     # 1.0
    xs = (2.0 ** rng.integers(-8, 8, (6, M))).astype(np.float32)
    y = nb.fp8_gemm(torch.from_numpy(xc).cuda().view(torch.float8_e4m3fn), torch.from_numpy(xs).cuda(), wc, ws,
                    out_dtype=torch.float32).cpu().numpy()
    w = fp8.dequant_tiles(codes, ws.cpu().numpy())
    assert np.array_equal(y, (w[:, at] * xs[at // 128, np.arange(M)]).T.astype(np.float32))


@pytest.mark.parametrize("M", [3, 40, 300])
def test_gemm_nan_and_inf_stay_in_their_rows(nb, M):
    N, K = 200, 272
    xc, xs, wc, ws = operands(nb, np.random.default_rng(3), M, N, K)
    clean = nb.fp8_gemm(xc, xs, wc, ws)
    xc.view(torch.uint8)[1, 130] = 0x7F
    xs[0, 2] = float("inf")
    wc.view(torch.uint8)[150, 7] = 0xFF
    y = nb.fp8_gemm(xc, xs, wc, ws)
    assert bool(y[1].isnan().all()) and bool(y[:, 150].isnan().all())
    assert not bool(y[2, :150].isfinite().any())
    keep = [m for m in range(M) if m not in (1, 2)]
    cols = [n for n in range(N) if n != 150]
    assert torch.equal(y[keep][:, cols], clean[keep][:, cols])


def test_gemm_rows_do_not_depend_on_the_batch_beside_them(nb):
    """Determinism, and no row of another call's scratch: the same call twice, with others between."""
    xc, xs, wc, ws = operands(nb, np.random.default_rng(4), 20, 512, 1040)
    a = nb.fp8_gemm(xc, xs, wc, ws)
    nb.fp8_gemm(*operands(nb, np.random.default_rng(5), 300, 700, 400))
    assert torch.equal(a, nb.fp8_gemm(xc, xs, wc, ws))


def test_gemm_many_calls_in_a_row(nb):
    """Thousands of launches back to back, of both forms and with K split and not: every block of
    every launch has to come to an end by itself, whatever runs before and after it."""
    sets = [operands(nb, np.random.default_rng(m), m, n, k) for m, n, k in ((333, 1000, 2064), (700, 640, 400), (3, 512, 1040))]
    want = [nb.fp8_gemm(*s) for s in sets]
    for i in range(3000):
        j = i % 3 if i % 100 < 50 else 0
        y = nb.fp8_gemm(*sets[j])
        if i % 500 == 0:
            assert torch.equal(y, want[j])
    assert torch.equal(y, want[j])
    assert nb.last_error() == 0


@pytest.mark.parametrize("M,N,K", [(129, 5120, 5120), (256, 5120, 5120), (257, 2048, 4096), (192, 5120, 13824),
                                   (130, 5200, 1040)])
def test_gemm_parts_of_k_in_the_rows_form_repeat_to_the_bit(nb, M, N, K):
    """The rows form with K split into parts of 3 to 36 blocks: the parts' sums take the place of the
    operands, which both halves of a tile's columns must have been multiplied from.  Against an FP64
    product, then the same bits in a thousand calls, alone and with another product under way."""
    xc, xs, wc, ws = operands(nb, np.random.default_rng(M + N + K), M, N, K)
    y = nb.fp8_gemm(xc, xs, wc, ws, out_dtype=torch.float32)
    x = xc.double() * xs.t().repeat_interleave(128, 1)[:, :K].double()
    w = wc.double() * ws.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K].double()
    S = x.abs() @ w.abs().t()
    assert bool(((y.double() - x @ w.t()).abs() <= (133 + -(-K // 128)) * 2.0 ** -23 * S).all())
    other, s = operands(nb, np.random.default_rng(1), 200, 1024, 2064), torch.cuda.Stream()
    torch.cuda.synchronize()
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(1000):
        if i % 2:
            nb.fp8_gemm(*other, stream=s)
        differ += (nb.fp8_gemm(xc, xs, wc, ws, out_dtype=torch.float32) != y).sum()
    assert int(differ) == 0
    assert nb.last_error() == 0


def test_gemm_out_argument_and_neighbours_untouched(nb):
    M, N, K = 5, 100, 144
    xc, xs, wc, ws = operands(nb, np.random.default_rng(6), M, N, K)
    for dtype in (torch.bfloat16, torch.float32):
        buf = torch.full((M * N + 2,), 7.0, dtype=dtype, device="cuda")
        out = buf[1:-1].view(M, N)                                 # not aligned to a vector store
        assert nb.fp8_gemm(xc, xs, wc, ws, out=out) is out
        assert torch.equal(out, nb.fp8_gemm(xc, xs, wc, ws, out_dtype=dtype))
        assert buf[0] == 7 and buf[-1] == 7


def test_empty_batch(nb):
    c, s = nb.fp8_quant_act(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"))
    wc, ws = nb.fp8_pack_weight(torch.ones((8, 64), device="cuda"))
    assert c.shape == (0, 64) and s.shape == (1, 0)
    assert nb.fp8_gemm(c, s, wc, ws).shape == (0, 8)


def test_gemm_binding_refusals(nb):
    xc, xs, wc, ws = operands(nb, np.random.default_rng(7), 4, 128, 256)
    for args in ((xc.t(), xs, wc, ws), (xc, xs.t(), wc, ws), (xc, xs, wc[:, :128], ws), (xc, xs, wc, ws[:, :1]),
                 (xc.view(torch.uint8), xs, wc, ws), (xc, xs.half(), wc, ws), (xc[0], xs, wc, ws)):
        with pytest.raises(ValueError):
            nb.fp8_gemm(*args)
    with pytest.raises(ValueError):
        nb.fp8_gemm(xc, xs, wc, ws, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        nb.fp8_gemm(xc, xs, wc, ws, out=torch.empty((4, 127), device="cuda"))
    with pytest.raises(nb.BilocoError):
        nb.fp8_quant_act(torch.zeros((2, 24), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        nb.fp8_quant_act(torch.zeros((32, 2), dtype=torch.bfloat16, device="cuda").t())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [
    (129, 2500, 144), (257, 1700, 528), (333, 1800, 2064), (512, 1288, 272), (700, 1100, 400), (128, 2368, 144),
    (129, 128, 2064), (300, 600, 272), (64, 200, 1040), (96, 130, 4096), (1000, 64, 256), (2048, 130, 384), (48, 5120, 256)])
def test_gemm_parity_between_the_forms(nb, M, N, K, dtype):
    """Few and many tiles above 128 tokens, and tiles of fewer columns than there are tokens."""
    xc, xs, wc, ws = operands(nb, np.random.default_rng(M + 7 * N + K), M, N, K)
    check(nb, xc, xs, wc, ws, nb.fp8_gemm(xc, xs, wc, ws, out_dtype=dtype))


@pytest.mark.parametrize("M,N,K", [(100, 20000, 128), (70, 30000, 144), (128, 40000, 64), (33, 24000, 256)])
def test_gemm_walks_over_small_tiles(nb, M, N, K):
    """Short sums over many weight rows: more tiles of few columns than run at once."""
    xc, xs, wc, ws = operands(nb, np.random.default_rng(N), M, N, K)
    y = nb.fp8_gemm(xc, xs, wc, ws, out_dtype=torch.float32).double()
    x = xc.double() * xs.t().repeat_interleave(128, 1)[:, :K].double()
    w = wc.double() * ws.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K].double()
    S = x.abs() @ w.abs().t()
    assert bool(((y - x @ w.t()).abs() <= (133 + -(-K // 128)) * 2.0 ** -23 * S).all())
    assert nb.last_error() == 0


@pytest.mark.parametrize("M,N", [(300, 2000), (130, 500), (70, 130)])
def test_gemm_one_hot_rows_are_exact_in_wide_products(nb, M, N):
    K = 656
    rng = np.random.default_rng(M + N)
    codes = rng.integers(0, 0x7F, (N, K)).astype(np.uint8) | (rng.integers(0, 2, (N, K)).astype(np.uint8) << 7)
    ws = 2.0 ** rng.integers(-8, 8, (-(-N // 128), 6)).astype(np.float32)
    at = rng.integers(0, K, M)
    xc = np.zeros((M, K), np.uint8)
    xc[np.arange(M), at] = 0x38                                     # 1.0
    xs = (2.0 ** rng.integers(-8, 8, (6, M))).astype(np.float32)
    xg, wg = (torch.from_numpy(c).cuda().view(torch.float8_e4m3fn) for c in (xc, codes))
    y = nb.fp8_gemm(xg, torch.from_numpy(xs).cuda(), wg, torch.from_numpy(ws).cuda(), out_dtype=torch.float32).cpu().numpy()
    assert np.array_equal(y, (fp8.dequant_tiles(codes, ws)[:, at] * xs[at // 128, np.arange(M)]).T.astype(np.float32))


def test_gemm_nan_and_inf_stay_in_their_rows_among_many_tiles(nb):
    M, N, K = 300, 1800, 272
    xc, xs, wc, ws = operands(nb, np.random.default_rng(3), M, N, K)
    clean = nb.fp8_gemm(xc, xs, wc, ws)
    xc.view(torch.uint8)[1, 130] = 0x7F
    xs[0, 200] = float("inf")
    wc.view(torch.uint8)[1150, 7] = 0xFF
    y = nb.fp8_gemm(xc, xs, wc, ws)
    assert bool(y[1].isnan().all()) and bool(y[:, 1150].isnan().all()) and not bool(y[200].isfinite().any())
    keep = [m for m in range(M) if m not in (1, 200)]
    cols = [n for n in range(N) if n != 1150]
    assert torch.equal(y[keep][:, cols], clean[keep][:, cols])


def test_gemm_many_calls_of_both_forms_in_a_row(nb):
    sets = [operands(nb, np.random.default_rng(m), m, n, k)
            for m, n, k in ((333, 1800, 2064), (700, 1100, 400), (333, 1000, 2064), (70, 512, 1040))]
    want = [nb.fp8_gemm(*s) for s in sets]
    for i in range(3000):
        j = i % 4 if i % 100 < 50 else 0
        y = nb.fp8_gemm(*sets[j])
        if i % 100 == 49:
            assert torch.equal(y, want[j])
    assert torch.equal(y, want[j])
    assert nb.last_error() == 0


@pytest.mark.parametrize("M", [1, 400])
def test_a_weight_packed_just_before_its_product(nb, M):
    """The product requests its weight early; a packer right in front of it has to come first all the same."""
    N, K = 2048, 2064
    x = nb.fp8_quant_act(activation(np.random.default_rng(13), M, K))
    ws = [torch.randn((N, K), generator=torch.Generator().manual_seed(i)).cuda() for i in range(3)]
    want = []
    for w in ws:
        packed = nb.fp8_pack_weight(w)
        torch.cuda.synchronize()
        want.append(nb.fp8_gemm(*x, *packed))
        torch.cuda.synchronize()
    del packed
    for i in range(150):                     # the same memory for every packed weight
        assert torch.equal(nb.fp8_gemm(*x, *nb.fp8_pack_weight(ws[i % 3])), want[i % 3])


@pytest.mark.parametrize("M", [1, 50, 400])
def test_a_weight_copied_just_before_its_product(nb, M):
    N, K = 1024, 1040
    sets = [operands(nb, np.random.default_rng(20 + i), M, N, K) for i in range(3)]
    want = [nb.fp8_gemm(*s) for s in sets]
    mine = [t.clone() for t in sets[0]]
    for i in range(150):
        for k in (0, 1, 3, 2):
            mine[k].copy_(sets[i % 3][k])
        assert torch.equal(nb.fp8_gemm(*mine), want[i % 3])


@pytest.mark.parametrize("M", [1, 50, 400])
def test_streams_and_graphs(nb, M):
    """Two calls at once on two streams, and a captured quantise + product replayed on new inputs."""
    N, K = 1024, 1040
    a = operands(nb, np.random.default_rng(8), M, N, K)
    b = operands(nb, np.random.default_rng(9), M, N, K)
    ya, yb = nb.fp8_gemm(*a), nb.fp8_gemm(*b)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        za, zb = nb.fp8_gemm(*a, stream=s1), nb.fp8_gemm(*b, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(ya, za) and torch.equal(yb, zb)

    x = activation(np.random.default_rng(10), M, K)
    x2 = activation(np.random.default_rng(12), M, K)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = nb.fp8_gemm(*nb.fp8_quant_act(x), *a[2:])
        graphs.append((g, out))
    x.copy_(x2)
    torch.cuda.synchronize()
    for (g, _), s in zip(graphs, (s1, s2)):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    want = nb.fp8_gemm(*nb.fp8_quant_act(x2), *a[2:])
    assert all(torch.equal(o, want) for _, o in graphs)
    assert nb.last_error() == 0
