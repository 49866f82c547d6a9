"""The experts' layer on the GPU, against the FP64 oracle.

Tolerance, from the number of roundings.  A sum over K: a block is eight MMA steps of 16
products (17 terms cut to the largest: 17 units of 2^-23 of the sum of magnitudes each), then
KB scaled blocks and the joins over warps and CTAs: (136 + KB + 80) 2^-23 of the sum of
magnitudes.  That bounds the gate and the up sums, dg and du; the hidden value is then off by
at most 1.1 |u| dg + |silu(g)| du + 2^-20 |h| (1.1 bounds silu's slope), and by 2^-11 |h| for its FP16
rounding (2^-25 of its strip's largest where that is more).  The down sum adds its own
(136 + KB + 80) 2^-23 of the magnitudes, BF16 half a step, 2^-8 |y|.

At the bottom of the range there are absolute limits.  The exponent that FP16 values are
stored relative to is at least -112, and FP16's smallest step is 2^-24, so a hidden value is
kept to 2^-137; below 2^-126, FP32 steps are 2^-149 (gate, up and their product: three of
them, inside the 2^-137 as well) and a BF16 output's 2^-133, half of which is 2^-134.
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


def layer(nb, T, D, F, E, shared=0, router_dtype=torch.bfloat16, bias=False, seed=0):
    g = torch.Generator().manual_seed(seed + 1000 * T + D + F + E)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = r(T, D)
    x[:, torch.randperm(D, generator=g)[:max(1, D // 100)]] *= 20
    n = E + shared
    w13, s13 = nb.fp8_pack_weight((r(n, 2 * F, D) * 0.05).cuda())
    w2, s2 = nb.fp8_pack_weight((r(n, D, F) * 0.05).cuda())
    return dict(x=x.to(torch.bfloat16).cuda(), router=(r(E, D) * 0.05).to(router_dtype).cuda(), w13=w13,
                w13_scales=s13, w2=w2, w2_scales=s2), (0.1 * r(E)).cuda() if bias else None


def dequant(c, s):
    return np.stack([fp8.dequant_tiles(c[e].view(torch.uint8).cpu().numpy(), s[e].cpu().numpy())
                     for e in range(c.shape[0])])


def verify(p, k, got, bias=None, score="softmax", renorm=True, route_scale=1.0):
    y, ids, w = got
    x, router = p["x"].double().cpu().numpy(), p["router"].double().cpu().numpy()
    E, n = router.shape[0], p["w13"].shape[0]
    b = None if bias is None else bias.double().cpu().numpy()
    rid, rw = fp8.route(x, router, k, score, b, renorm, route_scale)
    assert np.array_equal(ids.cpu().numpy(), rid)
    assert np.all(np.abs(w.double().cpu().numpy() - rw) <= 2.0 ** -20 * np.abs(rw) + 1e-30)
    W13, W2 = dequant(p["w13"], p["w13_scales"]), dequant(p["w2"], p["w2_scales"])
    F, D = W13.shape[1] // 2, x.shape[1]
    c1 = (136 + -(-D // 128) + 80) * 2.0 ** -23
    c2 = (136 + -(-F // 128) + 80) * 2.0 ** -23
    want = fp8.moe(x, rid, rw, W13, W2, n - E)
    tol = np.zeros_like(want)
    for t in range(x.shape[0]):
        for e, we in list(zip(rid[t], rw[t])) + [(e, 1.0) for e in range(E, n)]:
            a, ax = W13[e] @ x[t], np.abs(W13[e]) @ np.abs(x[t])
            g, u = a[:F], a[F:]
            sg = g / (1 + np.exp(-g))
            h = sg * u
            dh = 1.1 * np.abs(u) * c1 * ax[:F] + np.abs(sg) * c1 * ax[F:] + (2.0 ** -20 + 2.0 ** -11) * np.abs(h)
            dh += 2.0 ** -25 * np.repeat(np.abs(h).reshape(-1, 16).max(1), 16) + 2.0 ** -38 * np.abs(h).max()
            tol[t] += np.abs(we) * (np.abs(W2[e]) @ (dh + c2 * np.abs(h) + 2.0 ** -137))
    err = np.abs(y.double().cpu().numpy() - want)
    bad = err > tol * (1 + 2.0 ** -7) + 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -7) + 2.0 ** -133
    assert not bad.any(), f"{bad.sum()} of {bad.size}, first {np.argwhere(bad)[:3].tolist()}, worst {err.max()}"


@pytest.mark.parametrize("T,D,F,E,k,shared", [
    (1, 16, 16, 1, 1, 0), (1, 128, 64, 4, 2, 0), (2, 144, 48, 5, 3, 1), (3, 272, 272, 8, 2, 0), (1, 2048, 256, 16, 8, 1),
    (5, 400, 144, 33, 6, 2), (16, 512, 128, 8, 2, 0), (17, 256, 192, 8, 8, 0), (33, 160, 80, 3, 1, 1),
    (64, 336, 112, 6, 2, 4), (64, 128, 256, 64, 16, 0), (4, 1040, 1024, 2, 2, 0)])
def test_parity(nb, T, D, F, E, k, shared):
    p, _ = layer(nb, T, D, F, E, shared)
    verify(p, k, nb.fp8_moe(**p, top_k=k))


@pytest.mark.parametrize("T", [1, 20])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_scores(nb, T, score, bias, renorm):
    p, b = layer(nb, T, 256, 64, 40, bias=bias, router_dtype=torch.float32 if renorm else torch.bfloat16)
    kw = dict(score=score, bias=b, renorm=renorm, route_scale=2.5)
    verify(p, 6, nb.fp8_moe(**p, top_k=6, **kw), **kw)


def test_many_experts(nb):
    p, _ = layer(nb, 7, 64, 16, 512)
    verify(p, 16, nb.fp8_moe(**p, top_k=16))


def test_ties_take_the_lowest_index(nb):
    p, _ = layer(nb, 3, 64, 32, 6)
    p["router"][:] = p["router"][0]
    _, ids, w = nb.fp8_moe(**p, top_k=4)
    assert ids.tolist() == [[0, 1, 2, 3]] * 3 and bool((w == 0.25).all())


def test_all_tokens_on_one_expert(nb):
    """More than 16 tokens of an expert: several passes over its weights."""
    p, _ = layer(nb, 64, 128, 64, 4)
    p["x"] = p["x"].abs()
    p["router"][:] = -1
    p["router"][2] = 1
    got = nb.fp8_moe(**p, top_k=1)
    assert bool((got[1] == 2).all())
    verify(p, 1, got)


def test_tokens_of_an_expert_in_several_units(nb):
    """17 to 64 tokens of an expert are served by different CTAs, which all have to deal them out alike:
    no token missed or taken twice, and every call the same to the bit."""
    p, _ = layer(nb, 64, 512, 256, 8, shared=1, seed=7)
    got = nb.fp8_moe(**p, top_k=4)
    counts = torch.bincount(got[1].flatten().long(), minlength=8)
    assert int(counts.max()) > 32 and int(counts.min()) > 8
    verify(p, 4, got)
    for _ in range(50):
        again = nb.fp8_moe(**p, top_k=4)
    assert all(torch.equal(u, v) for u, v in zip(got, again))


def test_scales_of_the_operands(nb):
    """Rows of x far from 1, tiny and huge weights: the FP16 scaling must not overflow or vanish."""
    p, _ = layer(nb, 6, 128, 64, 3)
    p["x"] = (p["x"].float() * torch.tensor([1e-20, 1e-6, 1.0, 1e6, 0.0, 30.0], device="cuda")[:, None]).to(torch.bfloat16)
    p["w13_scales"] *= 0.01
    p["w2_scales"] *= 100.0
    p["router"] *= 1e-5
    verify(p, 2, nb.fp8_moe(**p, top_k=2))
    assert bool((nb.fp8_moe(**p, top_k=2)[0][4] == 0).all())


@pytest.mark.parametrize("T", [1, 20])
def test_hidden_values_up_to_the_largest_float(nb, T):
    """Gate and up of about 2^63 each: hidden values from 2^126 to 2^127.8 stay in the sum, and an
    infinite one spoils its own token only."""
    D = F = 128
    rng = np.random.default_rng(T)
    p, _ = layer(nb, T, D, F, 3)
    codes = rng.integers(0x38, 0x40, (3, 2 * F, D)).astype(np.uint8)               # 1 to 1.875
    codes[:, F:] |= rng.integers(0, 2, (3, F, D)).astype(np.uint8) << 7
    p["w13"] = torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn)
    p["w13_scales"] = torch.full((3, 2, 1), 2.0 ** 63, device="cuda")
    p["w2_scales"] = p["w2_scales"] * 2.0 ** -110
    x = torch.zeros((T, D))
    x[torch.arange(T), torch.from_numpy(rng.permutation(D)[:T])] = torch.tensor([1.0, 0.5, 2.0 ** -50, 1.0])[torch.arange(T) % 4]
    p["x"] = x.to(torch.bfloat16).cuda()
    got = nb.fp8_moe(**p, top_k=2)
    W = dequant(p["w13"], p["w13_scales"])[got[1][0, 0].item()] @ x[0].double().numpy()
    assert (np.abs(W[:F] * W[F:]) >= 2.0 ** 127).sum() > 20                        # the case is what it says
    verify(p, 2, got)
    if T > 1:
        p["x"][3] *= 4
        y = nb.fp8_moe(**p, top_k=2)[0]
        keep = [t for t in range(T) if t != 3]
        assert torch.equal(y[keep], got[0][keep]) and not bool(y[3].isfinite().all())


def test_a_bad_token_spoils_only_its_row(nb):
    p, _ = layer(nb, 20, 144, 48, 4)
    clean, ids, _ = nb.fp8_moe(**p, top_k=2)
    p["x"][3, 7] = float("nan")
    p["x"][5, 140] = float("inf")
    y, ids2, w = nb.fp8_moe(**p, top_k=2)
    keep = [t for t in range(20) if t not in (3, 5)]
    assert torch.equal(y[keep], clean[keep]) and torch.equal(ids[keep], ids2[keep])
    assert not bool(y[3].isfinite().any()) and not bool(y[5].isfinite().all())
    assert bool(((ids2 >= 0) & (ids2 < 4)).all()) and bool((ids2[:, 0] != ids2[:, 1]).all())


def test_strided_rows_streams_and_graphs(nb):
    p, _ = layer(nb, 9, 272, 80, 8, 1)
    q, _ = layer(nb, 9, 272, 80, 8, 1, seed=5)
    want, other = nb.fp8_moe(**p, top_k=3), nb.fp8_moe(**q, top_k=3)
    wide = torch.zeros((9, 320), dtype=torch.bfloat16, device="cuda")
    wide[:, 16:288] = p["x"]
    assert all(torch.equal(a, b) for a, b in zip(want, nb.fp8_moe(**{**p, "x": wide[:, 16:288]}, top_k=3)))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        a, b = nb.fp8_moe(**p, top_k=3, stream=s1), nb.fp8_moe(**q, top_k=3, stream=s2)
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(want, a)) and all(torch.equal(u, v) for u, v in zip(other, b))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = nb.fp8_moe(**p, top_k=3)
        graphs.append((g, out))
    p["x"].copy_(q["x"])
    want = nb.fp8_moe(**p, top_k=3)
    torch.cuda.synchronize()
    for (g, _), s in zip(graphs, (s1, s2)):
        with torch.cuda.stream(s):
            g.replay()
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for _, o in graphs for u, v in zip(want, o))


@pytest.mark.parametrize("T,k,shared", [(1, 3, 1), (40, 3, 1), (1, 8, 1)])
def test_two_streams_and_two_graphs_at_once(nb, T, k, shared):
    """One token (clusters of its experts, with and without the combine kernel) and units of 16."""
    p, _ = layer(nb, T, 272, 80, 8, shared)
    q, _ = layer(nb, T, 272, 80, 8, shared, seed=5)
    want, other = nb.fp8_moe(**p, top_k=k), nb.fp8_moe(**q, top_k=k)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(50):
        a, b = nb.fp8_moe(**p, top_k=k, stream=s1), nb.fp8_moe(**q, top_k=k, stream=s2)
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(want, a)) and all(torch.equal(u, v) for u, v in zip(other, b))
    graphs = []
    for w in (p, q):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = nb.fp8_moe(**w, top_k=k)
        graphs.append((g, out))
    for _ in range(20):
        for (g, _), s in zip(graphs, (s1, s2)):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (_, out), w in zip(graphs, (want, other)):
        assert all(torch.equal(u, v) for u, v in zip(out, w))


@pytest.mark.parametrize("T", [1, 20])
def test_operands_written_just_before_the_layer(nb, T):
    """router and w2 are read early; PyTorch's kernels and the packer right in front come first all the same."""
    layers = [layer(nb, T, 512, 256, 16, seed=s)[0] for s in range(3)]
    g = torch.Generator(device="cuda").manual_seed(1)
    raw = [torch.randn((16, 512, 256), generator=g, device="cuda") for _ in layers]
    want = []
    for p, r in zip(layers, raw):
        p["w2"], p["w2_scales"] = nb.fp8_pack_weight(r)
        torch.cuda.synchronize()
        want.append(nb.fp8_moe(**p, top_k=4))
        torch.cuda.synchronize()
    q = {k: v.clone() for k, v in layers[0].items()}
    for i in range(150):
        j = i % 3
        for k in ("x", "w13", "w13_scales", "w2", "w2_scales", "router"):
            q[k].copy_(layers[j][k])
        assert all(torch.equal(a, b) for a, b in zip(want[j], nb.fp8_moe(**q, top_k=4)))
    del q["w2"], q["w2_scales"]
    for i in range(150):                     # the same memory for every packed weight
        j = i % 3
        for k in ("x", "w13", "w13_scales", "router"):
            q[k].copy_(layers[j][k])
        w2, s2 = nb.fp8_pack_weight(raw[j])
        got = nb.fp8_moe(**q, w2=w2, w2_scales=s2, top_k=4)
        assert all(torch.equal(a, b) for a, b in zip(want[j], got))


@pytest.mark.parametrize("T", [1, 33])
def test_a_bias_of_minus_infinity_leaves_an_expert_out(nb, T):
    """Masked experts are picked only where nothing else is left, and then the lowest first."""
    p, _ = layer(nb, T, 128, 64, 40)
    b = torch.full((40,), float("-inf"), device="cuda")
    b[[7, 31]] = torch.tensor([0.25, -3.0], device="cuda")
    for score in ("softmax", "sigmoid"):
        got = nb.fp8_moe(**p, top_k=4, bias=b, score=score)
        assert got[1].tolist() == [[7, 31, 0, 1]] * T
        verify(p, 4, got, bias=b, score=score)


@pytest.mark.parametrize("T", [1, 17])
def test_the_largest_sizes(nb, T):
    """D and F at their limit; the formula and the tolerance in FP64 on the GPU."""
    D = F = 16384
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn((T, D), generator=g, device="cuda").to(torch.bfloat16)
    router = (torch.randn((2, D), generator=g, device="cuda") * 0.05).to(torch.bfloat16)
    w13, s13 = nb.fp8_pack_weight((torch.randn((2, 2 * F, D), generator=g, device="cuda") * 0.02).to(torch.bfloat16))
    w2, s2 = nb.fp8_pack_weight((torch.randn((2, D, F), generator=g, device="cuda") * 0.02).to(torch.bfloat16))
    y, ids, w = nb.fp8_moe(x, router, w13, s13, w2, s2, 1)
    assert torch.equal(ids[:, 0].long(), (x.double() @ router.double().t()).argmax(1)) and bool((w == 1).all())

    def wide(c, s):
        return c.double() * s.double().repeat_interleave(128, 0).repeat_interleave(128, 1)

    c = (136 + 128 + 80) * 2.0 ** -23
    for e in range(2):
        t = (ids[:, 0] == e).nonzero()[:, 0]
        if len(t) == 0:
            continue
        W, xe = wide(w13[e], s13[e]), x[t].double()
        a, ax = xe @ W.t(), xe.abs() @ W.abs().t()
        del W
        sg, u = torch.nn.functional.silu(a[:, :F]), a[:, F:]
        h = sg * u
        dh = 1.1 * u.abs() * c * ax[:, :F] + sg.abs() * c * ax[:, F:] + (2.0 ** -20 + 2.0 ** -11) * h.abs()
        dh += 2.0 ** -25 * h.abs().view(len(t), -1, 16).amax(2).repeat_interleave(16, 1) + 2.0 ** -38 * h.abs().max()
        V = wide(w2[e], s2[e])
        want, tol = h @ V.t(), (dh + c * h.abs()) @ V.abs().t()
        assert bool(((y[t].double() - want).abs() <= (tol + 2.0 ** -8 * want.abs()) * (1 + 2.0 ** -7)).all())


def test_empty_and_refusals(nb):
    p, _ = layer(nb, 2, 64, 32, 4)
    y, ids, w = nb.fp8_moe(**{**p, "x": p["x"][:0]}, top_k=2)
    assert y.shape == (0, 64) and ids.shape == (0, 2)
    for bad in (dict(top_k=0), dict(top_k=5), dict(score="relu"), dict(x=p["x"].float()), dict(w2=p["w2"][:3]),
                dict(w13_scales=p["w13_scales"][:, :0]), dict(router=p["router"][:, :32]), dict(x=p["x"].t()),
                dict(bias=torch.zeros(3, device="cuda")), dict(router=torch.zeros((6, 64), device="cuda"))):
        with pytest.raises(ValueError):
            nb.fp8_moe(**{**p, "top_k": 2, **bad})
    with pytest.raises(nb.BilocoError):
        nb.fp8_moe(**{**p, "x": torch.zeros((65, 64), dtype=torch.bfloat16, device="cuda")}, top_k=2)
