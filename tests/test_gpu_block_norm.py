"""The block norm on the GPU, against the FP64 oracle.

Tolerances, from the roundings: a row's sum of squares goes through at most 44 FP32 adds
(a thread's 32 elements, ten shuffles, the mean and eps), so rsqrt of it is off by at most
22 + 4 units of 2^-24, taken as 2^-19; each product adds 2^-24.  h' is within
2^-19 |gate u| + 2^-23 (|a h| + |gate u|), x within 2^-17 of |x| + |r w| (|a h| + |gate u|);
then half a step of the output's type (bf16 2^-8, fp32 2^-24 relative).
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


HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def case(M, D, h_type=torch.bfloat16, w_type=torch.bfloat16, post=True, gate=0, pre=True, seed=0):
    g = torch.Generator().manual_seed(seed + M + D)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(y=(r(M, D) * 3).to(torch.bfloat16).cuda(), h=(r(M, D) * 5).to(h_type).cuda(),
                post_weight=(1 + 0.2 * r(D)).to(w_type).cuda() if post else None,
                gate=r(gate, D).to(w_type).cuda() if gate else None,
                pre_weight=(1 + 0.2 * r(D)).to(w_type).cuda() if pre else None)


def verify(c, got, quant=False, **kw):
    y, h, g = f64(c["y"]), f64(c["h"]), f64(c["gate"])
    h2, x = fp8.block_norm(y, h, f64(c["post_weight"]), g, pre_weight=f64(c["pre_weight"]), **kw)
    a = kw.get("res_scale", 1.0)
    ah = np.zeros_like(h2) if h is None else np.abs(a * h)
    gu = np.abs(h2 - (0 if h is None else a * h))
    h_out = got if x is None else got[0]
    assert np.all(np.abs(f64(h_out) - h2) <= (2.0 ** -19 + 2.0 ** -23) * gu + 2.0 ** -23 * ah
                  + HALF[h_out.dtype] * np.abs(h2) * (1 + 2.0 ** -10) + 1e-38)
    if x is None:
        return
    r = 1 / np.sqrt((h2 * h2).mean(axis=1, keepdims=True) + kw.get("eps", 1e-6))
    rw = r * np.abs(f64(c["pre_weight"]) + kw.get("offset", 0.0))
    tol = 2.0 ** -17 * (np.abs(x) + rw * (ah + gu))
    if not quant:
        assert np.all(np.abs(f64(got[1]) - x) <= tol + 2.0 ** -8 * np.abs(x) * (1 + 2.0 ** -10) + 1e-38)
        return
    codes, scales = got[1].view(torch.uint8).cpu().numpy(), got[2].cpu().numpy()
    kb = -(-x.shape[1] // 128)
    amax = np.stack([np.abs(x[:, b * 128:(b + 1) * 128]).max(axis=1) for b in range(kb)])
    top = np.stack([tol[:, b * 128:(b + 1) * 128].max(axis=1) for b in range(kb)])
    assert np.all(np.abs(scales - np.maximum(amax, 2.0 ** -100) / 448) <= (top + 2.0 ** -22 * amax) / 448 + 1e-40)
    back = fp8.dequant_rows(codes, scales)
    step = np.repeat(scales.T.astype(np.float64), 128, axis=1)[:, :x.shape[1]] * 2.0 ** -10
    assert np.all(np.abs(back - x) <= (2.0 ** -4 * np.abs(x) + step) * (1 + 2.0 ** -10) + 2 * tol)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("h_type,w_type", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                           (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("M,D", [(1, 16), (3, 128), (2, 1168), (5, 2048), (6, 2064), (1, 5120), (4, 8208), (2, 32768)])
def test_parity(nb, M, D, h_type, w_type, quant):
    c = case(M, D, h_type, w_type)
    verify(c, nb.block_norm(**c, res_scale=0.9, quant=quant), quant, res_scale=0.9)


def test_width_of_eight(nb):
    for D in (8, 1160):
        c = case(7, D, torch.float32, gate=7)
        verify(c, nb.block_norm(**c))


@pytest.mark.parametrize("post,gate,pre,no_y,no_h", [
    (False, 0, True, False, False), (True, 1, True, False, False), (True, 6, True, False, False),
    (False, 3, False, False, False), (True, 0, False, False, False), (False, 0, True, True, False),
    (True, 2, True, False, True), (False, 0, False, True, False)])
def test_optional_parts(nb, post, gate, pre, no_y, no_h):
    c = case(6, 400, post=post, gate=gate, pre=pre)
    if no_y:
        c["y"] = None
    if no_h:
        c["h"] = None
    verify(c, nb.block_norm(**c, res_scale=1.25, offset=1.0, eps=1e-3), res_scale=1.25, offset=1.0, eps=1e-3)


def test_one_gate_row_as_a_vector(nb):
    c = case(5, 256, gate=1)
    want = nb.block_norm(**c)
    c["gate"] = c["gate"][0]
    assert all(torch.equal(a, b) for a, b in zip(want, nb.block_norm(**c)))


def test_rows_in_place_strided_and_on_another_stream(nb):
    c = case(9, 528, torch.float32, gate=3)
    want = nb.block_norm(**c, quant=True)
    wide_y = torch.zeros((9, 1000), dtype=torch.bfloat16, device="cuda")
    wide_h = torch.full((9, 600), 3.0, device="cuda")
    wide_y[:, 8:536] = c["y"]
    wide_h[:, 16:544] = c["h"]
    c["y"], c["h"] = wide_y[:, 8:536], wide_h[:, 16:544]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = nb.block_norm(**c, out_h=c["h"], quant=True, stream=s)
    torch.cuda.synchronize()
    assert got[0].data_ptr() == c["h"].data_ptr()
    assert torch.equal(want[0], got[0]) and torch.equal(want[2], got[2])
    assert torch.equal(want[1].view(torch.uint8), got[1].view(torch.uint8))
    assert bool((wide_h[:, :16] == 3).all()) and bool((wide_h[:, 544:] == 3).all())


def test_zero_rows_nan_rows_and_infinities(nb):
    c = case(5, 272)
    for t in (c["y"], c["h"]):
        t[0] = 0
    c["y"][1, 3] = float("nan")
    c["h"][2, 200] = float("inf")
    h2, x = nb.block_norm(**c)
    _, codes, scales = nb.block_norm(**c, quant=True)
    assert bool((h2[0] == 0).all()) and bool((x[0] == 0).all())
    assert bool((codes.view(torch.uint8)[0] == 0).all()) and bool((scales[:, 0] > 0).all())
    assert bool(h2[1].isnan().all()) and bool(x[1].isnan().all()) and bool(scales[:, 1].isnan().all())
    assert bool(h2[2, 200].isinf()) and bool(x[2, 200].isnan())
    assert bool(x[3:].isfinite().all())


def test_empty_and_refusals(nb):
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    h2, x = nb.block_norm(e, e, pre_weight=w)
    assert h2.shape == x.shape == (0, 64)
    c = case(4, 64)
    for bad in (dict(gate=torch.ones((3, 64), device="cuda")), dict(pre_weight=w[:32]), dict(h=c["h"].half()),
                dict(h=c["h"][:2]), dict(y=c["y"].t()), dict(post_weight=w.float()), dict(pre_weight=None, quant=True),
                dict(y=None), dict(out_h=c["h"].float())):
        with pytest.raises(ValueError):
            nb.block_norm(**{**c, **bad})
    with pytest.raises(nb.BilocoError):
        nb.block_norm(c["y"][:, :60], c["h"][:, :60], pre_weight=w[:60])


def verify_on_gpu(c, got, quant, res_scale=1.0, offset=0.0, eps=1e-6):
    """verify() for many rows, in FP64 on the GPU; the same tolerances."""
    y, h, post, g, pre = (None if c[k] is None else c[k].double() for k in ("y", "h", "post_weight", "gate", "pre_weight"))
    M, D = (h if y is None else y).shape
    u = torch.zeros((M, D), dtype=torch.float64, device="cuda") if y is None else y
    if post is not None:
        u = u / ((u * u).mean(1, keepdim=True) + eps).sqrt() * (post + offset)
    if g is not None:
        u = u * g.repeat_interleave(M // g.shape[0], 0)
    ah = torch.zeros_like(u) if h is None else res_scale * h
    h2, gu = ah + u, u.abs()
    h_out = got if pre is None else got[0]
    assert bool(((h_out.double() - h2).abs() <= (2.0 ** -19 + 2.0 ** -23) * gu + 2.0 ** -23 * ah.abs()
                 + HALF[h_out.dtype] * h2.abs() * (1 + 2.0 ** -10) + 1e-38).all())
    if pre is None:
        return
    rw = (pre + offset).abs() / ((h2 * h2).mean(1, keepdim=True) + eps).sqrt()
    x = h2 / ((h2 * h2).mean(1, keepdim=True) + eps).sqrt() * (pre + offset)
    tol = 2.0 ** -17 * (x.abs() + rw * (ah.abs() + gu))
    if not quant:
        assert bool(((got[1].double() - x).abs() <= tol + 2.0 ** -8 * x.abs() * (1 + 2.0 ** -10) + 1e-38).all())
        return
    KB = -(-D // 128)
    pad = lambda t: torch.nn.functional.pad(t, (0, KB * 128 - D)).view(M, KB, 128)  # noqa: E731
    amax, top, scales = pad(x.abs()).amax(2), pad(tol).amax(2), got[2].double().t()
    assert bool(((scales - amax.clamp(min=2.0 ** -100) / 448).abs() <= (top + 2.0 ** -22 * amax) / 448 + 1e-40).all())
    s = scales.repeat_interleave(128, 1)[:, :D]
    assert bool(((got[1].double() * s - x).abs() <= (2.0 ** -4 * x.abs() + s * 2.0 ** -10) * (1 + 2.0 ** -10) + 2 * tol).all())


def same(a, b):
    a, b = ((t,) if torch.is_tensor(t) else t for t in (a, b))
    return all(torch.equal(u.view(torch.uint8), v.view(torch.uint8)) for u, v in zip(a, b))


# More rows than CTAs run at once, so that each walks over several: one piece a thread (D up to 1024), two
# (up to 8192), four (above); the last rows of the walk are fewer than the CTAs.
WALKS = [(3000, 512), (5000, 16), (2000, 1160), (3001, 5120), (1500, 8192), (700, 8208), (401, 16400)]


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("h_type,w_type", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32)])
@pytest.mark.parametrize("M,D", WALKS)
def test_walks_over_rows(nb, M, D, h_type, w_type, quant):
    if quant and D % 16:
        D += 8
    c = case(M, D, h_type, w_type)
    got = nb.block_norm(**c, res_scale=0.9, quant=quant)
    verify_on_gpu(c, got, quant, res_scale=0.9)
    for _ in range(20):
        assert same(got, nb.block_norm(**c, res_scale=0.9, quant=quant))


@pytest.mark.parametrize("post,gate,pre,no_y,no_h", [
    (False, 0, True, False, False), (True, 1, True, False, False), (True, 500, True, False, False),
    (False, 4, False, False, False), (True, 0, False, False, False), (False, 0, True, True, False),
    (True, 2, True, False, True), (False, 0, False, True, False), (False, 2000, True, False, False)])
@pytest.mark.parametrize("D", [528, 2064, 8208])
def test_walks_with_optional_parts(nb, D, post, gate, pre, no_y, no_h):
    """One sum a row, none, and two: the barriers between rows are different ones."""
    c = case(2000, D, torch.float32, post=post, gate=gate, pre=pre)
    if no_y:
        c["y"] = None
    if no_h:
        c["h"] = None
    kw = dict(res_scale=1.25, offset=1.0, eps=1e-3)
    for quant in ([False, True] if pre else [False]):
        got = nb.block_norm(**c, **kw, quant=quant)
        verify_on_gpu(c, got, quant, **kw)
        for _ in range(20):
            assert same(got, nb.block_norm(**c, **kw, quant=quant))


@pytest.mark.parametrize("h_type", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,D", [(3000, 512), (2000, 1168), (3001, 5120), (700, 8208)])
def test_walks_in_place_and_over_strided_rows(nb, M, D, h_type):
    """h' over h, whose next row is loaded while this one is written; the columns beside stay."""
    c = case(M, D, h_type, h_type, gate=1)
    want = nb.block_norm(**c, quant=True)
    wide_y = torch.zeros((M, D + 24), dtype=torch.bfloat16, device="cuda")
    wide_h = torch.full((M, D + 40), 3.0, dtype=h_type, device="cuda")
    wide_y[:, 8:8 + D] = c["y"]
    wide_h[:, 16:16 + D] = c["h"]
    c["y"], c["h"] = wide_y[:, 8:8 + D], wide_h[:, 16:16 + D]
    got = nb.block_norm(**c, out_h=c["h"], quant=True)
    assert got[0].data_ptr() == c["h"].data_ptr()
    assert torch.equal(got[0], want[0]) and same(got[1:], want[1:])
    assert bool((wide_h[:, :16] == 3).all()) and bool((wide_h[:, 16 + D:] == 3).all())


@pytest.mark.parametrize("D", [512, 2064, 8208])
def test_bad_rows_of_a_walk_spoil_only_themselves(nb, D):
    M = 2000
    c = case(M, D)
    clean, cc, cs = nb.block_norm(**c, quant=True)
    bad = torch.arange(0, M, 7, device="cuda")
    c["y"][bad, 3] = float("nan")
    h2, codes, scales = nb.block_norm(**c, quant=True)
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[bad] = False
    assert bool(h2[bad].isnan().all()) and bool(scales[:, bad].isnan().all())
    assert torch.equal(h2[keep], clean[keep]) and torch.equal(scales[:, keep], cs[:, keep])
    assert torch.equal(codes[keep].view(torch.uint8), cc[keep].view(torch.uint8))
