"""The FP8 operators together, as a decode step and a prompt use them, and in the situations a
serving program puts them in: captured on first use, far offsets, a layer replayed."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import fp8

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def nb():
    import nvfp4_binary_rank_b200 as nb
    nb.load()
    return nb


class Layer:
    """One block of a model that holds its projections in FP8 and its experts' MLP in FP8, and
    one projection in NVFP4 with a sign correction."""

    def __init__(self, nb, D=512, F=256, E=8, r=32, seed=0):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.D, self.nb = D, nb
        self.norms = [(1 + 0.1 * rnd(D)).to(torch.bfloat16).cuda() for _ in range(4)]
        self.proj = nb.fp8_pack_weight((rnd(D, D) * 0.04).cuda())
        self.W, self.Wsf, self.gs = nb.pack_weight((rnd(D, D) * 0.04).cuda())
        self.Ub, self.Vb = nb.pack_signs(rnd(D, r).sign().cuda()), nb.pack_signs(rnd(r, D).sign().cuda())
        self.alpha = (0.01 * rnd(r).abs()).cuda()
        self.router = (rnd(E, D) * 0.05).to(torch.bfloat16).cuda()
        self.w13 = nb.fp8_pack_weight((rnd(E, 2 * F, D) * 0.04).cuda())
        self.w2 = nb.fp8_pack_weight((rnd(E, D, F) * 0.04).cuda())

    def run(self, y, h, gemm=None):
        """(h', next block's input): norm -> FP8 product -> norm -> NVFP4 product -> norm -> experts -> norm."""
        nb, n = self.nb, self.norms
        h, c, s = nb.block_norm(y, h, post_weight=n[0], pre_weight=n[1], quant=True)
        y = nb.fp8_gemm(c, s, *self.proj)
        h, x = nb.block_norm(y, h, pre_weight=n[2], res_scale=0.9)
        y = (gemm or nb.gemm)(x, self.W, self.Wsf, self.gs, self.Ub, self.Vb, self.alpha)
        h, x = nb.block_norm(y, h, post_weight=n[3], pre_weight=n[0])
        y, ids, w = nb.fp8_moe(x, self.router, *self.w13, *self.w2, 2)
        return (*nb.block_norm(y, h, pre_weight=n[1]), ids)


@pytest.mark.parametrize("T", [1, 3, 20, 64])
def test_a_layer_step_by_step(nb, T):
    """Each step of the layer against the oracle on the step's own inputs; the result stays finite."""
    L = Layer(nb)
    g = torch.Generator().manual_seed(T)
    y = torch.randn((T, L.D), generator=g).to(torch.bfloat16).cuda()
    h = torch.randn((T, L.D), generator=g).cuda()
    h2, c, s = nb.block_norm(y, h, post_weight=L.norms[0], pre_weight=L.norms[1], quant=True)
    want, S = fp8.gemm(c.view(torch.uint8).cpu().numpy(), s.cpu().numpy(), L.proj[0].view(torch.uint8).cpu().numpy(),
                       L.proj[1].cpu().numpy())
    got = nb.fp8_gemm(c, s, *L.proj).double().cpu().numpy()
    assert np.all(np.abs(got - want) <= (133 + 4) * 2.0 ** -23 * S + 2.0 ** -8 * np.abs(want))
    _, x = nb.block_norm(y, h, post_weight=L.norms[0], pre_weight=L.norms[1])
    # the FP8 blocks are those of the unrounded x: within a BF16 and an E4M3 rounding of the BF16 one's
    back = fp8.dequant_rows(c.view(torch.uint8).cpu().numpy(), s.cpu().numpy())
    x64 = x.double().cpu().numpy()
    step = np.repeat(s.cpu().numpy().T.astype(np.float64), 128, axis=1) * 2.0 ** -10
    assert np.all(np.abs(back - x64) <= (2.0 ** -4 + 2.0 ** -7) * np.abs(x64) + step * 1.01)
    out_h, out_x, ids = L.run(y, h)
    assert out_h.dtype == torch.float32 and out_x.dtype == torch.bfloat16
    assert bool(out_h.isfinite().all()) and bool(out_x.isfinite().all()) and ids.shape == (T, 2)
    again = L.run(y, h)
    assert all(torch.equal(a, b) for a, b in zip((out_h, out_x, ids), again))
    assert nb.last_error() == 0


@pytest.mark.parametrize("T", [1, 17])
def test_rows_of_a_batch_are_the_rows_alone(nb, T):
    """A padded batch: rows behind the sequences change nothing in the rows before them."""
    L = Layer(nb, seed=1)
    g = torch.Generator().manual_seed(5)
    y = torch.randn((T + 7, L.D), generator=g).to(torch.bfloat16).cuda()
    h = torch.randn((T + 7, L.D), generator=g).cuda()
    a = nb.block_norm(y, h, post_weight=L.norms[0], pre_weight=L.norms[1], quant=True)
    b = nb.block_norm(y[:T].contiguous(), h[:T].contiguous(), post_weight=L.norms[0], pre_weight=L.norms[1], quant=True)
    assert torch.equal(a[0][:T], b[0]) and torch.equal(a[2][:, :T], b[2])
    assert torch.equal(a[1][:T].view(torch.uint8), b[1].view(torch.uint8))


def test_a_captured_layer_replayed_on_new_inputs(nb):
    """The NVFP4 product by its no-allocation entry: biloco_gemm allocates scratch on a stream's first call."""
    L = Layer(nb, seed=2)
    T = 5
    mk = lambda s: (torch.randn((T, L.D), generator=torch.Generator().manual_seed(s)).to(torch.bfloat16).cuda(),  # noqa: E731
                    torch.randn((T, L.D), generator=torch.Generator().manual_seed(s + 1)).cuda())
    y, h = mk(0)
    L.run(y, h, nb.gemm_noalloc)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = L.run(y, h, nb.gemm_noalloc)
    for s in (10, 20):
        y2, h2 = mk(s)
        y.copy_(y2)
        h.copy_(h2)
        want = L.run(y2, h2, nb.gemm_noalloc)
        torch.cuda.synchronize()          # the no-allocation entry's calls must not overlap
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out))
    assert nb.last_error() == 0


FIRST_USE = """
import sys
sys.path.insert(0, {root!r})
import torch
import nvfp4_binary_rank_b200 as nb
x = torch.randn((40, 256), device="cuda").to(torch.bfloat16)
w = torch.ones(256, device="cuda", dtype=torch.bfloat16)
big = x.repeat(10, 1)
W, Ws = nb.fp8_pack_weight(torch.randn((384, 256), device="cuda"))
w13, s13 = nb.fp8_pack_weight(torch.randn((4, 64, 256), device="cuda"))
w2, s2 = nb.fp8_pack_weight(torch.randn((4, 256, 32), device="cuda"))
r = torch.randn((4, 256), device="cuda")
def step():
    return [nb.fp8_gemm(*nb.fp8_quant_act(x), W, Ws), nb.fp8_gemm(*nb.fp8_quant_act(big), W, Ws),
            *nb.block_norm(x, x, post_weight=w, pre_weight=w), *nb.fp8_moe(x, r, w13, s13, w2, s2, 2),
            *nb.fp8_moe(x[:1], r, w13, s13, w2, s2, 2)]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = step()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, step()))
assert nb.last_error() == 0
print("captured on first use")
"""


def test_first_use_inside_a_capture():
    r = subprocess.run([sys.executable, "-c", FIRST_USE.format(root=ROOT)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured on first use" in r.stdout, r.stdout + r.stderr


def test_offsets_past_32_bits(nb):
    """More than 2^31 elements: the last rows of a large call are those of a small one."""
    D = 4096
    M = (1 << 31) // D + 300
    y = torch.zeros((M, D), dtype=torch.bfloat16, device="cuda")
    y[-3:] = torch.randn((3, D), generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    w = torch.full((D,), 1.5, dtype=torch.bfloat16, device="cuda")
    c, s = nb.fp8_quant_act(y)
    c3, s3 = nb.fp8_quant_act(y[-3:].contiguous())
    assert torch.equal(c[-3:].view(torch.uint8), c3.view(torch.uint8)) and torch.equal(s[:, -3:], s3)
    h, x = nb.block_norm(y, None, post_weight=w, pre_weight=w)
    h3, x3 = nb.block_norm(y[-3:].contiguous(), None, post_weight=w, pre_weight=w)
    assert torch.equal(h[-3:], h3) and torch.equal(x[-3:], x3)
    del h, x, y
    # a weight of more than 2^31 codes, its last rows and those of an activation beside them
    N = M
    ws = torch.full(((N + 127) // 128, D // 128), 2.0, device="cuda")
    one = c[-2:].contiguous()
    got = nb.fp8_gemm(one, s[:, -2:].contiguous(), c, ws)
    few = nb.fp8_gemm(one, s[:, -2:].contiguous(), c[-300:].contiguous(), ws[:3])
    assert torch.equal(got[:, -300:], few)
    # an output of more than 2^31 elements
    wc = c3.repeat(1366, 1)[:4096].contiguous()
    big = nb.fp8_gemm(c, s, wc, ws[:32].contiguous())
    assert torch.equal(big[-300:], nb.fp8_gemm(c[-300:].contiguous(), s[:, -300:].contiguous(), wc, ws[:32].contiguous()))
    assert nb.last_error() == 0
