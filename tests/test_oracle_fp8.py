"""Pins for the FP8 oracle and the refusals of the FP8 entry points (CPU only)."""

import ctypes

import ml_dtypes
import numpy as np
import pytest
import torch

from oracle import fp8


def test_decode_matches_library():
    lib = np.arange(256, dtype=np.uint8).view(ml_dtypes.float8_e4m3fn).astype(np.float64)
    assert np.array_equal(np.isnan(lib), np.isnan(fp8.E4M3))
    ok = ~np.isnan(lib)
    assert np.array_equal(lib[ok], fp8.E4M3[ok])


def test_encode_matches_library_at_codes_midpoints_and_random_values():
    mags = fp8.E4M3[:127]
    mid = (mags[1:] + mags[:-1]) / 2
    rng = np.random.default_rng(0)
    v = np.concatenate([mags, mid, np.nextafter(mid, 0), np.nextafter(mid, 1e9), rng.standard_normal(4096) * 10.0,
                        rng.standard_normal(1024) * 2.0 ** -8])
    v = np.concatenate([v, -v])
    want = np.clip(v, -448, 448).astype(np.float32).astype(ml_dtypes.float8_e4m3fn).view(np.uint8)
    exact32 = v.astype(np.float32).astype(np.float64) == v           # the library rounds from FP32
    assert np.array_equal(fp8.encode(v)[exact32], want[exact32])
    assert fp8.decode(fp8.encode(np.array([1e9, -1e9, 449.0]))).tolist() == [448, -448, 448]


def test_quantisers_closed_forms():
    x = np.zeros((2, 160), np.float32)
    x[0, :128] = 448.0
    x[1, 130] = -7.0
    c, s = fp8.quant_rows(x)
    assert s.shape == (2, 2)
    assert s[0, 0] == 1.0 and np.all(fp8.decode(c[0, :128]) == 448)
    assert s[1, 1] == np.float32(7) / np.float32(448) and fp8.decode(c[1, 130:131])[0] == -448
    assert np.all(c[0, 128:] == 0) and s[1, 0] == np.float32(2.0 ** -100) / np.float32(448)
    rng = np.random.default_rng(1)
    w = rng.standard_normal((130, 272)).astype(np.float32)
    c, s = fp8.quant_tiles(w)
    assert s.shape == (2, 3)
    # half a step of four significant bits, or half a subnormal step
    back = fp8.dequant_tiles(c, s)
    step = np.repeat(np.repeat(s, 128, 0)[:130], 128, 1)[:, :272] * 2.0 ** -10
    assert np.all(np.abs(back - w) <= (np.abs(w) * 2.0 ** -4 + step) * (1 + 2.0 ** -20))


def test_gemm_is_the_dense_product():
    rng = np.random.default_rng(2)
    x, w = rng.standard_normal((3, 272)).astype(np.float32), rng.standard_normal((130, 272)).astype(np.float32)
    y, top = fp8.gemm(*fp8.quant_rows(x), *fp8.quant_tiles(w))
    assert np.linalg.norm(y - x @ w.T) < 0.06 * np.linalg.norm(y) and np.all(top >= np.abs(y))


def test_block_norm_against_torch():
    rng = np.random.default_rng(3)
    y, h, w = rng.standard_normal((4, 24)), rng.standard_normal((4, 24)), rng.standard_normal(24)
    g = rng.standard_normal((2, 24))
    h2, x = fp8.block_norm(y, h, post_weight=w, gate=g, res_scale=0.5, pre_weight=w, offset=1.0, eps=1e-3)
    t = torch.from_numpy
    u = torch.nn.functional.rms_norm(t(y), (24,), t(w) + 1.0, 1e-3) * t(g)[[0, 0, 1, 1]]
    want = 0.5 * t(h) + u
    assert np.allclose(h2, want.numpy(), rtol=1e-12, atol=1e-12)
    assert np.allclose(x, torch.nn.functional.rms_norm(want, (24,), t(w) + 1.0, 1e-3).numpy(), rtol=1e-12, atol=1e-12)


def test_route_ties_take_the_lowest_index_and_moe_of_one_expert_is_its_mlp():
    x = np.ones((2, 4))
    ids, w = fp8.route(x, np.ones((5, 4)), 2)
    assert ids.tolist() == [[0, 1], [0, 1]] and np.allclose(w, 0.5)
    rng = np.random.default_rng(4)
    w13, w2 = rng.standard_normal((1, 6, 4)), rng.standard_normal((1, 4, 3))
    y = fp8.moe(x, np.zeros((2, 1), int), np.ones((2, 1)), w13, w2)
    g = torch.nn.functional.silu(torch.from_numpy(w13[0, :3] @ x[0])).numpy() * (w13[0, 3:] @ x[0])
    assert np.allclose(y[0], w2[0] @ g)


# ---- refusals: checked on the host before any CUDA call

@pytest.fixture(scope="module")
def lib():
    from nvfp4_binary_rank_b200 import _lib, build
    build.build()
    return _lib.load()


P = ctypes.c_void_p
A, ODD = P(0x10000), P(0x10001)


def test_fp8_quant_refusals(lib):
    f = lib.biloco_fp8_quant_act
    assert f(None, 64, 1, 64, A, A, None) == -1
    assert f(A, 64, -1, 64, A, A, None) == -1
    assert f(A, 64, 1, 0, A, A, None) == -2
    assert f(A, 64, 1, 24, A, A, None) == -2
    assert f(A, 32, 1, 64, A, A, None) == -2          # rows overlap
    assert f(A, 68, 1, 64, A, A, None) == -2          # row stride not 16 bytes
    assert f(P(0x10008), 64, 1, 64, A, A, None) == -3
    assert f(A, 64, 1, 64, P(0x10008), A, None) == -3
    g = lib.biloco_fp8_pack_weight
    assert g(A, 2, 1, 128, 64, A, A, None) == -1
    assert g(A, 1, 0, 128, 64, A, A, None) == -2
    assert g(A, 1, 1, 0, 64, A, A, None) == -2
    assert g(A, 1, 1, 128, 40, A, A, None) == -2
    assert g(A, 1, 1, 128, 64, ODD, A, None) == -3


def test_fp8_gemm_refusals(lib):
    f = lib.biloco_fp8_gemm
    assert f(None, A, A, A, A, 0, 1, 128, 64, None) == -1
    assert f(A, A, A, A, None, 0, 1, 128, 64, None) == -1
    assert f(A, A, A, A, A, 2, 1, 128, 64, None) == -1
    assert f(A, A, A, A, A, 0, -1, 128, 64, None) == -1
    assert f(A, A, A, A, A, 0, 1, 0, 64, None) == -2
    assert f(A, A, A, A, A, 0, 1, 128, 8, None) == -2
    assert f(A, A, A, A, A, 0, 1, 128, 72, None) == -2
    assert f(A, A, A, A, A, 0, 1, (1 << 24) + 1, 64, None) == -2
    assert f(P(0x10008), A, A, A, A, 0, 1, 128, 64, None) == -3
    assert f(A, A, A, A, ODD, 0, 1, 128, 64, None) == -3
    assert f(A, A, A, A, P(0x10002), 1, 1, 128, 64, None) == -3


def _norm(lib, y=A, ldy=64, h=A, ldh=64, ht=0, post=None, pre=A, wt=0, gate=None, gt=0, G=1, M=4, D=64, ho=A, ldho=64,
          x=A, codes=None, scales=None):
    return lib.biloco_block_norm(y, ldy, h, ldh, ht, post, pre, wt, gate, gt, G, 1.0, 0.0, 1e-6, M, D, ho, ldho, x,
                                 codes, scales, None)


def test_block_norm_refusals(lib):
    assert _norm(lib, y=None, h=None) == -1
    assert _norm(lib, y=None, post=A) == -1
    assert _norm(lib, y=None, gate=A) == -1
    assert _norm(lib, ho=None, x=None) == -1
    assert _norm(lib, pre=None) == -1
    assert _norm(lib, x=None) == -1
    assert _norm(lib, x=None, codes=A) == -1
    assert _norm(lib, ht=3) == -1
    assert _norm(lib, M=-1) == -1
    assert _norm(lib, D=0) == -2
    assert _norm(lib, D=60) == -2
    assert _norm(lib, D=32776, ldy=32776, ldh=32776, ldho=32776) == -2
    assert _norm(lib, D=72, ldy=72, ldh=72, ldho=72, codes=A, scales=A) == -2
    assert _norm(lib, ldy=32) == -2
    assert _norm(lib, ldh=68) == -2
    assert _norm(lib, gate=A, G=3) == -2
    assert _norm(lib, gate=A, G=0) == -2
    assert _norm(lib, post=P(0x10008)) == -3


def _moe(lib, x=A, ldx=64, router=A, rt=0, w13=A, T=2, D=64, F=32, E=4, k=2, sh=0, score=0, y=A, ws=A, nbytes=1 << 30):
    return lib.biloco_fp8_moe(x, ldx, router, rt, None, w13, A, A, A, T, D, F, E, k, sh, score, 1, 1.0, y, A, A, ws,
                              nbytes, None)


def test_fp8_moe_refusals(lib):
    assert _moe(lib, x=None) == -1
    assert _moe(lib, ws=None) == -1
    assert _moe(lib, rt=5) == -1
    assert _moe(lib, score=2) == -1
    assert _moe(lib, T=-1) == -1
    assert _moe(lib, nbytes=64) == -1
    assert _moe(lib, T=65) == -2
    assert _moe(lib, D=72, ldx=72) == -2
    assert _moe(lib, F=24) == -2
    assert _moe(lib, F=16400) == -2
    assert _moe(lib, k=5) == -2
    assert _moe(lib, k=0) == -2
    assert _moe(lib, E=513) == -2
    assert _moe(lib, k=17, E=32) == -2
    assert _moe(lib, sh=5) == -2
    assert _moe(lib, ldx=48) == -2
    assert _moe(lib, x=P(0x10008)) == -3
    assert _moe(lib, w13=P(0x10008)) == -3
    assert _moe(lib, ws=P(0x10010)) == -3
    assert _moe(lib, T=0, x=None, ws=None) == 0
    assert lib.biloco_fp8_moe_workspace_bytes(1, 64, 32, 2, 0) > 0
    assert lib.biloco_fp8_moe_workspace_bytes(0, 64, 32, 2, 0) == 0


def test_binding_refuses_host_tensors():
    import nvfp4_binary_rank_b200 as nb
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        nb.fp8_quant_act(x)
    with pytest.raises(ValueError):
        nb.fp8_pack_weight(x)
    with pytest.raises(ValueError):
        nb.block_norm(x, None)
    with pytest.raises(ValueError):
        nb.block_norm(None, None)
