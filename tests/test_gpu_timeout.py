"""The failure path on the GPU, made on purpose without a fault: a bounded wait
that nothing completes gives up, the kernel records BILOCO_ERR_TIMEOUT in the
stream's status word, the host reads it, and the stream stays usable.

Two forms: a one-warp self-test kernel, and the GEMM itself with some of its
grid-wide arrivals left out (biloco_selftest_drop_arrivals), so that the fused
kernel's own abort protocol runs: the waiting CTAs give up, leave together,
drain their copies and MMAs, free their tensor memory and return; the host then
resets the counters and the next call on the stream is correct."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import workloads
from gpu_common import assert_y_close, device_problem, oracle_for, y_to_numpy

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def nb():
    import nvfp4_binary_rank_b200 as nb
    nb.load()
    return nb


def test_expired_wait_is_reported_and_cleared(nb):
    s = torch.cuda.Stream()
    assert nb.last_error(s) == 0
    nb.selftest_wait_timeout(s)
    assert nb.last_error(s) == nb._lib.ERR_TIMEOUT
    assert nb.last_error(s) == 0                          # read once, then cleared
    # the context and the stream still work
    w = workloads.CONFIGS["tiny"]
    d, ref = oracle_for(w)
    prob = device_problem(w, d)
    with torch.cuda.stream(s):
        y = nb.gemm(prob["x"], prob["W"], prob["sf"], prob["g"], prob["Ub"], prob["Vb"], prob["alpha"])
    s.synchronize()
    assert nb.last_error(s) == 0
    assert_y_close(y_to_numpy(y), ref["y"], "tiny after a timeout")


# (mask, M, N, K): 1 drops the z arrivals (1 row: the completing CTA's U side
# waits; 16 rows: the per-contributor tensor-core U side waits), 2 the
# activation-image arrivals (8 rows; from 17 rows the producers' wait on the
# streamed image), 3 both.  The 64- and 128-row cases run the column-chunked
# epilogue's abort path; at N = K = 5120 their CTAs hold two tiles, so the
# 128-row class's single U-side product buffer is waited on for a second segment.
@pytest.mark.timeout(120, method="thread")
@pytest.mark.parametrize("entry", ["gemm", "gemm_noalloc"])
@pytest.mark.parametrize("mask,M,N,K", [(1, 1, 1280, 2048), (1, 16, 1280, 2048), (2, 8, 1280, 2048),
                                        (3, 16, 1280, 2048), (2, 24, 1280, 2048), (1, 32, 1280, 2048),
                                        (1, 64, 1280, 2048), (3, 64, 5120, 5120), (2, 100, 1280, 2048),
                                        (1, 128, 5120, 5120)])
def test_dropped_arrivals_expire_inside_the_gemm(nb, entry, mask, M, N, K):
    if entry == "gemm_noalloc" and M > 64 and N * K > 1280 * 2048:
        pytest.skip("the 128-row class's scratch at this size exceeds the no-allocation array")
    w = workloads.Workload(f"drop_{M}", M, N, K, 256, 60 + M)
    d, ref = oracle_for(w)
    prob = device_problem(w, d)
    args = (prob["x"], prob["W"], prob["sf"], prob["g"], prob["Ub"], prob["Vb"], prob["alpha"])
    fn = getattr(nb, entry)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y0 = fn(*args)                                    # a correct call first
    assert nb.last_error(s) == 0
    nb.selftest_drop_arrivals(mask)
    with torch.cuda.stream(s):
        fn(*args)                                         # its waits expire after ~1 s
    assert nb.last_error(s) == nb._lib.ERR_TIMEOUT
    assert nb.last_error(s) == 0
    with torch.cuda.stream(s):
        y1 = fn(*args)
        y2 = fn(*args)
    assert nb.last_error(s) == 0
    assert_y_close(y_to_numpy(y1), ref["y"], "first call after the timeout")
    np.testing.assert_array_equal(y_to_numpy(y1), y_to_numpy(y0))
    np.testing.assert_array_equal(y_to_numpy(y2), y_to_numpy(y0))


# swapped form: one tile a cluster of 8 parts, tiles of 32 to 128 columns, several tiles a CTA; rows form: K split
# over pairs, one tile a pair, several tiles a pair
@pytest.mark.timeout(120, method="thread")
@pytest.mark.parametrize("M,N,K", [(1, 512, 5120), (40, 1000, 2064), (60, 5120, 1024), (128, 5120, 5120), (3, 60000, 1024),
                                   (129, 5120, 5120), (333, 1800, 2064), (2048, 5120, 1024)])
def test_scales_that_never_arrive_expire_inside_the_fp8_product(nb, M, N, K):
    g = torch.Generator().manual_seed(M)
    w = nb.fp8_pack_weight(torch.randn((N, K), generator=g).cuda())
    x = nb.fp8_quant_act(torch.randn((M, K), generator=g).to(torch.bfloat16).cuda())
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    y0 = nb.fp8_gemm(*x, *w, stream=s)                    # a correct call first
    assert nb.last_error(s) == 0
    nb.selftest_drop_scales()
    nb.fp8_gemm(*x, *w, stream=s)                         # its waits expire after ~1 s
    assert nb.last_error(s) == nb._lib.ERR_TIMEOUT
    assert nb.last_error(s) == 0
    y1, y2 = nb.fp8_gemm(*x, *w, stream=s), nb.fp8_gemm(*x, *w, stream=s)
    assert nb.last_error(s) == 0
    assert torch.equal(y0, y1) and torch.equal(y0, y2)


def expire(nb, s, M=3, N=256, K=1024):
    x = nb.fp8_quant_act(torch.ones((M, K), dtype=torch.bfloat16, device="cuda"))
    w = nb.fp8_pack_weight(torch.ones((N, K), device="cuda"))
    torch.cuda.synchronize()
    nb.selftest_drop_scales()
    nb.fp8_gemm(*x, *w, stream=s)
    return x, w


def test_an_expired_fp8_product_is_its_own_streams_error(nb):
    """Other streams, asked before and after the kernel has given up, report nothing and clear nothing."""
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    nb.last_error(a)
    x, w = expire(nb, a)
    y = nb.fp8_gemm(*x, *w, stream=b)
    assert nb.last_error(b) == 0                           # the other stream's kernel still waits
    a.synchronize()
    assert nb.last_error(b) == 0 and nb.last_error() == 0
    assert nb.last_error(a) == nb._lib.ERR_TIMEOUT
    assert nb.last_error(a) == 0
    assert torch.equal(y, nb.fp8_gemm(*x, *w))
    # two streams, each its own
    expire(nb, a)
    expire(nb, b)
    assert nb.last_error(b) == nb._lib.ERR_TIMEOUT and nb.last_error() == 0
    assert nb.last_error(a) == nb._lib.ERR_TIMEOUT
    assert nb.last_error(a) == 0 and nb.last_error(b) == 0


def test_an_expired_fp8_product_in_a_graph_is_reported(nb):
    """A captured product may be replayed on any stream: whichever asks first is told, once."""
    x = nb.fp8_quant_act(torch.ones((3, 1024), dtype=torch.bfloat16, device="cuda"))
    w = nb.fp8_pack_weight(torch.ones((256, 1024), device="cuda"))
    want = nb.fp8_gemm(*x, *w)
    graphs = []
    for drop in (True, False):
        if drop:
            nb.selftest_drop_scales()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = nb.fp8_gemm(*x, *w)
        graphs.append((g, y))
    s, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        graphs[0][0].replay()
    assert nb.last_error(other) == nb._lib.ERR_TIMEOUT    # it waited for the replay
    assert nb.last_error(s) == 0 and nb.last_error() == 0
    with torch.cuda.stream(s):
        graphs[1][0].replay()
    assert nb.last_error(s) == 0
    assert torch.equal(graphs[1][1], want)


MANY_STREAMS = """
import ctypes, sys
sys.path.insert(0, {root!r})
import torch
import nvfp4_binary_rank_b200 as nb
x = nb.fp8_quant_act(torch.ones((3, 1024), dtype=torch.bfloat16, device="cuda"))
w = nb.fp8_pack_weight(torch.ones((256, 1024), device="cuda"))
want = nb.fp8_gemm(*x, *w)
torch.cuda.synchronize()
streams = []
for _ in range(1100):
    h = ctypes.c_void_p()
    assert int(torch.cuda.cudart().cudaStreamCreate(ctypes.addressof(h))) == 0
    streams.append(torch.cuda.ExternalStream(h.value))
y = [nb.fp8_gemm(*x, *w, stream=s) for s in streams]
torch.cuda.synchronize()
assert all(torch.equal(t, want) for t in y)
assert all(nb.last_error(s) == 0 for s in streams)
for i, asked in ((500, 500), (1080, 1099)):
    nb.selftest_drop_scales()
    nb.fp8_gemm(*x, *w, stream=streams[i])
    if i == asked:
        assert nb.last_error(streams[i + 1]) == 0
    assert nb.last_error(streams[asked]) == nb._lib.ERR_TIMEOUT
    assert nb.last_error(streams[i]) == 0
print("a thousand streams")
"""


def test_more_streams_than_error_words(nb):
    """The first 1023 streams have a word each, those beyond one together."""
    r = subprocess.run([sys.executable, "-c", MANY_STREAMS.format(root=ROOT)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "a thousand streams" in r.stdout, r.stdout + r.stderr


def test_drop_request_is_consumed_by_one_call(nb):
    # a request made before a call that does not take the decode kernel (here the
    # local-z schedule, which runs the general kernel) is consumed by that call and
    # affects nothing
    w = workloads.Workload("drop_general", 40, 256, 512, 32, 77)
    d, ref = oracle_for(w)
    prob = device_problem(w, d)
    nb.set_mode(nb.MODE_LOCAL_Z)
    try:
        assert nb.gemm_kernel_count(w.M, w.N, w.K, w.r) == 2
        nb.selftest_drop_arrivals(1)
        y = nb.gemm(prob["x"], prob["W"], prob["sf"], prob["g"], prob["Ub"], prob["Vb"], prob["alpha"])
    finally:
        nb.set_mode(nb.MODE_AUTO)
    assert nb.last_error() == 0
    assert_y_close(y_to_numpy(y), ref["y"], w.name)
