"""The FP8 calls' fast path: built for the PyTorch that runs, and not needed for a call."""

import os
import sys
import types
import warnings

import pytest
import torch

import nvfp4_binary_rank_b200 as nb
from nvfp4_binary_rank_b200 import _fp8, build

NAME = "nvfp4_binary_rank_b200._binding"


def misfit(kind):
    if kind == "missing":
        return None                                        # the import system's mark for "not there"
    m = types.ModuleType(NAME)
    if kind == "other":
        m.torch_version = "1.0.0"
    # called with this PyTorch's tensors, such a module would read them by another one's layout
    m.quant_act = m.gemm = m.norm = m.moe = lambda *args: pytest.fail("a fast path of another PyTorch was called")
    return m


@pytest.fixture(params=["missing", "other", "unmarked"])
def unfit(request, monkeypatch):
    build.build()
    monkeypatch.setitem(sys.modules, NAME, misfit(request.param))
    monkeypatch.delattr(nb, "_binding", raising=False)
    if request.param != "missing":
        monkeypatch.setattr(nb, "_binding", sys.modules[NAME], raising=False)
    monkeypatch.setattr(_fp8, "_fast", None)


def test_a_fast_path_that_does_not_fit_is_left_out_with_one_warning(unfit):
    with pytest.warns(RuntimeWarning, match="_binding.so"):
        with pytest.raises(ValueError):                    # a host tensor: checked as ever
            nb.fp8_quant_act(torch.zeros((2, 64), dtype=torch.bfloat16))
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(ValueError):
            nb.fp8_gemm(*[torch.zeros((2, 64))] * 4)
        with pytest.raises(ValueError):
            nb.block_norm(torch.zeros((2, 64), dtype=torch.bfloat16), None)


def test_the_built_fast_path_fits(monkeypatch):
    build.build()
    monkeypatch.setattr(_fp8, "_fast", None)
    assert _fp8._load_fast().torch_version == torch.__version__


def test_a_fast_path_of_another_pytorch_is_built_anew(monkeypatch, tmp_path):
    """Whatever the files' times: an older PyTorch installed later has older files."""
    calls = []

    def compiler(cmd, **kw):
        calls.append(cmd)
        open(cmd[cmd.index("-o") + 1], "wb").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(build, "OBJ", str(tmp_path))
    monkeypatch.setattr(build.subprocess, "run", compiler)
    build._build_binding(False, False)
    build._build_binding(False, False)
    assert len(calls) == 1
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    build._build_binding(False, False)
    assert len(calls) == 2
    build._build_binding(False, False)
    assert len(calls) == 2 and os.path.exists(build.BINDING)


def test_the_library_is_built_without_a_compiler_for_the_fast_path(monkeypatch, tmp_path, capsys):
    build.build()
    (tmp_path / "_binding.so").write_bytes(b"from before")
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(build, "OBJ", str(tmp_path))
    monkeypatch.setattr(build, "_build_library", lambda force, verbose: build.LIB)
    monkeypatch.setattr(build.subprocess, "run",
                        lambda cmd, **kw: types.SimpleNamespace(returncode=1, stdout="", stderr="no Python.h"))
    assert build.build() == build.LIB
    assert "fast path" in capsys.readouterr().err and not os.path.exists(build.BINDING)


@pytest.mark.gpu
def test_calls_without_the_fast_path_give_the_same(unfit, monkeypatch):
    g = torch.Generator().manual_seed(0)
    x = torch.randn((5, 256), generator=g).to(torch.bfloat16).cuda()
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    W = nb.fp8_pack_weight(torch.randn((384, 256), generator=g).cuda())
    w13 = nb.fp8_pack_weight(torch.randn((4, 64, 256), generator=g).cuda())
    w2 = nb.fp8_pack_weight(torch.randn((4, 256, 32), generator=g).cuda())
    r = torch.randn((4, 256), generator=g).cuda()

    def run():
        c, s = nb.fp8_quant_act(x)
        return [c.view(torch.uint8), s, nb.fp8_gemm(c, s, *W), *nb.block_norm(x, x, post_weight=w, pre_weight=w),
                *nb.fp8_moe(x, r, *w13, *w2, 2)]

    with pytest.warns(RuntimeWarning):
        plain = run()
    monkeypatch.undo()
    _fp8._fast = None
    assert all(torch.equal(a, b) for a, b in zip(plain, run()))
    assert _fp8._fast.torch_version == torch.__version__
