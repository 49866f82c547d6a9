"""Binding of the FP8 block-format operators and the block norm (include/biloco.h).

Inference only: operands that require a gradient are taken, and the outputs carry none.

Argument checks and marshalling only.  Outputs are allocated on the stream the call
runs on, and the call runs on its tensors' device whatever the current one is.

A decode step calls these once per layer with microseconds of GPU work, so a plain call
(contiguous operands, the current device and stream) goes through _binding.so, which checks
it, allocates its outputs and calls the library.  What that does not take comes back as None
and is checked here: strided rows, another stream or device, an output to write into, and
every call that is refused.  Where _binding.so is missing or was built for another PyTorch, every
call is made from here, after one warning.
"""

from __future__ import annotations

import importlib
import warnings

import torch

from . import _lib
from ._lib import _check

_BF16, _F32, _FP8, _I32, _U8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int32, torch.uint8
_TYPE = {_BF16: 0, _F32: 1}
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_empty = torch.empty
_SCORE = {"softmax": 0, "sigmoid": 1}
_fast = None


class _NoFast:
    """Stands in for the fast path's module: takes no call."""

    @staticmethod
    def _none(*args):
        return None

    quant_act = gemm = norm = moe = _none


def _load_fast():
    """The fast path's module (loads the library first: it links to it)."""
    global _fast
    _lib.load()
    try:
        m = importlib.import_module(__package__ + "._binding")
        why = None if getattr(m, "torch_version", None) == torch.__version__ else "was built for another PyTorch"
    except ImportError as e:
        m, why = None, f"cannot be loaded ({e})"
    if why:
        warnings.warn(f"_binding.so {why}; the FP8 calls take several microseconds more without it: build it with "
                      "`python -m nvfp4_binary_rank_b200.build`", RuntimeWarning, stacklevel=3)
        m = _NoFast
    _fast = m
    return m


def _done(r, fn: str):
    """A fast call's outputs; its status, if it is one, raised."""
    if r.__class__ is int:
        _check(fn, r)
    return r


def _refuse(dev: int, *operands):
    """Raise for the first operand (value, name, dtypes, shape) that is not a contiguous CUDA
    tensor of that type and shape on device `dev`.  A shape of None, or an entry of it, is free; dense=False
    (a fifth entry) asks for contiguous rows only."""
    for t, name, dtypes, shape, *dense in operands:
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dtype not in dtypes:
            raise ValueError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
        if t.dim() != len(shape) or any(b is not None and a != b for a, b in zip(t.shape, shape)):
            raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
        if dense and dense[0] is False:
            if t.shape[-1] > 1 and t.stride(-1) != 1:
                raise ValueError(f"{name} must have contiguous rows")
        elif not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.get_device() != dev:
            raise ValueError(f"{name} is on cuda:{t.get_device()}, the other operands on cuda:{dev}")
    raise ValueError("operands do not go together")


def _elsewhere(dev: int, stream, fn, *args, **kw):
    """fn(*args) with device `dev` and `stream` (None: that device's current one) made current."""
    if stream is not None and stream.device_index != dev:
        raise ValueError(f"stream is on cuda:{stream.device_index}, the operands on cuda:{dev}")
    with torch.cuda.device(dev):
        if stream is None:
            return fn(*args, **kw)
        with torch.cuda.stream(stream):
            return fn(*args, **kw)


def _rows_ok(t, dtype, dev) -> bool:
    """2-D tensor with contiguous rows."""
    return (isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == 2 and t.get_device() == dev
            and (t.is_contiguous() or t.shape[1] <= 1 or t.stride(1) == 1))


def fp8_quant_act(x: torch.Tensor, stream=None):
    """BF16 [M, K] (rows contiguous, any row stride that is a multiple of 8) ->
    (codes float8_e4m3fn [M, K], scales float32 [ceil(K/128), M]), without a gradient."""
    if stream is None:
        r = (_fast or _load_fast()).quant_act(x)
        if r is not None:
            return _done(r, "biloco_fp8_quant_act")
    dev = x.get_device() if isinstance(x, torch.Tensor) else -1
    if dev < 0 or not _rows_ok(x, _BF16, dev):
        _refuse(dev, (x, "x", (_BF16,), (None, None), False))
    if stream is not None or dev != _current_device():
        return _elsewhere(dev, stream, fp8_quant_act, x)
    M, K = x.shape
    codes = x.new_empty((M, K), dtype=_FP8)
    scales = x.new_empty(((K + 127) // 128, M), dtype=_F32)
    st = (_lib._lib or _lib.load()).biloco_fp8_quant_act(
        x.data_ptr(), x.stride(0) if M > 1 else K, M, K, codes.data_ptr(), scales.data_ptr(), _raw_stream(dev))
    if st:
        _check("biloco_fp8_quant_act", st)
    return codes, scales


def fp8_pack_weight(W: torch.Tensor, stream=None):
    """BF16 or float32 [N, K] or [E, N, K] -> (codes float8_e4m3fn of W's shape,
    scales float32 [(E,) ceil(N/128), ceil(K/128)]), without a gradient."""
    dev = W.get_device() if isinstance(W, torch.Tensor) else -1
    if dev < 0 or W.dtype not in _TYPE or W.dim() not in (2, 3) or not W.is_contiguous():
        _refuse(dev, (W, "W", (_BF16, _F32), (None,) * (3 if isinstance(W, torch.Tensor) and W.dim() == 3 else 2)))
    if stream is not None or dev != _current_device():
        return _elsewhere(dev, stream, fp8_pack_weight, W)
    N, K = W.shape[-2:]
    lead = tuple(W.shape[:-2])
    codes = W.new_empty(W.shape, dtype=_FP8)
    scales = W.new_empty((*lead, (N + 127) // 128, (K + 127) // 128), dtype=_F32)
    _check("biloco_fp8_pack_weight", _lib.load().biloco_fp8_pack_weight(
        W.data_ptr(), _TYPE[W.dtype], lead[0] if lead else 1, N, K, codes.data_ptr(), scales.data_ptr(),
        _raw_stream(dev)))
    return codes, scales


def fp8_gemm(x_codes: torch.Tensor, x_scales: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor,
             out: torch.Tensor | None = None, out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """y[m, n] = sum_b x_scales[b, m] w_scales[n/128, b] (x[m] . w[n])_b over blocks b of 128
    along K, for any number of rows; y is bfloat16 or float32 and carries no gradient.  w_codes
    may be read while earlier calls of this library on the stream still run: none of them but
    fp8_pack_weight may have written it since PyTorch's last kernel there."""
    if stream is None and (out is not None or out_dtype in _TYPE):
        r = (_fast or _load_fast()).gemm(x_codes, x_scales, w_codes, w_scales, out,
                                         (out_dtype if out is None else getattr(out, "dtype", None)) is _F32)
        if r is not None:
            return _done(r, "biloco_fp8_gemm")
    try:
        dev = x_codes.get_device()
        M, K = x_codes.shape
        N = w_codes.shape[0]
        KB = (K + 127) // 128
        good = (dev >= 0 and x_codes.dtype is _FP8 and w_codes.dtype is _FP8 and x_scales.dtype is _F32
                and w_scales.dtype is _F32 and w_codes.shape == (N, K) and x_scales.shape == (KB, M)
                and w_scales.shape == ((N + 127) // 128, KB) and x_codes.is_contiguous() and w_codes.is_contiguous()
                and x_scales.is_contiguous() and w_scales.is_contiguous() and w_codes.get_device() == dev
                and x_scales.get_device() == dev and w_scales.get_device() == dev)
        if out is not None:
            out_dtype = out.dtype
            good = good and out.shape == (M, N) and out.is_contiguous() and out.get_device() == dev
        good = good and out_dtype in _TYPE
    except (AttributeError, ValueError, IndexError, RuntimeError):
        good = False
    if not good:
        for t, name in ((x_codes, "x_codes"), (w_codes, "w_codes")):
            if not isinstance(t, torch.Tensor) or t.dim() != 2:
                raise ValueError(f"{name} must be a 2-D CUDA tensor")
        M, K, N, dev = *x_codes.shape, w_codes.shape[0], x_codes.get_device()
        KB = (K + 127) // 128
        if out is None and out_dtype not in _TYPE:
            raise ValueError(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
        more = [] if out is None else [(out, "out", (_BF16, _F32), (M, N))]
        _refuse(dev, (x_codes, "x_codes", (_FP8,), (M, K)), (x_scales, "x_scales", (_F32,), (KB, M)),
                (w_codes, "w_codes", (_FP8,), (N, K)), (w_scales, "w_scales", (_F32,), ((N + 127) // 128, KB)), *more)
    if stream is not None or dev != _current_device():
        return _elsewhere(dev, stream, fp8_gemm, x_codes, x_scales, w_codes, w_scales, out, out_dtype)
    if out is None:
        out = x_scales.new_empty((M, N), dtype=out_dtype)
    st = (_lib._lib or _lib.load()).biloco_fp8_gemm(
        x_codes.data_ptr(), x_scales.data_ptr(), w_codes.data_ptr(), w_scales.data_ptr(), out.data_ptr(),
        0 if out_dtype is _BF16 else 1, M, N, K, _raw_stream(dev))
    if st:
        _check("biloco_fp8_gemm", st)
    return out


def block_norm(y: torch.Tensor | None, h: torch.Tensor | None, *, post_weight: torch.Tensor | None = None,
               gate: torch.Tensor | None = None, res_scale: float = 1.0, pre_weight: torch.Tensor | None = None,
               offset: float = 0.0, eps: float = 1e-6, quant: bool = False, out_h: torch.Tensor | None = None,
               stream=None):
    """The norm after a block, its gate, the scaled residual and the norm before the next:

        u  = y rsqrt(mean(y^2) + eps) (post_weight + offset)     (u = y without post_weight)
        h' = res_scale h + gate u
        x  = h' rsqrt(mean(h'^2) + eps) (pre_weight + offset)

    y is bfloat16 [M, D] (None: no block before, u = 0), h bfloat16 or float32 [M, D]
    (None: no residual yet; h' is then bfloat16), gate [D] or [G, D] with M % G == 0
    (each row serves M / G consecutive rows).  Returns (h', x), (h', codes, scales) with
    `quant` (as fp8_quant_act lays them out), or h' alone without pre_weight; none carries a
    gradient.  out_h may be h itself, and must not overlap the inputs otherwise."""
    if stream is None and out_h is None:
        r = (_fast or _load_fast()).norm(y, h, post_weight, pre_weight, gate, res_scale, offset, eps, bool(quant))
        if r is not None:
            return _done(r, "biloco_block_norm")
    ref = h if y is None else y
    if ref is None:
        raise ValueError("y or h must be given")
    if y is None and (post_weight is not None or gate is not None):
        raise ValueError("post_weight and gate act on y, which is None")
    if quant and pre_weight is None:
        raise ValueError("quant needs pre_weight")
    dev = ref.get_device() if isinstance(ref, torch.Tensor) and ref.dim() == 2 else -1
    if dev < 0:
        _refuse(dev, (ref, "h" if y is None else "y", (_BF16, _F32), (None, None), False))
    M, D = ref.shape
    h_dtype = _BF16 if h is None else h.dtype
    w_dtype, g_type, G = _BF16, 0, 1
    p_y = p_h = p_post = p_pre = p_gate = None
    ldy = ldh = 0
    if y is not None:
        if not _rows_ok(y, _BF16, dev):
            _refuse(dev, (y, "y", (_BF16,), (M, D), False))
        p_y, ldy = y.data_ptr(), y.stride(0) if M > 1 else D
    if h is not None:
        if h_dtype not in _TYPE or not _rows_ok(h, h_dtype, dev) or h.shape != (M, D):
            _refuse(dev, (h, "h", (_BF16, _F32), (M, D), False))
        p_h, ldh = h.data_ptr(), h.stride(0) if M > 1 else D
    if pre_weight is not None:
        w_dtype = pre_weight.dtype
        if w_dtype not in _TYPE or pre_weight.shape != (D,) or not pre_weight.is_contiguous() or pre_weight.get_device() != dev:
            _refuse(dev, (pre_weight, "pre_weight", (_BF16, _F32), (D,)))
        p_pre = pre_weight.data_ptr()
    if post_weight is not None:
        if pre_weight is not None and post_weight.dtype is not w_dtype:
            raise ValueError("post_weight and pre_weight must have one type")
        w_dtype = post_weight.dtype
        if w_dtype not in _TYPE or post_weight.shape != (D,) or not post_weight.is_contiguous() or post_weight.get_device() != dev:
            _refuse(dev, (post_weight, "post_weight", (_BF16, _F32), (D,)))
        p_post = post_weight.data_ptr()
    if gate is not None:
        if gate.dtype not in _TYPE or gate.dim() not in (1, 2) or gate.shape[-1] != D or not gate.is_contiguous() or gate.get_device() != dev:
            _refuse(dev, (gate, "gate", (_BF16, _F32), (None, D) if gate.dim() == 2 else (D,)))
        G = gate.shape[0] if gate.dim() == 2 else 1
        if G < 1 or M % G:
            raise ValueError(f"gate has {G} rows, which do not divide {M}")
        p_gate, g_type = gate.data_ptr(), _TYPE[gate.dtype]
    if out_h is not None and (not _rows_ok(out_h, h_dtype, dev) or out_h.shape != (M, D)):
        _refuse(dev, (out_h, "out_h", (h_dtype,), (M, D), False))
    if stream is not None or dev != _current_device():
        return _elsewhere(dev, stream, block_norm, y, h, post_weight=post_weight, gate=gate, res_scale=res_scale,
                          pre_weight=pre_weight, offset=offset, eps=eps, quant=quant, out_h=out_h)
    if out_h is None:
        out_h = ref.new_empty((M, D), dtype=h_dtype)
        ldo = D
    else:
        ldo = out_h.stride(0) if M > 1 else D
    x = codes = scales = p_x = p_c = p_s = None
    if quant:
        codes = ref.new_empty((M, D), dtype=_FP8)
        scales = ref.new_empty(((D + 127) // 128, M), dtype=_F32)
        p_c, p_s = codes.data_ptr(), scales.data_ptr()
    elif pre_weight is not None:
        x = ref.new_empty((M, D), dtype=_BF16)
        p_x = x.data_ptr()
    st = (_lib._lib or _lib.load()).biloco_block_norm(
        p_y, ldy, p_h, ldh, _TYPE[h_dtype], p_post, p_pre, _TYPE[w_dtype], p_gate, g_type, G, res_scale, offset, eps,
        M, D, out_h.data_ptr(), ldo, p_x, p_c, p_s, _raw_stream(dev))
    if st:
        _check("biloco_block_norm", st)
    if quant:
        return out_h, codes, scales
    return out_h if x is None else (out_h, x)


def fp8_moe(x: torch.Tensor, router: torch.Tensor, w13: torch.Tensor, w13_scales: torch.Tensor, w2: torch.Tensor,
            w2_scales: torch.Tensor, top_k: int, *, score: str = "softmax", bias: torch.Tensor | None = None,
            renorm: bool = True, route_scale: float = 1.0, stream=None):
    """A whole mixture-of-experts layer for up to 64 tokens:

        y[t] = sum over t's top_k experts e of weight[t, e] W2_e (silu(W1_e x[t]) * (W3_e x[t]))

    x bfloat16 [T, D]; router bfloat16 or float32 [E, D]; w13 [n, 2F, D] ([W1; W3] stacked)
    and w2 [n, D, F] with their scales from fp8_pack_weight.  The n - E last experts are
    shared: they serve every token with weight 1.  `score` is "softmax" (over the experts)
    or "sigmoid"; bias float32 [E] is added for the choice only.  Returns (y bfloat16
    [T, D], ids int32 [T, top_k], weights float32 [T, top_k]), none with a gradient.  The hidden
    values are held in FP16.  router and w2 may be read while earlier calls of this library on the
    stream still run: none of them but fp8_pack_weight may have written them since PyTorch's last
    kernel there."""
    if stream is None and score in _SCORE:
        r = (_fast or _load_fast()).moe(x, router, w13, w13_scales, w2, w2_scales, bias, top_k, _SCORE[score], bool(renorm),
                                        route_scale)
        if r is not None:
            return _done(r, "biloco_fp8_moe")
    for t, name, nd in ((x, "x", 2), (router, "router", 2), (w13, "w13", 3)):
        if not isinstance(t, torch.Tensor) or t.dim() != nd:
            raise ValueError(f"{name} must be a {nd}-D CUDA tensor")
    dev = x.get_device()
    T, D = x.shape
    E = router.shape[0]
    n, F = w13.shape[0], w13.shape[1] // 2
    KD, KF = (D + 127) // 128, (F + 127) // 128
    if not (dev >= 0 and _rows_ok(x, _BF16, dev) and router.dtype in _TYPE and router.shape == (E, D)
            and router.is_contiguous() and router.get_device() == dev and w13.dtype is _FP8 and w13.shape == (n, 2 * F, D)
            and w13.is_contiguous() and w13.get_device() == dev and w13_scales.dtype is _F32
            and w13_scales.shape == (n, (2 * F + 127) // 128, KD) and w13_scales.is_contiguous()
            and w13_scales.get_device() == dev and w2.dtype is _FP8 and w2.shape == (n, D, F) and w2.is_contiguous()
            and w2.get_device() == dev and w2_scales.dtype is _F32 and w2_scales.shape == (n, KD, KF)
            and w2_scales.is_contiguous() and w2_scales.get_device() == dev
            and (bias is None or (bias.dtype is _F32 and bias.shape == (E,) and bias.is_contiguous() and bias.get_device() == dev))):
        _refuse(dev, (x, "x", (_BF16,), (T, D), False), (router, "router", (_BF16, _F32), (E, D)),
                (w13, "w13", (_FP8,), (n, 2 * F, D)), (w13_scales, "w13_scales", (_F32,), (n, (2 * F + 127) // 128, KD)),
                (w2, "w2", (_FP8,), (n, D, F)), (w2_scales, "w2_scales", (_F32,), (n, KD, KF)),
                *(() if bias is None else ((bias, "bias", (_F32,), (E,)),)))
    if n < E:
        raise ValueError(f"router has {E} experts, w13 {n}")
    if not 1 <= top_k <= E:
        raise ValueError(f"top_k must be 1 to {E}, got {top_k}")
    if score not in _SCORE:
        raise ValueError(f"score must be one of {sorted(_SCORE)}, got {score!r}")
    if stream is not None or dev != _current_device():
        return _elsewhere(dev, stream, fp8_moe, x, router, w13, w13_scales, w2, w2_scales, top_k, score=score, bias=bias,
                          renorm=renorm, route_scale=route_scale)
    lib = _lib._lib or _lib.load()
    y = x.new_empty((T, D))
    ids = x.new_empty((T, top_k), dtype=_I32)
    weights = x.new_empty((T, top_k), dtype=_F32)
    nbytes = lib.biloco_fp8_moe_workspace_bytes(T, D, F, top_k, n - E) if T else 1
    if nbytes == 0:
        raise _lib.BilocoError("biloco_fp8_moe_workspace_bytes", _lib.ERR_SHAPE)
    ws = x.new_empty((nbytes,), dtype=_U8)
    st = lib.biloco_fp8_moe(
        x.data_ptr(), x.stride(0) if T > 1 else D, router.data_ptr(), _TYPE[router.dtype],
        None if bias is None else bias.data_ptr(), w13.data_ptr(), w13_scales.data_ptr(), w2.data_ptr(),
        w2_scales.data_ptr(), T, D, F, E, top_k, n - E, _SCORE[score], renorm, route_scale, y.data_ptr(), ids.data_ptr(),
        weights.data_ptr(), ws.data_ptr(), nbytes, _raw_stream(dev))
    if st:
        _check("biloco_fp8_moe", st)
    return y, ids, weights
