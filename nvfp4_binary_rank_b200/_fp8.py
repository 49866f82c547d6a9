"""Binding of the FP8 block-format operators and the block norm (include/biloco.h).

Argument checks and marshalling only.  Outputs are allocated on the stream the call
runs on, and the call runs on its tensors' device whatever the current one is.
"""

from __future__ import annotations

import torch

from . import _lib
from ._lib import _check

BLOCK = 128
_BF16, _F32, _FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
_TYPE = {_BF16: 0, _F32: 1}
_raw_stream = torch._C._cuda_getCurrentRawStream


def _tensor(t, name: str, dtypes, ndim: int):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {tuple(t.shape)}")


def _dense(t, name: str, dtypes, shape, dev):
    _tensor(t, name, dtypes, len(shape))
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, the other operands on {dev}")


def _rows(t, name: str) -> int:
    """Row stride of a 2-D tensor whose rows are contiguous."""
    M, K = t.shape
    if K > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    return t.stride(0) if M > 1 else max(K, 1)


class _on:
    """The device and stream of a call: entered only where they are not the current ones."""

    __slots__ = ("guards",)

    def __init__(self, dev, stream):
        self.guards = []
        if dev.index != torch.cuda.current_device():
            self.guards.append(torch.cuda.device(dev))
        if stream is not None:
            if stream.device != dev:
                raise ValueError(f"stream is on {stream.device}, the operands on {dev}")
            self.guards.append(torch.cuda.stream(stream))

    def __enter__(self):
        for g in self.guards:
            g.__enter__()

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)


def fp8_quant_act(x: torch.Tensor, stream=None):
    """BF16 [M, K] (rows contiguous, any row stride that is a multiple of 8) ->
    (codes float8_e4m3fn [M, K], scales float32 [ceil(K/128), M])."""
    _tensor(x, "x", (_BF16,), 2)
    M, K = x.shape
    ld = _rows(x, "x")
    dev = x.device
    with _on(dev, stream):
        codes = torch.empty((M, K), dtype=_FP8, device=dev)
        scales = torch.empty(((K + 127) // 128, M), dtype=_F32, device=dev)
        _check("biloco_fp8_quant_act", _lib.load().biloco_fp8_quant_act(
            x.data_ptr(), ld, M, K, codes.data_ptr(), scales.data_ptr(), _raw_stream(dev.index)))
    return codes, scales


def fp8_pack_weight(W: torch.Tensor, stream=None):
    """BF16 or float32 [N, K] or [E, N, K] -> (codes float8_e4m3fn of W's shape,
    scales float32 [(E,) ceil(N/128), ceil(K/128)])."""
    _tensor(W, "W", (_BF16, _F32), 3 if W.dim() == 3 else 2)
    if not W.is_contiguous():
        raise ValueError("W must be contiguous")
    N, K = W.shape[-2:]
    lead = tuple(W.shape[:-2])
    dev = W.device
    with _on(dev, stream):
        codes = torch.empty(W.shape, dtype=_FP8, device=dev)
        scales = torch.empty((*lead, (N + 127) // 128, (K + 127) // 128), dtype=_F32, device=dev)
        _check("biloco_fp8_pack_weight", _lib.load().biloco_fp8_pack_weight(
            W.data_ptr(), _TYPE[W.dtype], lead[0] if lead else 1, N, K, codes.data_ptr(), scales.data_ptr(),
            _raw_stream(dev.index)))
    return codes, scales


def fp8_gemm(x_codes: torch.Tensor, x_scales: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor,
             out: torch.Tensor | None = None, out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """y[m, n] = sum_b x_scales[b, m] w_scales[n/128, b] (x[m] . w[n])_b over blocks b of 128
    along K, for any number of rows; y is bfloat16 or float32."""
    _tensor(x_codes, "x_codes", (_FP8,), 2)
    _tensor(w_codes, "w_codes", (_FP8,), 2)
    M, K = x_codes.shape
    N = w_codes.shape[0]
    KB = (K + 127) // 128
    dev = x_codes.device
    _dense(x_codes, "x_codes", (_FP8,), (M, K), dev)
    _dense(x_scales, "x_scales", (_F32,), (KB, M), dev)
    _dense(w_codes, "w_codes", (_FP8,), (N, K), dev)
    _dense(w_scales, "w_scales", (_F32,), ((N + 127) // 128, KB), dev)
    if out is not None:
        out_dtype = out.dtype
        _dense(out, "out", (_BF16, _F32), (M, N), dev)
    elif out_dtype not in _TYPE:
        raise ValueError(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
    with _on(dev, stream):
        if out is None:
            out = torch.empty((M, N), dtype=out_dtype, device=dev)
        _check("biloco_fp8_gemm", _lib.load().biloco_fp8_gemm(
            x_codes.data_ptr(), x_scales.data_ptr(), w_codes.data_ptr(), w_scales.data_ptr(), out.data_ptr(),
            _TYPE[out_dtype], M, N, K, _raw_stream(dev.index)))
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
    `quant` (as fp8_quant_act lays them out), or h' alone without pre_weight.  out_h may
    be h itself."""
    if y is None and h is None:
        raise ValueError("y or h must be given")
    if y is None and (post_weight is not None or gate is not None):
        raise ValueError("post_weight and gate act on y, which is None")
    if quant and pre_weight is None:
        raise ValueError("quant needs pre_weight")
    ref = h if y is None else y
    if y is not None:
        _tensor(y, "y", (_BF16,), 2)
    if h is not None:
        _tensor(h, "h", (_BF16, _F32), 2)
    M, D = ref.shape
    dev = ref.device
    if h is not None and (h.shape != (M, D) or h.device != dev):
        raise ValueError(f"h must be {(M, D)} on {dev}")
    ldy = 0 if y is None else _rows(y, "y")
    ldh = 0 if h is None else _rows(h, "h")
    h_dtype = _BF16 if h is None else h.dtype
    w_dtype = _BF16
    for w, name in ((post_weight, "post_weight"), (pre_weight, "pre_weight")):
        if w is not None:
            _dense(w, name, (_BF16, _F32), (D,), dev)
            w_dtype = w.dtype
    if post_weight is not None and pre_weight is not None and post_weight.dtype != pre_weight.dtype:
        raise ValueError("post_weight and pre_weight must have one type")
    G, g_type = 1, 0
    if gate is not None:
        G = gate.shape[0] if gate.dim() == 2 else 1
        _dense(gate, "gate", (_BF16, _F32), (G, D) if gate.dim() == 2 else (D,), dev)
        if G < 1 or M % G:
            raise ValueError(f"gate has {G} rows, which do not divide {M}")
        g_type = _TYPE[gate.dtype]
    if out_h is not None:
        _tensor(out_h, "out_h", (h_dtype,), 2)
        if out_h.shape != (M, D) or out_h.device != dev:
            raise ValueError(f"out_h must be {(M, D)} on {dev}")
    with _on(dev, stream):
        if out_h is None:
            out_h = torch.empty((M, D), dtype=h_dtype, device=dev)
        x = codes = scales = None
        if quant:
            codes = torch.empty((M, D), dtype=_FP8, device=dev)
            scales = torch.empty(((D + 127) // 128, M), dtype=_F32, device=dev)
        elif pre_weight is not None:
            x = torch.empty((M, D), dtype=_BF16, device=dev)
        _check("biloco_block_norm", _lib.load().biloco_block_norm(
            y if y is None else y.data_ptr(), ldy, h if h is None else h.data_ptr(), ldh, _TYPE[h_dtype],
            None if post_weight is None else post_weight.data_ptr(),
            None if pre_weight is None else pre_weight.data_ptr(), _TYPE[w_dtype],
            None if gate is None else gate.data_ptr(), g_type, G, res_scale, offset, eps, M, D, out_h.data_ptr(),
            _rows(out_h, "out_h"), None if x is None else x.data_ptr(), None if codes is None else codes.data_ptr(),
            None if scales is None else scales.data_ptr(), _raw_stream(dev.index)))
    if quant:
        return out_h, codes, scales
    return out_h if x is None else (out_h, x)


_SCORE = {"softmax": 0, "sigmoid": 1}


def fp8_moe(x: torch.Tensor, router: torch.Tensor, w13: torch.Tensor, w13_scales: torch.Tensor, w2: torch.Tensor,
            w2_scales: torch.Tensor, top_k: int, *, score: str = "softmax", bias: torch.Tensor | None = None,
            renorm: bool = True, route_scale: float = 1.0, stream=None):
    """A whole mixture-of-experts layer for up to 64 tokens:

        y[t] = sum over t's top_k experts e of weight[t, e] W2_e (silu(W1_e x[t]) * (W3_e x[t]))

    x bfloat16 [T, D]; router bfloat16 or float32 [E, D]; w13 [n, 2F, D] ([W1; W3] stacked)
    and w2 [n, D, F] with their scales from fp8_pack_weight.  The n - E last experts are
    shared: they serve every token with weight 1.  `score` is "softmax" (over the experts)
    or "sigmoid"; bias float32 [E] is added for the choice only.  Returns (y bfloat16
    [T, D], ids int32 [T, top_k], weights float32 [T, top_k])."""
    _tensor(x, "x", (_BF16,), 2)
    _tensor(router, "router", (_BF16, _F32), 2)
    _tensor(w13, "w13", (_FP8,), 3)
    T, D = x.shape
    E, n, F = router.shape[0], w13.shape[0], w13.shape[1] // 2
    dev = x.device
    ld = _rows(x, "x")
    KD, KF = (D + 127) // 128, (F + 127) // 128
    _dense(router, "router", (_BF16, _F32), (E, D), dev)
    _dense(w13, "w13", (_FP8,), (n, 2 * F, D), dev)
    _dense(w13_scales, "w13_scales", (_F32,), (n, (2 * F + 127) // 128, KD), dev)
    _dense(w2, "w2", (_FP8,), (n, D, F), dev)
    _dense(w2_scales, "w2_scales", (_F32,), (n, KD, KF), dev)
    if n < E:
        raise ValueError(f"router has {E} experts, w13 {n}")
    if bias is not None:
        _dense(bias, "bias", (_F32,), (E,), dev)
    if not 1 <= top_k <= E:
        raise ValueError(f"top_k must be 1 to {E}, got {top_k}")
    if score not in _SCORE:
        raise ValueError(f"score must be one of {sorted(_SCORE)}, got {score!r}")
    lib = _lib.load()
    with _on(dev, stream):
        y = torch.empty((T, D), dtype=_BF16, device=dev)
        ids = torch.empty((T, top_k), dtype=torch.int32, device=dev)
        weights = torch.empty((T, top_k), dtype=_F32, device=dev)
        nbytes = lib.biloco_fp8_moe_workspace_bytes(T, D, F, top_k, n - E) if T else 1
        if nbytes == 0:
            raise _lib.BilocoError("biloco_fp8_moe_workspace_bytes", _lib.ERR_SHAPE)
        ws = torch.empty((nbytes,), dtype=torch.uint8, device=dev)
        _check("biloco_fp8_moe", lib.biloco_fp8_moe(
            x.data_ptr(), ld, router.data_ptr(), _TYPE[router.dtype], None if bias is None else bias.data_ptr(),
            w13.data_ptr(), w13_scales.data_ptr(), w2.data_ptr(), w2_scales.data_ptr(), T, D, F, E, top_k, n - E,
            _SCORE[score], int(renorm), route_scale, y.data_ptr(), ids.data_ptr(), weights.data_ptr(), ws.data_ptr(),
            nbytes, _raw_stream(dev.index)))
    return y, ids, weights
