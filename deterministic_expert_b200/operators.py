"""Handle-free expert-layer operators: routing and its gradient, grouping, E4M3
quantisation with one scale per 128 elements, block-scaled E4M3 products, and the
weighted combine with its gradient (include/moe.h documents the entry points).

Like the rest of the binding these functions only check and marshal arguments.
Outputs are allocated where they are not given; ``stream`` (default: the current
stream of the tensors' device) is where the kernels run, and where outputs are
allocated.  A stream that is given does not wait for the current one: the caller
orders them (``wait_stream``) before the call, and before outputs are used elsewhere;
the call's tensors may be dropped at once, their memory is kept until that stream is
done with it (a stream given by its raw handle has to outlive them).  Tensors of a call live on one CUDA device, which need not be the
current one.

Autograd does not see these calls: gradients are operators of their own
(``route_backward``, ``combine_rows_backward``, ...).  A tensor that requires a
gradient is refused while gradients are recorded; pass it detached, or call under
``torch.no_grad()`` or in an ``autograd.Function``.
"""
from __future__ import annotations

import ctypes
import functools

import torch

import deterministic_expert_b200 as _moe

DTYPE_BF16, DTYPE_F32 = 0, 1
_DTYPES = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}
BLOCK = 128          # elements that share a scale


class moe_route_config(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int), ("k", ctypes.c_int), ("scores", ctypes.c_int), ("n_groups", ctypes.c_int),
                ("topk_groups", ctypes.c_int), ("group_top", ctypes.c_int), ("renormalize", ctypes.c_int),
                ("routed_scale", ctypes.c_float), ("logits_dtype", ctypes.c_int)]


class moe_glu_config(ctypes.Structure):
    _fields_ = [("activation", ctypes.c_int), ("gate_clamp_max", ctypes.c_float), ("up_clamp", ctypes.c_float),
                ("situ_beta_gate", ctypes.c_float), ("situ_beta_up", ctypes.c_float)]


_vp, _i, _ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong
ARGTYPES = {
    "moe_route": [ctypes.POINTER(moe_route_config), _i, _vp, _ll, _vp, _vp, _vp, _vp],
    "moe_route_backward": [ctypes.POINTER(moe_route_config), _i, _vp, _ll, _vp, _vp, _vp, _ll, _vp],
    "moe_group_rows": [_i, _i, _i, _vp, _vp, _vp, _vp, _vp],
    "moe_quantize_rows_fp8": [_i, _i, _vp, _i, _ll, _i, _vp, _vp, _vp, _vp, _ll, _vp],
    "moe_quantize_weights_fp8": [_i, _i, _i, _vp, _vp, _vp, _vp],
    "moe_glu_quantize_fp8": [ctypes.POINTER(moe_glu_config), _i, _i, _vp, _ll, _vp, _vp, _vp, _ll, _vp],
    "moe_glu_backward_quantize_fp8": [ctypes.POINTER(moe_glu_config), _i, _i, _vp, _ll, _vp, _ll, _vp, _vp, _vp,
                                      _ll, _vp],
    "moe_matmul_fp8": [_i, _i, _vp, _i, _i, _i, _vp, _vp, _ll, _vp, _vp, _vp, _i, _ll, _vp],
    "moe_combine_rows": [_i, _i, _i, _i, _vp, _i, _ll, _vp, _vp, _vp, _vp, _i, _vp],
    "moe_combine_rows_backward": [_i, _i, _i, _i, _vp, _vp, _i, _ll, _vp, _vp, _vp, _vp, _vp],
    "moe_get_operator_error": [_vp],
    "moe_selftest_matmul_timeout": [_i, _i, _i, _i, _vp],
}
_fns: dict = {}
_Tensor = torch.Tensor
_grad_enabled = torch.is_grad_enabled
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _fn(name):
    f = _fns.get(name)
    if f is None:
        f = getattr(_moe.lib(), name)
        f.argtypes = ARGTYPES[name]
        _fns[name] = f
    return f


def _call(name, device, stream, used, *args):
    """Run an entry point with the tensors' device current, on `stream`; `used`: its
    tensors (or None), which the allocator keeps for a stream that is not theirs."""
    f = _fns.get(name) or _fn(name)
    if stream is None:
        s = _raw_stream(device.index)
    else:
        s = _handle(stream)
        on = _moe._torch_stream(stream, device)
        for t in used:
            if t is not None:
                t.record_stream(on)
    if device.index == torch.cuda.current_device():
        rc = f(*args, s)
    else:
        with torch.cuda.device(device):
            rc = f(*args, s)
    if rc != 0:
        raise _moe.MoEError(rc, name)


def _handle(stream):
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _empty(stream, device, *specs):
    """New tensors (shape, dtype); they belong to the stream that writes them."""
    if stream is None:
        return [torch.empty(shape, dtype=dtype, device=device) for shape, dtype in specs]
    with torch.cuda.stream(_moe._torch_stream(stream, device)):
        return [torch.empty(shape, dtype=dtype, device=device) for shape, dtype in specs]


def _need(cond, what):
    if not cond:
        raise ValueError(what)


def _tensor(t, name, device, dtypes, shape=None, contiguous=True):
    """Refuse a tensor the library would read or write wrongly."""
    if (isinstance(t, _Tensor) and t.is_cuda and (device is None or t.device == device) and t.dtype in dtypes
            and (shape is None or t.shape == shape) and (not contiguous or t.is_contiguous())
            and not (t.requires_grad and _grad_enabled())):
        return
    _need(isinstance(t, _Tensor), f"{name}: expected a tensor")
    _need(not (t.requires_grad and _grad_enabled()),
          f"{name}: requires a gradient, which this call would not record: detach it, or call under torch.no_grad()")
    _need(t.is_cuda and (device is None or t.device == device),
          f"{name}: expected a CUDA tensor" + (f" on {device}, got {t.device}" if device is not None else ""))
    _need(t.dtype in dtypes, f"{name}: expected {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    _need(shape is None or t.shape == shape, f"{name}: expected shape {shape}, got {tuple(t.shape)}")
    raise ValueError(f"{name}: expected a contiguous tensor")


def _rows(t, name):
    """Row pitch of a matrix whose rows are dense."""
    if t.dim() == 2:
        rows, width = t.shape
        pitch, step = t.stride()
        if width <= 1 or step == 1:
            if rows <= 1:
                return max(width, 1)
            if pitch >= width:
                return pitch
    _need(t.dim() == 2, f"{name}: expected two dimensions, got {t.dim()}")
    _need(t.shape[1] <= 1 or t.stride(1) == 1, f"{name}: expected rows of neighbouring elements")
    raise ValueError(f"{name}: rows overlap")


_CODES = (torch.uint8, torch.float8_e4m3fn)
_I32, _F32, _BF16 = (torch.int32,), (torch.float32,), (torch.bfloat16,)


@functools.lru_cache(maxsize=256)
def _route_struct(E, k, dtype, softmax, n_groups, topk_groups, group_top, renormalize, routed_scale):
    return moe_route_config(E, k, _moe.ROUTER_SOFTMAX if softmax else _moe.ROUTER_SIGMOID_BIAS, n_groups, topk_groups,
                            group_top, renormalize, routed_scale, _DTYPES[dtype])


def _route_config(E, k, dtype, scores, n_groups, topk_groups, group_top, renormalize, routed_scale):
    _need(scores == "softmax" or scores == "sigmoid", f"scores: expected 'softmax' or 'sigmoid', got {scores!r}")
    # Plain numbers only: the structures are kept by value.
    return _route_struct(E, int(k), dtype, scores == "softmax", int(n_groups), int(topk_groups), int(group_top),
                         1 if renormalize else 0, float(routed_scale))


def route(logits, k: int, *, scores: str = "softmax", bias=None, n_groups: int = 1, topk_groups: int = 1,
          group_top: int = 2, renormalize: bool = False, routed_scale: float = 1.0, out_idx=None, out_w=None,
          stream=None):
    """moe_route: the k experts of every row of ``logits`` [T, E] (bf16 or fp32) and
    their weights: (idx int32 [T, k], w fp32 [T, k])."""
    _tensor(logits, "logits", None, tuple(_DTYPES), contiguous=False)
    ld = _rows(logits, "logits")
    dev = logits.device
    T, E = int(logits.shape[0]), int(logits.shape[1])
    if bias is not None:
        _tensor(bias, "bias", dev, _F32, (E,))
    cfg = _route_config(E, k, logits.dtype, scores, n_groups, topk_groups, group_top, renormalize, routed_scale)
    _need(cfg.k >= 0, "k: negative")
    if out_idx is None:
        out_idx, = _empty(stream, dev, ((T, cfg.k), torch.int32))
    else:
        _tensor(out_idx, "out_idx", dev, _I32, (T, cfg.k))
    if out_w is None:
        out_w, = _empty(stream, dev, ((T, cfg.k), torch.float32))
    else:
        _tensor(out_w, "out_w", dev, _F32, (T, cfg.k))
    _call("moe_route", dev, stream, (logits, bias, out_idx, out_w),
          ctypes.byref(cfg), T, logits.data_ptr(), ld,
          None if bias is None else bias.data_ptr(), out_idx.data_ptr(), out_w.data_ptr())
    return out_idx, out_w


def route_backward(logits, idx, dw, *, scores: str = "softmax", n_groups: int = 1, topk_groups: int = 1,
                   group_top: int = 2, renormalize: bool = False, routed_scale: float = 1.0, out=None, stream=None):
    """moe_route_backward: the gradient of ``logits`` from ``dw``, that of the weights
    ``route`` gave for the experts ``idx`` with the same arguments."""
    _tensor(logits, "logits", None, tuple(_DTYPES), contiguous=False)
    ld = _rows(logits, "logits")
    dev = logits.device
    T, E = int(logits.shape[0]), int(logits.shape[1])
    _need(idx.dim() == 2, "idx: expected two dimensions")
    k = int(idx.shape[1])
    _tensor(idx, "idx", dev, _I32, (T, k))
    _tensor(dw, "dw", dev, _F32, (T, k))
    cfg = _route_config(E, k, logits.dtype, scores, n_groups, topk_groups, group_top, renormalize, routed_scale)
    if out is None:
        out, = _empty(stream, dev, ((T, E), logits.dtype))
    _tensor(out, "out", dev, (logits.dtype,), (T, E), contiguous=False)
    _call("moe_route_backward", dev, stream, (logits, idx, dw, out),
          ctypes.byref(cfg), T, logits.data_ptr(), ld, idx.data_ptr(),
          dw.data_ptr(), out.data_ptr(), _rows(out, "out"))
    return out


def group_rows(idx, E: int, *, out=None, stream=None):
    """moe_group_rows: ``idx`` [T, k] int32 -> (offsets [E + 1], token_of_row [T k],
    row_of_slot [T, k]), all int32.  ``out``: the three tensors to write."""
    _tensor(idx, "idx", None, _I32)
    _need(idx.dim() == 2, "idx: expected two dimensions")
    dev = idx.device
    T, k = int(idx.shape[0]), int(idx.shape[1])
    if out is None:
        offsets, token_of_row, row_of_slot = _empty(stream, dev, ((max(int(E), 0) + 1,), torch.int32),
                                                    ((T * k,), torch.int32), ((T, k), torch.int32))
    else:
        offsets, token_of_row, row_of_slot = out
        _tensor(offsets, "offsets", dev, _I32, (int(E) + 1,))
        _tensor(token_of_row, "token_of_row", dev, _I32, (T * k,))
        _tensor(row_of_slot, "row_of_slot", dev, _I32, (T, k))
    _call("moe_group_rows", dev, stream, (idx, offsets, token_of_row, row_of_slot),
          T, k, int(E), idx.data_ptr(), offsets.data_ptr(), token_of_row.data_ptr(),
          row_of_slot.data_ptr())
    return offsets, token_of_row, row_of_slot


def _quant_out(R, K, out_codes, out_scales, dev, stream):
    nb = -(-K // BLOCK)
    if out_codes is None:
        out_codes, = _empty(stream, dev, ((R, K), torch.uint8))
    else:
        _tensor(out_codes, "out_codes", dev, _CODES, (R, K))
    if out_scales is None:
        out_scales, = _empty(stream, dev, ((nb, R), torch.float32))
    else:
        _tensor(out_scales, "out_scales", dev, _F32, (nb, R), contiguous=False)
    return out_codes, out_scales, _rows(out_scales, "out_scales")


def _count(n_rows, dev):
    if n_rows is None:
        return None
    _tensor(n_rows, "n_rows", dev, _I32)
    _need(n_rows.numel() == 1, "n_rows: expected one element")
    return n_rows.data_ptr()


def quantize_rows_fp8(x, *, token_of_row=None, n_rows=None, out_codes=None, out_scales=None, stream=None):
    """moe_quantize_rows_fp8: rows of ``x`` [M, K] (bf16 or fp32; row r from row
    token_of_row[r] if given) -> (E4M3 codes uint8 [R, K], scales fp32
    [ceil(K / 128), R])."""
    _tensor(x, "x", None, tuple(_DTYPES), contiguous=False)
    ld = _rows(x, "x")
    dev = x.device
    M, K = int(x.shape[0]), int(x.shape[1])
    R = M
    if token_of_row is not None:
        _need(token_of_row.dim() == 1, "token_of_row: expected one dimension")
        _tensor(token_of_row, "token_of_row", dev, _I32)
        R = int(token_of_row.shape[0])
    out_codes, out_scales, ld_s = _quant_out(R, K, out_codes, out_scales, dev, stream)
    _call("moe_quantize_rows_fp8", dev, stream, (x, token_of_row, n_rows, out_codes, out_scales),
          R, K, x.data_ptr(), _DTYPES[x.dtype], ld, M,
          None if token_of_row is None else token_of_row.data_ptr(), _count(n_rows, dev), out_codes.data_ptr(),
          out_scales.data_ptr(), max(ld_s, R))
    return out_codes, out_scales


def quantize_weights_fp8(w, *, out_codes=None, out_scales=None, stream=None):
    """moe_quantize_weights_fp8: bf16 weights [G, N, K] (or [N, K]) -> (E4M3 codes
    uint8 of the same shape, scales fp32 [G, ceil(N / 128), ceil(K / 128)])."""
    _tensor(w, "w", None, _BF16)
    _need(w.dim() in (2, 3), "w: expected two or three dimensions")
    dev = w.device
    N, K = int(w.shape[-2]), int(w.shape[-1])
    G = int(w.shape[0]) if w.dim() == 3 else 1
    sshape = tuple(w.shape[:-2]) + (-(-N // BLOCK), -(-K // BLOCK))
    if out_codes is None:
        out_codes, = _empty(stream, dev, (w.shape, torch.uint8))
    if out_scales is None:
        out_scales, = _empty(stream, dev, (sshape, torch.float32))
    _tensor(out_codes, "out_codes", dev, _CODES, w.shape)
    _tensor(out_scales, "out_scales", dev, _F32, sshape)
    _call("moe_quantize_weights_fp8", dev, stream, (w, out_codes, out_scales),
          G, N, K, w.data_ptr(), out_codes.data_ptr(), out_scales.data_ptr())
    return out_codes, out_scales


_glu_struct = functools.lru_cache(maxsize=256)(moe_glu_config)


def _glu_config(activation, gate_clamp_max, up_clamp, situ_beta_gate, situ_beta_up):
    # Plain numbers only: the structures are kept by value.
    return _glu_struct(int(activation), float(gate_clamp_max), float(up_clamp), float(situ_beta_gate),
                       float(situ_beta_up))


def _gate_up(gu):
    _tensor(gu, "gu", None, _BF16, contiguous=False)
    ld = _rows(gu, "gu")
    _need(gu.shape[1] % 2 == 0, "gu: expected [gate | up] columns")
    return ld, int(gu.shape[0]), int(gu.shape[1]) // 2


def glu_quantize_fp8(gu, *, activation: int = 0, gate_clamp_max: float = float("inf"), up_clamp: float = float("inf"),
                     situ_beta_gate: float = 4.0, situ_beta_up: float = 25.0, n_rows=None, out_codes=None,
                     out_scales=None, stream=None):
    """moe_glu_quantize_fp8: rows [gate | up] (bf16 [R, 2 I]) -> the gated unit as
    (E4M3 codes [R, I], scales [ceil(I / 128), R])."""
    ld, R, I = _gate_up(gu)
    dev = gu.device
    cfg = _glu_config(activation, gate_clamp_max, up_clamp, situ_beta_gate, situ_beta_up)
    out_codes, out_scales, ld_s = _quant_out(R, I, out_codes, out_scales, dev, stream)
    _call("moe_glu_quantize_fp8", dev, stream, (gu, n_rows, out_codes, out_scales),
          ctypes.byref(cfg), R, I, gu.data_ptr(), ld, _count(n_rows, dev),
          out_codes.data_ptr(), out_scales.data_ptr(), max(ld_s, R))
    return out_codes, out_scales


def glu_backward_quantize_fp8(gu, dh, *, activation: int = 0, gate_clamp_max: float = float("inf"),
                              up_clamp: float = float("inf"), situ_beta_gate: float = 4.0, situ_beta_up: float = 25.0,
                              n_rows=None, out_codes=None, out_scales=None, stream=None):
    """moe_glu_backward_quantize_fp8: the gradient of ``gu`` from ``dh`` (bf16 [R, I]),
    that of the gated unit, as (E4M3 codes [R, 2 I], scales [2 I / 128, R])."""
    ld, R, I = _gate_up(gu)
    dev = gu.device
    _tensor(dh, "dh", dev, _BF16, (R, I), contiguous=False)
    cfg = _glu_config(activation, gate_clamp_max, up_clamp, situ_beta_gate, situ_beta_up)
    out_codes, out_scales, ld_s = _quant_out(R, 2 * I, out_codes, out_scales, dev, stream)
    _call("moe_glu_backward_quantize_fp8", dev, stream, (gu, dh, n_rows, out_codes, out_scales),
          ctypes.byref(cfg), R, I, gu.data_ptr(), ld, dh.data_ptr(),
          _rows(dh, "dh"), _count(n_rows, dev), out_codes.data_ptr(), out_scales.data_ptr(), max(ld_s, R))
    return out_codes, out_scales


def matmul_fp8(a, a_scale, w, w_scale, *, offsets=None, transposed: bool = False, out=None,
               out_dtype=torch.bfloat16, stream=None):
    """moe_matmul_fp8: E4M3 rows ``a`` [M, K] with ``a_scale`` [ceil(K / 128), M] times
    E4M3 weights ``w`` [G, N, K] (or [N, K]) with ``w_scale`` [G, ceil(N / 128),
    ceil(K / 128)] -> [M, N]; transposed: ``a`` [M, N] -> [M, K].  ``offsets`` int32
    [G + 1]: the rows that meet each group."""
    _tensor(a, "a", None, _CODES)
    _need(a.dim() == 2, "a: expected two dimensions")
    dev = a.device
    _tensor(w, "w", dev, _CODES)
    _need(w.dim() in (2, 3), "w: expected two or three dimensions")
    M, con = int(a.shape[0]), int(a.shape[1])
    N, K = int(w.shape[-2]), int(w.shape[-1])
    G = int(w.shape[0]) if w.dim() == 3 else 1
    width = K if transposed else N
    _need(con == (N if transposed else K), f"a: expected {N if transposed else K} columns, got {con}")
    _tensor(a_scale, "a_scale", dev, _F32, (-(-con // BLOCK), M), contiguous=False)
    ld_as = _rows(a_scale, "a_scale")
    _tensor(w_scale, "w_scale", dev, _F32, tuple(w.shape[:-2]) + (-(-N // BLOCK), -(-K // BLOCK)))
    if offsets is not None:
        _tensor(offsets, "offsets", dev, _I32, (G + 1,))
    else:
        _need(G == 1, "offsets: needed with more than one group")
    if out is None:
        _need(out_dtype in _DTYPES, f"out_dtype: expected bfloat16 or float32, got {out_dtype}")
        out, = _empty(stream, dev, ((M, width), out_dtype))
    _tensor(out, "out", dev, tuple(_DTYPES), (M, width), contiguous=False)
    _call("moe_matmul_fp8", dev, stream, (a, a_scale, w, w_scale, offsets, out),
          1 if transposed else 0, G, None if offsets is None else offsets.data_ptr(),
          M, N, K, a.data_ptr(), a_scale.data_ptr(), max(ld_as, M), w.data_ptr(), w_scale.data_ptr(), out.data_ptr(),
          _DTYPES[out.dtype], max(_rows(out, "out"), width))
    return out


def _slots(row_of_slot, w, dev):
    _need(row_of_slot.dim() == 2, "row_of_slot: expected two dimensions")
    T, k = int(row_of_slot.shape[0]), int(row_of_slot.shape[1])
    _tensor(row_of_slot, "row_of_slot", dev, _I32, (T, k))
    if w is not None:
        _tensor(w, "w", dev, _F32, (T, k))
    return T, k


def combine_rows(y, row_of_slot, w=None, *, addend=None, out=None, out_dtype=torch.bfloat16, stream=None):
    """moe_combine_rows: out[t] = addend[t] + sum_j w[t, j] y[row_of_slot[t, j]]
    (``w`` None: every slot 1), fp32 sums, [T, D] of ``out_dtype``."""
    _tensor(y, "y", None, tuple(_DTYPES), contiguous=False)
    ld = _rows(y, "y")
    dev = y.device
    rows, D = int(y.shape[0]), int(y.shape[1])
    T, k = _slots(row_of_slot, w, dev)
    if addend is not None:
        _tensor(addend, "addend", dev, _BF16, (T, D))
    if out is None:
        _need(out_dtype in _DTYPES, f"out_dtype: expected bfloat16 or float32, got {out_dtype}")
        out, = _empty(stream, dev, ((T, D), out_dtype))
    _tensor(out, "out", dev, tuple(_DTYPES), (T, D))
    _call("moe_combine_rows", dev, stream, (y, row_of_slot, w, addend, out),
          T, k, D, rows, y.data_ptr(), _DTYPES[y.dtype], max(ld, D),
          row_of_slot.data_ptr(), None if w is None else w.data_ptr(),
          None if addend is None else addend.data_ptr(), out.data_ptr(), _DTYPES[out.dtype])
    return out


def combine_rows_backward(dout, y, row_of_slot, w=None, *, need_dw: bool = True, out_dy=None, out_dw=None,
                          stream=None):
    """moe_combine_rows_backward: (dy, dw) from ``dout`` (bf16 [T, D]), the gradient of
    ``combine_rows(y, row_of_slot, w)``; dy has the type of ``y``, dw is fp32 [T, k]
    (None with need_dw False)."""
    _tensor(y, "y", None, tuple(_DTYPES), contiguous=False)
    ld = _rows(y, "y")
    dev = y.device
    rows, D = int(y.shape[0]), int(y.shape[1])
    T, k = _slots(row_of_slot, w, dev)
    _tensor(dout, "dout", dev, _BF16, (T, D))
    if out_dy is None:
        # The pitch of y, as the entry point has one for both.
        out_dy, = _empty(stream, dev, ((rows, ld), y.dtype))
        if ld != D:
            out_dy = out_dy[:, :D]
    if need_dw and out_dw is None:
        out_dw, = _empty(stream, dev, ((T, k), torch.float32))
    _tensor(out_dy, "out_dy", dev, (y.dtype,), (rows, D), contiguous=False)
    _need(rows <= 1 or _rows(out_dy, "out_dy") == ld, "out_dy: expected the row pitch of y")
    if need_dw:
        _tensor(out_dw, "out_dw", dev, _F32, (T, k))
    _call("moe_combine_rows_backward", dev, stream, (dout, y, row_of_slot, w, out_dy, out_dw if need_dw else None),
          T, k, D, rows, dout.data_ptr(), y.data_ptr(), _DTYPES[y.dtype],
          max(ld, D), row_of_slot.data_ptr(), None if w is None else w.data_ptr(), out_dy.data_ptr(),
          out_dw.data_ptr() if need_dw else None)
    return out_dy, (out_dw if need_dw else None)


def operator_error(device=None, stream=None) -> int:
    """moe_get_operator_error on ``device`` (default: the current one): read and clear
    the error word of matmul_fp8.  Synchronises the stream."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(dev):
        s = _raw_stream(torch.cuda.current_device()) if stream is None else _handle(stream)
        return int(_fn("moe_get_operator_error")(s))


def selftest_matmul_timeout(M: int, N: int, K: int, load_blocks: int, stream=None) -> int:
    """moe_selftest_matmul_timeout on the current device: the status after a product
    whose loads stop early (MOE_ETIMEOUT: its bounded waits ran out)."""
    s = _raw_stream(torch.cuda.current_device()) if stream is None else _handle(stream)
    return int(_fn("moe_selftest_matmul_timeout")(M, N, K, load_blocks, s))
