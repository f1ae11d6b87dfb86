"""Binding of the 8-bit rows and products and of the rows sorted by expert
(their section of include/qgemm.h).  Argument checks and one call each.

A call costs a few microseconds of host time, which bounds the small ones, so
the checks ask the tensors for little, and the raw stream (0.1 us) rather than
a Stream object (2 us) is taken.

`stream` is a torch.cuda.Stream of the tensors' device, the current one if not
given.  A call on another stream than the current one is ordered against
nothing else: the caller has it wait for the inputs' producers, keeps tensors
of other streams alive until it has run (Tensor.record_stream), and has the
consumers wait for it.  Outputs that a function allocates belong to the stream
of the call."""

from __future__ import annotations

from contextlib import nullcontext

import torch

from . import FORMATS, OK, _check, lib, weight_bytes

_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_DTYPES = {torch.float32: 0, torch.bfloat16: 1}
_OUT = {"f32": torch.float32, "bf16": torch.bfloat16}
_I32, _F32, _I8, _U8 = torch.int32, torch.float32, torch.int8, torch.uint8
_LIB = lib()
_CURRENT = nullcontext()


# ------------------------------------------------------------ arguments

def _on(stream):
    """Where a call's outputs are allocated: they belong to the stream that it
    is launched on, like tensors made under torch.cuda.stream(stream)."""
    return _CURRENT if stream is None else torch.cuda.stream(stream)


def _gpu(t):
    """Index of a tensor's GPU."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensors must be on a CUDA (HIP) device")
    return dev


def _addr(t, name, dev):
    """Address of a contiguous tensor on GPU dev."""
    if t.get_device() != dev:
        raise ValueError("%s must be on the CUDA (HIP) device of the others" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _call(f, dev, stream, *args):
    """One call of an entry point, whose last argument is the stream, with GPU
    dev as the current device: kernels, the status word and streams are its."""
    if _current_device() != dev:
        before = _current_device()
        torch.cuda.set_device(dev)
        try:
            return _call(f, dev, stream, *args)
        finally:
            torch.cuda.set_device(before)
    if stream is None:
        raw = _raw_stream(dev)
    elif stream.device_index != dev:
        raise ValueError("stream must be on the CUDA (HIP) device of the tensors")
    else:
        raw = stream.cuda_stream
    status = f(*args, raw)
    if status != OK:
        _check(status)


def _dtype(t, name):
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise TypeError("%s must be float32 or bfloat16, not %s" % (name, t.dtype))
    return dt


def _rows(t, name):
    """(rows, columns) of a matrix."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError("%s must be a matrix, not %s" % (name, tuple(shape)))
    return shape


def _rows_like(t, like, cols, name):
    """Rows of a matrix of `cols` columns and like's type."""
    if t.dtype != like.dtype:
        raise TypeError("dtype mismatch: %s %s" % (name, t.dtype))
    n, c = _rows(t, name)
    if c != cols:
        raise ValueError("%s must be rows of %d" % (name, cols))
    return n


def _topk(pos, T):
    shape = pos.shape
    if pos.dtype != _I32 or len(shape) != 2 or shape[0] != T:
        raise TypeError("pos must be int32 [T][topk]")
    return shape[1]


def _weights(w, pos, name="weights"):
    if w.dtype != _F32 or w.shape != pos.shape:
        raise TypeError("%s must be float32 [T][topk]" % name)


def code_stride(K: int) -> int:
    """The pitch at which quantize_rows allocates rows of K codes."""
    return (K + 15) // 16 * 16


def new_codes(R, K, device):
    return torch.empty((R, code_stride(K)), dtype=_I8, device=device)[:, :K]


def _codes(codes, scales, K, written=False):
    """(rows, pitch) of a tensor of codes, checked with its scales.  Rows that
    are written get zeros up to their pitch, so that has to be theirs."""
    if codes.dtype != _I8 or scales.dtype != _F32:
        raise TypeError("codes must be int8 and scales float32, not %s and %s" % (codes.dtype, scales.dtype))
    B, cols = _rows(codes, "codes")
    if cols != K:
        raise ValueError("codes must be rows of %d" % K)
    ldc, step = codes.stride()
    # one row, or none, carries no pitch of its own; one without padding is read
    # with the bytes behind it, which do not matter, but not written with them
    if B <= 1 and not (B and written and K % 16 and ldc < code_stride(K)):
        ldc = max(ldc, code_stride(K))
    if (step != 1 and K > 1) or ldc % 16 or ldc < K:
        raise ValueError("codes must be rows of stride 1 at a pitch that is a multiple of 16 and at least K")
    if B and codes.untyped_storage().nbytes() - codes.storage_offset() < B * ldc:
        raise ValueError("the last row of codes must have room for its whole pitch (%d bytes)" % ldc)
    if scales.numel() < B:
        raise ValueError("scales too small")
    return B, ldc


def _codes_addr(codes, dev):
    if codes.get_device() != dev:
        raise ValueError("codes must be on the CUDA (HIP) device of the others")
    return codes.data_ptr()


# ------------------------------------------------------------- products

def _workspace(plan, workspace, B, dev, stream):
    """(address, bytes) of a call's workspace: the caller's, none, or ("auto")
    the plan's, asked for again only when the width, the device or the stream
    is not the last eager call's.  A captured call always asks and leaves no
    answer behind: the plan does not record the capture's stream for it, which
    the next eager call on that stream has to have done."""
    if workspace is None:
        return 0, 0
    if not isinstance(workspace, str):
        return _addr(workspace, "workspace", dev), workspace.numel()
    if B == 0:
        return 0, 0
    key = (B, dev, _raw_stream(dev) if stream is None else stream.cuda_stream)
    last = plan.__dict__.get("_ws_last")
    capturing = torch.cuda.is_current_stream_capturing()
    if last is None or last[0] != key or capturing:
        st = torch.cuda.current_stream(dev) if stream is None else stream
        ws = plan._workspace(B, torch.device("cuda", dev), st)
        if ws is None:  # a width or a plan that the library refuses
            return 0, 0
        last = (key, ws.data_ptr(), ws.numel())
        plan._ws_last = None if capturing else last
    return last[1], last[2]


def run(plan, x, w, y, stream, B, workspace):
    """Plan.run of int8 weights: the rows are quantised into the workspace."""
    dev = _gpu(x)
    wsp, wsn = _workspace(plan, workspace, B, dev, stream)
    _call(_LIB.qgemm_run_ws, dev, stream, plan._h, B, _addr(w, "w", dev), _addr(x, "x", dev), _addr(y, "y", dev),
          wsp, wsn)
    return y


def run_codes(plan, codes, scales, w, y, stream, workspace):
    B, ldc = _codes(codes, scales, plan.K)
    if y.dtype != _OUT[plan.out] or w.dtype != _U8:
        raise TypeError("dtype mismatch: w %s, y %s" % (w.dtype, y.dtype))
    if y.numel() < B * plan.out_cols:
        raise ValueError("y too small for B")
    if w.numel() < plan.weight_bytes:
        raise ValueError("packed weight buffer too small")
    dev = _gpu(codes)
    if isinstance(workspace, str) and plan.tier(B) == "skinny":
        workspace = None  # nothing to split
    wsp, wsn = _workspace(plan, workspace, B, dev, stream)
    _call(_LIB.qgemm_run_codes, dev, stream, plan._h, B, _addr(w, "w", dev), codes.data_ptr(), ldc,
          _addr(scales, "scales", dev), _addr(y, "y", dev), wsp, wsn)
    return y


def run_grouped_codes(plan, codes, scales, w_table, offsets, y, stream):
    T, ldc = _codes(codes, scales, plan.K)
    E = w_table.numel()
    if y.dtype != _OUT[plan.out]:
        raise TypeError("dtype mismatch: y %s" % y.dtype)
    if w_table.dtype != torch.int64 or offsets.dtype != _I32 or offsets.numel() != E + 1:
        raise TypeError("w_table must be int64 [E], offsets int32 [E + 1]")
    if y.numel() < T * plan.out_cols:
        raise ValueError("y too small")
    dev = _gpu(codes)
    _call(_LIB.qgemm_run_grouped_codes, dev, stream, plan._h, E, T, _addr(w_table, "w_table", dev),
          _addr(offsets, "offsets", dev), codes.data_ptr(), ldc, _addr(scales, "scales", dev), _addr(y, "y", dev))
    return y


def pack_int8(codes, scales, out=None, stream=None):
    """qgemm_pack_device: int8 codes [N][K] and float32 scales [N] on the GPU
    to the packed buffer (uint8, allocated unless given)."""
    if codes.dtype != _I8 or scales.dtype != _F32:
        raise TypeError("codes must be int8 and scales float32, not %s and %s" % (codes.dtype, scales.dtype))
    N, K = _rows(codes, "codes")
    if scales.shape != codes.shape[:1]:
        raise ValueError("scales must be [N]")
    nbytes = weight_bytes("int8", N, K)
    if out is None:
        with _on(stream):
            out = torch.empty(nbytes, dtype=_U8, device=codes.device)
    if out.dtype != _U8 or out.numel() < nbytes:
        raise ValueError("out must be uint8, at least %d bytes" % nbytes)
    dev = _gpu(codes)
    _call(_LIB.qgemm_pack_device, dev, stream, FORMATS["int8"], N, K, _addr(codes, "codes", dev),
          _addr(scales, "scales", dev), _addr(out, "out", dev), out.numel())
    return out


def quantize_rows(x, codes=None, scales=None, stream=None):
    """qgemm_quantize_rows: float32 or bfloat16 rows x [B][K] to int8 codes
    [B][K] (at a pitch of code_stride(K)) and float32 scales [B]; outputs are
    allocated unless given.  Codes at a larger pitch get zeros up to it."""
    dt = _dtype(x, "x")
    B, K = _rows(x, "x")
    if codes is None or scales is None:
        with _on(stream):
            if codes is None:
                codes = new_codes(B, K, x.device)
            if scales is None:
                scales = torch.empty(B, dtype=_F32, device=x.device)
    rows, ldc = _codes(codes, scales, K, True)
    if rows != B:
        raise ValueError("codes must have x's rows")
    dev = _gpu(x)
    _call(_LIB.qgemm_quantize_rows, dev, stream, dt, B, K, _addr(x, "x", dev), _codes_addr(codes, dev), ldc,
          _addr(scales, "scales", dev))
    return codes, scales


# ------------------------------------------------- rows sorted by expert

def route(ids, E: int, offsets=None, pos=None, stream=None):
    """qgemm_route: the router's choices ids (int32 [T][topk]; ids outside
    0..E-1 are dropped) to the offsets (int32 [E + 1]) that run_grouped and
    run_grouped_codes take and the sorted row of each choice, pos (int32
    [T][topk], -1 for a dropped one); outputs are allocated unless given."""
    shape = ids.shape
    if ids.dtype != _I32 or len(shape) != 2:
        raise TypeError("ids must be int32 [T][topk]")
    if offsets is None or pos is None:
        with _on(stream):
            if offsets is None:
                offsets = torch.empty(E + 1, dtype=_I32, device=ids.device)
            if pos is None:
                pos = torch.empty_like(ids)
    if offsets.dtype != _I32 or pos.dtype != _I32:
        raise TypeError("offsets and pos must be int32")
    if offsets.numel() != E + 1 or pos.shape != shape:
        raise ValueError("offsets must be [E + 1], pos as ids")
    dev = _gpu(ids)
    _call(_LIB.qgemm_route, dev, stream, E, shape[0], shape[1], _addr(ids, "ids", dev),
          _addr(offsets, "offsets", dev), _addr(pos, "pos", dev))
    return offsets, pos


def dispatch(x, pos, xs, stream=None):
    """qgemm_dispatch: xs[pos[t][j]] = x[t], x [T][H] and xs [R][H] float32
    or bfloat16.  Rows of xs that no choice names are left as they were."""
    dt = _dtype(x, "x")
    T, H = _rows(x, "x")
    R = _rows_like(xs, x, H, "xs")
    k = _topk(pos, T)
    dev = _gpu(x)
    _call(_LIB.qgemm_dispatch, dev, stream, dt, T, k, H, R, _addr(x, "x", dev), _addr(pos, "pos", dev),
          _addr(xs, "xs", dev))
    return xs


def dispatch_codes(x, pos, codes, scales, stream=None):
    """qgemm_dispatch_codes: quantize_rows and dispatch in one pass: x [T][K]
    to the sorted rows of codes [R][K] and scales [R]."""
    dt = _dtype(x, "x")
    T, K = _rows(x, "x")
    k = _topk(pos, T)
    R, ldc = _codes(codes, scales, K, True)
    dev = _gpu(x)
    _call(_LIB.qgemm_dispatch_codes, dev, stream, dt, T, k, K, R, _addr(x, "x", dev), _addr(pos, "pos", dev),
          _codes_addr(codes, dev), ldc, _addr(scales, "scales", dev))
    return codes, scales


def combine(ys, pos, weights, y, stream=None):
    """qgemm_combine: y[t] = sum_j weights[t][j] * ys[pos[t][j]], ys [R][H]
    and y [T][H] float32 or bfloat16, weights float32 [T][topk] or None (ones)."""
    dt = _dtype(ys, "ys")
    R, H = _rows(ys, "ys")
    T = _rows_like(y, ys, H, "y")
    k = _topk(pos, T)
    if weights is not None:
        _weights(weights, pos)
    dev = _gpu(ys)
    _call(_LIB.qgemm_combine, dev, stream, dt, T, k, H, R, _addr(ys, "ys", dev), _addr(pos, "pos", dev),
          None if weights is None else _addr(weights, "weights", dev), _addr(y, "y", dev))
    return y


def dispatch_grad(dxs, pos, dx, stream=None):
    """The gradient of dispatch: dx[t] = sum_j dxs[pos[t][j]]."""
    return combine(dxs, pos, None, dx, stream)


def combine_grad(dy, ys, pos, weights, dys, dw, stream=None):
    """qgemm_combine_grad: dys[pos[t][j]] = weights[t][j] * dy[t] and
    dw[t][j] = dy[t] . ys[pos[t][j]] (float32, 0 for a dropped choice); rows
    of dys that no choice names are left as they were."""
    dt = _dtype(dy, "dy")
    T, H = _rows(dy, "dy")
    R = _rows_like(ys, dy, H, "ys")
    if _rows_like(dys, dy, H, "dys") != R:
        raise ValueError("dys must have ys's rows")
    k = _topk(pos, T)
    _weights(weights, pos)
    _weights(dw, pos, "dw")
    dev = _gpu(dy)
    _call(_LIB.qgemm_combine_grad, dev, stream, dt, T, k, H, R, _addr(dy, "dy", dev), _addr(ys, "ys", dev),
          _addr(pos, "pos", dev), _addr(weights, "weights", dev), _addr(dys, "dys", dev), _addr(dw, "dw", dev))
    return dys, dw
