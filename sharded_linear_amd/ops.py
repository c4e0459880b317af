"""Thin torch binding of the C ABI: argument marshalling only, every step runs in the HIP library.

Function names match the C entry points.  Tensors must be CUDA (HIP) tensors on one device,
contiguous, with the dtypes of include/sharded_linear.h; work is enqueued on torch's current
stream of that device.  Outputs not supplied are allocated with torch.empty (plumbing).
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from ._lib import check, lib

BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
SL_EALIGN, SL_ESHAPE, SL_EWORKSPACE = -2, -3, -4


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(dev):
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _want(t, name, dtype, shape, dev):
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == dev and t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _device(t):
    if not t.is_cuda:
        raise ValueError("the HIP library works on GPU tensors only; got a CPU tensor")
    return t.device


# knobs of sl_set_tuning, in the order of the header's SL_TUNE_* enum
TUNE_KNOBS = {"fwd": 0, "dgrad": 1, "wgrad": 2, "splitk": 3, "f8": 4}


def sl_set_tuning(knob: str, value: int) -> int:
    """Force a tuning choice (-1 restores the built-in one); returns the previous value."""
    prev = ctypes.c_int32(0)
    check("sl_set_tuning", lib().sl_set_tuning(TUNE_KNOBS[knob], int(value), ctypes.byref(prev)))
    return prev.value


@contextlib.contextmanager
def tuning(**knobs):
    """Within the block, force the given knobs (names of TUNE_KNOBS; ``gemm=n`` sets the tile
    configuration of all three bf16 products, so it takes 0..24; the forward-only 256x192
    configuration 25 is forced with ``fwd=25``); the previous values come back on exit."""
    if "gemm" in knobs:
        cfg = knobs.pop("gemm")
        knobs = {"fwd": cfg, "dgrad": cfg, "wgrad": cfg, **knobs}
    saved = []
    try:
        for k, v in knobs.items():
            saved.append((k, sl_set_tuning(k, v)))
        yield
    finally:
        for k, v in reversed(saved):
            sl_set_tuning(k, v)


def sl_grad_buffer_zero(grad_data: torch.Tensor) -> torch.Tensor:
    dev = _device(grad_data)
    _want(grad_data, "grad_data", F32, (grad_data.numel(),), dev)
    check("sl_grad_buffer_zero", lib().sl_grad_buffer_zero(_stream(dev), _ptr(grad_data), grad_data.numel()))
    return grad_data


def sl_linear_fwd(X: torch.Tensor, W: torch.Tensor, Y: torch.Tensor | None = None) -> torch.Tensor:
    """Y[T,out] = X[T,in] . W[out,in]^T (bf16)."""
    dev = _device(X)
    T, n_in = X.shape
    n_out = W.shape[0]
    _want(X, "X", BF16, (T, n_in), dev)
    _want(W, "W", BF16, (n_out, n_in), dev)
    if Y is None:
        Y = torch.empty((T, n_out), dtype=BF16, device=dev)
    _want(Y, "Y", BF16, (T, n_out), dev)
    check("sl_linear_fwd", lib().sl_linear_fwd(_stream(dev), _ptr(X), _ptr(W), _ptr(Y), T, n_in, n_out))
    return Y


def sl_linear_dgrad(dY: torch.Tensor, W: torch.Tensor, dX: torch.Tensor | None = None) -> torch.Tensor:
    """dX[T,in] = dY[T,out] . W[out,in] (bf16)."""
    dev = _device(dY)
    T, n_out = dY.shape
    n_in = W.shape[1]
    _want(dY, "dY", BF16, (T, n_out), dev)
    _want(W, "W", BF16, (n_out, n_in), dev)
    if dX is None:
        dX = torch.empty((T, n_in), dtype=BF16, device=dev)
    _want(dX, "dX", BF16, (T, n_in), dev)
    check("sl_linear_dgrad", lib().sl_linear_dgrad(_stream(dev), _ptr(dY), _ptr(W), _ptr(dX), T, n_in, n_out))
    return dX


def sl_wgrad_workspace_bytes(T: int, n_in: int, n_out: int) -> int:
    return int(lib().sl_wgrad_workspace_bytes(T, n_in, n_out))


def wgrad_workspace(dev: torch.device, nbytes: int) -> torch.Tensor:
    """A workspace of ``nbytes`` for one call on the current stream of ``dev`` (its contents do not matter to
    the kernels).  A call fills it in one launch and reads it in the next, and other host threads run
    meanwhile, so no two calls share one; dropped after the call it goes back to the stream's allocator,
    which hands it on in stream order, and under graph capture it belongs to the graph."""
    return torch.empty(nbytes, dtype=U8, device=dev)


def sl_linear_wgrad_accum(X: torch.Tensor, dY: torch.Tensor, main_grad: torch.Tensor,
                          workspace: torch.Tensor | None = None) -> torch.Tensor:
    """main_grad[out,in] += dY[T,out]^T . X[T,in] in fp32, in place."""
    dev = _device(X)
    T, n_in = X.shape
    n_out = dY.shape[1]
    _want(X, "X", BF16, (T, n_in), dev)
    _want(dY, "dY", BF16, (T, n_out), dev)
    _want(main_grad, "main_grad", F32, (n_out, n_in), dev)
    need = sl_wgrad_workspace_bytes(T, n_in, n_out)
    if workspace is None:
        workspace = wgrad_workspace(dev, need) if need else None
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    check("sl_linear_wgrad_accum", lib().sl_linear_wgrad_accum(
        _stream(dev), _ptr(X), _ptr(dY), _ptr(main_grad), T, n_in, n_out, _ptr(workspace), nbytes))
    return main_grad


def sl_linear_wgrad_accum_noalloc(X: torch.Tensor, dY: torch.Tensor, main_grad: torch.Tensor) -> torch.Tensor:
    """main_grad += dY^T . X in fp32, in place, with the split-K planes in the library's own device
    array (no workspace, no allocation)."""
    dev = _device(X)
    T, n_in = X.shape
    n_out = dY.shape[1]
    _want(X, "X", BF16, (T, n_in), dev)
    _want(dY, "dY", BF16, (T, n_out), dev)
    _want(main_grad, "main_grad", F32, (n_out, n_in), dev)
    check("sl_linear_wgrad_accum_noalloc", lib().sl_linear_wgrad_accum_noalloc(
        _stream(dev), _ptr(X), _ptr(dY), _ptr(main_grad), T, n_in, n_out))
    return main_grad


def sl_linear_fwd_mxfp8(Xq, Xs, Wq, Ws, Y=None):
    """Y = deq(Xq, Xs) . deq(Wq, Ws)^T (bf16 out); codes and scales are uint8."""
    dev = _device(Xq)
    T, n_in = Xq.shape
    n_out = Wq.shape[0]
    _want(Xq, "Xq", U8, (T, n_in), dev)
    _want(Xs, "Xs", U8, (T, n_in // 32), dev)
    _want(Wq, "Wq", U8, (n_out, n_in), dev)
    _want(Ws, "Ws", U8, (n_out, n_in // 32), dev)
    if Y is None:
        Y = torch.empty((T, n_out), dtype=BF16, device=dev)
    _want(Y, "Y", BF16, (T, n_out), dev)
    check("sl_linear_fwd_mxfp8", lib().sl_linear_fwd_mxfp8(
        _stream(dev), _ptr(Xq), _ptr(Xs), _ptr(Wq), _ptr(Ws), _ptr(Y), T, n_in, n_out))
    return Y


def sl_mxfp8_workspace_bytes(T: int, n_in: int, n_out: int) -> int:
    return int(lib().sl_mxfp8_workspace_bytes(T, n_in, n_out))


def sl_linear_dgrad_mxfp8w(dY, Wq, Ws, dX=None, workspace=None):
    """dX = dY . deq(Wq, Ws) (bf16 in/out)."""
    dev = _device(dY)
    T, n_out = dY.shape
    n_in = Wq.shape[1]
    _want(dY, "dY", BF16, (T, n_out), dev)
    _want(Wq, "Wq", U8, (n_out, n_in), dev)
    _want(Ws, "Ws", U8, (n_out, n_in // 32), dev)
    if dX is None:
        dX = torch.empty((T, n_in), dtype=BF16, device=dev)
    _want(dX, "dX", BF16, (T, n_in), dev)
    need = sl_mxfp8_workspace_bytes(T, n_in, n_out)
    if workspace is None:
        workspace = wgrad_workspace(dev, need) if need else None
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    check("sl_linear_dgrad_mxfp8w", lib().sl_linear_dgrad_mxfp8w(
        _stream(dev), _ptr(dY), _ptr(Wq), _ptr(Ws), _ptr(dX), T, n_in, n_out, _ptr(workspace), nbytes))
    return dX


def sl_linear_wgrad_accum_mxfp8x(Xq, Xs, dY, main_grad, workspace=None):
    """main_grad += dY^T . deq(Xq, Xs) in fp32, in place."""
    dev = _device(Xq)
    T, n_in = Xq.shape
    n_out = dY.shape[1]
    _want(Xq, "Xq", U8, (T, n_in), dev)
    _want(Xs, "Xs", U8, (T, n_in // 32), dev)
    _want(dY, "dY", BF16, (T, n_out), dev)
    _want(main_grad, "main_grad", F32, (n_out, n_in), dev)
    need = sl_mxfp8_workspace_bytes(T, n_in, n_out)
    if workspace is None:
        workspace = wgrad_workspace(dev, need) if need else None
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    check("sl_linear_wgrad_accum_mxfp8x", lib().sl_linear_wgrad_accum_mxfp8x(
        _stream(dev), _ptr(Xq), _ptr(Xs), _ptr(dY), _ptr(main_grad), T, n_in, n_out, _ptr(workspace), nbytes))
    return main_grad


def sl_mxfp8_dequantize(q, s, out=None):
    """bf16 out[r, c] = E4M3(q[r, c]) * 2^(s[r, c/32] - 127) for codes q[R, C] and scales s[R, C/32]."""
    dev = _device(q)
    R, C = q.shape
    _want(q, "q", U8, (R, C), dev)
    _want(s, "s", U8, (R, C // 32), dev)
    if out is None:
        out = torch.empty(R, C, dtype=BF16, device=dev)
    else:
        _want(out, "out", BF16, (R, C), dev)
    _launch("sl_mxfp8_dequantize", dev, _addr(q), _addr(s), _addr(out), R, C)
    return out


# ---- all-MXFP8 step ---------------------------------------------------------------------------

def sl_mxfp8_quantize(x, rows=True, cols=True, out=None):
    """MX-quantise bf16 x[R, C]: returns (q_rows, s_rows, q_cols, s_cols); a copy not asked for is
    None.  Rowwise blocks run along C ([R, C] codes, [R, C/32] scales); columnwise blocks run down
    the columns and are stored transposed ([C, R] codes, [C, R/32] scales).  ``out`` may supply
    the four tensors."""
    dev = _device(x)
    R, C = x.shape
    _want(x, "x", BF16, (R, C), dev)
    if out is None:
        out = (torch.empty((R, C), dtype=U8, device=dev) if rows else None,
               torch.empty((R, C // 32), dtype=U8, device=dev) if rows else None,
               torch.empty((C, R), dtype=U8, device=dev) if cols else None,
               torch.empty((C, R // 32), dtype=U8, device=dev) if cols else None)
    qr, sr, qc, sc = out
    if qr is not None:
        _want(qr, "q_rows", U8, (R, C), dev)
        _want(sr, "s_rows", U8, (R, C // 32), dev)
    if qc is not None:
        _want(qc, "q_cols", U8, (C, R), dev)
        _want(sc, "s_cols", U8, (C, R // 32), dev)
    check("sl_mxfp8_quantize", lib().sl_mxfp8_quantize(
        _stream(dev), _ptr(x), R, C, _ptr(qr), _ptr(sr), _ptr(qc), _ptr(sc)))
    return qr, sr, qc, sc


def sl_linear_dgrad_mxfp8(dYq, dYs, WqT, WsT, dX=None):
    """dX[T,in] = deq(dYq, dYs)[T,out] . deq(WqT, WsT)[in,out]^T (bf16 out)."""
    dev = _device(dYq)
    T, n_out = dYq.shape
    n_in = WqT.shape[0]
    _want(dYq, "dYq", U8, (T, n_out), dev)
    _want(dYs, "dYs", U8, (T, n_out // 32), dev)
    _want(WqT, "WqT", U8, (n_in, n_out), dev)
    _want(WsT, "WsT", U8, (n_in, n_out // 32), dev)
    if dX is None:
        dX = torch.empty((T, n_in), dtype=BF16, device=dev)
    _want(dX, "dX", BF16, (T, n_in), dev)
    check("sl_linear_dgrad_mxfp8", lib().sl_linear_dgrad_mxfp8(
        _stream(dev), _ptr(dYq), _ptr(dYs), _ptr(WqT), _ptr(WsT), _ptr(dX), T, n_in, n_out))
    return dX


def sl_mxfp8_wgrad_workspace_bytes(T: int, n_in: int, n_out: int) -> int:
    return int(lib().sl_mxfp8_wgrad_workspace_bytes(T, n_in, n_out))


def sl_linear_wgrad_accum_mxfp8(dYqT, dYsT, XqT, XsT, main_grad, workspace=None):
    """main_grad[out,in] += deq(dYqT, dYsT)[out,T] . deq(XqT, XsT)[in,T]^T in fp32, in place."""
    dev = _device(dYqT)
    n_out, T = dYqT.shape
    n_in = XqT.shape[0]
    _want(dYqT, "dYqT", U8, (n_out, T), dev)
    _want(dYsT, "dYsT", U8, (n_out, T // 32), dev)
    _want(XqT, "XqT", U8, (n_in, T), dev)
    _want(XsT, "XsT", U8, (n_in, T // 32), dev)
    _want(main_grad, "main_grad", F32, (n_out, n_in), dev)
    need = sl_mxfp8_wgrad_workspace_bytes(T, n_in, n_out)
    if workspace is None:
        workspace = wgrad_workspace(dev, need) if need else None
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    check("sl_linear_wgrad_accum_mxfp8", lib().sl_linear_wgrad_accum_mxfp8(
        _stream(dev), _ptr(dYqT), _ptr(dYsT), _ptr(XqT), _ptr(XsT), _ptr(main_grad), T, n_in, n_out,
        _ptr(workspace), nbytes))
    return main_grad


# ---- NVFP4 weights ------------------------------------------------------------------------------

def sl_nvfp4_materialize(Wq, Ws, Wm=None):
    """Wm[rows, cols] (bf16) = E2M1(Wq) * E4M3(Ws) per 16-element block, exactly; the tensor scale
    is not applied.  Wq [rows, cols/2] packed codes (element 2j in the low nibble of byte j),
    Ws [rows, cols/16] scale bytes."""
    dev = _device(Wq)
    rows, half = Wq.shape
    cols = 2 * half
    _want(Wq, "Wq", U8, (rows, half), dev)
    _want(Ws, "Ws", U8, (rows, cols // 16), dev)
    if Wm is None:
        Wm = torch.empty((rows, cols), dtype=BF16, device=dev)
    _want(Wm, "Wm", BF16, (rows, cols), dev)
    check("sl_nvfp4_materialize", lib().sl_nvfp4_materialize(
        _stream(dev), _ptr(Wq), _ptr(Ws), _ptr(Wm), rows, cols))
    return Wm


def sl_linear_fwd_nvfp4w(X, Wm, w_scale: float, Y=None):
    """Y[T,out] = w_scale * (X[T,in] . Wm[out,in]^T), scaled in fp32, rounded to bf16."""
    dev = _device(X)
    T, n_in = X.shape
    n_out = Wm.shape[0]
    _want(X, "X", BF16, (T, n_in), dev)
    _want(Wm, "Wm", BF16, (n_out, n_in), dev)
    if Y is None:
        Y = torch.empty((T, n_out), dtype=BF16, device=dev)
    _want(Y, "Y", BF16, (T, n_out), dev)
    check("sl_linear_fwd_nvfp4w", lib().sl_linear_fwd_nvfp4w(
        _stream(dev), _ptr(X), _ptr(Wm), float(w_scale), _ptr(Y), T, n_in, n_out))
    return Y


def sl_linear_dgrad_nvfp4w(dY, Wm, w_scale: float, dX=None):
    """dX[T,in] = w_scale * (dY[T,out] . Wm[out,in]), scaled in fp32, rounded to bf16."""
    dev = _device(dY)
    T, n_out = dY.shape
    n_in = Wm.shape[1]
    _want(dY, "dY", BF16, (T, n_out), dev)
    _want(Wm, "Wm", BF16, (n_out, n_in), dev)
    if dX is None:
        dX = torch.empty((T, n_in), dtype=BF16, device=dev)
    _want(dX, "dX", BF16, (T, n_in), dev)
    check("sl_linear_dgrad_nvfp4w", lib().sl_linear_dgrad_nvfp4w(
        _stream(dev), _ptr(dY), _ptr(Wm), float(w_scale), _ptr(dX), T, n_in, n_out))
    return dX


# ---- MXFP4 --------------------------------------------------------------------------------------
# Matrices [r, k] as packed codes [r, k/2] and scales [r, k/32] (uint8), k a multiple of 32.

# A token's forward runs a few microseconds, so the calls below take the short way: pointers as ints, the
# stream's handle without a Stream object, and no allocation beyond the result.

_raw_stream = torch._C._cuda_getCurrentRawStream


def _addr(t):
    return None if t is None else t.data_ptr()


def _launch(name, dev, *args):
    """Calls the entry point on the current stream of ``dev``, with ``dev`` current."""
    fn = getattr(lib(), name)
    if dev.index == torch.cuda.current_device():
        st = fn(_raw_stream(dev.index), *args)
    else:
        with torch.cuda.device(dev):
            st = fn(_raw_stream(dev.index), *args)
    if st:
        check(name, st)


def _scratch(dev, need, workspace):
    """(tensor, bytes) of the caller's workspace, or of one for this call alone."""
    if workspace is None:
        if not need:
            return None, 0
        workspace = wgrad_workspace(dev, need)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {dev}")
    return workspace, workspace.numel() * workspace.element_size()


_FEW = 16  # tokens up to which the MXFP4 products need no workspace (the gradient through a frozen weight apart)


def _want_mxfp4(q, s, names, dev):
    """Checks codes and scales against each other; returns (rows, k)."""
    if not isinstance(q, torch.Tensor) or q.dim() != 2:
        raise ValueError(f"{names[0]} must be a matrix of packed codes [rows, k / 2]")
    rows, half = q.shape
    if half % 16:
        raise ValueError(f"{names[0]} has {2 * half} elements to a row, which is no multiple of 32")
    _want(q, names[0], U8, (rows, half), dev)
    _want(s, names[1], U8, (rows, half // 16), dev)
    return rows, 2 * half


def _same(a, b, what):
    if a != b:
        raise ValueError(f"{what} differ: {a} and {b}")


def sl_mxfp4_quantize(x, rows=True, cols=True, seed=None, out=None):
    """MXFP4 copies of bf16 x[R, C] (C % 8 == 0): returns (q_rows, s_rows, q_cols, s_cols); a copy not
    asked for is None.  Rowwise blocks of 32 run along C, columnwise ones down the columns, stored
    transposed; the last block of a row or column is padded with zeros, so the copies are
    [R, Cp/2] + [R, Cp/32] and [C, Rp/2] + [C, Rp/32] with the extents rounded up to 32.

    ``seed`` None rounds to nearest (OCP MX).  An int, or a one-element int64 tensor on x's device
    (read when the kernel runs, so a replayed graph can take another), rounds stochastically: the
    same seed gives the same codes.  ``out`` may supply the four tensors."""
    dev = _device(x)
    if x.dim() != 2:
        raise ValueError(f"x has shape {tuple(x.shape)}, expected a matrix")
    R, C = x.shape
    _want(x, "x", BF16, (R, C), dev)
    if C % 8:
        raise ValueError(f"x has {C} columns, which is no multiple of 8")
    Rp, Cp = (R + 31) // 32 * 32, (C + 31) // 32 * 32
    if out is None:
        new = lambda *shape: torch.empty(shape, dtype=U8, device=dev)  # noqa: E731
        out = ((new(R, Cp // 2), new(R, Cp // 32)) if rows else (None, None)) + \
              ((new(C, Rp // 2), new(C, Rp // 32)) if cols else (None, None))
    qr, sr, qc, sc = out
    if qr is not None:
        _want(qr, "q_rows", U8, (R, Cp // 2), dev)
        _want(sr, "s_rows", U8, (R, Cp // 32), dev)
    if qc is not None:
        _want(qc, "q_cols", U8, (C, Rp // 2), dev)
        _want(sc, "s_cols", U8, (C, Rp // 32), dev)
    offset, key = None, 0
    if isinstance(seed, torch.Tensor):
        offset = seed
        if offset.numel() != 1:
            raise ValueError("a seed tensor has one element")
        _want(offset, "seed", torch.int64, offset.shape, dev)
    elif seed is not None:
        key = int(seed) & 0xFFFFFFFFFFFFFFFF
    _launch("sl_mxfp4_quantize", dev, _addr(x), R, C, _addr(qr), _addr(sr), _addr(qc), _addr(sc),
            int(seed is not None), key, _addr(offset))
    return qr, sr, qc, sc


def sl_mxfp4_dequantize(q, s, out=None):
    """bf16 out[r, k] = E2M1(code) * 2^(s[r, k/32] - 127) of packed codes q[R, K/2] and scales s[R, K/32]."""
    dev = _device(q)
    R, K = _want_mxfp4(q, s, ("q", "s"), dev)
    if out is None:
        out = torch.empty((R, K), dtype=BF16, device=dev)
    _want(out, "out", BF16, (R, K), dev)
    _launch("sl_mxfp4_dequantize", dev, _addr(q), _addr(s), _addr(out), R, K)
    return out


def sl_mxfp4_fwd_workspace_bytes(T: int, n_in: int, n_out: int) -> int:
    return int(lib().sl_mxfp4_fwd_workspace_bytes(T, n_in, n_out))


def sl_linear_fwd_mxfp4(Xq, Xs, Wq, Ws, Y=None, workspace=None):
    """Y[T,out] = deq(Xq, Xs)[T,in] . deq(Wq, Ws)[out,in]^T (bf16 out)."""
    dev = _device(Xq)
    T, n_in = _want_mxfp4(Xq, Xs, ("Xq", "Xs"), dev)
    n_out, k = _want_mxfp4(Wq, Ws, ("Wq", "Ws"), dev)
    _same(n_in, k, "the contracted extents of Xq and Wq")
    if Y is None:
        Y = torch.empty((T, n_out), dtype=BF16, device=dev)
    else:
        _want(Y, "Y", BF16, (T, n_out), dev)
    need = sl_mxfp4_fwd_workspace_bytes(T, n_in, n_out) if T > _FEW else 0
    workspace, nbytes = _scratch(dev, need, workspace)
    _launch("sl_linear_fwd_mxfp4", dev, _addr(Xq), _addr(Xs), _addr(Wq), _addr(Ws), _addr(Y), T, n_in, n_out,
            _addr(workspace), nbytes)
    return Y


def sl_mxfp4_dgrad_workspace_bytes(T: int, n_in: int, n_out: int) -> int:
    return int(lib().sl_mxfp4_dgrad_workspace_bytes(T, n_in, n_out))


def sl_linear_dgrad_mxfp4(dYq, dYs, WqT, WsT, dX=None, workspace=None):
    """dX[T,in] = deq(dYq, dYs)[T,out] . deq(WqT, WsT)[in,out]^T (bf16 out)."""
    dev = _device(dYq)
    T, n_out = _want_mxfp4(dYq, dYs, ("dYq", "dYs"), dev)
    n_in, k = _want_mxfp4(WqT, WsT, ("WqT", "WsT"), dev)
    _same(n_out, k, "the contracted extents of dYq and WqT")
    if dX is None:
        dX = torch.empty((T, n_in), dtype=BF16, device=dev)
    else:
        _want(dX, "dX", BF16, (T, n_in), dev)
    need = sl_mxfp4_dgrad_workspace_bytes(T, n_in, n_out) if T > _FEW else 0
    workspace, nbytes = _scratch(dev, need, workspace)
    _launch("sl_linear_dgrad_mxfp4", dev, _addr(dYq), _addr(dYs), _addr(WqT), _addr(WsT), _addr(dX), T, n_in, n_out,
            _addr(workspace), nbytes)
    return dX


def sl_mxfp4_wgrad_workspace_bytes(T: int, n_in: int, n_out: int) -> int:
    return int(lib().sl_mxfp4_wgrad_workspace_bytes(T, n_in, n_out))


def sl_linear_wgrad_accum_mxfp4(dYqT, dYsT, XqT, XsT, main_grad, workspace=None):
    """main_grad[out,in] += deq(dYqT, dYsT)[out,T] . deq(XqT, XsT)[in,T]^T in fp32, in place."""
    dev = _device(dYqT)
    n_out, T = _want_mxfp4(dYqT, dYsT, ("dYqT", "dYsT"), dev)
    n_in, k = _want_mxfp4(XqT, XsT, ("XqT", "XsT"), dev)
    _same(T, k, "the contracted extents of dYqT and XqT")
    _want(main_grad, "main_grad", F32, (n_out, n_in), dev)
    workspace, nbytes = _scratch(dev, sl_mxfp4_wgrad_workspace_bytes(T, n_in, n_out), workspace)
    _launch("sl_linear_wgrad_accum_mxfp4", dev, _addr(dYqT), _addr(dYsT), _addr(XqT), _addr(XsT), _addr(main_grad), T, n_in,
            n_out, _addr(workspace), nbytes)
    return main_grad


def sl_mxfp4w_fwd_workspace_bytes(T: int, n_in: int, n_out: int) -> int:
    return int(lib().sl_mxfp4w_fwd_workspace_bytes(T, n_in, n_out))


def sl_linear_fwd_mxfp4w(X, Wq, Ws, Y=None, workspace=None):
    """Y[T,out] = X[T,in] . deq(Wq, Ws)[out,in]^T with bf16 X and Y, from one token on.  The workspace of many
    tokens (1024, fewer by a wide weight) is a bf16 copy of the weight, 2 out in bytes for the call's time."""
    dev = _device(X)
    n_out, n_in = _want_mxfp4(Wq, Ws, ("Wq", "Ws"), dev)
    T = X.shape[0]
    _want(X, "X", BF16, (T, n_in), dev)
    if Y is None:
        Y = torch.empty((T, n_out), dtype=BF16, device=dev)
    else:
        _want(Y, "Y", BF16, (T, n_out), dev)
    need = sl_mxfp4w_fwd_workspace_bytes(T, n_in, n_out) if T > _FEW else 0
    workspace, nbytes = _scratch(dev, need, workspace)
    _launch("sl_linear_fwd_mxfp4w", dev, _addr(X), _addr(Wq), _addr(Ws), _addr(Y), T, n_in, n_out, _addr(workspace), nbytes)
    return Y


def sl_mxfp4w_dgrad_workspace_bytes(T: int, n_in: int, n_out: int) -> int:
    return int(lib().sl_mxfp4w_dgrad_workspace_bytes(T, n_in, n_out))


def sl_linear_dgrad_mxfp4w(dY, Wq, Ws, dX=None, workspace=None):
    """dX[T,in] = dY[T,out] . deq(Wq, Ws)[out,in] with bf16 dY and dX (a frozen MXFP4 weight's input gradient).
    Workspaces are as sl_linear_fwd_mxfp4w's."""
    dev = _device(dY)
    n_out, n_in = _want_mxfp4(Wq, Ws, ("Wq", "Ws"), dev)
    T = dY.shape[0]
    _want(dY, "dY", BF16, (T, n_out), dev)
    if dX is None:
        dX = torch.empty((T, n_in), dtype=BF16, device=dev)
    else:
        _want(dX, "dX", BF16, (T, n_in), dev)
    workspace, nbytes = _scratch(dev, sl_mxfp4w_dgrad_workspace_bytes(T, n_in, n_out), workspace)
    _launch("sl_linear_dgrad_mxfp4w", dev, _addr(dY), _addr(Wq), _addr(Ws), _addr(dX), T, n_in, n_out, _addr(workspace),
            nbytes)
    return dX


# ---- vocabulary-parallel embedding --------------------------------------------------------------

def _want_ids(ids, dev):
    """Checks token ids of any shape; returns the bytes of one."""
    size = 4 if ids.dtype is torch.int32 else 8
    if size == 8 and ids.dtype is not torch.int64:
        raise TypeError(f"ids must be torch.int32 or torch.int64, got {ids.dtype}")
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous")
    return size


def _want_matrix(t, name, dtype, dev):
    """Checks a matrix of any extents; returns them."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a matrix")
    shape = t.shape
    if t.dtype is not dtype or t.device != dev or not t.is_contiguous():
        _want(t, name, dtype, shape, dev)
    return shape


def sl_embedding_fwd(ids, W, Y=None, vocab_start=0, scale=1.0):
    """Y[*ids.shape, H] = bf16(scale * W[ids - vocab_start]) of the table shard W[V, H] (bf16); zeros where an id
    is not in vocab_start .. vocab_start + V - 1 (another rank's)."""
    dev = _device(ids)
    size = _want_ids(ids, dev)
    V, H = _want_matrix(W, "W", BF16, dev)
    T = ids.numel()
    if Y is None:
        Y = torch.empty(*ids.shape, H, dtype=BF16, device=dev)
    else:
        _want(Y, "Y", BF16, (*ids.shape, H), dev)
    _launch("sl_embedding_fwd", dev, _addr(ids), size, _addr(W), _addr(Y), T, V, H, vocab_start, scale)
    return Y


def sl_embedding_wgrad_workspace_bytes(T: int, V: int, H: int) -> int:
    return int(lib().sl_embedding_wgrad_workspace_bytes(T, V, H))


def sl_embedding_wgrad_accum(ids, dY, main_grad, vocab_start=0, scale=1.0, workspace=None):
    """main_grad[V, H] += scale * the sums of dY[*ids.shape, H] (bf16) over equal ids, fp32, in place."""
    dev = _device(ids)
    size = _want_ids(ids, dev)
    V, H = _want_matrix(main_grad, "main_grad", F32, dev)
    _want(dY, "dY", BF16, (*ids.shape, H), dev)
    T = ids.numel()
    workspace, nbytes = _scratch(dev, sl_embedding_wgrad_workspace_bytes(T, V, H), workspace)
    _launch("sl_embedding_wgrad_accum", dev, _addr(ids), size, _addr(dY), _addr(main_grad), T, V, H, vocab_start, scale,
            _addr(workspace), nbytes)
    return main_grad


# ---- root-mean-square norm ----------------------------------------------------------------------

def _norm_inputs(x, w, residual, h, parts=1):
    """Checks a norm's inputs; returns (device, T, H, h, rstd[parts * T]), h being x itself without a residual."""
    dev = _device(x)
    T, H = _want_matrix(x, "x", BF16, dev)
    _want(w, "w", BF16, (H,), dev)
    if residual is None:
        if h is not None:
            raise ValueError("h is the sum with a residual, and none is given")
        h = x
    else:
        _want(residual, "residual", BF16, (T, H), dev)
        if h is None:
            h = torch.empty(T, H, dtype=BF16, device=dev)
        else:
            _want(h, "h", BF16, (T, H), dev)
    return dev, T, H, h, torch.empty(parts * T, dtype=F32, device=dev)


def sl_rmsnorm_fwd(x, w, eps, residual=None, y=None, h=None):
    """Returns (y, h, rstd) of x[T, H]: h = bf16(x + residual) (x itself without one), rstd = (mean(h^2) + eps)^-1/2
    (fp32 [T]), y = bf16(h * rstd * w)."""
    dev, T, H, h, rstd = _norm_inputs(x, w, residual, h)
    if y is None:
        y = torch.empty(T, H, dtype=BF16, device=dev)
    else:
        _want(y, "y", BF16, (T, H), dev)
    _launch("sl_rmsnorm_fwd", dev, _addr(x), _addr(residual), _addr(w), eps, _addr(y), None if residual is None else _addr(h),
            _addr(rstd), T, H)
    return y, h, rstd


def sl_rmsnorm_fwd_mxfp8(x, w, eps, residual=None, rows=True, cols=True, out=None, h=None):
    """sl_rmsnorm_fwd with y in MXFP8, rounded once: returns (q_rows, s_rows, q_cols, s_cols, h, rstd); a copy not
    asked for is None.  The copies are laid out as sl_mxfp8_quantize's: rowwise [T, H] + [T, H/32] (H % 32 == 0), columnwise,
    stored transposed, [H, T] + [H, T/32] (T % 32 == 0).  ``out`` may supply the four tensors."""
    if out is not None:
        cols = out[2] is not None
    dev, T, H, h, rstd = _norm_inputs(x, w, residual, h, 2 if cols else 1)
    if out is None:
        new = lambda *shape: torch.empty(*shape, dtype=U8, device=dev)  # noqa: E731
        qr, sr = (new(T, H), new(T, H // 32)) if rows else (None, None)
        qc, sc = (new(H, T), new(H, T // 32)) if cols else (None, None)
    else:
        qr, sr, qc, sc = out
        if qr is not None:
            _want(qr, "q_rows", U8, (T, H), dev)
            _want(sr, "s_rows", U8, (T, H // 32), dev)
        if qc is not None:
            _want(qc, "q_cols", U8, (H, T), dev)
            _want(sc, "s_cols", U8, (H, T // 32), dev)
    _launch("sl_rmsnorm_fwd_mxfp8", dev, _addr(x), _addr(residual), _addr(w), eps, _addr(qr), _addr(sr), _addr(qc), _addr(sc),
            None if residual is None else _addr(h), _addr(rstd), T, H)
    return qr, sr, qc, sc, h, rstd[:T] if cols else rstd


def sl_rmsnorm_bwd_workspace_bytes(T: int, H: int) -> int:
    return int(lib().sl_rmsnorm_bwd_workspace_bytes(T, H))


def sl_rmsnorm_bwd(dY, h, w, rstd, w_grad, dresidual=None, dX=None, workspace=None):
    """dX[T, H] (bf16) of sl_rmsnorm_fwd, the gradient of x and of the residual alike, from the h and rstd it returned;
    dresidual is the gradient that reaches h by other ways.  w_grad[H] += the weight's gradient (fp32, in place);
    None leaves it out."""
    dev = _device(dY)
    T, H = _want_matrix(dY, "dY", BF16, dev)
    _want(h, "h", BF16, (T, H), dev)
    _want(w, "w", BF16, (H,), dev)
    _want(rstd, "rstd", F32, (T,), dev)
    if w_grad is not None:
        _want(w_grad, "w_grad", F32, (H,), dev)
    if dresidual is not None:
        _want(dresidual, "dresidual", BF16, (T, H), dev)
    if dX is None:
        dX = torch.empty(T, H, dtype=BF16, device=dev)
    else:
        _want(dX, "dX", BF16, (T, H), dev)
    workspace, nbytes = _scratch(dev, 0 if w_grad is None else sl_rmsnorm_bwd_workspace_bytes(T, H), workspace)
    _launch("sl_rmsnorm_bwd", dev, _addr(dY), _addr(h), _addr(w), _addr(rstd), _addr(dresidual), _addr(dX), _addr(w_grad), T, H,
            _addr(workspace), nbytes)
    return dX


# ---- orthogonalised updates ---------------------------------------------------------------------

NEWTON_SCHULZ = (3.4445, -4.7750, 2.0315)      # moves singular values of 0.01 .. 1 to 0.7 .. 1.2 in 5 steps


def _coefficients(steps, coefficients):
    """(steps, a C array of a, b, c for each); one triple serves every step."""
    if steps < 0:
        raise ValueError(f"steps is {steps}")
    flat = [float(v) for c in coefficients for v in (c if isinstance(c, (tuple, list)) else (c,))]
    if len(flat) == 3:
        flat = flat * steps
    if len(flat) != 3 * steps:
        raise ValueError(f"coefficients are one triple, or one for each of the {steps} steps")
    return steps, (ctypes.c_float * max(1, len(flat)))(*flat)


def sl_orthogonalize_workspace_bytes(L: int, rows: int, cols: int) -> int:
    return int(lib().sl_orthogonalize_workspace_bytes(L, rows, cols))


def sl_orthogonalize_tiles(L: int, rows: int, cols: int):
    """For measurement and tests: how the products X X^T, A A and P X of a step are taken apart, for each (tiles of 256x256, of
    128x128, of the latter with split sums, their parts); None where the steps go to the kernels for few rows."""
    t = (ctypes.c_int64 * 12)()
    check("sl_orthogonalize_tiles", lib().sl_orthogonalize_tiles(L, rows, cols, t))
    return [tuple(t[4 * k:4 * k + 4]) for k in range(3)] if any(t) else None


def sl_orthogonalize(G, out=None, steps=5, coefficients=NEWTON_SCHULZ, workspace=None):
    """bf16 Newton-Schulz iterate of G[rows, cols] or of each of G[L, rows, cols] (fp32 or bf16): X = G / |G|_F, and
    ``steps`` times X <- a X + (b A + c A A) X with A = X X^T."""
    dev = _device(G)
    if G.dim() not in (2, 3) or G.dtype not in (F32, BF16):
        raise ValueError(f"G must be one or a batch of fp32 or bf16 matrices, got {G.dtype} {tuple(G.shape)}")
    _want(G, "G", G.dtype, G.shape, dev)
    rows, cols = G.shape[-2:]
    L = G.shape[0] if G.dim() == 3 else 1
    if out is None:
        out = torch.empty(G.shape, dtype=BF16, device=dev)
    else:
        _want(out, "out", BF16, G.shape, dev)
    steps, k = _coefficients(steps, coefficients)
    workspace, nbytes = _scratch(dev, sl_orthogonalize_workspace_bytes(L, rows, cols), workspace)
    _launch("sl_orthogonalize", dev, _addr(G), G.element_size(), _addr(out), L, rows, cols, steps, k, _addr(workspace), nbytes)
    return out


def _want_apart(written, read):
    """No matrix that a call writes overlaps another of its matrices; those that it only reads may be the same."""
    end, last_written = 0, False
    for start, stop, w in sorted((t.data_ptr(), t.data_ptr() + t.nbytes, w) for ts, w in ((written, True), (read, False)) for t in ts):
        if start < end and (w or last_written):
            raise ValueError("a weight, momentum or master overlaps another of the matrices, or is given twice")
        if stop >= end:
            end, last_written = stop, w


def _muon_call(weights, main_grads, momenta, lr, momentum=0.95, nesterov=True, weight_decay=0.0, scale=None, masters=None, steps=5,
               coefficients=NEWTON_SCHULZ, workspace=None):
    """Checks sl_muon_step's arguments and launches nothing: (the matrices that it writes, those that it reads, the call itself)."""
    lists = [[t] if isinstance(t, torch.Tensor) else list(t) for t in (weights, main_grads, momenta)]
    lists.append(None if masters is None else [masters] if isinstance(masters, torch.Tensor) else list(masters))
    W = lists[0]
    if any(x is not None and len(x) != len(W) for x in lists):
        raise ValueError("weights, main_grads, momenta and masters differ in number")
    if not W:
        return [], [], lambda: None
    dev = _device(W[0])
    rows, cols = _want_matrix(W[0], "a weight", BF16, dev)
    for x, name, dtype in zip(lists, ("a weight", "a main_grad", "a momentum", "a master"), (BF16, F32, F32, F32)):
        for t in x or ():
            _want(t, name, dtype, (rows, cols), dev)
    if scale is None:
        scale = max(1.0, rows / cols) ** 0.5 if cols else 1.0
    steps, k = _coefficients(steps, coefficients)
    table = lambda x: None if x is None else (ctypes.c_void_p * len(x))(*(t.data_ptr() for t in x))  # noqa: E731
    need = sl_orthogonalize_workspace_bytes(len(W), rows, cols)

    def call():
        w, g, m, p = (table(x) for x in lists)
        ws, nbytes = _scratch(dev, need, workspace)
        _launch("sl_muon_step", dev, w, p, g, m, len(W), rows, cols, lr, momentum, int(nesterov), weight_decay, scale, steps, k,
                _addr(ws), nbytes)
        # as any update in place: a graph that saved a weight refuses to use the new one for the old
        torch.autograd.graph.increment_version([t for t in written if not t.is_inference()])

    written = [t for x in (lists[0], lists[2], lists[3]) for t in x or ()]
    return written, lists[1], call


def sl_muon_step(weights, main_grads, momenta, lr, momentum=0.95, nesterov=True, weight_decay=0.0, scale=None, masters=None,
                 steps=5, coefficients=NEWTON_SCHULZ, workspace=None):
    """One step of bf16 weights of one shape, in place, from their fp32 main_grads: M <- momentum M + G, U = G + momentum M
    (``nesterov``) or M, W <- (1 - lr weight_decay) W - lr scale orthogonalize(U).  Arguments are matrices or lists of them; a
    list's products run together, so weights of one shape belong in one call.  ``masters`` are fp32 weights that take the step in W's
    place; W is then their rounding.  ``scale`` None is sqrt(max(1, rows / cols))."""
    written, read, call = _muon_call(weights, main_grads, momenta, lr, momentum, nesterov, weight_decay, scale, masters, steps,
                                     coefficients, workspace)
    _want_apart(written, read)
    call()


def _muon_steps(groups, lr, momentum=0.95, nesterov=True, weight_decay=0.0, scale=None, steps=5, coefficients=NEWTON_SCHULZ,
                workspace=None):
    """sl_muon_step of each (weights, main_grads, momenta, masters) of ``groups``; all are checked before the first is launched, so
    that a refusal leaves every weight and momentum as it was."""
    calls = [_muon_call(w, g, m, lr, momentum, nesterov, weight_decay, scale, p, steps, coefficients, workspace) for w, g, m, p in groups]
    _want_apart([t for c in calls for t in c[0]], [t for c in calls for t in c[1]])
    # as slices of an aligned batch are: by whole groups of four elements, or by elements
    unit = lambda t: t.element_size() if t.shape[1] % 4 else 8 if t.nbytes % 16 else 16  # noqa: E731
    if any(t.data_ptr() % unit(t) for c in calls for t in c[0] + c[1] if t.numel()):
        check("sl_muon_step", SL_EALIGN)
    for w, _, _, _ in groups:
        if w[0].numel():
            need = sl_orthogonalize_workspace_bytes(len(w), *w[0].shape)
            if not need:
                check("sl_muon_step", SL_ESHAPE)
            if workspace is not None and _scratch(w[0].device, need, workspace)[1] < need:
                check("sl_muon_step", SL_EWORKSPACE)
    for _, _, call in calls:
        call()
