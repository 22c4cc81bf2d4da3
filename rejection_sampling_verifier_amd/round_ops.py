"""Binding of the operators around a verification round (spec_verify.h, "Operators
around a verification round"): torch tensors in, device pointers out.

As in ``binding``, every step runs in the library's HIP kernels, a call is
enqueued on the current (or given) stream and nothing is synchronised.
Outputs and workspaces that a call allocates belong to the stream it runs on.
"""

from __future__ import annotations

import ctypes

import torch

from .binding import (SvControls, _check, _dtype_code, _OnStream, _stream_handle, load_library)


class _OnDevice:
    """Makes `dev` the current device for a call if another one is."""

    def __init__(self, dev):
        self.ctx = None if dev.index is None or dev.index == torch.cuda.current_device() else torch.cuda.device(dev)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def _gpu(t, name):
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError(f"{name} must be a tensor on a GPU device")
    return t.device


def _need(name, t, shape, dtype, dev):
    """A contiguous tensor of this shape (None: any size there), type and device."""
    if (not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != dev or t.dim() != len(shape)
            or any(w is not None and n != w for n, w in zip(t.shape, shape)) or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape "
                         f"({', '.join('any' if w is None else str(w) for w in shape)}) on {dev}")


def _maybe(name, t, shape, dtype, dev):
    if t is not None:
        _need(name, t, shape, dtype, dev)


def _rows(name, t, B, dtype, dev):
    """A [B, n] tensor whose rows are contiguous; its row pitch in elements."""
    if (not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != dev or t.dim() != 2 or t.shape[0] != B
            or (t.shape[1] > 1 and t.stride(1) != 1) or (B > 1 and t.stride(0) < t.shape[1])):
        raise ValueError(f"{name} must be a {dtype} tensor of shape ({B}, any) on {dev} with contiguous rows")
    return t.stride(0) if B > 1 else t.shape[1]


def _p(t):
    return None if t is None else t.data_ptr()


def _logit_strides(name, t):
    """(row, position) strides of a [B, P, V] tensor with contiguous logits."""
    B, P, V = t.shape
    pos = t.stride(1) if P > 1 else V
    row = t.stride(0) if B > 1 else P * pos
    if (V > 1 and t.stride(2) != 1) or pos < V or row < (P - 1) * pos + V:
        raise ValueError(f"{name} must have contiguous, non-overlapping rows of logits")
    return row, pos


def adjust_logits(logits, tokens=None, *, parents=None, history=None, history_lens=None, prompt_lens=None,
                  repetition=None, presence=None, frequency=None, bias_ids=None, bias_values=None, bias_lens=None,
                  mask=None, mask_rows=None, out=None, stream=None):
    """spec_verify_adjust_logits: penalties, biases and grammar masks on the
    logits of a round (see the header for the formulas).

    logits [B, P, V] bf16 or fp32 with contiguous rows (a slice of a padded
    vocabulary will do); tokens [B, >= P - 1] int32 of a chain, or [B, P] node
    tokens with parents [B, P] of a tree; history [B, any] int32 with
    history_lens [B] and prompt_lens [B] int32; repetition, presence,
    frequency [B] fp32; bias_ids int32 and bias_values fp32 [B, any], bias_lens
    [B] int32; mask [R, ceil(V / 32)] int32 words, mask_rows [B, P] int32 (-1:
    no mask; without mask_rows position (b, i) goes by mask row b P + i).

    Returns ``out`` (a new contiguous [B, P, V] tensor if None; ``out=logits``
    works in place).
    """
    dev = _gpu(logits, "logits")
    if logits.dim() != 3 or 0 in logits.shape:
        raise ValueError("logits must be [B, P, V]")
    B, P, V = logits.shape
    dt = _dtype_code(logits)
    in_row, in_pos = _logit_strides("logits", logits)
    i32, f32 = torch.int32, torch.float32
    c = SvControls()
    tok_stride = 0
    for name, t in (("repetition", repetition), ("presence", presence), ("frequency", frequency)):
        if t is not None:
            _need(name, t, (B,), f32, dev)
            setattr(c, name, t.data_ptr())
    penalties = repetition is not None or presence is not None or frequency is not None
    if tokens is not None:
        tok_stride = _rows("tokens", tokens, B, i32, dev)
    need = P if parents is not None else P - 1
    if penalties and P > 1 and (tokens is None or tokens.shape[1] < need):
        raise ValueError(f"tokens must hold at least {need} drafted tokens per row")
    _maybe("parents", parents, (B, P), i32, dev)
    if history is not None:
        c.history_stride = _rows("history", history, B, i32, dev)
        if history_lens is None:
            raise ValueError("history needs history_lens")
        _need("history_lens", history_lens, (B,), i32, dev)
        _maybe("prompt_lens", prompt_lens, (B,), i32, dev)
        c.history, c.history_lens, c.prompt_lens = history.data_ptr(), history_lens.data_ptr(), _p(prompt_lens)
    if bias_ids is not None:
        _need("bias_ids", bias_ids, (B, None), i32, dev)
        _need("bias_values", bias_values, tuple(bias_ids.shape), f32, dev)
        _maybe("bias_lens", bias_lens, (B,), i32, dev)
        c.bias_ids, c.bias_values, c.bias_lens = bias_ids.data_ptr(), bias_values.data_ptr(), _p(bias_lens)
        c.bias_stride = bias_ids.shape[1]
    if mask is not None:
        _need("mask", mask, (None, (V + 31) // 32), i32, dev)
        _maybe("mask_rows", mask_rows, (B, P), i32, dev)
        if mask_rows is None and mask.shape[0] < B * P:
            raise ValueError(f"mask must hold {B * P} rows without mask_rows")
        c.mask, c.mask_rows, c.num_masks = mask.data_ptr(), _p(mask_rows), mask.shape[0]
    handle = _stream_handle(dev, stream)
    if out is None:
        with _OnStream(dev, handle):
            out = torch.empty((B, P, V), dtype=logits.dtype, device=dev)
    elif (not isinstance(out, torch.Tensor) or tuple(out.shape) != (B, P, V) or out.dtype != logits.dtype
          or out.device != dev):
        raise ValueError(f"out must be a {logits.dtype} tensor of shape {(B, P, V)} on {dev}")
    out_row, out_pos = _logit_strides("out", out)
    with _OnDevice(dev):
        _check(load_library().spec_verify_adjust_logits(
            logits.data_ptr(), in_row, in_pos, _p(tokens), tok_stride, _p(parents), ctypes.byref(c), B, P, V, dt,
            out.data_ptr(), out_row, out_pos, handle))
    return out
