"""The fused LoRA layer as PyTorch operators with autograd, and a module.

    Y = X W^T + s (X A^T) B^T,   s = alpha / r   (or an explicit scale)

fastaf 0.1.0, "FWD kernel speedup" / "BWD kernel speedup": the layer and its
backward for a frozen base weight W; section "torch.compile compatibility":
each kernel is a torch.library custom op with a fake implementation, so the
compiler traces through the layer without a graph break (checked with
torch._dynamo.explain).  Here:

* ``torch.ops.lora_b200.lora_linear(X, W, A, B, scale)`` runs
  ``lora_fwd_scaled``;
* ``torch.ops.lora_b200.lora_linear_bwd(X, W, A, B, dY, scale, fp32_grads)``
  runs ``lora_bwd_scaled`` and returns (dX, dA, dB), dA and dB in fp32 when
  ``fp32_grads`` (the unrounded reductions, e.g. for fp32 optimizer states
  or a data-parallel sum before rounding), else bf16;
* ``torch.ops.lora_b200.lora_linear_train(X, W, A, B, scale)`` runs
  ``lora_fwd_save_scaled`` and returns (Y, saved): Y as ``lora_linear`` (bit
  for bit) and the backward's workspace with T = X A^T already in it; its
  backward, ``lora_linear_bwd_saved``, runs ``lora_bwd_scaled`` with
  ``LORA_BWD_T_SAVED`` and so reads X once less (``LoRALinear`` uses this
  pair whenever autograd will need the backward);
* all have fake (meta) implementations, so they trace under FakeTensorMode
  and torch.compile without graph breaks, and ``lora_linear`` and
  ``lora_linear_train`` are differentiable in X, A and B through their
  backward ops.  W is frozen: it gets no gradient.

* ``torch.ops.lora_b200.lora_linear_adapter(X, W, W_scales, A, B, scale, p,
  rng, save)`` is the layer with dropout on the adapter branch (``lora_fwd_dropout``)
  or, with ``W_scales`` (W then holds e4m3 codes), over an 8-bit base
  (``lora_fwd_fp8``), with or without dropout.  It returns (Y, saved), saved
  being T for ``lora_linear_adapter_bwd``.  The mask is drawn from ``rng``, an
  int64 tensor [seed, offset] on the device, and never stored: the backward
  draws it again.  ``quantize_weight`` and ``dequantize_weight`` convert a
  weight.

The scale is passed explicitly, so rsLoRA's alpha / sqrt(r) (unsloth fork
commit log, scripts/benchmarks/qwen3_flex_inference.py: PEFT keeps the
adapter's scaling, alpha / sqrt(r) under rsLoRA, in the module) is as easy
to use as alpha / r.  The operators call the library's explicit-scale entry
points (``lora_fwd_scaled``, ``lora_fwd_save_scaled``, ``lora_bwd_scaled``),
which take s itself (rounded once to fp32) rather than alpha.

Argument marshalling only: all arithmetic runs in the library's kernels.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple

import torch

from . import (LORA_BWD_FP32_GRADS, LORA_BWD_T_SAVED, lora_bwd_dropout, lora_bwd_fp8, lora_bwd_scaled,
               lora_bwd_workspace_size, lora_dequantize_fp8, lora_fp8_workspace_size, lora_fwd_dropout, lora_fwd_fp8,
               lora_fwd_save_scaled, lora_fwd_scaled, lora_quantize_fp8)

_LIB = "lora_b200"


def _check(X: torch.Tensor, W: torch.Tensor, A: torch.Tensor, B: torch.Tensor) -> Tuple[int, int, int, int]:
    if X.dim() != 2 or W.dim() != 2 or A.dim() != 2 or B.dim() != 2:
        raise ValueError("lora_linear takes 2-D X [M, d_in], W [d_out, d_in], A [r, d_in], B [d_out, r]")
    M, d_in = X.shape
    d_out, r = B.shape
    if tuple(W.shape) != (d_out, d_in) or tuple(A.shape) != (r, d_in):
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, W {tuple(W.shape)}, A {tuple(A.shape)}, "
                         f"B {tuple(B.shape)}")
    return M, d_in, d_out, r


@torch.library.custom_op(f"{_LIB}::lora_linear", mutates_args=())
def lora_linear(X: torch.Tensor, W: torch.Tensor, A: torch.Tensor, B: torch.Tensor, scale: float) -> torch.Tensor:
    """Y = X W^T + scale (X A^T) B^T (bf16, 2-D, contiguous CUDA tensors)."""
    M, d_in, d_out, r = _check(X, W, A, B)
    Y = torch.empty((M, d_out), dtype=X.dtype, device=X.device)
    lora_fwd_scaled(X.contiguous(), W.contiguous(), A.contiguous(), B.contiguous(), Y, scale)
    return Y


@lora_linear.register_fake
def _lora_linear_fake(X, W, A, B, scale):
    M, d_in, d_out, r = _check(X, W, A, B)
    return X.new_empty((M, d_out))


@torch.library.custom_op(f"{_LIB}::lora_linear_bwd", mutates_args=())
def lora_linear_bwd(X: torch.Tensor, W: torch.Tensor, A: torch.Tensor, B: torch.Tensor, dY: torch.Tensor,
                    scale: float, fp32_grads: bool = False) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(dX, dA, dB) of Y = X W^T + scale (X A^T) B^T for the gradient dY;
    dA and dB in fp32 when fp32_grads, else in the dtype of A and B."""
    M, d_in, d_out, r = _check(X, W, A, B)
    gdt = torch.float32 if fp32_grads else A.dtype
    dX = torch.empty((M, d_in), dtype=X.dtype, device=X.device)
    dA = torch.empty((r, d_in), dtype=gdt, device=A.device)
    dB = torch.empty((d_out, r), dtype=gdt, device=B.device)
    ws = torch.empty(max(lora_bwd_workspace_size(M, d_in, d_out, r), 1), dtype=torch.uint8, device=X.device)
    lora_bwd_scaled(X.contiguous(), W.contiguous(), A.contiguous(), B.contiguous(), dY.contiguous(), dX, dA, dB,
                    scale, ws, LORA_BWD_FP32_GRADS if fp32_grads else 0)
    return dX, dA, dB


@lora_linear_bwd.register_fake
def _lora_linear_bwd_fake(X, W, A, B, dY, scale, fp32_grads=False):
    M, d_in, d_out, r = _check(X, W, A, B)
    gdt = torch.float32 if fp32_grads else A.dtype
    return X.new_empty((M, d_in)), A.new_empty((r, d_in), dtype=gdt), B.new_empty((d_out, r), dtype=gdt)


def _workspace_bytes(M, r: int):
    """Bytes of lora_bwd_workspace_size(M, ., ., r) from its documented
    layout (T and dT as bf16 [M, r_pad], r_pad = r rounded up to 16, each
    padded to 256 bytes); usable on symbolic M, where the library cannot be
    asked.  0 when M == 0."""
    r_pad = (r + 15) // 16 * 16
    return 2 * ((M * r_pad * 2 + 255) // 256 * 256)


@torch.library.custom_op(f"{_LIB}::lora_linear_train", mutates_args=())
def lora_linear_train(X: torch.Tensor, W: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                      scale: float) -> Tuple[torch.Tensor, torch.Tensor]:
    """(Y, saved): Y = X W^T + scale (X A^T) B^T and the backward's
    workspace (uint8) holding T = X A^T for lora_linear_bwd_saved."""
    M, d_in, d_out, r = _check(X, W, A, B)
    nbytes = _workspace_bytes(M, r)
    if nbytes < lora_bwd_workspace_size(M, d_in, d_out, r):
        raise RuntimeError("lora_linear_train: the library needs a larger workspace than its documented layout")
    Y = torch.empty((M, d_out), dtype=X.dtype, device=X.device)
    ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=X.device)
    lora_fwd_save_scaled(X.contiguous(), W.contiguous(), A.contiguous(), B.contiguous(), Y, scale, ws)
    return Y, ws


@lora_linear_train.register_fake
def _lora_linear_train_fake(X, W, A, B, scale):
    M, d_in, d_out, r = _check(X, W, A, B)
    return X.new_empty((M, d_out)), X.new_empty((max(_workspace_bytes(M, r), 1),), dtype=torch.uint8)


@torch.library.custom_op(f"{_LIB}::lora_linear_bwd_saved", mutates_args=("saved",))
def lora_linear_bwd_saved(X: torch.Tensor, W: torch.Tensor, A: torch.Tensor, B: torch.Tensor, dY: torch.Tensor,
                          saved: torch.Tensor, scale: float,
                          fp32_grads: bool = False) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """lora_linear_bwd with T taken from ``saved`` (the workspace that
    lora_linear_train returned for the same X, A); writes dT into ``saved``
    beside T and leaves T as it was."""
    M, d_in, d_out, r = _check(X, W, A, B)
    gdt = torch.float32 if fp32_grads else A.dtype
    dX = torch.empty((M, d_in), dtype=X.dtype, device=X.device)
    dA = torch.empty((r, d_in), dtype=gdt, device=A.device)
    dB = torch.empty((d_out, r), dtype=gdt, device=B.device)
    flags = LORA_BWD_T_SAVED | (LORA_BWD_FP32_GRADS if fp32_grads else 0)
    lora_bwd_scaled(X.contiguous(), W.contiguous(), A.contiguous(), B.contiguous(), dY.contiguous(), dX, dA, dB,
                    scale, saved, flags)
    return dX, dA, dB


@lora_linear_bwd_saved.register_fake
def _lora_linear_bwd_saved_fake(X, W, A, B, dY, saved, scale, fp32_grads=False):
    return _lora_linear_bwd_fake(X, W, A, B, dY, scale, fp32_grads)


def _setup_context_train(ctx, inputs, output):
    X, W, A, B, scale = inputs
    if W.requires_grad:
        raise RuntimeError("lora_linear: the base weight W is frozen and gets no gradient; "
                           "call W.requires_grad_(False)")
    ctx.save_for_backward(X, W, A, B, output[1])
    ctx.scale = scale


def _backward_train(ctx, dY, _d_saved):
    X, W, A, B, saved = ctx.saved_tensors
    dX, dA, dB = torch.ops.lora_b200.lora_linear_bwd_saved(X, W, A, B, dY.contiguous(), saved, ctx.scale)
    return (dX if ctx.needs_input_grad[0] else None, None, dA if ctx.needs_input_grad[2] else None,
            dB if ctx.needs_input_grad[3] else None, None)


lora_linear_train.register_autograd(_backward_train, setup_context=_setup_context_train)


def _setup_context(ctx, inputs, output):
    X, W, A, B, scale = inputs
    if W.requires_grad:
        raise RuntimeError("lora_linear: the base weight W is frozen and gets no gradient; "
                           "call W.requires_grad_(False)")
    ctx.save_for_backward(X, W, A, B)
    ctx.scale = scale


def _backward(ctx, dY):
    X, W, A, B = ctx.saved_tensors
    dX, dA, dB = torch.ops.lora_b200.lora_linear_bwd(X, W, A, B, dY.contiguous(), ctx.scale)
    return (dX if ctx.needs_input_grad[0] else None, None, dA if ctx.needs_input_grad[2] else None,
            dB if ctx.needs_input_grad[3] else None, None)


lora_linear.register_autograd(_backward, setup_context=_setup_context)


# ------------------------------------- dropout and the 8-bit base ----

def _empty_codes(d_out: int, d_in: int, device) -> Tuple[torch.Tensor, torch.Tensor]:
    return (torch.empty((d_out, d_in), dtype=torch.float8_e4m3fn, device=device),
            torch.empty(((d_out + 127) // 128, (d_in + 127) // 128), dtype=torch.float8_e8m0fnu, device=device))


def quantize_weight(W: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """(codes float8_e4m3fn [d_out, d_in], scales float8_e8m0fnu, one power of
    two for each 128 x 128 block) of a bf16 weight (``lora_quantize_fp8``)."""
    d_out, d_in = W.shape
    codes, scales = _empty_codes(d_out, d_in, W.device)
    lora_quantize_fp8(W.contiguous(), codes, scales)
    return codes, scales


def dequantize_weight(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """The bf16 weight that codes and scales stand for (``lora_dequantize_fp8``)."""
    W = torch.empty(codes.shape, dtype=torch.bfloat16, device=codes.device)
    lora_dequantize_fp8(codes, scales, W)
    return W


def _saved_bytes(M, r: int):
    """Bytes that the forward leaves for the backward: T, at the start of
    either workspace.  (The rest is scratch, with an 8-bit base of M *
    max(d_in, d_out) bytes and more.)"""
    return _workspace_bytes(M, r) // 2


def _check_rng(p: float, rng: Optional[torch.Tensor]):
    if p > 0 and rng is None:
        raise ValueError("dropout needs rng, an int64 tensor [seed, offset] on the layer's device")


@torch.library.custom_op(f"{_LIB}::lora_linear_adapter", mutates_args=())
def lora_linear_adapter(X: torch.Tensor, W: torch.Tensor, W_scales: Optional[torch.Tensor], A: torch.Tensor,
                        B: torch.Tensor, scale: float, p: float, rng: Optional[torch.Tensor],
                        save: bool = True) -> Tuple[torch.Tensor, torch.Tensor]:
    """(Y, saved): Y = X W^T + T B^T, T = scale/(1-p) (m * X) A^T, over a bf16
    base or, with W_scales, over e4m3 codes W.  Without ``save`` (no backward
    will follow) saved is empty and T is not copied out; a backward then
    computes it again."""
    M, d_in, d_out, r = _check(X, W, A, B)
    _check_rng(p, rng)
    fp8 = W_scales is not None
    nbytes = lora_fp8_workspace_size(M, d_in, d_out, r) if fp8 else _workspace_bytes(M, r)
    if not fp8 and nbytes < lora_bwd_workspace_size(M, d_in, d_out, r):
        raise RuntimeError("lora_linear_adapter: the library needs a larger workspace than its documented layout")
    Y = torch.empty((M, d_out), dtype=X.dtype, device=X.device)
    ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=X.device)
    args = (X.contiguous(), W.contiguous())
    ab = (A.contiguous(), B.contiguous(), Y, scale)
    if fp8:
        lora_fwd_fp8(*args, W_scales.contiguous(), *ab, ws, p, rng)
    else:
        lora_fwd_dropout(*args, *ab, p, rng, ws)
    if not save:
        return Y, torch.empty(0, dtype=torch.uint8, device=X.device)
    return Y, ws[:max(_saved_bytes(M, r), 1)].clone()


@lora_linear_adapter.register_fake
def _lora_linear_adapter_fake(X, W, W_scales, A, B, scale, p, rng, save=True):
    M, d_in, d_out, r = _check(X, W, A, B)
    _check_rng(p, rng)
    return X.new_empty((M, d_out)), X.new_empty((max(_saved_bytes(M, r), 1) if save else 0,), dtype=torch.uint8)


@torch.library.custom_op(f"{_LIB}::lora_linear_adapter_bwd", mutates_args=())
def lora_linear_adapter_bwd(X: torch.Tensor, W: torch.Tensor, W_scales: Optional[torch.Tensor], A: torch.Tensor,
                            B: torch.Tensor, dY: torch.Tensor, saved: torch.Tensor, scale: float, p: float,
                            rng: Optional[torch.Tensor],
                            fp32_grads: bool = False) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(dX, dA, dB) of lora_linear_adapter for the same rng values, with T from
    ``saved``, which stays as it is (a graph may be gone through twice); an
    empty ``saved`` has T computed again."""
    M, d_in, d_out, r = _check(X, W, A, B)
    gdt = torch.float32 if fp32_grads else A.dtype
    dX = torch.empty((M, d_in), dtype=X.dtype, device=X.device)
    dA = torch.empty((r, d_in), dtype=gdt, device=A.device)
    dB = torch.empty((d_out, r), dtype=gdt, device=B.device)
    flags = LORA_BWD_FP32_GRADS if fp32_grads else 0
    args = (X.contiguous(), W.contiguous())
    rest = (A.contiguous(), B.contiguous(), dY.contiguous(), dX, dA, dB, scale)
    fp8 = W_scales is not None
    nbytes = lora_fp8_workspace_size(M, d_in, d_out, r) if fp8 else _workspace_bytes(M, r)
    ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=X.device)
    if saved.numel() > 0:
        flags |= LORA_BWD_T_SAVED
        t_bytes = _saved_bytes(M, r)
        ws[:t_bytes].copy_(saved[:t_bytes])
    if fp8:
        lora_bwd_fp8(*args, W_scales.contiguous(), *rest, ws, p, rng, flags)
    else:
        lora_bwd_dropout(*args, *rest, p, rng, ws, flags)
    return dX, dA, dB


@lora_linear_adapter_bwd.register_fake
def _lora_linear_adapter_bwd_fake(X, W, W_scales, A, B, dY, saved, scale, p, rng, fp32_grads=False):
    return _lora_linear_bwd_fake(X, W, A, B, dY, scale, fp32_grads)


def _setup_context_adapter(ctx, inputs, output):
    X, W, W_scales, A, B, scale, p, rng, _ = inputs
    if W.requires_grad:
        raise RuntimeError("lora_linear: the base weight W is frozen and gets no gradient; "
                           "call W.requires_grad_(False)")
    ctx.save_for_backward(X, W, W_scales, A, B, rng, output[1])
    ctx.scale, ctx.p = scale, p


def _backward_adapter(ctx, dY, _d_saved):
    X, W, W_scales, A, B, rng, saved = ctx.saved_tensors
    dX, dA, dB = torch.ops.lora_b200.lora_linear_adapter_bwd(X, W, W_scales, A, B, dY.contiguous(), saved, ctx.scale,
                                                             ctx.p, rng)
    need = ctx.needs_input_grad
    return (dX if need[0] else None, None, None, dA if need[3] else None, dB if need[4] else None,
            None, None, None, None)


lora_linear_adapter.register_autograd(_backward_adapter, setup_context=_setup_context_adapter)


class LoRALinear(torch.nn.Module):
    """A linear layer with a frozen base weight and a trainable rank-r adapter:
    y = x W^T + s (x A^T) B^T over the last dimension of x (any leading
    dimensions).  s = alpha / r, or alpha / sqrt(r) with ``rslora=True``.
    A is initialised N(0, 1/d_in) (variance), B to zero (the adapter starts
    as the identity map of the base layer); all parameters are bf16.

    ``dropout``: in training the adapter (not the base) sees x with each value
    dropped with this probability and the rest scaled by 1/(1 - dropout).  The
    mask's seed and offset are drawn from torch's generator of the device for
    each call, so torch.manual_seed repeats a run, activation checkpointing
    repeats a mask, and a captured step draws a new mask at each replay.

    ``quantize_base()`` turns the base weight into 8 bits (e4m3 codes, one
    power-of-two scale for each 128 x 128 block), as buffers ``weight_codes``
    and ``weight_scales`` in place of ``weight``: half the memory, and 8-bit
    products in forward and backward.  A cast of the module (``.to(dtype)``,
    ``.half()``) leaves these two as they are, and a checkpoint that has them
    turns a layer with a bf16 base into the 8-bit form as it loads."""

    dropout = 0.0  # (of a layer that was pickled before it had one)

    def __init__(self, d_in: int, d_out: int, r: int, alpha: float, rslora: bool = False,
                 device: Optional[torch.device] = None, generator: Optional[torch.Generator] = None,
                 dropout: float = 0.0):
        super().__init__()
        self.d_in, self.d_out, self.r, self.alpha = int(d_in), int(d_out), int(r), float(alpha)
        # (as the library holds it: fp32, then a multiple of 1/65536)
        if not 0.0 <= ctypes.c_float(dropout).value < 1.0 - 2.0 ** -17:
            raise ValueError(f"dropout must be in [0, 1), and below 1 as a multiple of 1/65536, got {dropout}")
        self.dropout = float(dropout)
        self.scale = self.alpha / (math.sqrt(self.r) if rslora else self.r)
        kw = dict(dtype=torch.bfloat16, device=device)
        self.weight = torch.nn.Parameter(
            (torch.randn(d_out, d_in, generator=generator) * d_in ** -0.5).to(**kw), requires_grad=False)
        self.lora_A = torch.nn.Parameter((torch.randn(r, d_in, generator=generator) * d_in ** -0.5).to(**kw))
        self.lora_B = torch.nn.Parameter(torch.zeros(d_out, r, **kw))

    def quantize_base(self) -> "LoRALinear":
        """The base weight to 8 bits, in place; returns the layer.  d_in and
        d_out have to be multiples of 16 (the codes' rows, and those that dY
        is rounded to, are read 16 bytes at a time)."""
        if self.weight is not None:
            if self.d_in % 16 or self.d_out % 16:
                raise ValueError(f"an 8-bit base needs d_in and d_out as multiples of 16, got {self.d_in} and "
                                 f"{self.d_out}")
            self._hold_codes(*quantize_weight(self.weight.detach()))
        return self

    def _hold_codes(self, codes: torch.Tensor, scales: torch.Tensor):
        self.weight = None
        self.register_buffer("weight_codes", codes)
        self.register_buffer("weight_scales", scales)

    def _load_from_state_dict(self, state_dict, prefix, *args):
        given = [state_dict.get(prefix + name) for name in ("weight_codes", "weight_scales")]
        if self.weight is not None and all(g is not None for g in given):
            room = _empty_codes(self.d_out, self.d_in, self.weight.device)
            if all(g.shape == e.shape for g, e in zip(given, room)):  # (other sizes are refused below)
                self._hold_codes(*room)
        super()._load_from_state_dict(state_dict, prefix, *args)

    def _apply(self, fn, recurse=True):
        # codes and scales are bytes, not numbers of a precision: casts pass
        # them by (as uint8), moves take them along
        def keep(t):
            if t.dtype not in (torch.float8_e4m3fn, torch.float8_e8m0fnu):
                return fn(t)
            held = t.view(torch.uint8)
            moved = fn(held)
            return (moved if moved.dtype == torch.uint8 else held.to(moved.device)).view(t.dtype)

        return super()._apply(keep, recurse)

    def base_weight(self) -> torch.Tensor:
        """The base weight's values in bf16."""
        return self.weight if self.weight is not None else dequantize_weight(self.weight_codes, self.weight_scales)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        lead = x.shape[:-1]
        x2 = x.reshape(-1, self.d_in)
        p = self.dropout if self.training else 0.0
        # keep T for a backward (it then reads X once less)
        save = torch.is_grad_enabled() and (x.requires_grad or self.lora_A.requires_grad or self.lora_B.requires_grad)
        if p > 0 or self.weight is None:
            rng = torch.randint(0, 2 ** 62, (2,), dtype=torch.int64, device=x.device) if p > 0 else None
            codes = self.weight is None
            y, _ = torch.ops.lora_b200.lora_linear_adapter(
                x2, self.weight_codes if codes else self.weight, self.weight_scales if codes else None, self.lora_A,
                self.lora_B, self.scale, p, rng, save)
        elif save:
            y, _ = torch.ops.lora_b200.lora_linear_train(x2, self.weight, self.lora_A, self.lora_B, self.scale)
        else:
            y = torch.ops.lora_b200.lora_linear(x2, self.weight, self.lora_A, self.lora_B, self.scale)
        return y.reshape(*lead, self.d_out)

    def extra_repr(self) -> str:
        more = (f", dropout={self.dropout:g}" if self.dropout else "") + (", base=e4m3" if self.weight is None else "")
        return f"d_in={self.d_in}, d_out={self.d_out}, r={self.r}, scale={self.scale:g}{more}"
