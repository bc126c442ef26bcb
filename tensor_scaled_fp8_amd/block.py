"""Block-scaled FP8: a power-of-two scale for each block of 128 elements.

Python binding of the block entry points of include/fp8lin.h, and their
autograd forms:

  fp8_block_quantize / fp8_block_dequantize   8-bit store and restore
  fp8_block_gemm                              product of two stored matrices
  block_linear, BlockLinear                   training linear, both gradients
  prepare_block_weight, fp8_block_linear_fwd_cached, BlockInferenceLinear
                                              serving linear on a stored weight
  swiglu                                      SwiGLU whose backward reads 8-bit checkpoints
  block_mlp, BlockMLP                         a SwiGLU MLP of all of these

Matrices are bf16 on the device. Rows must be contiguous, with any pitch
and alignment; the autograd forms copy other strides first. Work runs on
the current stream of the tensors' device."""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Tuple

import torch

from ._lib import (FP8_BLOCK_NEED_DW, FP8_BLOCK_NEED_DW2, FP8_BLOCK_NEED_DX, check, load)
from .binding import _fmt, _stream

BLOCK = 128


def _round(n: int) -> int:
    return -(-n // BLOCK) * BLOCK


def _rows(t: torch.Tensor, name: str) -> Tuple[int, int]:
    """(pointer, row pitch) of a 2-D bf16 device matrix with contiguous rows."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor (no CPU path exists)")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    ld, step = t.stride()
    if step != 1 and t.shape[1] > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return t.data_ptr(), ld


def _same_device(a: torch.Tensor, b: torch.Tensor, name: str) -> None:
    if a.device != b.device:
        raise ValueError(f"{name} must be on {a.device}, got {b.device}")


def _as_rows(t: torch.Tensor) -> torch.Tensor:
    """t [..., n] as a matrix with contiguous rows (a view where it can be)."""
    if t.dim() != 2:
        t = t.reshape(t.shape[:-1].numel(), t.shape[-1])
    return t if t.stride(1) == 1 or t.shape[1] <= 1 else t.contiguous()


class BlockTensor:
    """A stored matrix [rows, cols]: codes (uint8 [rows, cols rounded up to
    128]), scales (uint8, in the library's order) and the FP8 format."""

    __slots__ = ("codes", "scales", "rows", "cols", "fmt")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, rows: int, cols: int, fmt: int):
        self.codes, self.scales, self.rows, self.cols, self.fmt = codes, scales, rows, cols, fmt

    @classmethod
    def empty(cls, rows: int, cols: int, fmt, device) -> "BlockTensor":
        pitch = _round(cols)
        codes = torch.empty((rows, pitch), dtype=torch.uint8, device=device)
        scales = torch.empty((pitch // BLOCK, _round(rows)), dtype=torch.uint8, device=device)
        return cls(codes, scales, rows, cols, _fmt(fmt))

    @property
    def shape(self) -> Tuple[int, int]:
        return self.rows, self.cols

    @property
    def device(self):
        return self.codes.device

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()

    def biases(self) -> torch.Tensor:
        """The scaling bias of each block: int32 [rows, blocks]; a code stands for code * 2^-bias."""
        nb, sr = self.scales.shape
        s = self.scales.reshape(nb, sr // BLOCK, 16, 8).transpose(2, 3).reshape(nb, sr)
        return 127 - s[:, :self.rows].t().to(torch.int32)

    def dequantize(self, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        return fp8_block_dequantize(self, out)


def fp8_block_quantize(x: torch.Tensor, fmt="e4m3", rowwise: bool = True, transposed: bool = False):
    """The stored form of a bf16 matrix x [rows, cols], blocks along its rows
    (rowwise), and of its transpose [cols, rows], blocks down the columns
    (transposed), from one read. Returns (BlockTensor or None, BlockTensor or None)."""
    p, ld = _rows(x, "x")
    rows, cols = x.shape
    f = _fmt(fmt)
    if not rowwise and not transposed:
        raise ValueError("neither form is wanted")
    q = BlockTensor.empty(rows, cols, f, x.device) if rowwise else None
    qt = BlockTensor.empty(cols, rows, f, x.device) if transposed else None
    check(load().fp8_block_quantize(p, rows, cols, ld, f, q.codes.data_ptr() if rowwise else None,
                                    q.scales.data_ptr() if rowwise else None,
                                    qt.codes.data_ptr() if transposed else None,
                                    qt.scales.data_ptr() if transposed else None, _stream(x)), "fp8_block_quantize")
    return q, qt


def fp8_block_dequantize(q: BlockTensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values of a stored matrix, bf16 [rows, cols]; out: any row pitch."""
    if out is None:
        out = torch.empty((q.rows, q.cols), dtype=torch.bfloat16, device=q.codes.device)
        p, ld = out.data_ptr(), q.cols
    else:
        if tuple(out.shape) != (q.rows, q.cols):
            raise ValueError("out has the wrong shape")
        p, ld = _rows(out, "out")
        _same_device(q.codes, out, "out")
    check(load().fp8_block_dequantize(q.codes.data_ptr(), q.scales.data_ptr(), q.rows, q.cols, q.fmt, p, ld,
                                      _stream(out)), "fp8_block_dequantize")
    return out


def fp8_block_gemm(a: BlockTensor, b: BlockTensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """C [M, N] (bf16) = A B^T of stored A [M, R] and B [N, R], any formats."""
    if a.cols != b.cols:
        raise ValueError(f"reduction mismatch: A {a.shape}, B {b.shape}")
    _same_device(a.codes, b.codes, "B")
    M, N, R = a.rows, b.rows, a.cols
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    if tuple(out.shape) != (M, N):
        raise ValueError("out has the wrong shape")
    p, ld = _rows(out, "out")
    _same_device(a.codes, out, "out")
    lib = load()
    nb = lib.fp8_block_gemm_workspace_bytes(M, N, R)
    ws = torch.empty(nb, dtype=torch.uint8, device=a.device) if nb else None
    check(lib.fp8_block_gemm(a.codes.data_ptr(), a.scales.data_ptr(), a.fmt, b.codes.data_ptr(), b.scales.data_ptr(),
                             b.fmt, M, N, R, p, ld, ws.data_ptr() if nb else None, nb, _stream(out)), "fp8_block_gemm")
    return out


@functools.lru_cache(maxsize=4096)
def _bytes(entry: str, a: int, b: int, c: int, flags: int) -> Tuple[int, int, int]:
    """Sizes of (kept, forward scratch, backward scratch) of a linear or an MLP."""
    k, f, w = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    check(getattr(load(), entry)(a, b, c, flags, ctypes.byref(k), ctypes.byref(f), ctypes.byref(w)), entry)
    return k.value, f.value, w.value


def _space(n: int, device) -> torch.Tensor:
    return torch.empty(n, dtype=torch.uint8, device=device)


def _flags(ctx) -> int:
    need = ctx.needs_input_grad
    return sum(f for f, n in zip((FP8_BLOCK_NEED_DX, FP8_BLOCK_NEED_DW, FP8_BLOCK_NEED_DW2), need) if n)


def _grad_rows(dy: torch.Tensor) -> torch.Tensor:
    if dy.dtype != torch.bfloat16:
        dy = dy.to(torch.bfloat16)
    return _as_rows(dy)


class _BlockLinearFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, W):
        X2, W2 = _as_rows(X), _as_rows(W)
        (px, ldx), (pw, ldw) = _rows(X2, "X"), _rows(W2, "W")
        M, K = X2.shape
        N = W2.shape[1]
        flags = _flags(ctx)
        nk, nf, _ = _bytes("fp8_block_linear_bytes", M, K, N, flags)
        kept = _space(nk, X.device)
        scratch = _space(nf, X.device)
        Y = torch.empty((*X.shape[:-1], N), dtype=torch.bfloat16, device=X.device)
        check(load().fp8_block_linear_fwd(px, ldx, pw, ldw, M, K, N, flags, kept.data_ptr(), nk, scratch.data_ptr(), nf,
                                          Y.data_ptr(), _stream(X)), "fp8_block_linear_fwd")
        if flags:
            ctx.save_for_backward(kept)
            ctx.flags, ctx.size, ctx.lead = flags, (M, K, N), X.shape[:-1]
        return Y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dY):
        kept, = ctx.saved_tensors
        M, K, N = ctx.size
        flags = ctx.flags
        dY2 = _grad_rows(dY)
        p, ld = _rows(dY2, "dY")
        nk, _, nb = _bytes("fp8_block_linear_bytes", M, K, N, flags)
        scratch = _space(nb, dY.device)
        new = dict(dtype=torch.bfloat16, device=dY.device)
        dX = torch.empty((*ctx.lead, K), **new) if flags & FP8_BLOCK_NEED_DX else None
        dW = torch.empty((K, N), **new) if flags & FP8_BLOCK_NEED_DW else None
        check(load().fp8_block_linear_bwd(p, ld, M, K, N, flags, kept.data_ptr(), nk, scratch.data_ptr(), nb,
                                          None if dX is None else dX.data_ptr(), None if dW is None else dW.data_ptr(),
                                          _stream(dY)), "fp8_block_linear_bwd")
        return dX, dW


def block_linear(X: torch.Tensor, W: torch.Tensor) -> torch.Tensor:
    """Y [..., N] = X [..., K] W [K, N] with block-scaled FP8 operands (E4M3
    X and W, E5M2 dY). The backward reads 8-bit forms kept by the forward,
    only those that the wanted gradients need."""
    if X.dim() < 1 or W.dim() != 2 or X.shape[-1] != W.shape[0]:
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, W {tuple(W.shape)}")
    _same_device(X, W, "W")
    return _BlockLinearFn.apply(X, W)


class BlockLinear(torch.nn.Module):
    """Block-scaled FP8 linear (no bias term); weight stored [in, out] in bf16."""

    def __init__(self, in_features: int, out_features: int, device=None):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.empty((in_features, out_features), dtype=torch.bfloat16, device=device))
        torch.nn.init.normal_(self.weight, std=0.02)

    def forward(self, x):
        return block_linear(x, self.weight)


def prepare_block_weight(W: torch.Tensor) -> BlockTensor:
    """A bf16 weight W [K, N] stored once for inference: E4M3, transposed [N, K]."""
    return fp8_block_quantize(W, "e4m3", rowwise=False, transposed=True)[1]


def fp8_block_linear_fwd_cached(X: torch.Tensor, w: BlockTensor, Y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y [M, N] = X [M, K] W from a stored weight (prepare_block_weight)."""
    p, ld = _rows(X, "X")
    M, K = X.shape
    N = w.rows
    if w.cols != K or w.fmt != 0:
        raise ValueError(f"X {tuple(X.shape)} does not go with the stored weight {w.shape} (E4M3, transposed)")
    _same_device(X, w.codes, "w")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    elif tuple(Y.shape) != (M, N) or Y.dtype != torch.bfloat16 or not Y.is_contiguous() or Y.device != X.device:
        raise ValueError("Y must be a contiguous bf16 [M, N] on X's device")
    lib = load()
    nb = lib.fp8_block_linear_cached_bytes(M, K, N)
    scratch = _space(nb, X.device)
    check(lib.fp8_block_linear_fwd_cached(p, ld, M, K, N, w.codes.data_ptr(), w.scales.data_ptr(), scratch.data_ptr(),
                                          nb, Y.data_ptr(), _stream(X)), "fp8_block_linear_fwd_cached")
    return Y


class BlockInferenceLinear(torch.nn.Module):
    """Forward-only block-scaled FP8 linear on a weight stored once."""

    def __init__(self, W: torch.Tensor):
        super().__init__()
        q = prepare_block_weight(W)
        self.register_buffer("codes", q.codes)
        self.register_buffer("scales", q.scales)
        self.in_features, self.out_features = q.cols, q.rows

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        w = BlockTensor(self.codes, self.scales, self.out_features, self.in_features, 0)
        return fp8_block_linear_fwd_cached(_as_rows(x), w).reshape(*x.shape[:-1], self.out_features)


class _SwigluFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gate, up):
        g2, u2 = _as_rows(gate), _as_rows(up)
        (pg, ldg), (pu, ldu) = _rows(g2, "gate"), _rows(u2, "up")
        rows, cols = g2.shape
        lib = load()
        n = 0
        kept = None
        if any(ctx.needs_input_grad):
            n = lib.fp8_swiglu_kept_bytes(rows, cols)
            kept = _space(n, gate.device)
            ctx.save_for_backward(kept)
            ctx.size, ctx.shape = (rows, cols), gate.shape
        h = torch.empty(gate.shape, dtype=torch.bfloat16, device=gate.device)
        check(lib.fp8_swiglu_fwd(pg, ldg, pu, ldu, rows, cols, h.data_ptr(), kept.data_ptr() if n else None, n,
                                 _stream(gate)), "fp8_swiglu_fwd")
        return h

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dh):
        kept, = ctx.saved_tensors
        rows, cols = ctx.size
        dh2 = _grad_rows(dh)
        p, ld = _rows(dh2, "dh")
        new = dict(dtype=torch.bfloat16, device=dh.device)
        dg = torch.empty(ctx.shape, **new) if ctx.needs_input_grad[0] else None
        du = torch.empty(ctx.shape, **new) if ctx.needs_input_grad[1] else None
        check(load().fp8_swiglu_bwd(p, ld, rows, cols, kept.data_ptr(), kept.numel(),
                                    None if dg is None else dg.data_ptr(), None if du is None else du.data_ptr(),
                                    _stream(dh)), "fp8_swiglu_bwd")
        return dg, du


def swiglu(gate: torch.Tensor, up: torch.Tensor) -> torch.Tensor:
    """h = gate sigmoid(gate) up, [..., F] bf16. For its backward it keeps
    gate and up in 8 bits (block-scaled E4M3), and computes the gradients at
    those values."""
    if gate.shape != up.shape or gate.dim() < 1:
        raise ValueError(f"shape mismatch: gate {tuple(gate.shape)}, up {tuple(up.shape)}")
    _same_device(gate, up, "up")
    return _SwigluFn.apply(gate, up)


class _BlockMlpFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, Wgu, Wd):
        X2, G2, D2 = _as_rows(X), _as_rows(Wgu), _as_rows(Wd)
        (px, ldx), (pg, ldg), (pd, ldd) = _rows(X2, "X"), _rows(G2, "Wgu"), _rows(D2, "Wd")
        M, K = X2.shape
        F = D2.shape[0]
        flags = _flags(ctx)
        nk, nf, _ = _bytes("fp8_block_mlp_bytes", M, K, F, flags)
        kept = _space(nk, X.device)
        scratch = _space(nf, X.device)
        Y = torch.empty(X.shape, dtype=torch.bfloat16, device=X.device)
        check(load().fp8_block_mlp_fwd(px, ldx, pg, ldg, pd, ldd, M, K, F, flags, kept.data_ptr(), nk,
                                       scratch.data_ptr(), nf, Y.data_ptr(), _stream(X)), "fp8_block_mlp_fwd")
        if flags:
            ctx.save_for_backward(kept)
            ctx.flags, ctx.size, ctx.shape = flags, (M, K, F), X.shape
        return Y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dY):
        kept, = ctx.saved_tensors
        M, K, F = ctx.size
        flags = ctx.flags
        dY2 = _grad_rows(dY)
        p, ld = _rows(dY2, "dY")
        nk, _, nb = _bytes("fp8_block_mlp_bytes", M, K, F, flags)
        scratch = _space(nb, dY.device)
        new = dict(dtype=torch.bfloat16, device=dY.device)
        dX = torch.empty(ctx.shape, **new) if flags & FP8_BLOCK_NEED_DX else None
        dWgu = torch.empty((K, 2 * F), **new) if flags & FP8_BLOCK_NEED_DW else None
        dWd = torch.empty((F, K), **new) if flags & FP8_BLOCK_NEED_DW2 else None
        check(load().fp8_block_mlp_bwd(p, ld, M, K, F, flags, kept.data_ptr(), nk, scratch.data_ptr(), nb,
                                       *[None if t is None else t.data_ptr() for t in (dX, dWgu, dWd)], _stream(dY)),
              "fp8_block_mlp_bwd")
        return dX, dWgu, dWd


def block_mlp(X: torch.Tensor, Wgu: torch.Tensor, Wd: torch.Tensor) -> torch.Tensor:
    """A SwiGLU MLP on block-scaled FP8 operands: X [..., K], Wgu [K, 2 F]
    (gate columns, then up columns), Wd [F, K] -> [..., K]. For the backward
    it keeps X, the gate and up activations and the weights in 8 bits."""
    if (X.dim() < 1 or Wgu.dim() != 2 or Wd.dim() != 2 or X.shape[-1] != Wgu.shape[0] or
            Wgu.shape[1] != 2 * Wd.shape[0] or Wd.shape[1] != X.shape[-1]):
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, Wgu {tuple(Wgu.shape)}, Wd {tuple(Wd.shape)}")
    _same_device(X, Wgu, "Wgu")
    _same_device(X, Wd, "Wd")
    return _BlockMlpFn.apply(X, Wgu, Wd)


class BlockMLP(torch.nn.Module):
    """SwiGLU MLP of a transformer layer on block-scaled FP8 operands (no biases)."""

    def __init__(self, hidden: int, intermediate: int, device=None):
        super().__init__()
        new = dict(dtype=torch.bfloat16, device=device)
        self.gate_up = torch.nn.Parameter(torch.empty((hidden, 2 * intermediate), **new))
        self.down = torch.nn.Parameter(torch.empty((intermediate, hidden), **new))
        torch.nn.init.normal_(self.gate_up, std=0.02)
        torch.nn.init.normal_(self.down, std=0.02)

    def forward(self, x):
        return block_mlp(x, self.gate_up, self.down)
