"""Block-scaled FP8: a power-of-two scale for each block of 128 elements.

Python binding of the block entry points of include/fp8lin.h, and their
autograd forms (compiled: csrc/block_binding.cpp):

  fp8_block_quantize / fp8_block_dequantize   8-bit store and restore
  fp8_block_gemm                              product of two stored matrices
  block_linear, BlockLinear                   training linear, both gradients
  prepare_block_weight, fp8_block_linear_fwd_cached, BlockInferenceLinear
                                              serving linear on a stored weight
  swiglu                                      SwiGLU whose backward reads 8-bit checkpoints
  block_mlp, BlockMLP                         a SwiGLU MLP of all of these

Matrices are bf16 on the device. Rows must be contiguous, with any pitch
and alignment; the autograd forms copy other strides first. Their
derivatives are first-order and reverse-mode: a gradient of a gradient and
forward-mode tangents are refused. Work runs on the current stream of the
tensors' device."""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Tuple

import torch
from torch.autograd import forward_ad

from ._lib import check, load
from .binding import _at, _fmt, _launch

BLOCK = 128
_BF16, _U8 = torch.bfloat16, torch.uint8


def _round(n: int) -> int:
    return -(-n // BLOCK) * BLOCK


def _check_bf16(t: torch.Tensor, name: str) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor (no CPU path exists)")
    if t.dtype is not _BF16:
        raise ValueError(f"{name} must be {_BF16}, got {t.dtype}")


def _check_rows(t: torch.Tensor, name: str) -> None:
    """A 2-D bf16 device matrix with contiguous rows."""
    _check_bf16(t, name)
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"{name} must have contiguous rows")


def _as_rows(t: torch.Tensor, name: str):
    """t [..., n] bf16 as a matrix with contiguous rows (a view where it can
    be): (the matrix, pointer, row pitch, rows, columns)."""
    _check_bf16(t, name)
    if t.dim() != 2:
        t = t.reshape(t.shape[:-1].numel(), t.shape[-1])
    rows, cols = t.shape
    ld, step = t.stride()
    if step != 1 and cols > 1:
        t = t.contiguous()
        ld = cols
    return t, t.data_ptr(), ld, rows, cols


def _same_device(a: torch.Tensor, b: torch.Tensor, name: str) -> None:
    if a.device != b.device:
        raise ValueError(f"{name} must be on {a.device}, got {b.device}")


@functools.lru_cache(maxsize=4096)
def _stored_bytes(rows: int, cols: int) -> int:
    pitch = _round(cols)
    return rows * pitch + _round(rows) * (pitch // BLOCK)


def _check_data(data: torch.Tensor, rows: int, cols: int, name: str) -> None:
    if rows < 0 or cols < 0:
        raise ValueError(f"{name}: negative size [{rows}, {cols}]")
    if data.numel() != _stored_bytes(rows, cols) or data.dtype is not _U8 or data.dim() != 1 or not data.is_contiguous():
        raise ValueError(f"{name} must be {_stored_bytes(rows, cols)} contiguous bytes (uint8, 1-D) for "
                         f"[{rows}, {cols}], got {data.dtype} {tuple(data.shape)}")


def _check_stored(q: "BlockTensor", name: str) -> None:
    _check_data(q.data, q.rows, q.cols, name)
    if not q.data.is_cuda:
        raise ValueError(f"{name} must be on the device (no CPU path exists)")


class BlockTensor:
    """A stored matrix [rows, cols] of an FP8 format: data (uint8) holds the
    codes, [rows, cols rounded up to 128], then the scales in the library's
    order."""

    __slots__ = ("data", "rows", "cols", "fmt")

    def __init__(self, data: torch.Tensor, rows: int, cols: int, fmt):
        _check_data(data, rows, cols, "data")
        self.data, self.rows, self.cols, self.fmt = data, rows, cols, _fmt(fmt)

    @classmethod
    def empty(cls, rows: int, cols: int, fmt, device) -> "BlockTensor":
        return cls(torch.empty(_stored_bytes(rows, cols), dtype=_U8, device=device), rows, cols, fmt)

    @classmethod
    def _made(cls, data: torch.Tensor, rows: int, cols: int, fmt: int) -> "BlockTensor":
        """Of data that was allocated for it: nothing to check."""
        q = cls.__new__(cls)
        q.data, q.rows, q.cols, q.fmt = data, rows, cols, fmt
        return q

    @property
    def shape(self) -> Tuple[int, int]:
        return self.rows, self.cols

    @property
    def device(self):
        return self.data.device

    @property
    def nbytes(self) -> int:
        return self.data.numel()

    @property
    def codes(self) -> torch.Tensor:
        """uint8 [rows, cols rounded up to 128], a view."""
        pitch = _round(self.cols)
        return self.data[:self.rows * pitch].view(self.rows, pitch)

    @property
    def scales(self) -> torch.Tensor:
        """uint8 [blocks, rows rounded up to 128] in the library's order, a view."""
        pitch = _round(self.cols)
        return self.data[self.rows * pitch:].view(pitch // BLOCK, _round(self.rows))

    def pointers(self) -> Tuple[int, int]:
        p = self.data.data_ptr()
        return p, p + self.rows * _round(self.cols)

    def biases(self) -> torch.Tensor:
        """The scaling bias of each block: int32 [rows, blocks]; a code stands for code * 2^-bias."""
        s = self.scales
        nb, sr = s.shape
        s = s.reshape(nb, sr // BLOCK, 16, 8).transpose(2, 3).reshape(nb, sr)
        return 127 - s[:, :self.rows].t().to(torch.int32)

    def dequantize(self, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        return fp8_block_dequantize(self, out)


def fp8_block_quantize(x: torch.Tensor, fmt="e4m3", rowwise: bool = True, transposed: bool = False):
    """The stored form of a bf16 matrix x [rows, cols], blocks along its rows
    (rowwise), and of its transpose [cols, rows], blocks down the columns
    (transposed), from one read. Returns (BlockTensor or None, BlockTensor or None)."""
    _check_rows(x, "x")
    rows, cols = x.shape
    f = _fmt(fmt)
    if not rowwise and not transposed:
        raise ValueError("neither form is wanted")
    q, qt = _at(x, _binding().quantize, x, f, rowwise, transposed)
    return (None if q is None else BlockTensor._made(q, rows, cols, f),
            None if qt is None else BlockTensor._made(qt, cols, rows, f))


def fp8_block_dequantize(q: BlockTensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values of a stored matrix, bf16 [rows, cols]; out: any row pitch."""
    if not q.data.is_cuda:
        raise ValueError("q must be on the device (no CPU path exists)")
    if out is not None:
        if tuple(out.shape) != (q.rows, q.cols):
            raise ValueError("out has the wrong shape")
        _check_rows(out, "out")
        _same_device(q.data, out, "out")
    return _at(q.data, _binding().dequantize, q.data, q.rows, q.cols, q.fmt, out)


def fp8_block_gemm(a: BlockTensor, b: BlockTensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """C [M, N] (bf16) = A B^T of stored A [M, R] and B [N, R], any formats.
    The FP8 matrix instructions drop what of a product lies below 2^-13 of the
    largest of eight neighbours: about 1.5e-5 of a sum, below bf16's 2^-9."""
    if a.cols != b.cols:
        raise ValueError(f"reduction mismatch: A {a.shape}, B {b.shape}")
    _check_stored(a, "A")
    _check_data(b.data, b.rows, b.cols, "B")
    _same_device(a.data, b.data, "B")
    M, N, R = a.rows, b.rows, a.cols
    if out is None:
        out = torch.empty((M, N), dtype=_BF16, device=a.device)
    if tuple(out.shape) != (M, N):
        raise ValueError("out has the wrong shape")
    _check_rows(out, "out")
    _same_device(a.data, out, "out")
    nb = _gemm_bytes(M, N, R)
    ws = torch.empty(nb, dtype=_U8, device=a.device) if nb else None
    _launch(a.data, "fp8_block_gemm", *a.pointers(), a.fmt, *b.pointers(), b.fmt, M, N, R, out.data_ptr(),
            out.stride(0), ws.data_ptr() if nb else None, nb)
    return out


# Sizes of workspaces, by the sizes of the call
@functools.lru_cache(maxsize=4096)
def _gemm_bytes(M: int, N: int, R: int) -> int:
    return load().fp8_block_gemm_workspace_bytes(M, N, R)


def _space(n: int, device) -> torch.Tensor:
    return torch.empty(n, dtype=_U8, device=device)


def _wants_grad(*tensors) -> bool:
    # a dual tensor wants no gradient by requires_grad, and its tangent would be left behind
    if forward_ad._current_level >= 0 and any(forward_ad.unpack_dual(t).tangent is not None for t in tensors):
        raise NotImplementedError("the block-scaled operators have no forward-mode derivatives")
    return torch.is_grad_enabled() and any(t.requires_grad for t in tensors)


@functools.lru_cache(maxsize=None)
def _binding():
    """The compiled binding (csrc/block_binding.cpp)."""
    load()
    try:
        from . import _block_binding
    except ImportError as e:
        raise ImportError("the block-scaled operators' binding is not built; build it with "
                          f"`python -m tensor_scaled_fp8_amd.build` ({e})") from e
    return _block_binding


@functools.lru_cache(maxsize=4096)
def _forward_bytes(entry: str, a: int, b: int, c: int) -> int:
    """Scratch of a linear's or an MLP's forward that keeps nothing."""
    k, f, w = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    check(getattr(load(), entry)(a, b, c, 0, ctypes.byref(k), ctypes.byref(f), ctypes.byref(w)), entry)
    return f.value


def block_linear(X: torch.Tensor, W: torch.Tensor) -> torch.Tensor:
    """Y [..., N] = X [..., K] W [K, N] with block-scaled FP8 operands (E4M3
    X and W, E5M2 dY). The backward reads 8-bit forms kept by the forward,
    only those that the wanted gradients need."""
    if X.dim() < 1 or W.dim() != 2 or X.shape[-1] != W.shape[0]:
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, W {tuple(W.shape)}")
    _same_device(X, W, "W")
    if _wants_grad(X, W):
        _check_bf16(X, "X")
        _check_bf16(W, "W")
        return _at(X, _binding().linear, X, W)
    X2, px, ldx, M, K = _as_rows(X, "X")
    W2, pw, ldw, _, N = _as_rows(W, "W")
    n = _forward_bytes("fp8_block_linear_bytes", M, K, N)
    scratch = _space(n, X.device)
    Y = torch.empty((*X.shape[:-1], N), dtype=_BF16, device=X.device)
    _launch(X, "fp8_block_linear_fwd", px, ldx, pw, ldw, M, K, N, 0, None, 0, scratch.data_ptr(), n, Y.data_ptr())
    return Y


class BlockLinear(torch.nn.Module):
    """Block-scaled FP8 linear (no bias term); weight stored [in, out] in bf16."""

    def __init__(self, in_features: int, out_features: int, device=None):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.empty((in_features, out_features), dtype=_BF16, device=device))
        torch.nn.init.normal_(self.weight, std=0.02)

    def forward(self, x):
        return block_linear(x, self.weight)


def prepare_block_weight(W: torch.Tensor) -> BlockTensor:
    """A bf16 weight W [K, N] stored once for inference: E4M3, transposed [N, K]."""
    return fp8_block_quantize(W, "e4m3", rowwise=False, transposed=True)[1]


def fp8_block_linear_fwd_cached(X: torch.Tensor, w: BlockTensor, Y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y [M, N] = X [M, K] W from a stored weight (prepare_block_weight)."""
    _check_rows(X, "X")
    M, K = X.shape
    N = w.rows
    if w.cols != K or w.fmt != 0:
        raise ValueError(f"X {tuple(X.shape)} does not go with the stored weight {w.shape} (E4M3, transposed)")
    _same_device(X, w.data, "w")
    if Y is not None and (tuple(Y.shape) != (M, N) or Y.dtype is not _BF16 or not Y.is_contiguous() or
                          Y.device != X.device):
        raise ValueError("Y must be a contiguous bf16 [M, N] on X's device")
    return _at(X, _binding().serve, X, w.data, N, Y)


class BlockInferenceLinear(torch.nn.Module):
    """Forward-only block-scaled FP8 linear on a weight stored once."""

    def __init__(self, W: torch.Tensor):
        super().__init__()
        self.register_buffer("weight", prepare_block_weight(W).data)
        self.in_features, self.out_features = W.shape

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        w = BlockTensor(self.weight, self.out_features, self.in_features, 0)
        return fp8_block_linear_fwd_cached(_as_rows(x, "x")[0], w).reshape(*x.shape[:-1], self.out_features)


def swiglu(gate: torch.Tensor, up: torch.Tensor) -> torch.Tensor:
    """h = gate sigmoid(gate) up, [..., F] bf16. For its backward it keeps
    gate and up in 8 bits (block-scaled E4M3), and computes the gradients at
    those values."""
    if gate.shape != up.shape or gate.dim() < 1:
        raise ValueError(f"shape mismatch: gate {tuple(gate.shape)}, up {tuple(up.shape)}")
    _same_device(gate, up, "up")
    if _wants_grad(gate, up):
        _check_bf16(gate, "gate")
        _check_bf16(up, "up")
        return _at(gate, _binding().swiglu, gate, up)
    g2, pg, ldg, rows, cols = _as_rows(gate, "gate")
    u2, pu, ldu, _, _ = _as_rows(up, "up")
    h = torch.empty(gate.shape, dtype=_BF16, device=gate.device)
    _launch(gate, "fp8_swiglu_fwd", pg, ldg, pu, ldu, rows, cols, h.data_ptr(), None, 0)
    return h


def block_mlp(X: torch.Tensor, Wgu: torch.Tensor, Wd: torch.Tensor) -> torch.Tensor:
    """A SwiGLU MLP on block-scaled FP8 operands: X [..., K], Wgu [K, 2 F]
    (gate columns, then up columns), Wd [F, K] -> [..., K]. For the backward
    it keeps X, the gate and up activations and the weights in 8 bits. Outputs
    and gradients are 0.0021 to 0.0025 off the formulas (FP32 products: 0.0017):
    the FP8 products' own error, 1.5e-5, moves some intermediate values to a
    neighbour in 8 bits."""
    if (X.dim() < 1 or Wgu.dim() != 2 or Wd.dim() != 2 or X.shape[-1] != Wgu.shape[0] or
            Wgu.shape[1] != 2 * Wd.shape[0] or Wd.shape[1] != X.shape[-1]):
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, Wgu {tuple(Wgu.shape)}, Wd {tuple(Wd.shape)}")
    _same_device(X, Wgu, "Wgu")
    _same_device(X, Wd, "Wd")
    if _wants_grad(X, Wgu, Wd):
        for t, name in ((X, "X"), (Wgu, "Wgu"), (Wd, "Wd")):
            _check_bf16(t, name)
        return _at(X, _binding().mlp, X, Wgu, Wd)
    X2, px, ldx, M, K = _as_rows(X, "X")
    G2, pg, ldg, _, _ = _as_rows(Wgu, "Wgu")
    D2, pd, ldd, F, _ = _as_rows(Wd, "Wd")
    n = _forward_bytes("fp8_block_mlp_bytes", M, K, F)
    scratch = _space(n, X.device)
    Y = torch.empty(X.shape, dtype=_BF16, device=X.device)
    _launch(X, "fp8_block_mlp_fwd", px, ldx, pg, ldg, pd, ldd, M, K, F, 0, None, 0, scratch.data_ptr(), n, Y.data_ptr())
    return Y


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
