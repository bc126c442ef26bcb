"""Serving operators of an attention layer: a paged key/value cache in 8 bits,
the attention that reads it, and the linear on 4-bit weights.

Python binding of include/fp8lin_serve.h (compiled: csrc/serve_binding.cpp):

  BlockKVCache                                the cache: E4M3, a scale for 16 tokens and a head
  fp8_cache_append, fp8_cache_read            store (rotating on the way) and restore
  fp8_cache_attention                         attention of new tokens over the cache
  prepare_fp4_weight, FP4Tensor               a weight in 4 bits, a scale for 32 elements
  fp4_linear_fwd_cached, FP4InferenceLinear   serving linear on it
  InferenceAttention                          an attention layer of all of these

A batch is packed: sequence i's new tokens are rows starts[i] ..
starts[i + 1] - 1 of the tensors (without starts: one row a sequence), and
lengths[i] counts its tokens with them, so they are at positions up to
lengths[i] - 1. tables [sequences, pages of a sequence] names each sequence's
pages, -1 where it has none. All three are int32 on the device and are read
there: a call never waits, and a captured one replays with what they hold
then. A position without a page is neither stored nor seen, so a padded
sequence is one of length 0; rows behind the last sequence are left alone.

Tensors are bf16 on the device, [tokens, heads, head_dim] of any strides with
a contiguous last dimension. There are no derivatives: tensors that want a
gradient, outputs among them, are refused, and an output that is given counts
as changed in place. Work runs on the current stream of the cache's device."""
from __future__ import annotations

from typing import Optional, Tuple

import torch
from torch.autograd import forward_ad

from .binding import _at
from .block import BlockInferenceLinear, _as_rows, _binding, _wants_grad
from ._lib import load

_U8 = torch.uint8


def _call(t: torch.Tensor, entry: str, *args):
    """A function of the compiled binding with t's device current; it refuses tensors that are on none."""
    f = getattr(_binding(), entry)
    return _at(t, f, *args) if t.is_cuda else f(*args)


def _no_tangent(**tensors):
    """What is stored once is a constant from then on: a parameter may be, a tangent would be left behind."""
    for name, t in tensors.items():
        if forward_ad._current_level >= 0 and t is not None and forward_ad.unpack_dual(t).tangent is not None:
            raise NotImplementedError(f"{name} wants a gradient: the serving operators have none (its tangent would be lost)")


class BlockKVCache:
    """Keys and values of `heads` heads in `pages` pages of page_tokens tokens
    (a power of two, 16 .. 4096); head_dim 64, 128 or 256. E4M3 with a
    power-of-two scale for each 16 tokens of a page and each head: one byte an
    element and one for 16 head_dim. data (uint8) holds the keys' codes, the
    values', then the scales, in the library's order."""

    __slots__ = ("data", "pages", "page_tokens", "heads", "head_dim")

    def __init__(self, pages: int, page_tokens: int, heads: int, head_dim: int, device=None):
        if (page_tokens < 16 or page_tokens > 4096 or page_tokens & (page_tokens - 1) or head_dim not in (64, 128, 256) or
                not 0 < heads <= 1024 or not 0 <= pages < 2 ** 31):
            raise ValueError(f"no cache of {pages} pages of {page_tokens} tokens, {heads} heads of {head_dim}: a page holds "
                             "16 to 4096 tokens, a power of two; a head has 64, 128 or 256 elements")
        sizes = (pages, page_tokens, heads, head_dim)
        n = 2 * load().fp8_cache_codes_bytes(*sizes) + load().fp8_cache_scales_bytes(*sizes)
        self.data = torch.zeros(n, dtype=_U8, device=device)
        self.pages, self.page_tokens, self.heads, self.head_dim = sizes

    @property
    def device(self):
        return self.data.device

    @property
    def nbytes(self) -> int:
        return self.data.numel()

    def _of(self):
        return self.data, self.pages, self.page_tokens, self.heads, self.head_dim


def fp8_cache_append(cache: BlockKVCache, k: torch.Tensor, v: torch.Tensor, tables: torch.Tensor, lengths: torch.Tensor,
                     starts: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                     freqs: Optional[torch.Tensor] = None, interleaved: bool = False,
                     q_out: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """Stores k and v [tokens, heads, head_dim] as the sequences' last tokens.
    With freqs (float32, half as many as the rotated dimensions, a multiple of
    16 from the first on) k and q are rotated by position * freqs: pairs
    (j, j + half), or neighbours if interleaved. Returns q [tokens, any
    multiple of heads, head_dim] rotated, in q_out if given (which may be q
    itself and may not overlap q, k or v otherwise); None without q. Keys are rotated in 64 bits and rounded once. A block's
    scale follows its largest token; earlier tokens of it are rounded anew
    when it grows. A page that two sequences share must not be appended to."""
    return _call(cache.data, "cache_append", *cache._of(), k, v, tables, lengths, starts, q, freqs, interleaved,
               q_out)


def fp8_cache_read(cache: BlockKVCache, tables: torch.Tensor, lengths: torch.Tensor, starts: Optional[torch.Tensor] = None,
                   tokens: Optional[int] = None, k: Optional[torch.Tensor] = None,
                   v: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The sequences' last tokens (starts of `tokens` rows in all; without, one
    each) as the cache holds them: keys and values, bf16 [tokens, heads,
    head_dim], in k and v (which may not overlap) if given; zeros where there
    is no page."""
    if tokens is None:
        if starts is not None:
            raise ValueError("tokens (the rows of all sequences) must be given with starts")
        tokens = lengths.shape[0] if lengths.dim() else 0
    return _call(cache.data, "cache_read", *cache._of(), tables, lengths, starts, tokens, k, v)


def fp8_cache_attention(q: torch.Tensor, cache: BlockKVCache, tables: torch.Tensor, lengths: torch.Tensor,
                        starts: Optional[torch.Tensor] = None, scale: Optional[float] = None, softcap: float = 0.0,
                        window: int = 0, lse: bool = False, out: Optional[torch.Tensor] = None):
    """Attention of q [tokens, any multiple of heads, head_dim] over the cache,
    which holds these tokens' own keys and values already. The query at
    position p sees positions j <= p, and j > p - window if window > 0. Scores
    are scale (default head_dim^-0.5) q . k, then softcap tanh(score / softcap)
    if softcap > 0. Returns [tokens, heads of q, head_dim] (in out, if given,
    which may be q itself and may not overlap it otherwise), 0 where nothing is
    seen; with lse also the logarithms of the sums, float32 [tokens, heads of
    q], -inf there. One form takes the whole batch, chosen by its mean rows:
    decoded tokens over long contexts are faster in a call of their own than
    beside a prompt's chunk (63 of up to 32768 and 2048 tokens of one: 0.37 ms
    in two calls, 1.47 in one), where their softmax weights are rounded as the
    prompt's are (2^-9; 2^-17 alone)."""
    if scale is None:
        scale = cache.head_dim ** -0.5
    o, s = _call(cache.data, "cache_attention", *cache._of(), q, tables, lengths, starts, scale, softcap, window, lse,
               out)
    return (o, s) if lse else o


class FP4Tensor:
    """A stored weight W [K, N] in 4 bits (E2M1, a power-of-two scale for each
    32 elements along K): data (uint8) holds the codes, then the scales, in
    the library's order."""

    __slots__ = ("data", "K", "N")

    def __init__(self, data: torch.Tensor, K: int, N: int):
        n = load().fp4_codes_bytes(K, N) + load().fp4_scales_bytes(K, N) if K >= 0 and N >= 0 else -1
        if data.dtype is not _U8 or data.dim() != 1 or not data.is_contiguous() or data.numel() != n:
            raise ValueError(f"data must be {n} contiguous bytes (uint8, 1-D) for [{K}, {N}], got {data.dtype} "
                             f"{tuple(data.shape)}")
        self.data, self.K, self.N = data, K, N

    @property
    def shape(self) -> Tuple[int, int]:
        return self.K, self.N

    @property
    def device(self):
        return self.data.device

    @property
    def nbytes(self) -> int:
        return self.data.numel()

    def dequantize(self) -> torch.Tensor:
        """Its values, bf16 [K, N]."""
        return _call(self.data, "fp4_restore", self.data, self.K, self.N)


def prepare_fp4_weight(W: torch.Tensor) -> FP4Tensor:
    """A bf16 weight W [K, N] stored once for inference in 4 bits."""
    _no_tangent(W=W)
    data = _call(W, "fp4_store", W.detach())
    return FP4Tensor(data, *W.shape)


def fp4_linear_fwd_cached(X: torch.Tensor, w: FP4Tensor, Y: Optional[torch.Tensor] = None,
                          exact: bool = False) -> torch.Tensor:
    """Y [M, N] = X [M, K] W from a stored 4-bit weight (prepare_fp4_weight);
    X is quantised to E4M3, a scale for each 128 elements of a row. Y, if
    given, is contiguous and does not overlap X. exact: products are exact and
    sums 32-bit at any number of rows, for a Y that is rounded to 8 bits next;
    otherwise those of more than 32 rows are as near as fp8_block_gemm's."""
    return _call(X, "fp4_serve", X, w.data, w.K, w.N, Y, exact)


class FP4InferenceLinear(torch.nn.Module):
    """Forward-only linear on a weight [in, out] stored once in 4 bits; exact:
    as of fp4_linear_fwd_cached."""

    def __init__(self, W: torch.Tensor, exact: bool = False):
        super().__init__()
        self.exact = exact
        self.register_buffer("weight", prepare_fp4_weight(W).data)
        self.in_features, self.out_features = W.shape

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        y = _call(x, "fp4_serve", _as_rows(x, "x")[0], self.weight, self.in_features, self.out_features, None,
                  self.exact)
        return y if x.dim() == 2 else y.reshape(*x.shape[:-1], self.out_features)


class InferenceAttention(torch.nn.Module):
    """Forward-only attention layer on a BlockKVCache: projection to queries,
    keys and values, rotation and append, attention, output projection. Wqkv
    [hidden, (heads + 2 kv_heads) head_dim] (queries, keys, values) and Wo
    [heads head_dim, hidden] are stored once, in 8 bits (a scale for each 128
    elements) or 4 (for each 32). Of 4 bits the projection's products are
    exact, and so are the cache's codes but for 1 in 10^6; of 8 bits they are
    fp8_block_linear_fwd_cached's, which leaves 1 in 1000 of the cache's values
    a step of their 8 bits off (0.001 of them, rms, beside the 0.027 of the 8
    bits' own rounding). Like the weights freqs stay as they are, float32,
    when the module's type is changed."""

    def __init__(self, Wqkv: torch.Tensor, Wo: torch.Tensor, heads: int, kv_heads: int, head_dim: int,
                 freqs: Optional[torch.Tensor] = None, interleaved: bool = False, scale: Optional[float] = None,
                 softcap: float = 0.0, window: int = 0, bits: int = 8):
        super().__init__()
        if Wqkv.dim() != 2 or Wqkv.shape[1] != (heads + 2 * kv_heads) * head_dim or Wo.dim() != 2 or \
                Wo.shape[0] != heads * head_dim:
            raise ValueError(f"shape mismatch: Wqkv {tuple(Wqkv.shape)}, Wo {tuple(Wo.shape)} for {heads} and {kv_heads} "
                             f"heads of {head_dim}")
        if bits not in (4, 8):
            raise ValueError(f"weights are stored in 4 or 8 bits, got {bits}")
        if freqs is not None and (freqs.dtype is not torch.float32 or freqs.dim() != 1):
            raise ValueError(f"freqs must be float32 and 1-D, got {freqs.dtype} {tuple(freqs.shape)}")
        # what the attention would refuse after the tokens are appended
        if kv_heads <= 0 or heads <= 0 or heads % kv_heads or head_dim not in (64, 128, 256):
            raise ValueError(f"{heads} and {kv_heads} heads of {head_dim}: query heads are a multiple of the key heads, a head "
                             "has 64, 128 or 256 elements")
        if freqs is not None and (freqs.numel() % 8 or 2 * freqs.numel() > head_dim):
            raise ValueError(f"freqs must be half as many as the rotated dimensions, a multiple of 16 up to {head_dim}, got "
                             f"{freqs.numel()}")
        if scale is not None and not abs(scale) <= 2.0 ** 64:
            raise ValueError("scale must be finite, up to 2^64")
        if not (softcap == 0 or 2.0 ** -64 <= softcap <= 2.0 ** 64):
            raise ValueError("softcap must be 0 or between 2^-64 and 2^64")
        if not 0 <= window < 2 ** 31:
            raise ValueError("window must be between 0 and 2^31 - 1")
        _no_tangent(Wqkv=Wqkv, Wo=Wo, freqs=freqs)
        # keys and values go to 8 bits next
        self.qkv = FP4InferenceLinear(Wqkv.detach(), exact=True) if bits == 4 else BlockInferenceLinear(Wqkv.detach())
        self.out = (FP4InferenceLinear if bits == 4 else BlockInferenceLinear)(Wo.detach())
        self.register_buffer("freq_bytes", None if freqs is None else freqs.detach().contiguous().view(_U8))
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.interleaved, self.scale, self.softcap, self.window = interleaved, scale, softcap, window

    @property
    def freqs(self) -> Optional[torch.Tensor]:
        return None if self.freq_bytes is None else self.freq_bytes.view(torch.float32)

    def forward(self, x: torch.Tensor, cache: BlockKVCache, tables: torch.Tensor, lengths: torch.Tensor,
                starts: Optional[torch.Tensor] = None) -> torch.Tensor:
        """x [tokens, hidden]: appends the tokens' keys and values to the cache and returns [tokens, out features]."""
        if x.dim() != 2:
            raise ValueError(f"x must be [tokens, hidden], got {tuple(x.shape)}")
        if _wants_grad(x):
            raise NotImplementedError("x wants a gradient: the serving operators have none (use torch.no_grad())")
        h, g, d = self.heads, self.kv_heads, self.head_dim
        qkv = self.qkv(x).view(-1, h + 2 * g, d)
        q, k, v = qkv[:, :h], qkv[:, h:h + g], qkv[:, h + g:]
        fp8_cache_append(cache, k, v, tables, lengths, starts, q, self.freqs, self.interleaved, q)
        o = fp8_cache_attention(q, cache, tables, lengths, starts, self.scale, self.softcap, self.window)
        return self.out(o.view(-1, h * d))
