"""The operators around the QLoRA linears of a decoder: rotary positions, a paged key/value
cache of 8 bits with its append and its attention, and the vocabulary head's softmax cross
entropy.  Thin binding over ``include/qlora_decoder.h``; the rules of the package hold (GPU
tensors, the current stream, no fallback, ``ValueError`` for a bad tensor and ``NF4Error``
for what the library refuses).

Rotary positions: Su et al., "RoFormer" (2021); the scalings "ntk" and "parts" for contexts
longer than a model was trained on follow the base change and the by-parts interpolation of
Peng et al., "YaRN" (2023).
"""
import ctypes
import functools
import math
from dataclasses import dataclass
from typing import Optional

import torch

from . import NF4_BF16, NF4_F32, _check, _dev, _ptr, _same_device, _stream, _workspace, load_library

__all__ = ["RopePlan", "rope_plan", "rope_fwd", "rope_bwd", "KVCache", "kv_cache", "kv_append", "kv_attention",
           "head_loss"]

_vp, _i64, _i32, _sz, _f = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float


class _Heads(ctypes.Structure):
    _fields_ = [("data", _vp), ("token_stride", _i64), ("head_stride", _i64), ("heads", _i32)]


class _Rope(ctypes.Structure):
    _fields_ = [("freq", _vp), ("rotary_dim", _i32), ("interleaved", _i32), ("magnitude", _f)]


class _Cache(ctypes.Structure):
    _fields_ = [("codes", _vp), ("scales", _vp), ("pages", _i64), ("kv_heads", _i32), ("page_size", _i32),
                ("head_dim", _i32)]


class _Batch(ctypes.Structure):
    _fields_ = [("starts", _vp), ("lengths", _vp), ("table", _vp), ("table_stride", _i64), ("tokens", _i64),
                ("seqs", _i32), ("table_width", _i32)]


_bound = None


def _library():
    global _bound
    if _bound is None:
        L = load_library()
        p = ctypes.POINTER
        L.qlora_rope_apply.restype = ctypes.c_int
        L.qlora_rope_apply.argtypes = [p(_Rope), _i32, _vp, _i64, _i32, ctypes.c_int, p(_Heads), p(_Heads), _i32, _vp]
        L.qlora_kv_append.restype = ctypes.c_int
        L.qlora_kv_append.argtypes = [p(_Cache), p(_Batch), p(_Heads), p(_Heads), p(_Rope), p(_Heads), p(_Heads), _vp]
        L.qlora_kv_attention_workspace_bytes.restype = _sz
        L.qlora_kv_attention_workspace_bytes.argtypes = [p(_Cache), p(_Batch), _i32, _i64, _i64]
        L.qlora_kv_attention.restype = ctypes.c_int
        L.qlora_kv_attention.argtypes = [p(_Cache), p(_Batch), p(_Heads), p(_Heads), _f, _i64, _i64, _vp, _sz, _vp]
        L.qlora_head_loss_workspace_bytes.restype = _sz
        L.qlora_head_loss_workspace_bytes.argtypes = [_i64, _i64, _i64, _i32, _i32]
        L.qlora_head_loss.restype = ctypes.c_int
        L.qlora_head_loss.argtypes = [_vp, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
        _bound = L
    return _bound


# The calls below serve single tokens, where the host's time counts: each tensor is asked
# once for its shape, strides, type and device, and the stream is taken as a raw handle.
def _on(t: torch.Tensor, name: str, dtype, dev: int) -> int:
    """Address of a dense tensor of the given type on device `dev`."""
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.get_device() != dev:
        raise ValueError("%s must be on the same GPU as the other operands, got %s" % (name, t.device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _device(t: torch.Tensor, name: str) -> int:
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor" % name)
    return t.get_device()


def _heads(t: torch.Tensor, name: str, dtype, tokens: int, dim: int, dev: int) -> _Heads:
    """A [tokens, heads, dim] tensor of any token and head strides."""
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.get_device() != dev:
        raise ValueError("%s must be on the same GPU as the other operands, got %s" % (name, t.device))
    shape = t.shape
    if len(shape) != 3 or shape[0] != tokens or shape[2] != dim or shape[1] < 1:
        raise ValueError("%s must be [%d, heads, %d], got %s" % (name, tokens, dim, tuple(shape)))
    token_stride, head_stride, last = t.stride()
    if last != 1 and tokens:
        raise ValueError("%s must be dense along its last dimension" % name)
    heads = shape[1]
    if heads == 1:                      # the stride of a dimension of one is not looked at
        head_stride = dim
    if tokens <= 1:
        token_stride = heads * head_stride
    return _Heads(t.data_ptr(), token_stride, head_stride, heads)


def _fresh_heads(like: torch.Tensor, tokens: int, dim: int):
    """A new dense tensor of `like`'s shape and type, and its description."""
    out = torch.empty(like.shape, dtype=like.dtype, device=like.device)
    heads = out.shape[1]
    return out, _Heads(out.data_ptr(), heads * dim, dim, heads)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


# ---------------------------------------------------------------------------
# Rotary positions
# ---------------------------------------------------------------------------
@dataclass
class RopePlan:
    """A rotation: the frequencies of its pairs (int64 on the GPU; 2^64 is one turn per
    position), the rotated size of a head, the layout of the pairs and the factor on them."""
    freq: torch.Tensor
    rotary_dim: int
    interleaved: bool = False
    magnitude: float = 1.0

    def _struct(self, dev):
        freq = self.freq
        if freq.numel() * 2 != self.rotary_dim:
            raise ValueError("freq must hold rotary_dim / 2 = %d values" % (self.rotary_dim // 2))
        return _Rope(_on(freq, "freq", torch.int64, dev), self.rotary_dim, self.interleaved, self.magnitude)


def rope_plan(rotary_dim: int, base: float = 10000.0, *, interleaved: bool = False, scaling: Optional[str] = None,
              factor: float = 1.0, original_length: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0,
              device="cuda") -> RopePlan:
    """The rotation of the first `rotary_dim` values of a head: pair i turns by
    base^(-2i/rotary_dim) per position.  Pairs are (i, i + rotary_dim/2), or (2i, 2i+1) if
    `interleaved`.  `scaling` stretches it to `factor` times the trained context:
      "linear"  every angle divided by factor
      "ntk"     base * factor^(rotary_dim/(rotary_dim-2))
      "parts"   pairs that turn fewer than beta_slow times over `original_length` positions are
                divided by factor, those that turn more than beta_fast times are left, with a
                linear ramp between; queries and keys are multiplied by 0.1 ln(factor) + 1"""
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and at least 2")
    if not (base > 0 and math.isfinite(base)) or not (factor > 0 and math.isfinite(factor)):
        raise ValueError("base and factor must be positive and finite")
    n, magnitude = rotary_dim // 2, 1.0
    if scaling == "ntk":
        if rotary_dim < 4:
            raise ValueError("ntk scaling needs rotary_dim of at least 4")
        base = base * factor ** (rotary_dim / (rotary_dim - 2.0))
    theta = [base ** (-2.0 * i / rotary_dim) for i in range(n)]
    if scaling == "linear":
        theta = [t / factor for t in theta]
    elif scaling == "parts":
        if original_length < 1 or not beta_fast > beta_slow > 0 or base <= 1:
            raise ValueError("parts scaling needs original_length, beta_fast > beta_slow > 0 and base > 1")
        at = [rotary_dim * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))
              for turns in (beta_fast, beta_slow)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rotary_dim - 1)
        ramp = [min(1.0, max(0.0, (i - low) / max(high - low, 1e-3))) for i in range(n)]
        theta = [t * (1 - r) + t / factor * r for t, r in zip(theta, ramp)]
        magnitude = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    elif scaling not in (None, "none", "ntk"):
        raise ValueError("scaling must be None, 'linear', 'ntk' or 'parts', got %r" % (scaling,))
    # whole turns per position drop out; 2^64 is one turn
    turns = [int((t / (2 * math.pi)) % 1.0 * 2.0 ** 64) for t in theta]
    freq = torch.tensor([t - (1 << 64) if t >= 1 << 63 else t for t in turns], dtype=torch.int64, device=device)
    return RopePlan(freq, rotary_dim, bool(interleaved), magnitude)


_Heads2 = _Heads * 2


def _rope(plan, positions, q, k, inplace, backward):
    dev = _device(q, "q")
    dtype = q.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise ValueError("q must be float32 or bfloat16, got %s" % dtype)
    M, dim = positions.numel(), q.shape[-1]
    at = _on(positions, "positions", torch.int32, dev)
    rope = plan._struct(dev)
    ins = _Heads2(_heads(q, "q", dtype, M, dim, dev))
    if k is not None:
        ins[1] = _heads(k, "k", dtype, M, dim, dev)
    yq, yk, outs = q, k, ins
    if not inplace:
        yq, hq = _fresh_heads(q, M, dim)
        outs = _Heads2(hq)
        if k is not None:
            yk, outs[1] = _fresh_heads(k, M, dim)
    _check(_library().qlora_rope_apply(rope, backward, at, M, dim, NF4_BF16 if dtype is torch.bfloat16 else NF4_F32, ins,
                                       outs, 1 if k is None else 2, _raw_stream(dev)))
    return yq if k is None else (yq, yk)


def rope_fwd(plan: RopePlan, positions: torch.Tensor, q: torch.Tensor, k: Optional[torch.Tensor] = None,
             inplace: bool = False):
    """Queries, and keys if given, rotated to their positions: q [tokens, heads, dim], k
    [tokens, kv_heads, dim] (fp32 or bf16, the same type; any strides with a dense last
    dimension), positions int32 [tokens].  Returns new dense tensors, or the same ones if `inplace`."""
    return _rope(plan, positions, q, k, inplace, 0)


def rope_bwd(plan: RopePlan, positions: torch.Tensor, dq: torch.Tensor, dk: Optional[torch.Tensor] = None,
             inplace: bool = False):
    """The gradient of rope_fwd: dq and dk turned back, times the same magnitude."""
    return _rope(plan, positions, dq, dk, inplace, 1)


# ---------------------------------------------------------------------------
# The paged 8-bit cache
# ---------------------------------------------------------------------------
@dataclass
class KVCache:
    """Keys and values in pages: codes uint8 [pages, 2, kv_heads, page_size, head_dim] (E4M3,
    index 0 the keys), scales float32 [pages, 2, kv_heads] (powers of two)."""
    codes: torch.Tensor
    scales: torch.Tensor

    def _struct(self, dev):
        codes, scales = self.codes, self.scales
        shape = codes.shape
        if len(shape) != 5 or shape[1] != 2:
            raise ValueError("codes must be [pages, 2, kv_heads, page_size, head_dim], got %s" % (tuple(shape),))
        if scales.shape != shape[:3]:
            raise ValueError("scales must be %s, got %s" % (tuple(shape[:3]), tuple(scales.shape)))
        return _Cache(_on(codes, "codes", torch.uint8, dev), _on(scales, "scales", torch.float32, dev), shape[0], shape[2],
                      shape[3], shape[4])

    def decode(self, dtype=torch.float32) -> torch.Tensor:
        """What the codes stand for, [pages, 2, kv_heads, page_size, head_dim] (for looking at)."""
        return (self.codes.view(torch.float8_e4m3fn).float() * self.scales[..., None, None]).to(dtype)


def kv_cache(pages: int, kv_heads: int, head_dim: int, page_size: int = 64, device="cuda") -> KVCache:
    """An empty cache of `pages` pages."""
    return KVCache(torch.zeros((pages, 2, kv_heads, page_size, head_dim), dtype=torch.uint8, device=device),
                   torch.ones((pages, 2, kv_heads), dtype=torch.float32, device=device))


def _batch(starts, lengths, table, tokens, dev):
    shape = table.shape
    if len(shape) != 2:
        raise ValueError("table must be [seqs, pages of a sequence], got %s" % (tuple(shape),))
    seqs, width = shape
    if tuple(lengths.shape) != (seqs,) or tuple(starts.shape) != (seqs + 1,):
        raise ValueError("lengths must be [%d] and starts [%d], as the table has %d rows" % (seqs, seqs + 1, seqs))
    stride, last = table.stride()
    if last != 1 and width > 1:
        raise ValueError("table must be dense along its rows")
    if table.dtype != torch.int32 or table.get_device() != dev:
        raise ValueError("table must be torch.int32 on the same GPU as the other operands, got %s on %s" % (table.dtype, table.device))
    return _Batch(_on(starts, "starts", torch.int32, dev), _on(lengths, "lengths", torch.int32, dev), table.data_ptr(),
                  stride if seqs > 1 else width, tokens, seqs, width)


def kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, starts: torch.Tensor, lengths: torch.Tensor,
              table: torch.Tensor, rope: Optional[RopePlan] = None, q: Optional[torch.Tensor] = None):
    """Appends the keys and values of new tokens, packed sequence after sequence, to their
    pages; `rope` rotates the keys on the way, and the queries `q` of the same tokens, which
    are returned (a new dense tensor; None without q).
      k, v     bf16 [tokens, kv_heads, head_dim], rows 16-byte aligned (slices of a fused projection serve)
      q        bf16 [tokens, heads, head_dim]
      starts   int32 [seqs + 1]: sequence b has the tokens starts[b] .. starts[b+1] - 1
      lengths  int32 [seqs]: tokens of each sequence before these (negative: an unused row)
      table    int32 [seqs, pages of a sequence]: the pool's page of each page_size positions
    The caller moves its lengths on by the new tokens after the attention of the same step."""
    dev = _device(k, "k")
    c = cache._struct(dev)
    T, dim = k.shape[0], c.head_dim
    b = _batch(starts, lengths, table, T, dev)
    kh, vh = _heads(k, "k", torch.bfloat16, T, dim, dev), _heads(v, "v", torch.bfloat16, T, dim, dev)
    out = qh = oh = None
    if q is not None:
        qh = _heads(q, "q", torch.bfloat16, T, dim, dev)
        out, oh = _fresh_heads(q, T, dim)
    _check(_library().qlora_kv_append(c, b, kh, vh, None if rope is None else rope._struct(dev), qh, oh, _raw_stream(dev)))
    return out


@functools.lru_cache(maxsize=1024)
def _attention_ws_bytes(kv_heads, page_size, head_dim, seqs, tokens, heads, max_new, max_length):
    """Workspace of an attention of these sizes (a plain function of them)."""
    some = 4096                         # addresses that are checked, not followed
    c = _Cache(some, some, 1, kv_heads, page_size, head_dim)
    b = _Batch(some, some, some, 1, tokens, seqs, 1)
    return _library().qlora_kv_attention_workspace_bytes(c, b, heads, max_new, max_length)


def kv_attention(cache: KVCache, q: torch.Tensor, starts: torch.Tensor, lengths: torch.Tensor, table: torch.Tensor,
                 scale: Optional[float] = None, max_new: Optional[int] = None,
                 max_length: Optional[int] = None) -> torch.Tensor:
    """Causal attention of new tokens, already appended, over the cache: bf16 [tokens, heads,
    head_dim].  Arguments as for kv_append (the same lengths: tokens before these); head h
    reads kv head h // (heads // kv_heads).  scale: 1/sqrt(head_dim) by default.  max_new (the
    most new tokens of a sequence) and max_length (its most positions, new ones included) size
    the launch: without them it is sized for `tokens` and for the table's width."""
    dev = _device(q, "q")
    c = cache._struct(dev)
    T, dim = q.shape[0], c.head_dim
    b = _batch(starts, lengths, table, T, dev)
    qh = _heads(q, "q", torch.bfloat16, T, dim, dev)
    out, oh = _fresh_heads(q, T, dim)
    max_new = max(1, T) if max_new is None else int(max_new)
    max_length = max(1, b.table_width * c.page_size) if max_length is None else int(max_length)
    wsb = _attention_ws_bytes(c.kv_heads, c.page_size, dim, b.seqs, T, qh.heads, max_new, max_length)
    ws = _workspace(wsb, q.device)
    _check(_library().qlora_kv_attention(c, b, qh, oh, dim ** -0.5 if scale is None else float(scale), max_new, max_length,
                                         None if ws is None else ws.data_ptr(), wsb, _raw_stream(dev)))
    return out


# ---------------------------------------------------------------------------
# The vocabulary head's loss
# ---------------------------------------------------------------------------
def head_loss(X: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, dloss: Optional[torch.Tensor] = None,
              need_dw: bool = False, ignore_index: int = -100):
    """Softmax cross entropy of the vocabulary head z = X W^T, without keeping the logits:
    (loss fp32 [M], dX bf16 [M, K] or None, dW bf16 [V, K] or None).
      X        bf16 [M, K], W bf16 [V, K], K a multiple of 64
      targets  int64 [M]; a row whose target is ignore_index, or outside 0 .. V-1, has loss 0
               and no gradient
      dloss    fp32 [M], the gradient of each row's loss (1/count for a mean): with it dX is
               computed in the same call, and dW if need_dw.  A later factor on a row's loss
               multiplies its row of dX."""
    L = _library()
    _dev(X, "X", torch.bfloat16)
    _dev(W, "W", torch.bfloat16)
    _dev(targets, "targets", torch.int64)
    if X.dim() != 2 or W.dim() != 2 or X.shape[1] != W.shape[1]:
        raise ValueError("X must be [M, K] and W [V, K]")
    M, K = X.shape
    V = W.shape[0]
    if tuple(targets.shape) != (M,):
        raise ValueError("targets must be [%d]" % M)
    if dloss is not None:
        _dev(dloss, "dloss", torch.float32)
        if tuple(dloss.shape) != (M,):
            raise ValueError("dloss must be [%d]" % M)
    elif need_dw:
        raise ValueError("need_dw needs dloss")
    _same_device(("X", X), ("W", W), ("targets", targets), ("dloss", dloss))
    loss = torch.empty(M, dtype=torch.float32, device=X.device)
    dX = torch.empty((M, K), dtype=torch.bfloat16, device=X.device) if dloss is not None else None
    dW = torch.empty((V, K), dtype=torch.bfloat16, device=X.device) if need_dw else None
    wsb = L.qlora_head_loss_workspace_bytes(M, K, V, dX is not None, dW is not None)
    ws = _workspace(wsb, X.device)
    _check(L.qlora_head_loss(_ptr(X), M, K, _ptr(W), V, _ptr(targets), ignore_index, _ptr(dloss), _ptr(loss), _ptr(dX),
                             _ptr(dW), _ptr(ws), wsb, _stream(X.device)))
    return loss, dX, dW
