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


def _heads(t: torch.Tensor, name: str, dtypes, tokens: int, dim: int) -> _Heads:
    """A [tokens, heads, dim] tensor of any token and head strides."""
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor" % name)
    if t.dtype not in dtypes:
        raise ValueError("%s must be %s, got %s" % (name, " or ".join(str(d) for d in dtypes), t.dtype))
    if t.dim() != 3 or t.shape[0] != tokens or t.shape[2] != dim or t.shape[1] < 1:
        raise ValueError("%s must be [%d, heads, %d], got %s" % (name, tokens, dim, tuple(t.shape)))
    if t.numel() and t.stride(2) != 1:
        raise ValueError("%s must be dense along its last dimension" % name)
    token_stride, head_stride = t.stride(0), t.stride(1)
    if t.shape[1] == 1:
        head_stride = dim
    if tokens <= 1:
        token_stride = t.shape[1] * head_stride
    return _Heads(t.data_ptr(), token_stride, head_stride, t.shape[1])


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

    def _struct(self):
        _dev(self.freq, "freq", torch.int64)
        if self.freq.numel() * 2 != self.rotary_dim:
            raise ValueError("freq must hold rotary_dim / 2 = %d values" % (self.rotary_dim // 2))
        return _Rope(self.freq.data_ptr(), self.rotary_dim, int(self.interleaved), self.magnitude)


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


def _rope(plan, positions, tensors, inplace, backward):
    L = _library()
    _dev(positions, "positions", torch.int32)
    M = positions.numel()
    given = [("q", tensors[0])] + ([("k", tensors[1])] if tensors[1] is not None else [])
    dtype, dim = tensors[0].dtype, tensors[0].shape[-1]
    if dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("q must be float32 or bfloat16, got %s" % dtype)
    ins, outs = (_Heads * 2)(), (_Heads * 2)()
    results = []
    for i, (name, t) in enumerate(given):
        ins[i] = _heads(t, name, (dtype,), M, dim)
        out = t if inplace else torch.empty(t.shape, dtype=dtype, device=t.device)
        outs[i] = ins[i] if inplace else _heads(out, name, (dtype,), M, dim)
        results.append(out)
    _same_device(("freq", plan.freq), ("positions", positions), *given)
    rope = plan._struct()
    _check(L.qlora_rope_apply(ctypes.byref(rope), int(backward), _ptr(positions), M, dim,
                              NF4_BF16 if dtype == torch.bfloat16 else NF4_F32, ins, outs, len(given),
                              _stream(tensors[0].device)))
    return tuple(results) if len(results) > 1 else results[0]


def rope_fwd(plan: RopePlan, positions: torch.Tensor, q: torch.Tensor, k: Optional[torch.Tensor] = None,
             inplace: bool = False):
    """Queries, and keys if given, rotated to their positions: q [tokens, heads, dim], k
    [tokens, kv_heads, dim] (fp32 or bf16, the same type; any strides with a dense last
    dimension), positions int32 [tokens].  Returns new dense tensors, or the same ones if `inplace`."""
    return _rope(plan, positions, (q, k), inplace, False)


def rope_bwd(plan: RopePlan, positions: torch.Tensor, dq: torch.Tensor, dk: Optional[torch.Tensor] = None,
             inplace: bool = False):
    """The gradient of rope_fwd: dq and dk turned back, times the same magnitude."""
    return _rope(plan, positions, (dq, dk), inplace, True)


# ---------------------------------------------------------------------------
# The paged 8-bit cache
# ---------------------------------------------------------------------------
@dataclass
class KVCache:
    """Keys and values in pages: codes uint8 [pages, 2, kv_heads, page_size, head_dim] (E4M3,
    index 0 the keys), scales float32 [pages, 2, kv_heads] (powers of two)."""
    codes: torch.Tensor
    scales: torch.Tensor

    def _struct(self):
        _dev(self.codes, "codes", torch.uint8)
        _dev(self.scales, "scales", torch.float32)
        if self.codes.dim() != 5 or self.codes.shape[1] != 2:
            raise ValueError("codes must be [pages, 2, kv_heads, page_size, head_dim], got %s" % (tuple(self.codes.shape),))
        if tuple(self.scales.shape) != tuple(self.codes.shape[:3]):
            raise ValueError("scales must be %s, got %s" % (tuple(self.codes.shape[:3]), tuple(self.scales.shape)))
        pages, _, kv_heads, page, dim = self.codes.shape
        return _Cache(self.codes.data_ptr(), self.scales.data_ptr(), pages, kv_heads, page, dim)

    def decode(self, dtype=torch.float32) -> torch.Tensor:
        """What the codes stand for, [pages, 2, kv_heads, page_size, head_dim] (for looking at)."""
        return (self.codes.view(torch.float8_e4m3fn).float() * self.scales[..., None, None]).to(dtype)


def kv_cache(pages: int, kv_heads: int, head_dim: int, page_size: int = 64, device="cuda") -> KVCache:
    """An empty cache of `pages` pages."""
    return KVCache(torch.zeros((pages, 2, kv_heads, page_size, head_dim), dtype=torch.uint8, device=device),
                   torch.ones((pages, 2, kv_heads), dtype=torch.float32, device=device))


def _batch(starts, lengths, table, tokens):
    for name, t in (("starts", starts), ("lengths", lengths), ("table", table)):
        if not t.is_cuda:
            raise ValueError("%s must be a GPU tensor" % name)
        if t.dtype != torch.int32:
            raise ValueError("%s must be torch.int32, got %s" % (name, t.dtype))
    _dev(starts, "starts")
    _dev(lengths, "lengths")
    seqs = lengths.numel()
    if lengths.dim() != 1 or starts.dim() != 1 or starts.numel() != seqs + 1:
        raise ValueError("lengths must be [seqs] and starts [seqs + 1]")
    if table.dim() != 2 or table.shape[0] != seqs or (table.numel() and table.stride(1) != 1):
        raise ValueError("table must be [%d, pages of a sequence], dense along its rows" % seqs)
    width = table.shape[1]
    return _Batch(starts.data_ptr(), lengths.data_ptr(), table.data_ptr(), table.stride(0) if seqs > 1 else width, tokens,
                  seqs, width)


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
    L = _library()
    c = cache._struct()
    T = k.shape[0]
    b = _batch(starts, lengths, table, T)
    bf16 = (torch.bfloat16,)
    kh, vh = _heads(k, "k", bf16, T, c.head_dim), _heads(v, "v", bf16, T, c.head_dim)
    named = [("cache", cache.codes), ("scales", cache.scales), ("k", k), ("v", v), ("starts", starts),
             ("lengths", lengths), ("table", table), ("q", q)]
    out = qh = oh = r = None
    if q is not None:
        qh = _heads(q, "q", bf16, T, c.head_dim)
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        oh = _heads(out, "q", bf16, T, c.head_dim)
    if rope is not None:
        r = rope._struct()
        named.append(("freq", rope.freq))
    _same_device(*named)
    ref = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    _check(L.qlora_kv_append(ref(c), ref(b), ref(kh), ref(vh), ref(r), ref(qh), ref(oh), _stream(k.device)))
    return out


def kv_attention(cache: KVCache, q: torch.Tensor, starts: torch.Tensor, lengths: torch.Tensor, table: torch.Tensor,
                 scale: Optional[float] = None, max_new: Optional[int] = None,
                 max_length: Optional[int] = None) -> torch.Tensor:
    """Causal attention of new tokens, already appended, over the cache: bf16 [tokens, heads,
    head_dim].  Arguments as for kv_append (the same lengths: tokens before these); head h
    reads kv head h // (heads // kv_heads).  scale: 1/sqrt(head_dim) by default.  max_new (the
    most new tokens of a sequence) and max_length (its most positions, new ones included) size
    the launch: without them it is sized for `tokens` and for the table's width."""
    L = _library()
    c = cache._struct()
    T = q.shape[0]
    b = _batch(starts, lengths, table, T)
    qh = _heads(q, "q", (torch.bfloat16,), T, c.head_dim)
    out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    oh = _heads(out, "out", (torch.bfloat16,), T, c.head_dim)
    _same_device(("cache", cache.codes), ("scales", cache.scales), ("q", q), ("starts", starts), ("lengths", lengths),
                 ("table", table))
    max_new = max(1, T) if max_new is None else int(max_new)
    max_length = max(1, b.table_width * c.page_size) if max_length is None else int(max_length)
    scale = 1.0 / math.sqrt(c.head_dim) if scale is None else float(scale)
    wsb = L.qlora_kv_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(b), qh.heads, max_new, max_length)
    ws = _workspace(wsb, q.device)
    _check(L.qlora_kv_attention(ctypes.byref(c), ctypes.byref(b), ctypes.byref(qh), ctypes.byref(oh), scale, max_new,
                                max_length, _ptr(ws), wsb, _stream(q.device)))
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
