"""The operators around the QLoRA linears of a decoder: rotary positions, a paged key/value
cache of 8 bits with its append and its attention, and the vocabulary head's softmax cross
entropy.  Thin binding over ``include/qlora_decoder.h``; the rules of the package hold (GPU
tensors, the current stream, no fallback, ``ValueError`` for a bad tensor and ``NF4Error``
for what the library refuses).

Rotary positions: Su et al., "RoFormer" (2021); the scalings "ntk" and "parts" for contexts
longer than a model was trained on follow the base change and the by-parts interpolation of
Peng et al., "YaRN" (2023).
"""
import importlib.util
import math
import os
from dataclasses import dataclass
from typing import Optional

import torch

from . import NF4_ERR_HIP, NF4Error, lib_path, load_library

__all__ = ["RopePlan", "rope_plan", "rope_fwd", "rope_bwd", "KVCache", "kv_cache", "kv_append", "kv_attention",
           "head_loss"]

_bound = None


def binding_path() -> str:
    return os.path.join(os.path.dirname(lib_path()), "qlora_decoder_binding.so")


def _binding():
    """The compiled calls (raises NF4Error if they have not been built).  They check each tensor's
    type, shape, strides and device, allocate outputs and workspaces with torch, and call the library
    on torch's current stream."""
    global _bound
    if _bound is None:
        load_library()
        path = binding_path()
        if not os.path.exists(path):
            raise NF4Error(NF4_ERR_HIP, "binding not built (%s); run __graft_entry__.build()" % path)
        spec = importlib.util.spec_from_file_location("qlora_decoder_binding", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        module.setup(NF4Error, stream or (lambda device: torch.cuda.current_stream(device).cuda_stream))
        _bound = module
    return _bound


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


def rope_fwd(plan: RopePlan, positions: torch.Tensor, q: torch.Tensor, k: Optional[torch.Tensor] = None,
             inplace: bool = False):
    """Queries, and keys if given, rotated to their positions: q [tokens, heads, dim], k
    [tokens, kv_heads, dim] (fp32 or bf16, the same type; any strides with a dense last
    dimension), positions int32 [tokens].  Returns new dense tensors, or the same ones if `inplace`
    (not of tensors that autograd records; rows may not share memory)."""
    return (_bound or _binding()).rope(plan.freq, plan.rotary_dim, plan.interleaved, plan.magnitude, False, positions, q, k, inplace)


def rope_bwd(plan: RopePlan, positions: torch.Tensor, dq: torch.Tensor, dk: Optional[torch.Tensor] = None,
             inplace: bool = False):
    """The gradient of rope_fwd: dq and dk turned back, times the same magnitude."""
    return (_bound or _binding()).rope(plan.freq, plan.rotary_dim, plan.interleaved, plan.magnitude, True, positions, dq, dk, inplace)


# ---------------------------------------------------------------------------
# The paged 8-bit cache
# ---------------------------------------------------------------------------
@dataclass
class KVCache:
    """Keys and values in pages: codes uint8 [pages, 2, kv_heads, page_size, head_dim] (E4M3,
    index 0 the keys), scales float32 [pages, 2, kv_heads] (powers of two)."""
    codes: torch.Tensor
    scales: torch.Tensor

    def decode(self, dtype=torch.float32) -> torch.Tensor:
        """What the codes stand for, [pages, 2, kv_heads, page_size, head_dim] (for looking at)."""
        return (self.codes.view(torch.float8_e4m3fn).float() * self.scales[..., None, None]).to(dtype)


def kv_cache(pages: int, kv_heads: int, head_dim: int, page_size: int = 64, device="cuda") -> KVCache:
    """An empty cache of `pages` pages."""
    return KVCache(torch.zeros((pages, 2, kv_heads, page_size, head_dim), dtype=torch.uint8, device=device),
                   torch.ones((pages, 2, kv_heads), dtype=torch.float32, device=device))


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
    call = (_bound or _binding()).append
    if rope is None:
        return call(cache.codes, cache.scales, k, v, starts, lengths, table, q, None, 0, False, 1.0)
    return call(cache.codes, cache.scales, k, v, starts, lengths, table, q, rope.freq, rope.rotary_dim, rope.interleaved,
                rope.magnitude)


def kv_attention(cache: KVCache, q: torch.Tensor, starts: torch.Tensor, lengths: torch.Tensor, table: torch.Tensor,
                 scale: Optional[float] = None, max_new: Optional[int] = None,
                 max_length: Optional[int] = None) -> torch.Tensor:
    """Causal attention of new tokens, already appended, over the cache: bf16 [tokens, heads,
    head_dim].  Arguments as for kv_append (the same lengths: tokens before these); head h
    reads kv head h // (heads // kv_heads).  scale: 1/sqrt(head_dim) by default.  max_new (the
    most new tokens of a sequence) and max_length (its most positions, new ones included) size
    the launch: without them it is sized for `tokens` and for the table's width, which costs single
    tokens up to twice the time (24 sequences of up to 4096 keys, 64 heads on 8: 32 us stated, 57 not)."""
    return (_bound or _binding()).attention(cache.codes, cache.scales, q, starts, lengths, table, scale, max_new, max_length)


# ---------------------------------------------------------------------------
# The vocabulary head's loss
# ---------------------------------------------------------------------------
def head_loss(X: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, dloss: Optional[torch.Tensor] = None,
              need_dw: bool = False, ignore_index: int = -100):
    """Softmax cross entropy of the vocabulary head z = X W^T:
    (loss fp32 [M], dX bf16 [M, K] or None, dW bf16 [V, K] or None).  Loss and dX do not keep the
    logits; need_dw keeps their exponentials, three bytes each, while they are up to 2^29 (more memory
    than bf16 logits), and computes the logits twice beyond.
      X        bf16 [M, K], W bf16 [V, K], K a multiple of 64
      targets  int64 [M]; a row whose target is ignore_index, or outside 0 .. V-1, has loss 0
               and no gradient, whatever X and dloss hold there
      dloss    fp32 [M], the gradient of each row's loss (1/count for a mean): with it dX is
               computed in the same call, and dW if need_dw.  A later factor on a row's loss
               multiplies its row of dX."""
    return (_bound or _binding()).head_loss(X, W, targets, dloss, need_dw, ignore_index)
