"""The operators around the QLoRA linears of a decoder: rotary positions, a paged key/value
cache of 8 bits with its append and its attention, the vocabulary head's softmax cross
entropy, the norms around a block, the gradients' norm and clipping, and the penalties and masks
of logits.  Thin binding over ``include/qlora_decoder.h`` and ``include/qlora_step.h``; the rules
of the package hold (GPU tensors, the current stream, no fallback, ``ValueError`` for a bad
tensor and ``NF4Error`` for what the library refuses).

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
           "head_loss", "block_norm_fwd", "block_norm_bwd", "grad_norm", "clip_grads", "shape_logits"]

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
                 max_length: Optional[int] = None, window: Optional[int] = None, sinks: int = 0) -> torch.Tensor:
    """Causal attention of new tokens, already appended, over the cache: bf16 [tokens, heads,
    head_dim].  Arguments as for kv_append (the same lengths: tokens before these); head h
    reads kv head h // (heads // kv_heads).  scale: 1/sqrt(head_dim) by default.  max_new (the
    most new tokens of a sequence) and max_length (its most positions, new ones included) size
    the launch: without them it is sized for `tokens` and for the table's width, which costs single
    tokens up to twice the time (24 sequences of up to 4096 keys, 64 heads on 8: 32 us stated, 57 not).
    window: a token sees the last `window` keys up to its own, and the first `sinks` of its sequence (None: all up
    to its own).  Pages that no token of the batch sees are not read: they may be given back, their table entries
    -1 (lengths and positions go on as if they were there)."""
    return (_bound or _binding()).attention(cache.codes, cache.scales, q, starts, lengths, table, scale, max_new, max_length, window, sinks)


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


# ---------------------------------------------------------------------------
# The norms around a block
# ---------------------------------------------------------------------------
def block_norm_fwd(h: torch.Tensor, x: Optional[torch.Tensor] = None, pre=True, post=None,
                   gate: Optional[torch.Tensor] = None, scale: float = 1.0, eps: float = 1e-6, inplace: bool = False):
    """From a block's output to the next block's input, in one pass: (the stream after the block, its norm):
      h' = h + scale * gate * (n(x) post),   y = n(h') pre,   n(a) = a / sqrt(mean(a^2) + eps)
      h      the stream [tokens, width], fp32 or bf16, any row stride; width up to 32768
      x      the block's output, bf16 [tokens, width]; None: no block, h' is h itself
      pre    the weight [width] of the norm before the next block, True for a norm without one, None for no norm (y is None)
      post   the same for a norm of the block's output; None: x as it is
      gate   [width], or [rows, width] where each row belongs to tokens / rows neighbouring tokens (a row for each
             sequence of a batch of equal lengths, or for each token); None: ones
    pre, post and gate are fp32 or bf16, all of one type.  h' is of the stream's type (h itself is written if `inplace`;
    not of tensors that autograd records, nor where h shares memory with another operand), and y, bf16, is the norm of h'
    as it was rounded."""
    return (_bound or _binding()).block_norm_fwd(h, x, pre, post, gate, scale, eps, inplace)


def block_norm_bwd(h: torch.Tensor, dy: Optional[torch.Tensor] = None, dh: Optional[torch.Tensor] = None,
                   x: Optional[torch.Tensor] = None, pre=True, post=None, gate: Optional[torch.Tensor] = None,
                   scale: float = 1.0, eps: float = 1e-6, need_weights: bool = True):
    """The gradients of block_norm_fwd: (dh of the stream before the block, dx bf16, dpre, dpost, dgate); None where there is
    nothing to have one.
      h      the stream after the block (what block_norm_fwd returned first)
      dy     the gradient of y, bf16 (with pre)
      dh     the gradient of the stream after the block from later blocks, of the stream's type; None: zero
      x, pre, post, gate, scale, eps   as in the forward call
    dpre, dpost [width] and dgate (the gate's shape) are fp32 sums over the tokens, in a fixed order; need_weights=False
    (frozen norms) leaves them out."""
    return (_bound or _binding()).block_norm_bwd(h, dy, dh, x, need_weights, pre, post, gate, scale, eps)


# ---------------------------------------------------------------------------
# The gradients' global norm
# ---------------------------------------------------------------------------
def grad_norm(grads) -> torch.Tensor:
    """The root of the sum of the squares of all values of a list of tensors (fp32 or bf16, dense, of any sizes, on one
    GPU): a fp32 number on the GPU.  Squares are added in 64 bits, in a fixed order."""
    return (_bound or _binding()).grad_norm(grads, math.inf)[0]


def norm_and_factor(grads, max_norm: float):
    """grad_norm, and the factor min(1, max_norm / norm) (both fp32 numbers on the GPU), for the optimizer."""
    return (_bound or _binding()).grad_norm(grads, max_norm)


def clip_grads(grads, max_norm: float, out=None) -> torch.Tensor:
    """Gradients times min(1, max_norm / norm), in place, or into the tensors of `out` (of the same sizes and types; none
    may share memory).  Returns the norm before (a fp32 number on the GPU); nothing waits for it.  A norm of infinity or
    NaN gives the products that the formula says (zeros and NaN)."""
    return (_bound or _binding()).clip_grads(grads, max_norm, out)


# ---------------------------------------------------------------------------
# Logits before the choice of a token
# ---------------------------------------------------------------------------
def shape_logits(logits: torch.Tensor, history: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                 prompts: Optional[torch.Tensor] = None, repetition=1.0, presence=0.0, frequency=0.0,
                 bias_ids: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                 allowed: Optional[torch.Tensor] = None, inplace: bool = False) -> torch.Tensor:
    """Logits [rows, vocabulary] (fp32 or bf16, any row stride) with, in this order and rounded once:
      - those of tokens in the row's history divided by `repetition` where positive, multiplied by it elsewhere,
      - less frequency * count + presence for tokens that are count > 0 times in the history after the prompt,
      - plus `bias` at `bias_ids` (of an id that is given twice, the last entry counts),
      - -inf where the bit v % 32 of word v // 32 of `allowed` is 0.
      history   int32 [rows, width]: a row's tokens so far are its first lengths[row] (None: all), of which
                the first prompts[row] are the prompt's (None: none); ids outside the vocabulary are passed over
      repetition, presence, frequency   numbers, or fp32 [rows]
      bias_ids, bias   int32 and fp32 [rows, biases]; ids outside the vocabulary are unused
      allowed   int32 [rows, at least vocabulary / 32, rounded up]
    history, bias_ids, bias and allowed may have a single row for all.  Returns a new dense tensor, or the same one if
    `inplace` (not of tensors that autograd records, nor of those that share memory with another operand)."""
    return (_bound or _binding()).shape_logits(logits, history, lengths, prompts, repetition, presence, frequency, bias_ids, bias,
                                               allowed, inplace)
