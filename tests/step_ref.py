"""Plain float64 forms of the operators of include/qlora_step.h, for the tests: written from the definitions
there, on the CPU, with numpy and torch.float64."""
import math

import numpy as np
import torch

import decoder_ref as ref


def unit(a, eps):
    """(rows over the root of their mean square, 1 / that root)."""
    s = 1.0 / torch.sqrt((a * a).mean(-1, keepdim=True) + eps)
    return a * s, s


def rows_of(gate, M):
    """A gate's rows, one for each of M tokens (1 without a gate)."""
    if gate is None:
        return torch.ones((1, 1), dtype=torch.float64)
    gate = gate.double()
    gate = gate[None] if gate.dim() == 1 else gate
    return gate.repeat_interleave(M // gate.shape[0], 0)


def weight(w):
    return torch.ones((), dtype=torch.float64) if w is True else w.double()


def block_norm(h, x=None, pre=True, post=None, gate=None, scale=1.0, eps=1e-6):
    """(the stream after the block before it is rounded, a function that gives y from the stream)."""
    h = h.double()
    if x is not None:
        p = x.double()
        if post is not None:
            p = unit(p, eps)[0] * weight(post)
        h = h + scale * rows_of(gate, len(h)) * p
    return h, (lambda s: None if pre is None else unit(s.double(), eps)[0] * weight(pre))


def block_norm_back(h, dy=None, dh=None, x=None, pre=True, post=None, gate=None, scale=1.0, eps=1e-6):
    """Gradients dict(dh, dx, dpre, dpost, dgate), and for each the size of what its rounding goes by."""
    M, K = h.shape
    g, size = {}, {}
    d = torch.zeros((M, K), dtype=torch.float64) if dh is None else dh.double().clone()
    dsize = torch.zeros_like(d)
    if pre is not None:
        a, s = unit(h.double(), eps)
        t = dy.double() * weight(pre)
        d = d + s * (t - a * (t * a).mean(-1, keepdim=True))
        dsize = s * (t.abs() + a.abs() * (t * a).abs().mean(-1, keepdim=True))
        if pre is not True:
            g["dpre"], size["dpre"] = (dy.double() * a).sum(0), (dy.double() * a).abs().sum(0)
    g["dh"], size["dh"] = d, dsize + (0 if dh is None else 0.125 * dh.double().abs())
    if x is not None:
        x = x.double()
        e = scale * rows_of(gate, M)
        q, qsize = e * d, e.abs() * (size["dh"] + 0.125 * d.abs())
        p = x
        if post is not None:
            b, r = unit(x, eps)
            w = weight(post)
            p, u, usize = b * w, q * w, qsize * w.abs()
            g["dx"] = r * (u - b * (u * b).mean(-1, keepdim=True))
            size["dx"] = r * (usize + b.abs() * (usize * b.abs()).mean(-1, keepdim=True) + u.abs() + b.abs() * (u * b).abs().mean(-1, keepdim=True))
            if post is not True:
                g["dpost"], size["dpost"] = (q * b).sum(0), ((qsize + q.abs()) * b.abs()).sum(0)
        else:
            g["dx"], size["dx"] = q, qsize
        if gate is not None:
            n = 1 if gate.dim() == 1 else gate.shape[0]
            v, vs = scale * p * d, abs(scale) * p.abs() * (size["dh"] + d.abs())
            g["dgate"] = v.view(n, M // n, K).sum(1).view(gate.shape)
            size["dgate"] = vs.view(n, M // n, K).sum(1).view(gate.shape)
    return g, size


def attention(codes, scales, q, starts, lengths, table, scale, window, sinks):
    """(out float64, the largest |value| each row can see) of the causal attention with a window."""
    pages, _, H, P, D = codes.shape
    value = ref.e4m3_values()
    T, Hq, _ = q.shape
    out, reach = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    for b in range(len(lengths)):
        for t in range(starts[b], starts[b + 1]):
            pos = lengths[b] + t - starts[b]
            if pos < 0 or pos >= table.shape[1] * P:
                continue
            j = np.arange(pos + 1)
            j = j[(j > pos - window) | (j < sinks)]
            page = table[b][j // P]
            held = (page >= 0) & (page < pages)
            if not held.any():
                continue
            j, page = j[held], page[held]
            for h in range(H):
                own = slice(h * (Hq // H), (h + 1) * (Hq // H))
                kk = value[codes[page, 0, h, j % P]] * scales[page, 0, h][:, None]
                vv = value[codes[page, 1, h, j % P]] * scales[page, 1, h][:, None]
                x = q[t, own].astype(np.float64) @ kk.T * scale
                p = np.exp(x - x.max(-1, keepdims=True))
                out[t, own] = (p / p.sum(-1, keepdims=True)) @ vv
                reach[t, own] = np.abs(vv).max()
    return out, reach


def shape_logits(z, history=None, lengths=None, prompts=None, repetition=1.0, presence=0.0, frequency=0.0, bias_ids=None,
                 bias=None, allowed=None):
    """float64 logits, and the size of what their rounding goes by (lists and numpy arrays in; numpy out)."""
    z = np.array(z, np.float64)
    R, V = z.shape
    size = np.abs(z)
    of = lambda v, r: float(v[r]) if np.ndim(v) else float(v)  # noqa: E731
    row = lambda v, r: v[r if len(v) > 1 else 0]  # noqa: E731
    for r in range(R):
        if history is not None:
            tokens = [int(t) for t in row(history, r)]
            n = len(tokens) if lengths is None else max(0, min(len(tokens), int(lengths[r])))
            counts, seen = {}, set()
            for i, t in enumerate(tokens[:n]):
                if not 0 <= t < V:
                    continue
                seen.add(t)
                if i >= (0 if prompts is None else int(prompts[r])):
                    counts[t] = counts.get(t, 0) + 1
            rep = of(repetition, r)
            for t in seen:
                z[r, t] = z[r, t] / rep if z[r, t] > 0 else z[r, t] * rep
            size[r] = np.maximum(size[r], np.abs(z[r]))
            for t, c in counts.items():
                less = of(frequency, r) * c + of(presence, r)
                z[r, t] -= less
                size[r, t] += abs(of(frequency, r)) * c + abs(of(presence, r))
        if bias_ids is not None:
            last = {int(t): float(b) for t, b in zip(row(bias_ids, r), row(bias, r)) if 0 <= t < V}
            for t, b in last.items():
                z[r, t] += b
                size[r, t] += abs(b)
        if allowed is not None:
            words = np.asarray(row(allowed, r)).astype(np.int64) & 0xFFFFFFFF
            v = np.arange(V)
            z[r][(words[v // 32] >> (v % 32) & 1) == 0] = -math.inf
    return z, size
