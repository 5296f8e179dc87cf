"""Plain float64 forms of the operators around the linears, for the tests: written from the
definitions in include/qlora_decoder.h, on the CPU, with numpy and torch.float64."""
import math

import numpy as np
import torch


def theta_of(rotary, base=10000.0, scaling=None, factor=1.0, original_length=0, beta_fast=32.0, beta_slow=1.0):
    """(angle per position of each pair in float64, magnitude)."""
    i = np.arange(rotary // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (rotary / (rotary - 2.0))
    theta = base ** (-2.0 * i / rotary)
    if scaling == "linear":
        return theta / factor, 1.0
    if scaling == "parts":
        edge = lambda turns: rotary * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        low, high = max(math.floor(edge(beta_fast)), 0), min(math.ceil(edge(beta_slow)), rotary - 1)
        r = np.clip((i - low) / max(high - low, 1e-3), 0.0, 1.0)
        return theta * (1 - r) + theta / factor * r, (0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0)
    return theta, 1.0


def pair_index(rotary, interleaved):
    n = rotary // 2
    return (np.arange(n) * 2, np.arange(n) * 2 + 1) if interleaved else (np.arange(n), np.arange(n) + n)


def rotate(x, positions, rotary, interleaved, theta, magnitude, back=False):
    """x float64 [tokens, heads, dim]."""
    a, b = pair_index(rotary, interleaved)
    angle = np.asarray(positions, np.float64)[:, None] * theta[None, :]
    c, s = np.cos(angle)[:, None, :] * magnitude, np.sin(angle)[:, None, :] * magnitude * (-1 if back else 1)
    y = np.array(x, np.float64)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    return y


def e4m3_values():
    """The value of each of the 256 codes (NaN for the two NaN codes)."""
    code = np.arange(256)
    e, m = (code >> 3) & 15, code & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * np.exp2(e.astype(np.float64) - 10))
    v[(code & 127) == 127] = np.nan
    return np.where(code >= 128, -v, v)


def e4m3_nearest(x):
    """E4M3 codes of float64 values within +-448, to nearest, ties to the even code."""
    x = np.asarray(x, np.float64)
    grid = e4m3_values()[:127]
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(grid, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - a, a - grid[lo]
    code = np.where(up < down, hi, np.where(up > down, lo, np.where(hi % 2 == 0, hi, lo)))
    return (code + np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def exponent(reach):
    """Smallest e of -50 .. 50 with reach <= 448 * 2^e."""
    e = -50
    while e < 50 and reach > 448.0 * 2.0 ** e:
        e += 1
    return e


def append(codes, scales, k, v, starts, lengths, table, rope=None):
    """The cache after an append, and the exact quotients that its new codes round:
    codes uint8 [pages, 2, heads, P, D], scales [pages, 2, heads] (copies are changed);
    rope: (rotary, interleaved, theta, magnitude) or None."""
    codes, scales = codes.copy(), scales.astype(np.float64)
    quotient = np.full(codes.shape, np.nan)
    pages, _, H, P, D = codes.shape
    value = e4m3_values()
    for b in range(len(lengths)):
        for h in range(H):
            at = starts[b]
            while at < starts[b + 1]:
                pos = lengths[b] + at - starts[b]
                if pos < 0:
                    at += 1
                    continue
                slot = pos % P
                n = min(P - slot, starts[b + 1] - at)
                page = table[b][pos // P] if pos // P < table.shape[1] else -1
                if 0 <= page < pages:
                    kt, vt = k[at:at + n, h].astype(np.float64), v[at:at + n, h].astype(np.float64)
                    bad = ~(np.isfinite(kt).all(-1) & np.isfinite(vt).all(-1))
                    y, reach = kt[:, None], np.abs(kt)
                    if rope is not None:
                        rotary, inter, theta, mag = rope
                        ia, ib = pair_index(rotary, inter)
                        norm = np.hypot(kt[:, ia], kt[:, ib]) * mag
                        reach[:, ia], reach[:, ib] = norm, norm
                        with np.errstate(invalid="ignore"):
                            y = rotate(y, np.arange(pos, pos + n), rotary, inter, theta, mag)
                    for kind, (x, r) in enumerate(((y[:, 0], reach), (vt, np.abs(vt)))):
                        e = exponent(r[~bad].max()) if (~bad).any() else -50
                        if slot > 0:
                            old = int(math.log2(scales[page, kind, h]))
                            if e > old:
                                held = value[codes[page, kind, h, :slot]] * 2.0 ** (old - e)
                                again = e4m3_nearest(held)
                                codes[page, kind, h, :slot] = np.where(np.isnan(held), codes[page, kind, h, :slot], again)
                            e = max(e, old)
                        scales[page, kind, h] = 2.0 ** e
                        with np.errstate(invalid="ignore"):
                            z = np.clip(x / 2.0 ** e, -448, 448)
                        z[bad] = 0.0
                        quotient[page, kind, h, slot:slot + n] = z
                        codes[page, kind, h, slot:slot + n] = np.where(bad[:, None], 127 if kind == 0 else 0, e4m3_nearest(z))
                at += n
    return codes, scales, quotient


def attention(codes, scales, q, starts, lengths, table, scale):
    """(out float64, the largest |value| each row can see) of the causal attention."""
    pages, _, H, P, D = codes.shape
    value = e4m3_values()
    T, Hq, _ = q.shape
    out, reach = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    for b in range(len(lengths)):
        for t in range(starts[b], starts[b + 1]):
            pos = lengths[b] + t - starts[b]
            if pos < 0 or pos >= table.shape[1] * P:
                continue
            j = np.arange(pos + 1)
            page = table[b][j // P]
            held = (page >= 0) & (page < pages)
            if not held.any():
                continue
            j, page = j[held], page[held]
            for h in range(Hq):
                g = h // (Hq // H)
                kk = value[codes[page, 0, g, j % P]] * scales[page, 0, g][:, None]
                vv = value[codes[page, 1, g, j % P]] * scales[page, 1, g][:, None]
                x = kk @ q[t, h].astype(np.float64) * scale
                p = np.exp(x - x.max())
                out[t, h] = (p / p.sum()) @ vv
                reach[t, h] = np.abs(vv).max()
    return out, reach


# Relative norm of dW's error over vocabulary rows that are no row's target.  Their G = dloss (p - 0) carries one rounding
# to bf16 and the output another.  Rounding to 8 significant bits leaves an error of 2^-8 / sqrt(3) of the power of two
# below (root of the mean square); mantissas spread evenly over the logarithm have a mean square of 1/m of 3 / (8 ln 2), so
# that is 1.66e-3 of a value, and errors of independent sign keep their relative norm in a sum: sqrt(2) 1.66e-3 =
# 2.35e-3.  Exponentials kept without their eight further bits add a third: sqrt(3) 1.66e-3 = 2.87e-3.  The limit is between.
DW_NORM = 2.6e-3


def kept_exponentials(E, low="right"):
    """fp32 exponentials after they were kept as bf16 and eight bits more; low: what happens to these."""
    top = E.bfloat16().float()
    bits = ((E.view(torch.int32) - top.view(torch.int32) + 0x80) >> 8).clamp(-128, 127)
    if low == "zero":
        return top
    if low == "misplaced":
        bits = bits.roll(1, 1)
    return (top.view(torch.int32) + (bits << 8)).view(torch.float32)


def head_loss(X, W, targets, dloss, ignore=-100):
    """loss, dX, dW and |G| in float64 (torch)."""
    x, w = X.double(), W.double()
    z = x @ w.t()
    lse = torch.logsumexp(z, dim=1)
    live = (targets >= 0) & (targets < W.shape[0]) & (targets != ignore)
    y = torch.where(live, targets, torch.zeros_like(targets))
    loss = torch.where(live, lse - z[torch.arange(len(y)), y], torch.zeros_like(lse))
    G = torch.exp(z - lse[:, None])
    rest = z.clone()                                                    # 1 - p_y without the cancellation of p_y - 1
    rest[torch.arange(len(y)), y] = -math.inf
    rest = torch.logsumexp(rest, dim=1) - z[torch.arange(len(y)), y]
    G[torch.arange(len(y)), y] = -torch.sigmoid(rest)
    G = torch.where(live[:, None], G * dloss.double()[:, None], torch.zeros_like(G))
    return loss, G @ w, G.t() @ x, G.abs(), z
