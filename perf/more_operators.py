"""More operators of a decoder around its QLoRA linears, as cases to time and to compare.

Four operators: the norms before and after a block with its gate, residual scale and residual
addition (forward and backward); the global norm of many gradients and their clipping;
attention over the paged 8-bit cache with a sliding window and first tokens that stay
visible; and the penalties, biases and grammar masks between a head's logits and the choice
of a token.  ``run`` computes a case in plain torch operations in 32 bits (sums of squares
over many tensors in 64), or, where ``own`` is true, by the calls a user makes of the
package.  ``exact`` gives a case's outputs from the definitions, in 64 bits.

Sizes follow the repository's LLaMA-7B (width 4096, 32 heads of 128) and LLaMA-65B (width
8192, 64 heads of 128, 80 layers, adapters of rank 64) layers, its few-token and 4096-token
steps, and its vocabularies of 32000 and 128256; grouped heads, windows and the odd sizes
are generic.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
CODE_MAX = 448.0          # the largest E4M3 value
EXP_MIN, EXP_MAX = -50, 50
EPS = 1e-6


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _norm(name, seqs, tokens, width, stream, weights, back, block, pre, post, gate, learn):
    """tokens: of each sequence; gate: "none", or one row of gates for all ("channel"), each sequence or each token;
    block: whether there is a block's output to add; learn: whether the weights' gradients are wanted."""
    return dict(name=name, op="norm", seqs=seqs, tokens=tokens, width=width, stream=stream, weights=weights, back=back,
                block=block, pre=pre, post=post, gate=gate, learn=learn)


def _clip(name, layers, rank, width, ffn, ragged, dtype, max_norm):
    """The adapters A [rank, in] and B [out, rank] of a layer's seven linears; ragged: odd ranks and widths among them."""
    return dict(name=name, op="clip", layers=layers, rank=rank, width=width, ffn=ffn, ragged=ragged, dtype=dtype,
                max_norm=max_norm)


def _attend(name, seqs, longest, new, heads, kv_heads, head_dim, page, window, sinks, freed):
    """freed: the pages between the first tokens and the window have been given back (table entries of -1)."""
    return dict(name=name, op="attend", seqs=seqs, longest=longest, new=new, heads=heads, kv_heads=kv_heads,
                head_dim=head_dim, page=page, window=window, sinks=sinks, freed=freed)


def _logits(name, rows, vocab, dtype, history, biases, grammar, each):
    """history: the most tokens of a row (0: no penalties); biases: of a row; each: penalties of every row's own."""
    return dict(name=name, op="logits", rows=rows, vocab=vocab, dtype=dtype, history=history, biases=biases,
                grammar=grammar, each=each)


def listed():
    return [
        # between two blocks of a decoding step (16 rows, 7B width): latency
        _norm("norm few tokens", 16, 1, 4096, "bfloat16", "bfloat16", False, True, True, False, "none", False),
        # between two blocks of a 4096-token training step of the 65B width: a norm after the block, a gate for each channel
        _norm("norm 4096 tokens", 1, 4096, 8192, "bfloat16", "bfloat16", False, True, True, True, "channel", False),
        # its gradient, the norms' weights and the gate trained
        _norm("norm gradient", 1, 4096, 8192, "bfloat16", "bfloat16", True, True, True, True, "channel", True),
        # odd sizes: seven sequences with a gate each, an fp32 stream and fp32 weights, gradients of all
        _norm("norm gradient of sequences", 7, 143, 2501, "float32", "float32", True, True, True, True, "sequence", True),
        # the adapters of a small decoder: latency
        _clip("clip a small decoder", 2, 16, 512, 1024, False, "float32", 0.3),
        # the adapters of the 65B shape: 1120 tensors, 3.2 GB
        _clip("clip the 65B adapters", 80, 64, 8192, 22016, False, "float32", 0.3),
        # one token of a short conversation: latency (7B heads)
        _attend("attend one window", 1, 3000, 1, 32, 32, 128, 16, 512, 4, False),
        # a batch of long conversations, one token each, whose old pages have been given back (grouped 65B heads)
        _attend("attend windows", 24, 40000, 1, 64, 8, 128, 64, 4096, 4, True),
        # chunks of prompts behind a cached beginning
        _attend("attend window of prompts", 3, 3000, 1500, 32, 8, 128, 32, 1024, 16, False),
        # one answer's next token with a grammar (7B vocabulary): latency
        _logits("logits of an answer", 1, 32000, "bfloat16", 700, 0, True, False),
        # a batch of answers with penalties and biases of their own, no grammar
        _logits("logits of a batch", 16, 32000, "float32", 4000, 300, False, True),
        # a large batch over a large vocabulary, everything at once
        _logits("logits of a large batch", 256, 128256, "float32", 8000, 100, True, True),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "clip", "attend", "logits"])
    if op == "norm":
        seqs = rng.choice([1, 1, _spread(rng, 2, 32)])
        width = 64 * _spread(rng, 1, 128) if rng.random() < 0.6 else _spread(rng, 33, 8192)
        back, block = rng.random() < 0.5, rng.random() < 0.85
        post = block and rng.random() < 0.5
        c = _norm("", seqs, _spread(rng, 1, max(1, min(6000, 4096 * 8192 // (seqs * width)))), width,
                  rng.choice(["bfloat16", "float32"]), rng.choice(["bfloat16", "float32"]), back, block,
                  not block or rng.random() < 0.85, post, rng.choice(["none", "channel", "sequence", "token"]) if block else "none",
                  back and rng.random() < 0.6)
    elif op == "clip":
        c = _clip("", _spread(rng, 1, 40), _spread(rng, 4, 64), 64 * _spread(rng, 4, 128), 64 * _spread(rng, 8, 344),
                  rng.random() < 0.5, rng.choice(["float32", "float32", "bfloat16", "mixed"]), rng.choice([0.3, 1.0, 1e9]))
    elif op == "attend":
        kv = rng.choice([1, 2, 4, 8, 16, 32])
        heads = kv * rng.choice([1, 2, 3, 4, 7, 8])
        while heads > 64:
            heads -= kv
        head_dim = rng.choice([64, 128, 128, 256])
        new = rng.choice([1, 1, _spread(rng, 2, 1500)])
        seqs = _spread(rng, 1, 48 if new < 16 else 4)
        room = (24 * 20000 * 8 * 128) // (seqs * kv * head_dim)
        longest = _spread(rng, 16, max(16, min(60000 if new < 16 else 4000, room)))
        wide = max(1, min(8192 if new < 16 else 2500, (24 * 4096 * 8 * 128) // (seqs * kv * head_dim)))
        c = _attend("", seqs, longest, new, heads, kv, head_dim, rng.choice([16, 32, 64, 128]), _spread(rng, 1, wide),
                    rng.choice([0, 1, 4, 16, _spread(rng, 1, 200)]), rng.random() < 0.5)
    else:
        vocab = _spread(rng, 500, 150000)
        rows = _spread(rng, 1, min(512, max(1, 256 * 128256 // vocab)))
        c = _logits("", rows, vocab, rng.choice(["bfloat16", "float32"]),
                    rng.choice([0, _spread(rng, 1, 8000), _spread(rng, 1, 8000)]), rng.choice([0, _spread(rng, 1, 400)]),
                    rng.random() < 0.5, rng.random() < 0.5)
        c["biases"] = min(c["biases"], vocab)
        if c["history"] == 0 and c["biases"] == 0:
            c["grammar"] = True
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def _prepare_norm(case, g, s):
    K, M = case["width"], case["seqs"] * case["tokens"]
    stream, weights = getattr(torch, case["stream"]), getattr(torch, case["weights"])
    # channels of unlike sizes, as a trained stream has
    channel = torch.exp(0.7 * torch.randn((1, K), generator=g, device=DEV))
    s["h"] = _normal(g, (M, K), torch.float32, 2.0).mul_(channel).to(stream)
    s["x"] = _normal(g, (M, K), scale=0.7) if case["block"] else None
    near_one = lambda: (1.0 + 0.2 * torch.randn((K,), generator=g, device=DEV)).to(weights)  # noqa: E731
    s["pre"] = near_one() if case["pre"] else None
    s["post"] = near_one() if case["post"] else None
    rows = {"none": 0, "channel": 1, "sequence": case["seqs"], "token": M}[case["gate"]]
    s["gate"] = _normal(g, (rows, K), weights, 0.5) if rows else None
    s["scale"] = 1.0 / math.sqrt(2 * 80) if case["post"] else 1.0
    if case["back"]:
        s["dy"] = _normal(g, (M, K), scale=0.01) if case["pre"] else None
        s["dh"] = _normal(g, (M, K), stream, 0.02)


def _shapes(case):
    """The shapes of all adapters of the case."""
    r, w, f = case["rank"], case["width"], case["ffn"]
    sides = [(w, w)] * 4 + [(w, f)] * 2 + [(f, w)]
    out = []
    for layer in range(case["layers"]):
        for i, (k, n) in enumerate(sides):
            odd = (3 * layer + i) % 5 if case["ragged"] else 0
            out += [(r + odd, k - odd), (n + odd, r + odd)]
    return out


def _places(shapes):
    """Where each tensor begins in a buffer of all, on multiples of 64 values, and the buffer's size."""
    at, ends = 0, []
    for a, b in shapes:
        ends.append(at)
        at += (a * b + 63) // 64 * 64
    return ends, at


def _types(case, count):
    if case["dtype"] == "mixed":
        return [torch.float32 if i % 3 else torch.bfloat16 for i in range(count)]
    return [getattr(torch, case["dtype"])] * count


def _prepare_clip(case, g, s):
    shapes = _shapes(case)
    types = _types(case, len(shapes))
    # layers of unlike sizes
    s["grads"] = [_normal(g, shape, t, 1e-3 * (1 + i % 7)) for i, (shape, t) in enumerate(zip(shapes, types))]
    # where the clipped gradients go: views of one buffer for each type, as buckets of an all-reduce are
    s["buffers"] = {}
    ends, size = _places(shapes)
    for t in sorted(set(types), key=str):
        s["buffers"][str(t).split(".")[1]] = torch.zeros((size,), dtype=t, device=DEV)
    s["out"] = [s["buffers"][str(t).split(".")[1]][at:at + a * b].view(a, b) for at, (a, b), t in zip(ends, shapes, types)]


def _encode_pages(x):
    """Pages [..., tokens, dim] as E4M3 codes (bytes) with a power-of-two scale per page and head."""
    top = x.float().abs().amax(dim=(-1, -2))
    scale = torch.exp2(torch.ceil(torch.log2(top.clamp_min(1e-12) / CODE_MAX))).clamp(2.0 ** EXP_MIN, 2.0 ** EXP_MAX)
    return (x.float() / scale[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _ragged(case):
    """Ragged cached lengths (the longest among them) and new tokens of each sequence, one at least: sizes, so
    they go by the case alone."""
    seqs, longest, new = case["seqs"], case["longest"], case["new"]
    r = np.random.RandomState(seqs * 1000003 + longest)
    length = np.exp(r.uniform(math.log(max(1, longest // 8)), math.log(longest), seqs)).astype(np.int64)
    length[r.randint(seqs)] = longest
    count = np.ones(seqs, np.int64) if new == 1 else r.randint(max(1, new // 2), new + 1, seqs)
    return length, count


def _prepare_attend(case, seed, g, s):
    P, H, D = case["page"], case["kv_heads"], case["head_dim"]
    before, count = _ragged(case)
    need = -(-(before + count) // P)
    # pages that no new token sees: between the first tokens' and the first new token's window
    first, last = -(-case["sinks"] // P), np.maximum(0, before - case["window"] + 1) // P
    gone = np.maximum(0, last - first) if case["freed"] else np.zeros_like(need)
    total = int((need - gone).sum()) + 3
    order = np.random.RandomState((seed + 1) % (1 << 31)).permutation(total)
    table = np.full((len(need), int(need.max())), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        held = [p for p in range(n) if not first <= p < first + gone[b]]
        table[b, held] = order[at:at + len(held)]
        at += len(held)
    codes = torch.empty((total, 2, H, P, D), dtype=torch.uint8, device=DEV)
    scales = torch.empty((total, 2, H), dtype=torch.float32, device=DEV)
    step = max(1, (1 << 28) // (2 * H * P * D))
    channel = torch.exp(0.5 * torch.randn((1, 2, H, 1, D), generator=g, device=DEV))   # channels of unlike sizes
    for a in range(0, total, step):
        n = min(step, total - a)
        codes[a:a + n], scales[a:a + n] = _encode_pages(torch.randn((n, 2, H, P, D), generator=g, device=DEV) * channel)
    starts = np.concatenate([[0], np.cumsum(count)]).astype(np.int32)
    put = lambda v: torch.from_numpy(np.ascontiguousarray(v)).to(DEV)  # noqa: E731
    s.update(codes=codes, scales=scales, table=put(table), lengths=put(before.astype(np.int32)), starts=put(starts),
             tokens=int(starts[-1]), longest=int((before + count).max()), most_new=int(count.max()))
    s["q"] = _normal(g, (s["tokens"], case["heads"], D))


def _prepare_logits(case, g, s):
    R, V, L, B = case["rows"], case["vocab"], case["history"], case["biases"]
    uniform = lambda *shape: torch.rand(shape, generator=g, device=DEV)  # noqa: E731
    s["logits"] = _normal(g, (R, V), getattr(torch, case["dtype"]), 3.0)
    s["history"] = s["lengths"] = s["prompts"] = s["bias_ids"] = s["bias"] = s["allowed"] = None
    s["repetition"], s["presence"], s["frequency"] = 1.0, 0.0, 0.0
    if L:
        # a text's tokens: few of them often; rows end raggedly, and a part of each is its prompt
        s["history"] = (V * uniform(R, L) ** 3).to(torch.int32).clamp_(max=V - 1)
        s["lengths"] = (L * (0.25 + 0.75 * uniform(R))).to(torch.int32).clamp_(min=1)
        s["prompts"] = (s["lengths"] * uniform(R)).to(torch.int32)
        if case["each"]:
            s["repetition"], s["presence"], s["frequency"] = 1.0 + 0.3 * uniform(R), 0.5 * uniform(R), 0.2 * uniform(R)
        else:
            s["repetition"], s["presence"], s["frequency"] = 1.15, 0.25, 0.125
    if B:
        # ids of a row differ: one of each of B equal stretches of the vocabulary
        width = V // B
        s["bias_ids"] = (torch.arange(B, device=DEV) * width + (width * uniform(R, B)).long().clamp_(max=width - 1)).to(torch.int32)
        s["bias"] = _normal(g, (R, B), torch.float32, 4.0)
    if case["grammar"]:
        # some rows may go on with little, some with much
        words = -(-V // 32)
        allowed = uniform(R, words * 32) < 0.9 * uniform(R, 1) ** 4 + 0.01
        weight = (2 ** torch.arange(32, device=DEV))[None, None, :]
        word = (allowed.view(R, words, 32) * weight).sum(-1)
        s["allowed"] = torch.where(word >= 1 << 31, word - (1 << 32), word).to(torch.int32)


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case=case)
    if case["op"] == "norm":
        _prepare_norm(case, g, s)
    elif case["op"] == "clip":
        _prepare_clip(case, g, s)
    elif case["op"] == "attend":
        _prepare_attend(case, seed, g, s)
    else:
        _prepare_logits(case, g, s)
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def _factor(a):
    """1 / root of the mean square of each row."""
    return torch.rsqrt(a.square().mean(-1, keepdim=True) + EPS)


def _by_row(gate, rows):
    """A gate's rows, one of each token."""
    return gate.float().repeat_interleave(rows // gate.shape[0], 0)


def _plain_norm(s):
    c = s["case"]
    h = s["h"].float()
    if not c["back"]:
        out = []
        if c["block"]:
            p = s["x"].float()
            if c["post"]:
                p = p * _factor(p) * s["post"].float()
            if s["gate"] is not None:
                p = p * _by_row(s["gate"], len(p))
            new = (h + s["scale"] * p).to(s["h"].dtype)
            out.append(new)
            h = new.float()
        if c["pre"]:
            out.append((h * _factor(h) * s["pre"].float()).to(torch.bfloat16))
        return out
    # the gradient: h is the stream after the block
    out = []
    d = s["dh"].float()
    if c["pre"]:
        f = _factor(h)
        a, dy = h * f, s["dy"].float()
        t = dy * s["pre"].float()
        d = d + f * (t - a * (t * a).mean(-1, keepdim=True))
        if c["learn"]:
            out.append((dy * a).sum(0))
    out.append(d.to(s["h"].dtype))
    if c["block"]:
        x = s["x"].float()
        gate = _by_row(s["gate"], len(x)) if s["gate"] is not None else 1.0
        q = s["scale"] * gate * d
        p = x
        if c["post"]:
            f = _factor(x)
            b, w = x * f, s["post"].float()
            p, u = b * w, q * w
            out.append((f * (u - b * (u * b).mean(-1, keepdim=True))).to(torch.bfloat16))
            if c["learn"]:
                out.append((q * b).sum(0))
        else:
            out.append(q.to(torch.bfloat16))
        if c["learn"] and s["gate"] is not None:
            out.append((s["scale"] * p * d).view(s["gate"].shape[0], -1, c["width"]).sum(1))
    return out


def _plain_clip(s):
    norm = torch.stack([g.double().square().sum() for g in s["grads"]]).sum().sqrt()
    f = (s["case"]["max_norm"] / norm).clamp(max=1.0).float()
    _ = [o.copy_(g.float() * f) for g, o in zip(s["grads"], s["out"])]
    return {"norm": norm.float(), **s["buffers"]}


def _plain_attend(s):
    c = s["case"]
    P, S, W, n = c["page"], c["sinks"], c["window"], s["most_new"]
    starts, lengths = s["starts"].long(), s["lengths"].long()
    count = starts[1:] - starts[:-1]
    # the keys that any new token of a sequence sees: the first ones, then those of its windows
    first = (lengths - W + 1).clamp_min(S)
    t = torch.arange(min(s["longest"], S + W + n - 1), device=DEV)[None, :]
    t = torch.where(t < S, t, first[:, None] + t - S)                               # [seqs, keys]
    page = s["table"].long().gather(1, (t // P).clamp_max(s["table"].shape[1] - 1)).clamp_min(0)
    kv = s["codes"][page, :, :, t % P].view(torch.float8_e4m3fn)                     # [seqs, keys, 2, heads, dim]
    kv = kv.float() * s["scales"][page][..., None]
    k, v = kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)
    j = torch.arange(n, device=DEV)
    q = s["q"][(starts[:-1, None] + j).clamp_max(s["tokens"] - 1)].float().transpose(1, 2)
    position = (lengths[:, None] + j)[:, :, None]
    seen = (t[:, None] <= position) & ((t[:, None] > position - W) | (t[:, None] < S))
    B, H, _, D = q.shape
    group = H // c["kv_heads"]
    z = torch.matmul(q.reshape(B, H // group, group * n, D), k.transpose(2, 3).contiguous()) * (1.0 / math.sqrt(D))
    z = z.view(B, H // group, group, n, -1).masked_fill_(~seen[:, None, None], float("-inf"))
    p = torch.exp(z - z.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, H // group, group * n, -1), v.contiguous()).view(B, H, n, D)
    return o.transpose(1, 2)[j[None, :] < count[:, None]].to(s["q"].dtype)


def _of_rows(v, rows):
    return v[:, None] if torch.is_tensor(v) else torch.full((rows, 1), v, device=DEV)


def _plain_logits(s):
    c = s["case"]
    R, V = c["rows"], c["vocab"]
    z = s["logits"].float()
    if c["history"]:
        at = torch.arange(c["history"], device=DEV)[None, :]
        held, answered = at < s["lengths"][:, None], at >= s["prompts"][:, None]
        ids = s["history"].long()
        seen = torch.zeros((R, V), device=DEV).scatter_add_(1, ids, held.float()) > 0
        count = torch.zeros((R, V), device=DEV).scatter_add_(1, ids, (held & answered).float())
        r = _of_rows(s["repetition"], R)
        z = torch.where(seen, torch.where(z > 0, z / r, z * r), z)
        z = z - (_of_rows(s["frequency"], R) * count + _of_rows(s["presence"], R) * (count > 0))
    if c["biases"]:
        z = z.scatter_add(1, s["bias_ids"].long(), s["bias"])
    if c["grammar"]:
        v = torch.arange(V, device=DEV)
        z = z.masked_fill((s["allowed"][:, v // 32] >> (v % 32) & 1) == 0, float("-inf"))
    return z.to(s["logits"].dtype)


def _own_run(s):
    import bit_nf4_quantized_09_amd as nf4
    c = s["case"]
    if c["op"] == "norm":
        how = dict(pre=s["pre"], post=s["post"], gate=s["gate"], scale=s["scale"], eps=EPS)
        if not c["back"]:
            h, y = nf4.block_norm_fwd(s["h"], s["x"], **how)
            return ([h] if c["block"] else []) + ([y] if c["pre"] else [])
        dh, dx, dpre, dpost, dgate = nf4.block_norm_bwd(s["h"], s["dy"], s["dh"], s["x"], need_weights=c["learn"], **how)
        return [v for v in (dpre, dh, dx, dpost, dgate) if v is not None]
    if c["op"] == "clip":
        return {"norm": nf4.clip_grads(s["grads"], c["max_norm"], out=s["out"]), **s["buffers"]}
    if c["op"] == "attend":
        return nf4.kv_attention(nf4.KVCache(s["codes"], s["scales"]), s["q"], s["starts"], s["lengths"], s["table"],
                                max_new=s["most_new"], max_length=s["longest"], window=c["window"], sinks=c["sinks"])
    return nf4.shape_logits(s["logits"], s["history"], s["lengths"], s["prompts"], repetition=s["repetition"],
                            presence=s["presence"], frequency=s["frequency"], bias_ids=s["bias_ids"], bias=s["bias"],
                            allowed=s["allowed"])


def run(state):
    if own:
        return _own_run(state)
    plain = {"norm": _plain_norm, "clip": _plain_clip, "attend": _plain_attend, "logits": _plain_logits}
    return plain[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "norm":
        K, M = case["width"], case["seqs"] * case["tokens"]
        stream, weight = (2 if case[k] == "bfloat16" else 4 for k in ("stream", "weights"))
        gates = {"none": 0, "channel": 1, "sequence": case["seqs"], "token": M}[case["gate"]]
        byte = weight * K * (case["pre"] + case["post"] + gates)
        if case["back"]:
            reads = stream * (1 + case["pre"]) + 2 * case["block"] + 2 * case["pre"]     # dh, and h for its norm; x; dy
            if not case["post"] and not case["learn"]:
                reads -= 2 * case["block"]                                                # x itself is not needed
            byte += M * K * (reads + stream + 2 * case["block"])
            if case["learn"]:
                byte += 4 * K * (case["pre"] + case["post"] + gates)
        else:
            byte += M * K * (stream + (2 + stream) * case["block"] + 2 * case["pre"])
        return {"bytes": float(byte), "flops": float(M * K * (4 + 4 * case["block"]) * (2 if case["back"] else 1))}
    if op == "clip":
        shapes = _shapes(case)
        sizes = [4 if t == torch.float32 else 2 for t in _types(case, len(shapes))]
        byte = sum(2 * a * b * z for (a, b), z in zip(shapes, sizes))
        return {"bytes": float(byte + 4), "flops": 3.0 * sum(a * b for a, b in shapes)}
    if op == "attend":
        before, count = _ragged(case)
        T, D, S, W = int(count.sum()), case["head_dim"], case["sinks"], case["window"]
        total = before + count
        held = np.minimum(total, np.minimum(S, np.maximum(0, before - W + 1)) + np.minimum(total, W + count - 1))
        position = np.concatenate([np.arange(b, b + n) for b, n in zip(before, count)])
        seen = np.minimum(position + 1, W) + np.minimum(S, np.maximum(0, position + 1 - W))
        return {"bytes": 2.0 * float(held.sum()) * case["kv_heads"] * D + 4.0 * T * case["heads"] * D,
                "flops": 4.0 * float(seen.sum()) * case["heads"] * D}
    R, V = case["rows"], case["vocab"]
    size = 2 if case["dtype"] == "bfloat16" else 4
    byte = R * (2 * V * size + 4 * case["history"] * 5 / 8 + 8 * case["biases"] + (V / 8 if case["grammar"] else 0))
    return {"bytes": float(byte), "flops": 4.0 * R * V}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _unit(a):
    """Rows over the root of their mean square, and that root."""
    root = torch.sqrt((a * a).sum(-1, keepdim=True) / a.shape[-1] + EPS)
    return a / root, root


def _through_norm(d, a):
    """The gradient of a norm's input from that of its output."""
    n, root = _unit(a)
    return (d - n * ((d * n).sum(-1, keepdim=True) / a.shape[-1])) / root


def _exact_norm(case, s):
    K, M, learn = case["width"], s["h"].shape[0], case["learn"]
    wide = lambda v: None if v is None else v.double()  # noqa: E731
    pre, post, gate = wide(s["pre"]), wide(s["post"]), wide(s["gate"])
    parts = []
    sums = {"pre": 0.0, "post": 0.0}
    gates = torch.zeros_like(gate) if gate is not None else None
    for a in range(0, M, 1024):                      # a slice of rows at a time
        rows = torch.arange(a, min(M, a + 1024), device=DEV)
        h, x = s["h"][rows].double(), None if s["x"] is None else s["x"][rows].double()
        owner = None if gate is None else rows // (M // gate.shape[0])
        g = s["scale"] * (1.0 if gate is None else gate[owner])
        piece = []
        if not case["back"]:
            if case["block"]:
                h = h + g * (_unit(x)[0] * post if case["post"] else x)
                piece.append(h)
                h = h.to(s["h"].dtype).double()      # the norm is of the stream as it is stored
            if case["pre"]:
                piece.append(_unit(h)[0] * pre)
        else:
            d = s["dh"][rows].double()
            if case["pre"]:
                dy = s["dy"][rows].double()
                d = d + _through_norm(dy * pre, h)
                sums["pre"] = sums["pre"] + (dy * _unit(h)[0]).sum(0)
            piece.append(d)
            if case["block"]:
                p = _unit(x)[0] if case["post"] else x
                piece.append(_through_norm(g * d * post, x) if case["post"] else g * d)
                if case["post"]:
                    sums["post"] = sums["post"] + (g * d * p).sum(0)
                if gate is not None:
                    gates.index_add_(0, owner, s["scale"] * d * (p * post if case["post"] else p))
        parts.append(piece)
    whole = [torch.cat(v) for v in zip(*parts)]
    if not case["back"]:
        return whole
    out = ([sums["pre"]] if learn and case["pre"] else []) + whole
    out += [sums["post"]] if learn and case["post"] else []
    return out + ([gates] if learn and gate is not None else [])


def _exact_clip(case, s):
    total = torch.zeros((), dtype=torch.float64, device=DEV)
    for g in s["grads"]:
        total += torch.dot(g.double().flatten(), g.double().flatten())
    norm = float(total) ** 0.5
    f = min(1.0, case["max_norm"] / norm)
    out = {name: torch.zeros(b.shape, dtype=torch.float64, device=DEV) for name, b in s["buffers"].items()}
    ends, _ = _places(_shapes(case))
    for at, g in zip(ends, s["grads"]):
        out[str(g.dtype).split(".")[1]][at:at + g.numel()] = g.double().flatten() * f
    return {"norm": torch.tensor(norm, dtype=torch.float64), **out}


def _exact_attend(case, s):
    P, H, Hk, D = case["page"], case["heads"], case["kv_heads"], case["head_dim"]
    starts, lengths, table = s["starts"].tolist(), s["lengths"].tolist(), s["table"].long()
    out = torch.empty((s["tokens"], H, D), dtype=torch.float64, device=DEV)
    for b, n in enumerate(lengths):
        a, z = starts[b], starts[b + 1]
        key = torch.arange(n + z - a, device=DEV)
        key = key[(key < case["sinks"]) | (key > n - case["window"])]
        row = torch.arange(n, n + z - a, device=DEV)[:, None]
        hidden = (key > row) | ((key >= case["sinks"]) & (key <= row - case["window"]))
        page, slot = table[b, key // P], key % P
        for h in range(Hk):
            k, v = (s["codes"][page, i, h, slot].view(torch.float8_e4m3fn).double() * s["scales"][page, i, h].double()[:, None]
                    for i in (0, 1))
            for q in range(h * (H // Hk), (h + 1) * (H // Hk)):
                score = (s["q"][a:z, q].double() @ k.t() / math.sqrt(D)).masked_fill(hidden, float("-inf"))
                out[a:z, q] = torch.softmax(score, dim=-1) @ v
    return out


def _exact_logits(case, s):
    R, V = case["rows"], case["vocab"]
    out = []
    number = lambda v, r: float(v[r]) if torch.is_tensor(v) else float(v)  # noqa: E731
    for r in range(R):
        z = s["logits"][r].double()
        if case["history"]:
            n, m = int(s["lengths"][r]), int(s["prompts"][r])
            ids = s["history"][r, :n].long()
            met, said = torch.bincount(ids, minlength=V) > 0, torch.bincount(ids[m:], minlength=V)
            rep = number(s["repetition"], r)
            z = torch.where(met, torch.where(z > 0, z / rep, z * rep), z)
            z = z - number(s["frequency"], r) * said - number(s["presence"], r) * (said > 0)
        if case["biases"]:
            z[s["bias_ids"][r].long()] += s["bias"][r].double()
        if case["grammar"]:
            bits = s["allowed"][r].cpu().numpy().view(np.uint8)
            may = torch.from_numpy(np.unpackbits(bits, bitorder="little")[:V].astype(bool)).to(DEV)
            z = torch.where(may, z, torch.full_like(z, -math.inf))
        out.append(z)
    return torch.stack(out)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(case, s)
    return {"norm": _exact_norm, "clip": _exact_clip, "logits": _exact_logits}[case["op"]](case, s)
