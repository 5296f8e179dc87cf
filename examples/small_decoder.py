"""A small decoder whose linears are QLoRA layers: trains its adapters, then answers from a paged cache.

    python examples/small_decoder.py

Random frozen NF4 weights stand in for a trained model's.  Training runs block_norm_fwd / block_norm_bwd between
the blocks, rope_fwd / rope_bwd around plain causal attention, head_loss for the loss with its gradient in one
call, and PagedAdamW on the adapters, their gradients clipped to a global norm.  Serving appends ragged prompts
and then single tokens with kv_append (which rotates queries and keys on the way) and attends with kv_attention,
over everything or a window, whose old pages it gives back; shape_logits keeps an answer from repeating itself.
Both read the same weights and adapters, so the answer's loss can be compared between them.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bit_nf4_quantized_09_amd as nf4  # noqa: E402

WIDTH, FFN, HEADS, KV_HEADS, DIM, VOCAB, LAYERS, RANK, ALPHA = 512, 1024, 8, 4, 64, 1000, 2, 16, 16.0


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, layer, A, B):
        y, t = nf4.qlora_linear_fwd(layer.weight, x, A, B, ALPHA)
        ctx.layer = layer
        ctx.save_for_backward(x, A, B, t)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, A, B, t = ctx.saved_tensors
        dx, dA, dB = nf4.qlora_linear_bwd(ctx.layer.weight, x, dy.contiguous(), A, B, ALPHA, T=t)
        ctx.layer.gradients = (dA, dB)              # fp32, as the optimizer takes them
        return dx, None, None, None


class _Rope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, plan, positions):
        ctx.plan, ctx.positions = plan, positions
        return nf4.rope_fwd(plan, positions, q, k)

    @staticmethod
    def backward(ctx, dq, dk):
        return (*nf4.rope_bwd(ctx.plan, ctx.positions, dq.contiguous(), dk.contiguous()), None, None)


class _Norm(torch.autograd.Function):
    """The norm of the stream h."""

    @staticmethod
    def forward(ctx, h):
        ctx.save_for_backward(h)
        return nf4.block_norm_fwd(h)[1]

    @staticmethod
    def backward(ctx, dy):
        return nf4.block_norm_bwd(ctx.saved_tensors[0], dy.contiguous())[0]


class _BlockNorm(torch.autograd.Function):
    """The stream after a block, and its norm."""

    @staticmethod
    def forward(ctx, h, x):
        h, y = nf4.block_norm_fwd(h, x)
        ctx.save_for_backward(h, x)
        return h, y

    @staticmethod
    def backward(ctx, dh, dy):
        h, x = ctx.saved_tensors
        return nf4.block_norm_bwd(h, dy.contiguous(), dh.contiguous(), x)[:2]


class _Loss(torch.autograd.Function):
    """The mean loss over the targets that count; its gradient is made in the same call."""

    @staticmethod
    def forward(ctx, x, head, targets):
        each = torch.full(targets.shape, 1.0, device=x.device) / (targets >= 0).sum().clamp(min=1)
        loss, dx, _ = nf4.head_loss(x, head, targets, dloss=each)
        ctx.save_for_backward(dx)
        return (loss * each).sum()

    @staticmethod
    def backward(ctx, d):
        return ctx.saved_tensors[0] * d, None, None


class Linear:
    def __init__(self, n, k, g):
        self.weight = nf4.quantize_weight(torch.randn((n, k), generator=g, device="cuda") / math.sqrt(k))
        self.A = (torch.randn((RANK, k), generator=g, device="cuda") / math.sqrt(k)).bfloat16()
        self.B = torch.zeros((n, RANK), device="cuda", dtype=torch.bfloat16)
        self.gradients = None

    def __call__(self, x):
        return _Linear.apply(x, self, self.A, self.B)


class Decoder:
    def __init__(self, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.table = torch.randn((VOCAB, WIDTH), generator=g, device="cuda").bfloat16()
        self.head = (torch.randn((VOCAB, WIDTH), generator=g, device="cuda") / math.sqrt(WIDTH)).bfloat16()
        self.layers = [dict(qkv=Linear((HEADS + 2 * KV_HEADS) * DIM, WIDTH, g), out=Linear(WIDTH, HEADS * DIM, g),
                            up=Linear(2 * FFN, WIDTH, g), down=Linear(WIDTH, FFN, g)) for _ in range(LAYERS)]
        self.plan = nf4.rope_plan(DIM)

    def linears(self):
        return [m for layer in self.layers for m in layer.values()]

    def hidden(self, tokens, attend):
        """Tokens [T] through the layers; attend(i, q, k, v) is layer i's attention, positions included."""
        h = self.table[tokens]
        y = _Norm.apply(h)
        for i, layer in enumerate(self.layers):
            qkv = layer["qkv"](y).view(-1, HEADS + 2 * KV_HEADS, DIM)
            q, k, v = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV_HEADS], qkv[:, HEADS + KV_HEADS:]
            h, y = _BlockNorm.apply(h, layer["out"](attend(i, q, k, v).reshape(-1, HEADS * DIM).contiguous()))
            gate, up = layer["up"](y).chunk(2, -1)
            h, y = _BlockNorm.apply(h, layer["down"]((torch.nn.functional.silu(gate.float()) * up.float()).bfloat16()))
        return y


def train_loss(model, tokens, targets):
    """Mean loss of one sequence, differentiable."""
    T = tokens.numel()
    positions = torch.arange(T, dtype=torch.int32, device="cuda")
    later = torch.ones((T, T), dtype=torch.bool, device="cuda").triu(1)

    def attend(i, q, k, v):
        q, k = _Rope.apply(q, k, model.plan, positions)
        q, k, v = (y.float().transpose(0, 1) for y in (q, k, v))
        k, v = (y.repeat_interleave(HEADS // KV_HEADS, 0) for y in (k, v))
        z = torch.matmul(q, k.transpose(1, 2).contiguous()) / math.sqrt(DIM)
        return torch.matmul(z.masked_fill(later, -math.inf).softmax(-1), v).transpose(0, 1).bfloat16()

    return _Loss.apply(model.hidden(tokens, attend), model.head, targets)


def train(model, tokens, targets, steps=20, lr=3e-3, max_norm=1.0, say=None):
    """Adapter steps on one sequence, the gradients clipped to a norm of max_norm (None: as they are); returns the
    losses.  say gets a line for each step."""
    linears = model.linears()
    opt = nf4.PagedAdamW([p for m in linears for p in (m.A, m.B)], lr=lr)
    model.table.requires_grad_(True)                # so that the first layer's gradient is asked for, like the others'
    losses = []
    for i in range(steps):
        loss = train_loss(model, tokens, targets)
        loss.backward()
        size = opt.step([d for m in linears for d in m.gradients], max_norm=max_norm)
        losses.append(float(loss.detach()))
        if say is not None:
            say("step %2d  loss %.4f%s" % (i, losses[-1], "" if size is None else "  gradients %.3f" % float(size)))
    model.table.requires_grad_(False)
    model.table.grad = None
    return losses


class Server:
    """Sequences of one model over one paged cache per layer.  With a window a token attends to the last `window`
    keys and the first `sinks`, and pages that no later token sees are given back (table entries of -1)."""

    def __init__(self, model, seqs, longest, page=16, window=None, sinks=4):
        self.model, self.page, self.window, self.sinks = model, page, window, sinks
        width = -(-longest // page)
        self.caches = [nf4.kv_cache(seqs * width, KV_HEADS, DIM, page) for _ in range(LAYERS)]
        self.pages = torch.randperm(seqs * width, device="cuda").to(torch.int32).view(seqs, width)
        self.lengths = torch.zeros(seqs, dtype=torch.int32, device="cuda")

    def step(self, new):
        """new: each sequence's new tokens (lists; possibly empty).  Hidden states of all, packed."""
        starts = [0]
        for n in new:
            starts.append(starts[-1] + len(n))
        tokens = torch.tensor([t for n in new for t in n], device="cuda")
        starts = torch.tensor(starts, dtype=torch.int32, device="cuda")

        def attend(i, q, k, v):
            q = nf4.kv_append(self.caches[i], k, v, starts, self.lengths, self.pages, rope=self.model.plan, q=q)
            return nf4.kv_attention(self.caches[i], q, starts, self.lengths, self.pages, max_new=max(map(len, new)),
                                    window=self.window, sinks=self.sinks)

        with torch.no_grad():
            x = self.model.hidden(tokens, attend)
        self.lengths += starts[1:] - starts[:-1]
        if self.window is not None:
            at = torch.arange(self.pages.shape[1], device="cuda") * self.page
            unseen = (at + self.page <= (self.lengths - self.window + 1)[:, None]) & (at >= self.sinks)
            self.pages.masked_fill_(unseen, -1)
        return x, starts

    def answer(self, prompts, count, repetition=1.0, allowed=None):
        """The next `count` tokens of each prompt, the likeliest each time; tokens that were there before are made
        less likely by `repetition`, and only those of the mask `allowed` are taken."""
        x, starts = self.step(prompts)
        last = x[starts[1:].long() - 1]
        out = [[] for _ in prompts]
        longest = max(map(len, prompts)) + count
        history = torch.zeros((len(prompts), longest), dtype=torch.int32)
        for row, p in zip(history, prompts):
            row[:len(p)] = torch.tensor(p)
        history = history.cuda()
        for i in range(count):
            lengths = torch.tensor([len(p) + i for p in prompts], dtype=torch.int32, device="cuda")
            logits = nf4.shape_logits(last.float() @ self.model.head.float().t(), history, lengths, repetition=repetition, allowed=allowed)
            choice = logits.argmax(-1)
            history.scatter_(1, lengths.long()[:, None], choice.to(torch.int32)[:, None])
            best = choice.tolist()
            for row, t in zip(out, best):
                row.append(t)
            if i + 1 < count:
                last, _ = self.step([[t] for t in best])
        return out

    def score(self, tokens, split):
        """Mean loss of tokens[split:] after tokens[:split], as one prompt and then token by token."""
        x, _ = self.step([tokens[:split]])
        states = [x[-1:]]
        for t in tokens[split:-1]:
            states.append(self.step([[t]])[0])
        loss, _, _ = nf4.head_loss(torch.cat(states), self.model.head, torch.tensor(tokens[split:], device="cuda"))
        return float(loss.mean())


def main():
    model = Decoder()
    g = torch.Generator().manual_seed(1)
    text = torch.randint(0, VOCAB, (97,), generator=g).tolist()
    tokens, targets = torch.tensor(text[:-1], device="cuda"), torch.tensor(text[1:], device="cuda")
    targets[:15] = -100                             # the prompt carries no loss
    train(model, tokens, targets, say=print)
    served = Server(model, 1, 128).score(text, 16)
    print("loss of the answer: trained form %.4f, from the paged cache %.4f" % (float(train_loss(model, tokens, targets)), served))
    prompts = [text[:16], text[:40], text[:23]]
    for p, a in zip(prompts, Server(model, 3, 128).answer(prompts, 8)):
        print("after %2d tokens: %s; the text has %s" % (len(p), a, text[len(p):len(p) + 8]))
    print("from a window of 24: %s" % Server(model, 1, 128, window=24).answer(prompts[:1], 8, repetition=1.3)[0])


if __name__ == "__main__":
    main()
