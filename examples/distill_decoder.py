"""A small decoder trained from a teacher's top logits, then served a token at a time.

    python examples/distill_decoder.py [--steps 150]

Training: every linear layer is an Int8MixedPrecisionActLinear (bias, SiLU and the
residual stream in the INT8 GEMMs' epilogue), query and key heads are views of one
packed projection turned by training.rotary, and the loss is
training.distill_loss against the teacher's kept logits, with the rest of its
distribution as one more class.  Serving: the weights are quantized once, each token
runs through operators.linear_wq_fwd, its heads are turned in place in the packed
projection, and keys and values stay in a cache.  The teacher is a table of next-token
logits, so what the student should answer is known."""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import int8_mixed_precision_rowwise_amd as i8  # noqa: E402
from int8_mixed_precision_rowwise_amd import training  # noqa: E402

VOCAB, KEPT, HIDDEN, FFN, LAYERS = 1021, 16, 256, 704, 2
HQ, HK, D = 4, 2, 64
TAU, CE = 2.0, 0.25
bf16 = torch.bfloat16


class Teacher:
    """Next-token logits by the current token: the top ones, and the whole row's log-sum-exp."""

    def __init__(self, device):
        g = torch.Generator(device=device).manual_seed(1)
        logits = torch.randn(VOCAB, VOCAB, generator=g, device=device)
        self.best = torch.randperm(VOCAB, generator=g, device=device)
        logits.scatter_(1, self.best[:, None], 9.0)
        self.probs = torch.softmax(logits, 1)
        top, idx = logits.topk(KEPT, 1)
        self.top, self.idx = top.to(bf16), idx.int()
        self.lse = torch.logsumexp(logits / TAU, 1)

    def sample(self, B, S):
        tokens = [torch.randint(0, VOCAB, (B, 1), device=self.best.device)]
        for _ in range(S):
            tokens.append(torch.multinomial(self.probs[tokens[-1][:, 0]], 1))
        return torch.cat(tokens, 1)


def norm(x):
    y = x.float()
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


def attend(q, k, v, mask):
    """q [B, S, HQ, D] over k, v [B, L, HK, D], softmax and products in fp32; mask [S, L]."""
    q, k, v = (t.float().transpose(1, 2).contiguous() for t in (q, k, v))
    k, v = (t.repeat_interleave(HQ // HK, 1) for t in (k, v))
    s = torch.matmul(q, k.transpose(2, 3).contiguous()) / math.sqrt(D)
    p = torch.softmax(s.masked_fill(~mask, -math.inf), -1)
    return torch.matmul(p, v).transpose(1, 2).flatten(2).to(bf16)


class Block(torch.nn.Module):
    def __init__(self, seed, device):
        super().__init__()
        make = lambda i, k, n, act="none": training.Int8MixedPrecisionActLinear(k, n, activation=act, seed=seed + i, device=device)  # noqa: E731
        self.qkv = make(0, HIDDEN, (HQ + 2 * HK) * D)
        self.out = make(1, HQ * D, HIDDEN)
        self.up = make(2, HIDDEN, FFN, "silu")
        self.down = make(3, FFN, HIDDEN)

    def forward(self, x, positions, freqs, mask):
        p = self.qkv(norm(x)).unflatten(-1, (HQ + 2 * HK, D))
        q, k = training.rotary(p[:, :, :HQ], p[:, :, HQ:HQ + HK], positions, freqs)
        x = self.out(attend(q, k, p[:, :, HQ + HK:], mask), residual=x)
        return self.down(self.up(norm(x)), residual=x)


class Student(torch.nn.Module):
    def __init__(self, device):
        super().__init__()
        self.embed = torch.nn.Parameter(torch.randn(VOCAB, HIDDEN, device=device).to(bf16))
        self.blocks = torch.nn.ModuleList(Block(10 * i, device) for i in range(LAYERS))
        self.head = training.Int8MixedPrecisionActLinear(HIDDEN, VOCAB, bias=False, seed=99, device=device)
        self.register_buffer("freqs", i8.rotary_frequencies(D, device=device))

    def forward(self, tokens):
        S = tokens.shape[1]
        positions = torch.arange(S, device=tokens.device)
        mask = positions[:, None] >= positions
        x = self.embed[tokens]
        for b in self.blocks:
            x = b(x, positions, self.freqs, mask)
        return self.head(norm(x))


class Server:
    """The student's weights quantized once, and a cache of keys and values."""

    def __init__(self, student, B, length):
        self.embed, self.freqs = student.embed.detach(), student.freqs
        fixed = lambda l: (*i8.quantize_rowwise(l.weight.detach()), None if l.bias is None else l.bias.detach(), l.activation)  # noqa: E731
        self.blocks = [[fixed(l) for l in (b.qkv, b.out, b.up, b.down)] for b in student.blocks]
        self.head = fixed(student.head)
        self.k, self.v = (torch.zeros(LAYERS, B, length, HK, D, dtype=bf16, device=self.embed.device) for _ in range(2))
        self.at = 0

    @staticmethod
    def linear(x, layer, residual=None):
        Wq, scale, bias, act = layer
        return i8.linear_wq_fwd(x, Wq, scale, bias=bias, activation=act, residual=residual)

    def step(self, tokens):
        """Logits [B, VOCAB] behind tokens [B]."""
        x, n = self.embed[tokens], self.at
        position = torch.full((1,), n, device=tokens.device)
        mask = torch.ones(1, n + 1, dtype=torch.bool, device=tokens.device)
        for (qkv, out, up, down), k_all, v_all in zip(self.blocks, self.k, self.v):
            p = self.linear(norm(x), qkv).view(-1, 1, HQ + 2 * HK, D)
            q, k = p[:, :, :HQ], p[:, :, HQ:HQ + HK]
            i8.rotary(q, k, position, self.freqs, out_q=q, out_k=k_all[:, n:n + 1])
            v_all[:, n] = p[:, 0, HQ + HK:]
            a = attend(q, k_all[:, :n + 1], v_all[:, :n + 1], mask).flatten(1)
            x = self.linear(a, out, residual=x)
            x = self.linear(self.linear(norm(x), up), down, residual=x)
        self.at += 1
        return self.linear(norm(x), self.head)


def run(steps=150, B=16, S=64, device="cuda", say=print):
    torch.manual_seed(0)
    teacher, student = Teacher(device), Student(device)
    optimizer = torch.optim.AdamW(student.parameters(), lr=2e-3, weight_decay=0.0)
    losses = []
    for step in range(steps):
        tokens = teacher.sample(B, S)
        now, then = tokens[:, :-1], tokens[:, 1:].reshape(-1)
        logits = student(now).flatten(0, 1)
        at = now.reshape(-1)
        rows = training.distill_loss(logits, teacher.top[at], teacher.idx[at], TAU, teacher.lse[at], then, CE)
        loss = rows.mean()
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        losses.append(loss.detach())
        if step % 25 == 0 or step == steps - 1:
            say(f"step {step}: loss {float(losses[-1]):.4f}", flush=True)
    # serving: eight sequences answered greedily, against the teacher's best next token
    server = Server(student, 8, 32)
    tokens = torch.randint(0, VOCAB, (8,), device=device)
    seen, served, right = [], [], 0
    for _ in range(32):
        seen.append(tokens)
        served.append(server.step(tokens))
        right += int((served[-1].argmax(1) == teacher.best[tokens]).sum())
        tokens = served[-1].argmax(1)
    with torch.no_grad():
        whole = student(torch.stack(seen, 1))
    apart = float((torch.stack(served, 1).float() - whole.float()).abs().max() / whole.float().abs().max())
    say(f"served: {right} of 256 tokens are the teacher's first choice; logits within {apart:.4f} of the whole sequences'", flush=True)
    return float(losses[0]), float(losses[-1]), right / 256, apart


if __name__ == "__main__":
    parser = argparse.ArgumentParser()
    parser.add_argument("--steps", type=int, default=150)
    run(parser.parse_args().steps)
