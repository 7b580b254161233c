"""A small recurrent language model on the operators beside the Based forward pass.

ids -> scaled embedding -> layers of [norm, projections, gated recurrence, group norm times an
activated gate, projection] -> logits with the embedding's table. It is trained on right-padded
sequences in which every token follows from the one before, and then generates from prompts of
different lengths: one pass over the padded prompts fills a pool of states, and each new token takes
one step of the recurrence. In a layer of kind "based" the token mixer is the Based forward pass
(without a backward pass, so such layers score text and are not trained). In a layer of kind "delta" it is the gated
delta rule, and the norm in front of it also adds what the layer before has left to add to the residual stream.
Tokens are the most likely ones, or sampled from given random numbers.

    python examples/language_model.py [--steps 60] [--kinds recurrence,delta] [--temperature 0.7 --top-p 0.9]
"""
import argparse
import math
import os
import sys

import torch
import torch.nn.functional as F

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from linear_attention_gb300 import (based_delta_fwd, based_delta_step, based_embed_fwd, based_fwd, based_norm_fwd,  # noqa: E402
                                    based_rms_fwd, based_sample, based_scan_fwd, based_scan_step)
from linear_attention_gb300.autograd import delta_rule, embedding, gated_scan, group_norm, rms_norm  # noqa: E402


class Layer(torch.nn.Module):
    def __init__(self, width: int, heads: int, kind: str, dtype, device):
        super().__init__()
        self.width, self.heads, self.kind = width, heads, kind
        new = lambda *s: torch.nn.Parameter(torch.empty(*s, dtype=dtype, device=device))  # noqa: E731
        # one projection: the recurrence's gate and input and the output gate, or q, k, v and the output gate
        mixed = 2 * width if kind == "recurrence" else heads * 32 + width
        self.proj_in, self.proj_out = new(mixed + width, width), new(width, width)
        self.norm_w, self.norm_b, self.head_w, self.head_b = (new(width) for _ in range(4))
        with torch.no_grad():
            for p in (self.proj_in, self.proj_out):
                p.normal_(0, width ** -0.5)
            for p, v in ((self.norm_w, 1), (self.head_w, 1), (self.norm_b, 0), (self.head_b, 0)):
                p.fill_(v)

    def split(self, x, norm):
        """The mixer's inputs, views of one projection, and the output gate."""
        p = F.linear(norm(x, 1, self.norm_w, self.norm_b, act="none"), self.proj_in)
        return p[..., :-self.width], p[..., -self.width:]

    def out(self, x, mixed, gate, norm):
        return x + F.linear(norm(mixed, self.heads, self.head_w, self.head_b, gate), self.proj_out)

    def train_forward(self, x, lengths):
        m, gate = self.split(x, group_norm)
        h, _ = gated_scan(m[..., :self.width] + 2.0, m[..., self.width:], lengths=lengths)
        return self.out(x, h, gate, group_norm)

    def prefill(self, x, lengths):
        """The layer on whole prompts, and the states behind them (None for the Based mixer)."""
        m, gate = self.split(x, based_norm_fwd)
        if self.kind == "based":
            B, T, _ = x.shape
            q, k, v = (t.reshape(B, T, self.heads, -1) for t in m.split([self.heads * 16, self.heads * 16, self.width], -1))
            o = based_fwd(q.contiguous(), k.contiguous(), v.contiguous())
            return self.out(x, o.view(B, T, self.width), gate, based_norm_fwd), None
        h, state, _ = based_scan_fwd(m[..., :self.width] + 2.0, m[..., self.width:], lengths=lengths)
        return self.out(x, h, gate, based_norm_fwd), state

    def step(self, x, pool, slots):
        """One token of each sequence; the pool's states move on."""
        m, gate = self.split(x, based_norm_fwd)
        return self.out(x, based_scan_step(m[:, :self.width] + 2.0, m[:, self.width:], pool, slots=slots), gate, based_norm_fwd)

    def pool(self, slots, device):
        return torch.zeros(slots, self.width, device=device)


def settled(x, update):
    """The stream with what is still to be added."""
    return x if update is None else x + update


class DeltaLayer(torch.nn.Module):
    """A layer of the gated delta rule. It takes the stream and what is still to be added to it, and returns the two."""

    def __init__(self, width: int, heads: int, dtype, device):
        super().__init__()
        self.width, self.heads, self.size = width, heads, width // heads
        new = lambda *s: torch.nn.Parameter(torch.empty(*s, dtype=dtype, device=device))  # noqa: E731
        # q, k, v, the output gate, and a gate and a step size for each head
        self.proj_in, self.proj_out = new(4 * width + 2 * heads, width), new(width, width)
        self.norm_w, self.head_w = new(width), new(width)
        with torch.no_grad():
            for p in (self.proj_in, self.proj_out):
                p.normal_(0, width ** -0.5)
            self.norm_w.fill_(1), self.head_w.fill_(1)

    def split(self, y):
        p = F.linear(y, self.proj_in)
        q, k, v, out, beta, gate = p.split([self.width] * 4 + [self.heads] * 2, -1)
        q, k, v = (t.unflatten(-1, (self.heads, self.size)) for t in (q, k, v))
        return F.normalize(q, dim=-1), F.normalize(k, dim=-1), v, torch.sigmoid(beta), F.logsigmoid(gate + 3.0), out

    def train_forward(self, x, update, lengths):
        y, x = rms_norm(x, self.norm_w) if update is None else rms_norm(update, self.norm_w, residual=x)
        *mix, out = self.split(y)
        o, _ = delta_rule(*mix, lengths=lengths)
        return x, F.linear(group_norm(o.flatten(-2), self.heads, self.head_w, gate=out), self.proj_out)

    def run(self, x, update, mixer):
        y, x, _ = based_rms_fwd(x, self.norm_w) if update is None else based_rms_fwd(update, self.norm_w, residual=x)
        *mix, out = self.split(y)
        o, state = mixer(*mix)
        return x, F.linear(based_norm_fwd(o.flatten(-2), self.heads, self.head_w, gate=out), self.proj_out), state

    def prefill(self, x, update, lengths):
        return self.run(x, update, lambda *mix: based_delta_fwd(*mix, lengths=lengths)[:2])

    def step(self, x, update, pool, slots):
        return self.run(x, update, lambda *mix: (based_delta_step(*mix, pool, slots=slots), None))[:2]

    def pool(self, slots, device):
        return torch.zeros(slots, self.heads, self.size, self.size, device=device)


class Model(torch.nn.Module):
    def __init__(self, vocab=512, width=256, heads=4, kinds=("recurrence", "recurrence"), dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.vocab, self.width, self.scale = vocab, width, math.sqrt(width)
        self.table = torch.nn.Parameter(torch.randn(vocab, width, device=device).mul_(width ** -0.5).to(dtype))
        self.layers = torch.nn.ModuleList(
            DeltaLayer(width, heads, dtype, device) if k == "delta" else Layer(width, heads, k, dtype, device) for k in kinds)
        self.last_w = torch.nn.Parameter(torch.ones(width, dtype=dtype, device=device))

    def logits(self, x, norm):
        return F.linear(norm(x, 1, self.last_w, act="none"), self.table).float()

    def loss(self, ids, lengths):
        """Mean loss of predicting each token from those before it; ids (B,T) hold -1 past the lengths."""
        x = embedding(ids[:, :-1], self.table, self.scale)
        update = None  # what a layer of kind "delta" leaves to the norm behind it to add
        for layer in self.layers:
            live = (lengths - 1).clamp(min=0).to(torch.int32)
            if isinstance(layer, DeltaLayer):
                x, update = layer.train_forward(x, update, live)
            else:
                x, update = layer.train_forward(settled(x, update), live), None
        x = settled(x, update)
        return F.cross_entropy(self.logits(x, group_norm).flatten(0, 1), ids[:, 1:].flatten().long(), ignore_index=-1)

    @torch.no_grad()
    def prefill(self, ids, lengths):
        """Logits of every position (B,T,vocab) and each layer's states (B,width)."""
        x, update, states = based_embed_fwd(ids, self.table, self.scale), None, []
        for layer in self.layers:
            if isinstance(layer, DeltaLayer):
                x, update, state = layer.prefill(x, update, lengths)
            else:
                (x, state), update = layer.prefill(settled(x, update), lengths), None
            states.append(state)
        return self.logits(settled(x, update), based_norm_fwd), states

    @torch.no_grad()
    def generate(self, ids, lengths, count, slots_in_pool=64, **limits):
        """`count` next tokens of each prompt: (B,count). The most likely ones, or, with any of the limits of based_sample
        (temperature, top_k, top_p, min_p), sampled from torch's random numbers."""
        logits, states = self.prefill(ids, lengths)
        B = ids.shape[0]
        # the sequences' places in a pool of states that a server shares among its requests
        slots = torch.randperm(slots_in_pool, device=ids.device)[:B].to(torch.int32)
        pools = []
        for layer, state in zip(self.layers, states):
            pool = layer.pool(slots_in_pool, ids.device)
            pool[slots.long()] = state
            pools.append(pool)

        def choose(logits):
            return based_sample(logits, torch.rand(B, device=ids.device), **limits)[0] if limits else logits.argmax(-1)

        token = choose(logits[torch.arange(B, device=ids.device), lengths.long() - 1])
        out = [token]
        for _ in range(count - 1):
            x, update = based_embed_fwd(token, self.table, self.scale), None
            for layer, pool in zip(self.layers, pools):
                if isinstance(layer, DeltaLayer):
                    x, update = layer.step(x, update, pool, slots)
                else:
                    x, update = layer.step(settled(x, update), pool, slots), None
            token = choose(self.logits(settled(x, update), based_norm_fwd))
            out.append(token)
        return torch.stack(out, 1)


def batch(vocab, B, T, gen, device="cuda"):
    """Sequences in which token t + 1 is (5 token_t + 3) mod vocab, padded with -1 past their lengths."""
    lengths = torch.randint(T // 2, T + 1, (B,), generator=gen)
    ids = torch.empty(B, T, dtype=torch.long)
    ids[:, 0] = torch.randint(0, vocab, (B,), generator=gen)
    for t in range(1, T):
        ids[:, t] = (5 * ids[:, t - 1] + 3) % vocab
    ids[torch.arange(T)[None] >= lengths[:, None]] = -1
    return ids.to(torch.int32).to(device), lengths.to(torch.int32).to(device)


def train(model, steps, gen, B=16, T=128):
    """The loss of each step."""
    opt = torch.optim.AdamW(model.parameters(), lr=3e-3, weight_decay=0.0)
    losses = []
    for _ in range(steps):
        loss = model.loss(*batch(model.vocab, B, T, gen))
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--kinds", default="recurrence,recurrence", help="the layers, by commas: recurrence or delta")
    for name, kind in (("temperature", float), ("top-k", int), ("top-p", float), ("min-p", float)):
        ap.add_argument("--" + name, type=kind, help="sample the tokens with this limit")
    a = ap.parse_args()
    torch.manual_seed(0)
    gen = torch.Generator().manual_seed(0)
    model = Model(kinds=tuple(a.kinds.split(",")))
    limits = {k: v for k, v in vars(a).items() if k not in ("steps", "kinds") and v is not None}
    losses = train(model, a.steps, gen)
    print("loss of the first and last five steps: %.3f %.3f" % (sum(losses[:5]) / 5, sum(losses[-5:]) / 5))
    ids, lengths = batch(model.vocab, 8, 40, gen)
    got = model.generate(ids, lengths, 12, **limits)
    last = ids[torch.arange(8, device=ids.device), lengths.long() - 1].long()
    right = 0
    for i in range(12):
        last = (5 * last + 3) % model.vocab
        right += int((got[:, i] == last).sum())
    print("%d of %d generated tokens follow the rule" % (right, got.numel()))


if __name__ == "__main__":
    main()
