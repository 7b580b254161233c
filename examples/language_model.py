"""A small recurrent language model on the operators beside the Based forward pass.

ids -> scaled embedding -> layers of [norm, projections, gated recurrence, group norm times an
activated gate, projection] -> logits with the embedding's table. It is trained on right-padded
sequences in which every token follows from the one before, and then generates from prompts of
different lengths: one pass over the padded prompts fills a pool of states, and each new token takes
one step of the recurrence. In a layer of kind "based" the token mixer is the Based forward pass
(without a backward pass, so such layers score text and are not trained).

    python examples/language_model.py [--steps 60]
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

from linear_attention_gb300 import based_embed_fwd, based_fwd, based_norm_fwd, based_scan_fwd, based_scan_step  # noqa: E402
from linear_attention_gb300.autograd import embedding, gated_scan, group_norm  # noqa: E402


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


class Model(torch.nn.Module):
    def __init__(self, vocab=512, width=256, heads=4, kinds=("recurrence", "recurrence"), dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.vocab, self.width, self.scale = vocab, width, math.sqrt(width)
        self.table = torch.nn.Parameter(torch.randn(vocab, width, device=device).mul_(width ** -0.5).to(dtype))
        self.layers = torch.nn.ModuleList(Layer(width, heads, k, dtype, device) for k in kinds)
        self.last_w = torch.nn.Parameter(torch.ones(width, dtype=dtype, device=device))

    def logits(self, x, norm):
        return F.linear(norm(x, 1, self.last_w, act="none"), self.table).float()

    def loss(self, ids, lengths):
        """Mean loss of predicting each token from those before it; ids (B,T) hold -1 past the lengths."""
        x = embedding(ids[:, :-1], self.table, self.scale)
        for layer in self.layers:
            x = layer.train_forward(x, (lengths - 1).clamp(min=0).to(torch.int32))
        return F.cross_entropy(self.logits(x, group_norm).flatten(0, 1), ids[:, 1:].flatten().long(), ignore_index=-1)

    @torch.no_grad()
    def prefill(self, ids, lengths):
        """Logits of every position (B,T,vocab) and each layer's states (B,width)."""
        x, states = based_embed_fwd(ids, self.table, self.scale), []
        for layer in self.layers:
            x, state = layer.prefill(x, lengths)
            states.append(state)
        return self.logits(x, based_norm_fwd), states

    @torch.no_grad()
    def generate(self, ids, lengths, count, slots_in_pool=64):
        """The `count` most likely next tokens of each prompt, greedily: (B,count)."""
        logits, states = self.prefill(ids, lengths)
        B = ids.shape[0]
        # the sequences' places in a pool of states that a server shares among its requests
        slots = torch.randperm(slots_in_pool, device=ids.device)[:B].to(torch.int32)
        pools = []
        for state in states:
            pool = torch.zeros(slots_in_pool, self.width, device=ids.device)
            pool[slots.long()] = state
            pools.append(pool)
        token = logits[torch.arange(B, device=ids.device), lengths.long() - 1].argmax(-1)
        out = [token]
        for _ in range(count - 1):
            x = based_embed_fwd(token, self.table, self.scale)
            for layer, pool in zip(self.layers, pools):
                x = layer.step(x, pool, slots)
            token = self.logits(x, based_norm_fwd).argmax(-1)
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
    a = ap.parse_args()
    torch.manual_seed(0)
    gen = torch.Generator().manual_seed(0)
    model = Model()
    losses = train(model, a.steps, gen)
    print("loss of the first and last five steps: %.3f %.3f" % (sum(losses[:5]) / 5, sum(losses[-5:]) / 5))
    ids, lengths = batch(model.vocab, 8, 40, gen)
    got = model.generate(ids, lengths, 12)
    last = ids[torch.arange(8, device=ids.device), lengths.long() - 1].long()
    right = 0
    for i in range(12):
        last = (5 * last + 3) % model.vocab
        right += int((got[:, i] == last).sum())
    print("%d of %d generated tokens follow the rule" % (right, got.numel()))


if __name__ == "__main__":
    main()
