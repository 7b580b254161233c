"""The delta rule, the residual stream's norm and sampling together: a layer against torch's autograd in 64 bits, the example's language
model in training and generation, and its steps captured into a graph."""
import importlib.util
import os

import pytest
import torch

from linear_attention_gb300 import based_delta_fwd, based_rms_fwd, based_sample
from linear_attention_gb300.autograd import delta_rule, group_norm, rms_norm

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("language_model", os.path.join(ROOT, "examples", "language_model.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def plain(x, stream, w, wq, wk, wv, wb, wg, lengths, heads):
    """Addition and norm, five projections, and the delta rule row by row."""
    s = x + stream
    y = s / torch.sqrt((s * s).mean(-1, keepdim=True) + 1e-6) * w
    cut = lambda t: t.unflatten(-1, (heads, -1))  # noqa: E731
    q, k, v = cut(y @ wq), cut(y @ wk), cut(y @ wv)
    k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + 1e-6)
    beta, a = torch.sigmoid(y @ wb), torch.sigmoid(y @ wg + 3)
    B, T = x.shape[:2]
    S = torch.zeros(B, heads, k.shape[-1], v.shape[-1], dtype=x.dtype)
    out = []
    for t in range(T):
        live = (t < lengths)[:, None, None]
        P = S * a[:, t, :, None, None]
        u = beta[:, t, :, None] * (v[:, t] - torch.einsum("bhkv,bhk->bhv", P, k[:, t]))
        S = torch.where(live[..., None], P + k[:, t, :, :, None] * u[:, :, None], S)
        o = torch.einsum("bhkv,bhk->bhv", S, q[:, t]) * k.shape[-1] ** -0.5
        out.append(torch.where(live, o, 0.0).flatten(1))
    return torch.stack(out, 1), s, S


def test_gradients_through_a_layer(cuda_device):
    gen = torch.Generator().manual_seed(1)
    B, T, D, heads = 3, 90, 48, 3
    rand = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    lengths = torch.tensor([90, 33, 64])
    leaves = [rand(B, T, D), rand(B, T, D), 1 + 0.1 * rand(D), *(rand(D, D) / 7 for _ in range(3)), rand(D, heads) / 7, rand(D, heads) / 7]
    cot, cot_s, cot_state = rand(B, T, D), rand(B, T, D), rand(B, heads, D // heads, D // heads)
    ref = [t.clone().requires_grad_() for t in leaves]
    o, s, S = plain(*ref, lengths, heads)
    ((o * cot).sum() + (s * cot_s).sum() + (S * cot_state).sum()).backward()
    mine = [t.float().cuda().requires_grad_() for t in leaves]
    x, stream, w, wq, wk, wv, wb, wg = mine
    y, total = rms_norm(x, w, stream)
    cut = lambda t: t.unflatten(-1, (heads, -1))  # noqa: E731
    q, k, v = cut(y @ wq), cut(y @ wk), cut(y @ wv)
    k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + 1e-6)
    o, S = delta_rule(q, k, v, torch.sigmoid(y @ wb), torch.nn.functional.logsigmoid(y @ wg + 3), lengths=lengths.to(torch.int32).cuda())
    ((o.flatten(2) * cot.float().cuda()).sum() + (total * cot_s.float().cuda()).sum() + (S * cot_state.float().cuda()).sum()).backward()
    # float32 against float64 through 90 dependent rows and products of 48 terms, gradients summed over 270 rows: some thousand
    # roundings of 2^-22 that are independent of one another, relative to the largest gradient
    for name, p, r in zip("x stream w wq wk wv wb wg".split(), mine, ref):
        assert ((p.grad.cpu().double() - r.grad).abs() <= 64 * 2.0 ** -22 * r.grad.abs().max()).all(), name


@pytest.mark.parametrize("kinds", [("delta", "delta"), ("recurrence", "delta", "recurrence")])
def test_model_trains_and_generates(cuda_device, kinds):
    m = example()
    torch.manual_seed(0)
    gen = torch.Generator().manual_seed(0)
    model = m.Model(vocab=64, width=128, heads=2, kinds=kinds)
    losses = m.train(model, 3, gen, B=4, T=100)
    assert all(0 < x < 20 for x in losses) and all(p.grad is not None and p.grad.isfinite().all() for p in model.parameters())
    ids, lengths = m.batch(64, 5, 70, gen)
    greedy = model.generate(ids, lengths, 9)
    # the first of the order is the most likely one
    assert torch.equal(model.generate(ids, lengths, 9, temperature=0.0), greedy) and torch.equal(model.generate(ids, lengths, 9, top_k=1), greedy)
    sampled = model.generate(ids, lengths, 9, temperature=1.3, top_p=0.9, min_p=0.01)
    assert sampled.shape == (5, 9) and (sampled >= 0).all() and (sampled < 64).all()


def test_generation_goes_on_where_a_longer_prompt_would(cuda_device):
    """Tokens one by one from the states give the logits that the whole sequence gives in one pass."""
    m = example()
    torch.manual_seed(1)
    gen = torch.Generator().manual_seed(1)
    model = m.Model(vocab=64, width=128, heads=2, kinds=("delta", "delta"), dtype=torch.float32)
    ids, lengths = m.batch(64, 3, 80, gen)
    tokens = model.generate(ids, lengths, 6)
    longer, more = torch.full((3, 86), -1, dtype=torch.int32, device="cuda"), lengths + 6
    longer[:, :80] = ids
    for b, n in enumerate(lengths.tolist()):
        longer[b, n:n + 6] = tokens[b].to(torch.int32)
    logits, _ = model.prefill(longer, more)
    for b, n in enumerate(lengths.tolist()):
        for i in range(6):
            row = logits[b, n - 1 + i]
            # the token that was taken is the best one, or one that float32's roundings in two layers (some thousand of 2^-22) do not tell from it
            assert row[tokens[b, i].long()] >= row.max() - 2.0 ** -10 * row.abs().max()


def test_training_step_captured(cuda_device):
    """A training step through the three operators, replayed, gives the gradients of an eager one."""
    B, T, heads, D = 2, 70, 2, 64
    torch.manual_seed(2)
    leaves = [torch.randn(D, device="cuda") * 0.1 + 1, *(torch.randn(D, D, device="cuda") / 8 for _ in range(3)), torch.randn(D, heads, device="cuda") / 8]
    leaves = [t.requires_grad_() for t in leaves]
    x, stream = (torch.randn(B, T, D, device="cuda") for _ in range(2))

    def step():
        w, wq, wk, wv, wb = leaves
        y, total = rms_norm(x, w, stream)
        cut = lambda t: t.unflatten(-1, (heads, -1))  # noqa: E731
        o, _ = delta_rule(cut(y @ wq), torch.nn.functional.normalize(cut(y @ wk), dim=-1), cut(y @ wv), torch.sigmoid(y @ wb), -torch.sigmoid(y @ wb))
        z = group_norm(o.flatten(2), heads)
        z, total = rms_norm(z, w, total)
        loss = (z.square().mean() + total.square().mean())
        return torch.autograd.grad(loss, leaves)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        got = step()
    x.normal_()
    g.replay()
    torch.cuda.synchronize()
    want = step()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_threads_call_at_once(cuda_device):
    import threading
    gen = torch.Generator().manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    q, k, v = (torch.nn.functional.normalize(rand(2, 90, 2, 32), dim=-1).cuda() for _ in range(3))
    beta, x, logits, u = torch.rand(2, 90, 2).cuda(), rand(100, 520).cuda(), rand(20, 3000).cuda(), torch.rand(20).cuda()
    calls = (lambda: based_delta_fwd(q, k, v, beta)[0], lambda: based_rms_fwd(x)[0], lambda: based_sample(logits, u, top_p=0.9)[0])
    want, wrong = [c() for c in calls], []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for n in range(30):
                j = (i + n) % 3
                if not torch.equal(calls[j](), want[j]):
                    wrong.append((i, n))
            torch.cuda.current_stream().synchronize()

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not wrong
