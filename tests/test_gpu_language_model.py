"""The operators together: the differentiable functions against torch's autograd in 64 bits, and the
example's language model in training and generation."""
import importlib.util
import os

import pytest
import torch

from linear_attention_gb300.autograd import embedding, gated_scan, group_norm

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("language_model", os.path.join(ROOT, "examples", "language_model.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def plain(ids, table, wg, wx, wz, state, weight, bias, lengths, groups):
    """One layer in plain torch: embedding, three projections, recurrence, gated group norm."""
    x = torch.where((ids >= 0)[..., None], table[ids.clamp(min=0)] * 3.0, 0.0)
    g, v, z = x @ wg, x @ wx, x @ wz
    a = torch.sigmoid(g)
    h, hs = state, []
    for t in range(ids.shape[1]):
        live = (t < lengths)[:, None]
        h = torch.where(live, a[:, t] * h + (1 - a[:, t]) * v[:, t], h)
        hs.append(torch.where(live, h, 0.0))
    y = torch.stack(hs, 1)
    n = y.unflatten(-1, (groups, -1))
    n = (n - n.mean(-1, keepdim=True)) / torch.sqrt(n.var(-1, unbiased=False, keepdim=True) + 1e-5)
    return (n.flatten(-2) * weight + bias) * torch.nn.functional.silu(z), h


def test_gradients_through_a_layer(cuda_device):
    gen = torch.Generator().manual_seed(1)
    B, T, D, V, groups = 3, 70, 48, 20, 3
    rand = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    ids = torch.randint(0, V, (B, T), generator=gen)
    lengths = torch.tensor([70, 33, 64])
    ids[torch.arange(T)[None] >= lengths[:, None]] = -1
    leaves = [rand(V, D), rand(D, D) / 7, rand(D, D) / 7, rand(D, D) / 7, rand(B, D), 1 + 0.1 * rand(D), 0.1 * rand(D)]
    cot, cot_state = rand(B, T, D), rand(B, D)
    ref = [t.clone().requires_grad_() for t in leaves]
    y, h = plain(ids, *ref, lengths, groups)
    ((y * cot).sum() + (h * cot_state).sum()).backward()
    mine = [t.float().cuda().requires_grad_() for t in leaves]
    table, wg, wx, wz, state, weight, bias = mine
    x = embedding(ids.cuda(), table, 3.0)
    s, final = gated_scan(x @ wg, x @ wx, state=state, lengths=lengths.to(torch.int32).cuda())
    out = group_norm(s, groups, weight, bias, x @ wz)
    ((out * cot.float().cuda()).sum() + (final * cot_state.float().cuda()).sum()).backward()
    # float32 against float64 through some 70 dependent rows and two products of 48 terms: a few
    # hundred roundings of 2^-24, relative to the largest gradient
    for name, p, q in zip("table wg wx wz state weight bias".split(), mine, ref):
        scale = q.grad.abs().max()
        assert (p.grad.cpu().double() - q.grad).abs().max() <= 2e-4 * scale, name
    assert (out.detach().cpu().double() - y.detach()).abs().max() <= 1e-4 * y.abs().max()


def test_gradients_that_are_broadcast_or_absent(cuda_device):
    g, x = (torch.randn(2, 30, 16, device="cuda", requires_grad=True) for _ in range(2))
    y, final = gated_scan(g, x)
    y.sum().backward()  # a gradient of stride 0 in every axis
    by_sum = (g.grad.clone(), x.grad.clone())
    g.grad = x.grad = None
    y, final = gated_scan(g, x)
    (y * torch.ones_like(y)).sum().backward()
    assert torch.equal(by_sum[0], g.grad) and torch.equal(by_sum[1], x.grad)
    g.grad = x.grad = None
    y, final = gated_scan(g, x)
    final.sum().backward()  # no gradient of y at all
    assert torch.isfinite(g.grad).all() and (x.grad.abs().sum() > 0)
    # a gate shared by all batch entries: autograd sums its gradient
    one = torch.randn(1, 30, 16, device="cuda", requires_grad=True)
    y, _ = gated_scan(one.expand(2, 30, 16), x.detach())
    y.sum().backward()
    assert one.grad.shape == (1, 30, 16)
    w = torch.ones(16, device="cuda", requires_grad=True)
    n = group_norm(x, 2, w, act="silu")
    n.transpose(0, 1).sum().backward()
    assert torch.isfinite(w.grad).all()
    table = torch.randn(9, 16, device="cuda", requires_grad=True)
    embedding(torch.tensor([[1, 2], [2, -1]], device="cuda"), table).sum().backward()
    assert table.grad[2].eq(2).all() and table.grad[1].eq(1).all() and table.grad[0].eq(0).all()


def test_nothing_is_kept_without_gradients(cuda_device):
    g, x = (torch.randn(1, 20, 16, device="cuda") for _ in range(2))
    y, final = gated_scan(g, x)
    assert not y.requires_grad and not final.requires_grad


def test_model_learns_and_generates(cuda_device):
    m = example()
    torch.manual_seed(0)
    gen = torch.Generator().manual_seed(0)
    model = m.Model()
    losses = m.train(model, 60, gen)
    assert losses[0] > 5.0 and sum(losses[-5:]) / 5 < 1.0, losses
    # generation step by step is the greedy continuation that whole passes give
    ids, lengths = m.batch(model.vocab, 5, 40, gen)
    got = model.generate(ids, lengths, 8)
    agree = 0
    for b in range(5):
        n = int(lengths[b])
        text = torch.cat([ids[b, :n].long(), got[b]]).to(torch.int32)[None]
        logits, _ = model.prefill(text, None)
        agree += int((logits[0, n - 1:-1].argmax(-1) == got[b]).sum())
    assert agree >= 38  # of 40: a bf16 rounding may tip a near tie


def test_based_layers_score(cuda_device):
    m = example()
    torch.manual_seed(0)
    model = m.Model(kinds=("based", "recurrence"))
    ids, lengths = m.batch(model.vocab, 3, 70, torch.Generator().manual_seed(2))
    logits, states = model.prefill(ids, lengths)
    assert logits.shape == (3, 70, 512) and torch.isfinite(logits).all() and states[0] is None
    # causal: later tokens change nothing before them
    other = ids.clone()
    other[:, 50:] = (other[:, 50:] + 1) % model.vocab
    again, _ = model.prefill(other, lengths)
    keep = int(min(50, int(lengths.min())))
    assert torch.equal(logits[:, :keep], again[:, :keep])


FIRST_CALLS = """
import torch
from linear_attention_gb300 import ops
dev = "cuda"
g, x, dy = (torch.randn(2, 200, 96, device=dev).bfloat16() for _ in range(3))
w = torch.ones(96, device=dev)
ids = torch.randint(0, 50, (3000,), device=dev, dtype=torch.int32)
table, de = torch.randn(50, 64, device=dev), torch.randn(3000, 64, device=dev)
pool = torch.randn(2, 96, device=dev)
kept = pool.clone()

def calls():
    y, final, saved = ops.based_scan_fwd(g, x, save=True)
    return (y, final, *ops.based_scan_bwd(g, x, dy, saved), ops.based_scan_step(g[:, 0], x[:, 0], pool),
            ops.based_norm_fwd(x, 2, w, w, g), *ops.based_norm_bwd(dy, x, 2, w, w, g),
            ops.based_embed_fwd(ids, table), ops.based_embed_bwd(ids, de, 50))

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    captured = calls()
graph.replay()
torch.cuda.synchronize()
captured = [t.clone() for t in captured]
pool.copy_(kept)
for a, b in zip(captured, calls()):
    assert torch.equal(a, b)
print("same")
"""


def test_first_calls_of_a_process_can_be_captured(cuda_device):
    import subprocess
    import sys
    out = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.strip() == "same", out.stderr[-2000:]


def test_two_threads_call_at_once(cuda_device):
    import threading

    from linear_attention_gb300 import ops
    inputs = [tuple(torch.randn(2, 100 + 70 * i, 64, device="cuda").bfloat16() for _ in range(2)) for i in range(4)]
    want = [ops.based_scan_fwd(g, x)[0] for g, x in inputs]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        stream = torch.cuda.Stream()
        for _ in range(50):
            y = ops.based_scan_fwd(*inputs[i], stream=stream)[0]
            stream.synchronize()
            if not torch.equal(y, want[i]):
                wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_empty_batches(cuda_device):
    from linear_attention_gb300 import ops
    z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    state = torch.randn(3, 8, device="cuda")
    side = torch.cuda.Stream()
    for stream in (None, side):
        for B, T in ((0, 5), (3, 0), (0, 0)):
            s = state[:B]
            y, final, saved = ops.based_scan_fwd(z(B, T, 8), z(B, T, 8), state=s, save=True, stream=stream)
            grads = ops.based_scan_bwd(z(B, T, 8), z(B, T, 8), z(B, T, 8), saved, dfinal=s, stream=stream)
            none = ops.based_scan_fwd(z(B, T, 8), z(B, T, 8), stream=stream)
            torch.cuda.synchronize()
            assert y.shape == grads[0].shape == grads[1].shape == (B, T, 8) and saved.shape == (B, (T + 63) // 64, 8)
            assert torch.equal(final, s) and torch.equal(grads[2], s) and final.data_ptr() != s.data_ptr() or B == 0
            assert none[1].shape == (B, 8) and (none[1] == 0).all()
        carry = state.clone()
        assert ops.based_scan_fwd(z(3, 0, 8), z(3, 0, 8), state=carry, final_state=carry, stream=stream)[1].data_ptr() == carry.data_ptr()
        torch.cuda.synchronize()
        assert torch.equal(carry, state)
        pool = state.clone()
        slots = torch.zeros(0, dtype=torch.int32, device="cuda")
        assert ops.based_scan_step(z(0, 8), z(0, 8), pool, slots=slots, stream=stream).shape == (0, 8) and torch.equal(pool, state)
        w = torch.ones(8, device="cuda")
        for shape in ((0, 8), (4, 0, 8)):
            assert ops.based_norm_fwd(z(*shape), 2, w, w, z(*shape), stream=stream).shape == shape
            dx, dgate, dw, db = ops.based_norm_bwd(z(*shape), z(*shape), 2, w, w, z(*shape), stream=stream)
            torch.cuda.synchronize()
            assert dx.shape == dgate.shape == shape and (dw == 0).all() and (db == 0).all() and dw.shape == db.shape == (8,)
        for shape in ((0,), (2, 0)):
            ids = torch.zeros(*shape, dtype=torch.int32, device="cuda")
            assert ops.based_embed_fwd(ids, state, stream=stream).shape == (*shape, 8)
            grad = ops.based_embed_bwd(ids, z(*shape, 8), 3, out=torch.ones(3, 8, device="cuda"), stream=stream)
            torch.cuda.synchronize()
            assert (grad == 0).all()
    # through autograd
    leaves = [t.requires_grad_() for t in (z(2, 0, 8), z(2, 0, 8), state[:2].clone(), w.clone(), state.clone())]
    y, final = gated_scan(leaves[0], leaves[1], state=leaves[2])
    x = embedding(torch.zeros(2, 0, dtype=torch.int64, device="cuda"), leaves[4])
    (group_norm(y + x, 2, leaves[3]).sum() + final.sum()).backward()
    assert (leaves[2].grad == 1).all() and (leaves[3].grad == 0).all() and (leaves[4].grad == 0).all()
    # a width of zero is still no width, and a table without rows no table
    from linear_attention_gb300.based import BasedError
    for call in (lambda: ops.based_scan_fwd(z(2, 3, 0), z(2, 3, 0)), lambda: ops.based_norm_fwd(z(2, 0), 1),
                 lambda: ops.based_embed_fwd(slots, z(0, 8))):
        with pytest.raises(BasedError):
            call()


def test_inputs_of_any_strides(cuda_device):
    # the same bits as from contiguous copies, forward and backward
    from linear_attention_gb300 import ops
    gen = torch.Generator().manual_seed(5)
    rand = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731

    def results(f, tensors):
        leaves = [t.detach().clone(memory_format=torch.preserve_format).requires_grad_() for t in tensors]
        outs = f(*leaves)
        outs = outs if isinstance(outs, tuple) else (outs,)
        sum((o * torch.arange(o.numel(), device="cuda").view(o.shape).cos()).sum() for o in outs).backward()
        return *outs, *(t.grad for t in leaves)

    def same(f, view, tensors):
        got = results(lambda *t: f(*map(view, t)), tensors)
        want = results(lambda *t: f(*(view(v).contiguous() for v in t)), tensors)
        assert all(torch.equal(p, q) for p, q in zip(got, want))

    for view in (lambda t: t[:, :-1], lambda t: t.transpose(0, 1), lambda t: t.transpose(1, 2), lambda t: t[..., ::2],
                 lambda t: t[:, ::3], lambda t: t[:1].expand_as(t), lambda t: t[..., :1].expand_as(t)):
        same(lambda g, x: gated_scan(g, x), view, (rand(4, 12, 16), rand(4, 12, 16)))
        same(lambda x, z: group_norm(x, 2, gate=z), view, (rand(4, 12, 16), rand(4, 12, 16)))
        same(lambda x: group_norm(x, 1, act="none"), view, (rand(4, 12, 16),))
    x, both = rand(4, 12, 16), rand(32, 2)
    same(lambda w, b: group_norm(x, 2, w[:16], b[16:]), lambda t: t[:, 0], (both, both))
    same(lambda s: gated_scan(x, x, state=s), lambda t: t.t(), (rand(16, 4),))
    lengths = torch.tensor([[3, 0], [12, 0], [7, 1], [0, 9]], device="cuda").to(torch.int32)
    assert torch.equal(gated_scan(x, x, lengths=lengths[:, 0])[0], gated_scan(x, x, lengths=lengths[:, 0].contiguous())[0])
    ids = torch.randint(-1, 9, (4, 13), generator=gen).cuda()
    for idt in (torch.int32, torch.int64):
        for part in (ids.to(idt)[:, :-1], ids.to(idt).t(), ids.to(idt)[::2, 1:]):
            same(lambda t: embedding(part, t, 2.0), lambda t: t.t(), (rand(16, 9),))
            dy = rand(*part.shape, 16)
            assert torch.equal(ops.based_embed_bwd(part, dy, 9), ops.based_embed_bwd(part.contiguous(), dy, 9))
            table = rand(9, 16)
            assert torch.equal(ops.based_embed_fwd(part, table), ops.based_embed_fwd(part.contiguous(), table))


def test_wrong_types_raise_type_error_and_wrong_shapes_value_error(cuda_device):
    from linear_attention_gb300 import ops
    x, s = torch.zeros(2, 5, 8, device="cuda"), torch.zeros(2, 8, device="cuda")
    w, ids = torch.ones(8, device="cuda"), torch.zeros(2, 5, dtype=torch.int32, device="cuda")
    n = torch.ones(2, dtype=torch.int32, device="cuda")
    saved = ops.based_scan_fwd(x, x, save=True)[2]
    calls = [  # a call of one argument, that argument right, of a wrong type, of a wrong shape
        (lambda t: ops.based_scan_fwd(x, x, state=t), s, s.half(), s[:1]),
        (lambda t: ops.based_scan_fwd(x, x, lengths=t), n, n.long(), n[:1]),
        (lambda t: ops.based_scan_fwd(x, x, out=t), x.clone(), x.half(), x[:, :4].clone()),
        (lambda t: ops.based_scan_fwd(x, x, final_state=t), s.clone(), s.double(), s.t().contiguous()),
        (lambda t: ops.based_scan_fwd(t, x), x, x.half(), x[:1]),
        (lambda t: ops.based_scan_bwd(x, x, x, t), saved, saved.half(), saved[:, :0]),
        (lambda t: ops.based_scan_bwd(x, x, x, saved, dfinal=t), s, s.half(), s[:1]),
        (lambda t: ops.based_scan_step(s, s, t), s.clone(), s.half(), s[:, :4].clone()),
        (lambda t: ops.based_scan_step(s, s, s.clone(), slots=t), n, n.long(), n[:1]),
        (lambda t: ops.based_norm_fwd(x, 2, w, t), w, w.half(), w[:4]),
        (lambda t: ops.based_norm_fwd(x, 2, out=t), x.clone(), x.half(), x[:1].clone()),
        (lambda t: ops.based_norm_bwd(t, x, 2, gate=x), x, x.half(), x[:1]),
        (lambda t: ops.based_embed_fwd(ids, s, out=t), x.clone(), x.half(), x[:1].clone()),
        (lambda t: ops.based_embed_bwd(t, x, 2), ids, ids.float(), ids[:1]),
        (lambda t: ops.based_embed_bwd(ids, x, 2, out=t), s.clone(), s.half(), s[:1].clone()),
    ]
    for call, right, type_, shape in calls:
        call(right)
        with pytest.raises(TypeError):
            call(type_)
        with pytest.raises(ValueError):
            call(shape)


CAPTURED_STEPS = """
import sys
import torch
sys.path[:0] = [".", "tests"]
from test_gpu_language_model import example

m = example()
ids, lengths = m.batch(64, 4, 40, torch.Generator().manual_seed(1))


def steps(model, count, capture):
    opt = torch.optim.SGD(model.parameters(), lr=0.05)

    def step():
        opt.zero_grad(set_to_none=True)
        loss = model.loss(ids, lengths)
        loss.backward()
        opt.step()
        return loss.detach()

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        losses = [step().clone() for _ in range(3)]  # their graphs are gone when the capture begins
    torch.cuda.current_stream().wait_stream(stream)
    if not capture:
        return losses + [step().clone() for _ in range(count)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        loss = step()
    for _ in range(count):
        graph.replay()
        losses.append(loss.clone())
    return losses


def run(capture):
    torch.manual_seed(0)
    model = m.Model(vocab=64, width=64, heads=2, dtype=torch.float32)
    losses = torch.stack(steps(model, 5, capture))
    return losses, [p.detach() for p in model.parameters()]


eager, captured = run(False), run(True)
assert torch.allclose(eager[0], captured[0], rtol=1e-4), (eager[0], captured[0])
for a, b in zip(eager[1], captured[1]):
    assert (a - b).abs().max() <= 1e-3 * a.abs().max()
assert eager[0][-1] < eager[0][0]
print("same")
"""


def test_training_steps_can_be_captured(cuda_device):
    # forward, backward and update as one graph, against the same steps without (products may choose other kernels)
    import subprocess
    import sys
    out = subprocess.run([sys.executable, "-c", CAPTURED_STEPS], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.strip() == "same", out.stderr[-2000:]
