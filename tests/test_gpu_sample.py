"""Sampling on the GPU against the definition in 64 bits, token by token."""
import math

import pytest
import torch

import more_ops_reference as ref
from linear_attention_gb300 import based_sample
from linear_attention_gb300.based import BasedError

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def numbers(order, prob, gen, count):
    """Random numbers in the middle of kept tokens' intervals, and the tokens: those off the borders by more than probabilities may be."""
    c = torch.cat([torch.zeros(1, dtype=torch.float64), prob.cumsum(0)])
    wide = torch.nonzero(prob > 1e-4)[:, 0]
    at = wide[torch.randint(0, wide.numel(), (count,), generator=gen)]
    at[0], at[-1] = wide[0], wide[-1]
    return ((c[at] + c[at + 1]) / 2).float(), order[at], prob[at]


def check(logits, temperature=1.0, top_k=None, top_p=None, min_p=None, seed=0, count=6):
    """One row, sampled `count` times in a batch of equal rows."""
    gen = torch.Generator().manual_seed(seed)
    order, prob = ref.sample_order(logits, temperature, top_k, top_p, min_p)
    u, want, p = numbers(order, prob, gen, count)
    rows = logits.cuda().expand(count, -1)
    got, probs = based_sample(rows, u.cuda(), temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)
    assert got.dtype == torch.int32 and got.cpu().tolist() == want.tolist()
    # a probability: the token's and the sum's weights, each to 2^-21 and arguments up to 64 rounded to 2^-24
    assert ((probs.cpu().double() - p).abs() <= p * 2.0 ** -17 + 2.0 ** -24).all()


def row(V, dtype, seed=0, spread=2.0):
    return (torch.randn(V, generator=torch.Generator().manual_seed(seed)) * spread).to(dtype)


@pytest.mark.parametrize("V", [1, 2, 7, 8, 31, 257, 1000, 1024, 4097, 20000, 50001])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_sizes(cuda_device, V, dtype):
    x = row(V, dtype, V)
    check(x)
    # a share between two of the cumulative ones
    p = torch.softmax(x.double(), 0).sort(descending=True)[0].cumsum(0)
    n = max(1, V // 3)
    share = float((p[n - 1] + (p[n] if n < V else 1.0)) / 2)
    if share < 1:
        check(x, top_p=share)
    check(x, top_k=max(1, V // 5), temperature=0.6)
    check(x, top_k=3, min_p=0.01)


@pytest.mark.parametrize("V", [130001, 300000])
def test_large_rows(cuda_device, V):
    x = row(V, F32, 1, 3.0)
    check(x, top_k=50)
    check(x, top_k=5000, temperature=0.5)  # more than are sorted
    check(x, min_p=0.2)
    check(row(V, BF16, 1, 3.0), top_k=1500)


def test_limits_of_each_row(cuda_device):
    gen = torch.Generator().manual_seed(5)
    N, V = 40, 3001
    x = torch.randn(N, V, generator=gen) * 2
    t, k = 0.3 + torch.rand(N, generator=gen), torch.randint(-1, 60, (N,), generator=gen).to(torch.int32)
    p, m = 0.3 + torch.rand(N, generator=gen), torch.rand(N, generator=gen) * 0.1 - 0.02
    u, want, prob = torch.empty(N), torch.empty(N, dtype=torch.int64), torch.empty(N, dtype=torch.float64)
    for i in range(N):
        order, q = ref.sample_order(x[i], float(t[i]), int(k[i]), float(p[i]), float(m[i]))
        a, b, c = numbers(order, q, gen, 2)
        u[i], want[i], prob[i] = a[0], b[0], c[0]
    got, probs = based_sample(x.cuda(), u.cuda(), t.cuda(), k.cuda(), p.cuda(), m.cuda())
    assert got.cpu().tolist() == want.tolist()
    assert ((probs.cpu().double() - prob).abs() <= prob * 2.0 ** -17 + 2.0 ** -24).all()


def test_ties_go_to_the_lowest_index(cuda_device):
    x = torch.zeros(5000)
    x[[7, 100, 3000]] = 4.0
    check(x, top_k=2)
    check(x, top_k=1)
    check(x, top_k=10)       # seven of the many equal ones, the first
    check(x, top_p=0.0)
    check(torch.full((9000,), -3.0).to(BF16), top_k=4000)  # more equal ones than are sorted
    check(torch.tensor([0.0, -0.0, 0.0, -0.0] * 50), top_k=5)
    got, _ = based_sample(x.cuda()[None], torch.zeros(1, device="cuda"), temperature=0.0)
    assert got.item() == 7
    # half the mass of equal tokens: the first half of them
    got, probs = based_sample(torch.zeros(1, 6000, device="cuda"), torch.full((1,), 0.9999, device="cuda"), top_p=0.50001)
    assert got.item() in (3000, 2999) and abs(probs.item() - 1 / 3001) < 1e-6


def test_masked_tokens_and_rows_without_any(cuda_device):
    x = row(4000, F32)
    x[::2] = -math.inf
    x[5] = math.nan
    check(x)
    check(x, top_k=3000)     # more than there are
    check(x, top_k=7, top_p=0.7003)
    low = torch.full((300,), torch.finfo(BF16).min).to(BF16)
    low[17] = 0.0
    check(low)
    check(torch.full((300,), torch.finfo(BF16).min).to(BF16), top_k=5)
    rows = torch.stack([torch.full((500,), -math.inf), torch.full((500,), math.nan), torch.zeros(500)])
    rows[2, 40] = rows[2, 90] = math.inf
    got, probs = based_sample(rows.cuda(), torch.full((3,), 0.5, device="cuda"), top_k=3, top_p=0.5)
    assert got.cpu().tolist() == [-1, -1, 40] and probs.cpu().tolist() == [0, 0, 1]


def test_numbers_at_the_ends(cuda_device):
    x = row(3000, F32).cuda().expand(5, -1)
    u = torch.tensor([0.0, 1.0 - 2.0 ** -24, 1.0, -1.0, math.nan], device="cuda")
    got, probs = based_sample(x, u)
    assert got[0] == 0 and got[3] == 0 and got[4] == 0 and got[1] == 2999 and got[2] == 2999 and (probs > 0).all()
    for t in (-1.0, 0.0, math.nan, 1e-30, 1e-42):
        assert (based_sample(x, torch.full((5,), 0.7, device="cuda"), temperature=t)[0] == x[0].argmax()).all()
    flat, _ = based_sample(x, torch.full((5,), 0.50001, device="cuda"), temperature=1e30)
    assert (flat == 1500).all()


def test_distribution(cuda_device):
    """Numbers on a grid hit each token as often as its probability says, to two of the grid's steps."""
    x, n = row(50, F32), 20000
    u = (torch.arange(n, device="cuda") + 0.5) / n
    got, _ = based_sample(x.cuda().expand(n, -1), u, temperature=0.8)
    share = torch.bincount(got.long().cpu(), minlength=50).double() / n
    assert ((share - torch.softmax(x.double() / 0.8, 0)).abs() <= 2.0 / n).all()


def test_strides_streams_and_outputs(cuda_device):
    wide = torch.randn(8, 2000, device="cuda")
    u = torch.rand(8, device="cuda")
    for view in (wide[:, :1000], wide[:, 3:1001], wide[::2], wide[:1].expand(8, 2000)):
        want = based_sample(view.contiguous(), u[:view.shape[0]], top_k=50, top_p=0.9)
        got = based_sample(view, u[:view.shape[0]], top_k=50, top_p=0.9)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    side, out = torch.cuda.Stream(), torch.empty(8, dtype=torch.int32, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    t, p = based_sample(wide, u, top_k=50, out=out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert t.data_ptr() == out.data_ptr() and torch.equal(out, based_sample(wide, u, top_k=50)[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        t, p = based_sample(wide, u, top_k=50, top_p=0.8, temperature=0.7)
    u.copy_(torch.rand(8, device="cuda"))
    g.replay()
    torch.cuda.synchronize()
    want = based_sample(wide, u, top_k=50, top_p=0.8, temperature=0.7)
    assert torch.equal(t, want[0]) and torch.equal(p, want[1])
    with pytest.raises(BasedError):
        based_sample(wide, u, out=u.view(torch.int32))
    assert based_sample(wide[:0], u[:0])[0].shape == (0,)


def test_batches_give_what_rows_alone_give(cuda_device):
    """Another number of rows is another number of CTAs to a row."""
    x, u = torch.randn(200, 30000, device="cuda"), torch.rand(200, device="cuda")
    for limits in (dict(top_k=40, top_p=0.9), dict(top_p=0.8), {}):
        got, probs = based_sample(x, u, **limits)
        for i in range(0, 200, 23):
            t, p = based_sample(x[i:i + 1], u[i:i + 1], **limits)
            # (without a cut the sums of eight tokens' masses may fall on other eights: the border moves by 2^-22)
            assert t.item() == got[i].item() and abs(p.item() - probs[i].item()) <= 2.0 ** -22 * p.item()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_few_kept_tokens_in_rows_of_any_order(cuda_device, dtype):
    """A small top_k is cut by the threads' largest tokens where those bound it well: rows that are in order, rows whose largest
    tokens lie side by side or in one thread's reach, and rows with fewer tokens than it are cut by all of them."""
    x = row(20000, F32, 3).sort()[0].to(dtype)
    for y in (x, x.flip(0), torch.roll(x, 777)):
        for k in (1, 2, 40, 255, 256, 257, 300, 511, 512, 513, 2047, 2049):
            check(y, top_k=k)
        check(y, top_k=64, top_p=0.9, min_p=0.02, temperature=0.7)
    y = torch.full((20000,), -math.inf).to(dtype)
    y[4096:4136] = row(40, dtype, 4)
    y[9] = math.nan
    for k in (1, 7, 39, 40, 41, 200):
        check(y, top_k=k)
        check(y, top_k=k, top_p=0.8)
    z = row(20000, dtype, 5)
    z[8000:8512] = z.max() + 1  # more equal ones than top_k
    check(z, top_k=100)
    check(z, top_k=100, top_p=0.5, min_p=0.5)
    z[8000:8512] -= torch.arange(512).to(dtype) * 2.0 ** -6
    check(z, top_k=100, top_p=0.9)
    check(z, top_k=100, temperature=1e-3)
    check(z, top_k=100, temperature=50.0)


def test_an_infinite_temperature_weighs_all_alike(cuda_device):
    x = row(3000, F32)
    x[:1000] = -math.inf
    for limits in ({}, dict(top_k=9), dict(top_k=2500), dict(top_p=0.5001), dict(top_k=600, top_p=0.3003)):
        check(x, temperature=math.inf, **limits)


@pytest.mark.parametrize("dtype", [F32, F16])
def test_rows_that_no_cluster_holds(cuda_device, dtype):
    x = row(4000003, dtype, 6, 3.0)
    for limits in (dict(top_k=60), dict(top_k=60, top_p=0.9, min_p=0.01), dict(top_k=300), dict(min_p=0.3), dict(temperature=0.0)):
        if limits.get("temperature") == 0.0:
            got, p = based_sample(x.cuda()[None], torch.full((1,), 0.3, device="cuda"), **limits)
            assert got.item() == int(x.float().argmax()) and p.item() == 1
        else:
            check(x, **limits)
