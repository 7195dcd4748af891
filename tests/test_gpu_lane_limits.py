"""The AdamW lane's layers at inputs where a kernel can be right and slow, or
right nearly everywhere: long runs and crowded classes of tokens, rows of huge
values, targets' entries of the head's gradients, frozen parameters."""
import math

import pytest
import torch

import matrix_orthogonalizing_optimizer_step_b200 as mo
from matrix_orthogonalizing_optimizer_step_b200 import layers
from tests import _lane_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def status_ok():
    assert mo.muon_device_status(DEV) == (mo.MUON_OK, -1)


def best_us(f, repeats=5):
    """Shortest of `repeats` timings of one call, after two calls."""
    f(), f()
    best = math.inf
    for _ in range(repeats):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3)
    return best


def integer_sums(t, g, vocab):
    """The table's gradient of integers: every order of additions gives it (sums below 2^24)."""
    return torch.zeros(vocab, g.shape[1], device=DEV, dtype=torch.float64).index_add_(0, t, g.double())


# ---- embedding gradient --------------------------------------------------------------


@pytest.mark.parametrize("n", [300_000, 700_001])
def test_embedding_backward_long_runs(n):
    """Runs of several hundred thousand equal tokens: from the first position,
    to the last, between others, and two that meet inside a chunk."""
    vocab, dim = 50, 24
    g = torch.randint(-3, 4, (n, dim), generator=gen(1), device=DEV).float()
    i = torch.arange(n, device=DEV)
    for t in (torch.full((n,), 7, device=DEV), torch.where(i < 5, 3, 7), torch.where(i < 77, 49, 7),
              torch.where(i % 2 == 0, 11, 12), torch.where(i % 1000 == 0, 1 + i // 1000 % 49, 20)):
        got = mo.muon_embedding_backward(t, g, vocab)
        assert torch.equal(got.double(), integer_sums(t, g, vocab))
    status_ok()


def test_embedding_backward_time_grows_with_the_run():
    """Four times the tokens in one run take about four times as long.  (A walk
    along the run from each of its chunks takes sixteen times as many steps.)"""
    times = []
    for n in (1 << 19, 1 << 21):
        g = torch.ones(n, 8, device=DEV)
        t = torch.zeros(n, dtype=torch.int64, device=DEV)
        times.append(best_us(lambda: mo.muon_embedding_backward(t, g, 4)))
    assert times[1] < 8 * times[0], times


def test_embedding_backward_time_of_one_class():
    """Tokens that one CTA of the first launch owns take that CTA a pass over
    them, not a pass per row: a few times the time of tokens spread over all CTAs."""
    sms = torch.cuda.get_device_properties(DEV).multi_processor_count
    n, vocab = 16384, 2000 * sms
    g = torch.ones(n, 8, device=DEV)
    i = torch.arange(n, device=DEV)
    spread = best_us(lambda t=i * 17 % vocab: mo.muon_embedding_backward(t, g, vocab))
    crowded = best_us(lambda t=i % 2000 * sms: mo.muon_embedding_backward(t, g, vocab))
    assert crowded < 8 * spread, (spread, crowded)


@pytest.mark.parametrize("vocab,dim", [(128256, 2001), (128256, 1000), (50257, 768)])
def test_embedding_backward_of_few_tokens_is_a_zero_fill(vocab, dim):
    """An fp32 table and 300 tokens: writing the zeros is all there is to do, and
    that goes as fast as torch's zeros with an index_add_ (a tenth for the clock)."""
    g = torch.randn(300, dim, generator=gen(5), device=DEV)
    t = torch.randint(0, vocab, (300,), generator=gen(6), device=DEV)
    plain = best_us(lambda: [torch.zeros(vocab, dim, device=DEV).index_add_(0, t, g) for _ in range(10)])
    own = best_us(lambda: [mo.muon_embedding_backward(t, g, vocab) for _ in range(10)])
    assert own < 1.1 * plain, (own / 10, plain / 10)


@pytest.mark.parametrize("vocab,dim,offset", [(70_001, 40, 0), (70_001, 333, 1), (400_003, 9, 3)])
@pytest.mark.parametrize("n", [0, 1, 300])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_embedding_backward_zeros_of_large_tables(vocab, dim, offset, n, dtype):
    """Zeros beside the ordering: any alignment of the table, every element of it
    and none around it, with tokens in the first and last row."""
    flat = torch.full((vocab * dim + 16,), 5.0, device=DEV, dtype=dtype)
    out = flat[offset:offset + vocab * dim].view(vocab, dim)
    g = torch.randint(-3, 4, (n, dim), generator=gen(7), device=DEV).to(dtype)
    t = torch.randint(0, vocab, (n,), generator=gen(8), device=DEV)
    t[:1], t[n // 2:n // 2 + 1] = vocab - 1, 0
    mo.muon_embedding_backward(t, g, vocab, out=out)
    assert torch.equal(out.double(), integer_sums(t, g, vocab))
    assert (flat[:offset] == 5).all() and (flat[offset + vocab * dim:] == 5).all()
    status_ok()


@pytest.mark.parametrize("n", [300, 20_000])
def test_embedding_backward_of_large_tables_in_graphs_and_streams(n):
    """The three launches of a large table's gradient (by classes and by sorting),
    captured twice and replayed on two streams at once, over tables that hold
    something else before."""
    vocab, dim = 130_001, 24
    sets = []
    for seed in (9, 10):
        g = torch.randint(-3, 4, (n, dim), generator=gen(seed), device=DEV).float()
        t = torch.randint(0, vocab, (n,), generator=gen(seed + 10), device=DEV)
        out = torch.empty(vocab, dim, device=DEV)
        mo.muon_embedding_backward(t, g, vocab, out=out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            mo.muon_embedding_backward(t, g, vocab, out=out)
        sets.append((t, g, out, graph, torch.cuda.Stream()))
    for repeat in range(3):
        for t, g, out, graph, stream in sets:
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                out.fill_(7)
                graph.replay()
                t.copy_(t.roll(1))  # after the call has read them
        torch.cuda.synchronize()
        for t, g, out, _, _ in sets:
            assert torch.equal(out.double(), integer_sums(t.roll(-1), g, vocab)), repeat
    # eager calls behind one another: each starts after the one before has ended
    for t, g, out, _, _ in sets:
        got = [mo.muon_embedding_backward(q, g, vocab, out=out).clone() for q in (t, t.flip(0), t // 2)]
        for a, q in zip(got, (t, t.flip(0), t // 2)):
            assert torch.equal(a.double(), integer_sums(q, g, vocab))
    status_ok()


# ---- LayerNorm -----------------------------------------------------------------


@pytest.mark.parametrize("dtype", [F32, BF])
def test_layer_norm_backward_of_huge_rows(dtype):
    """Equal values of 2^125: the row's mean times rstd passes fp32, the
    differences to the mean are 0.  The places behind the last column, where x
    counts as nothing, must not add a product of 0 and infinity."""
    for dim in (2, 4):
        x = torch.full((3, dim), 2.0 ** 125, device=DEV, dtype=dtype)
        y, mean, rstd = mo.muon_layer_norm(x)
        assert (y == 0).all() and (mean == 2.0 ** 125).all() and torch.isinf(mean * rstd).all()
        dy = torch.randn(3, dim, generator=gen(2), device=DEV).to(dtype)
        got = mo.muon_layer_norm_backward(dy, x, mean, rstd, torch.ones(dim, device=DEV))
        want, bound = ref.norm_grad(dy, x, mean, rstd, torch.ones(dim, device=DEV))
        for a, v, e in zip(got, want, bound):
            ref.close(a, v, e + ref.half(a.dtype) * (v.abs() + e))
    status_ok()


def test_layer_norm_backward_of_frozen_parameters():
    """Without a parameter to train there is nothing to add up over the rows:
    one launch.  The gradients that are asked for are the same."""
    x = torch.randn(50, 96, generator=gen(3), device=DEV)
    g = torch.randn(50, 96, generator=gen(4), device=DEV)

    def run(*trained):
        ps = [x.clone(), torch.full((96,), 1.5, device=DEV), torch.zeros(96, device=DEV)]
        for p, on in zip(ps, trained):
            p.requires_grad_(on)
        y = layers.layer_norm(*ps)
        before = mo.muon_launch_count()
        y.backward(g)
        return [p.grad for p in ps], mo.muon_launch_count() - before

    full, launches = run(True, True, True)
    assert launches == 2
    for trained in ((True, False, False), (True, True, False), (True, False, True), (False, True, True)):
        grads, launches = run(*trained)
        assert launches == (2 if trained[1] or trained[2] else 1), trained
        for on, got, want in zip(trained, grads, full):
            assert torch.equal(got, want) if on else got is None
    status_ok()


# ---- output head ---------------------------------------------------------------


def rounded_between(got, lo, hi):
    """got (bf16) is the rounding of a number in [lo, hi] (64 bits), element by element."""
    got = got.float()
    return (got >= lo.float().to(BF).float()) & (got <= hi.float().to(BF).float())


@pytest.mark.parametrize("n,ignored", [(40, 0.0), (300, 0.3), (900, 0.05)])
def test_head_loss_targets_entry_of_dhidden(n, ignored):
    """Row k of the weight is zero but in columns of its own, so those columns
    of dhidden, in a token whose target is k, are dloss (p - 1) w_k and nothing
    else: they must be its rounding, without the rounding of P.  p lies between
    0.1 and 0.4 of a vocabulary of 600, most of it zero rows."""
    vocab, used, width = 600, 8, 8
    dim = used * width
    rows = torch.arange(used, device=DEV) * 73 + 5  # in several 128-column stretches
    w = torch.zeros(vocab, dim, device=DEV)
    for k in range(used):
        w[rows[k], k * width:(k + 1) * width] = torch.randint(8, 16, (width,), generator=gen(20 + k), device=DEV) / 8
    k = torch.arange(n, device=DEV) % used
    # the own logit is about log(vocab p / (1 - p)); the others stay near zero
    p0 = 0.1 + 0.3 * torch.rand(n, generator=gen(30), device=DEV)
    own = torch.log(600 * p0 / (1 - p0))
    h = torch.zeros(n, used, width, device=DEV)
    h[torch.arange(n, device=DEV), k] = (own / w[rows[k]].sum(1))[:, None].expand(n, width)
    h = h.view(n, dim).to(BF)
    w = w.to(BF)
    t = rows[k].clone()
    dloss = torch.rand(n, generator=gen(31), device=DEV) * 2 - 0.7
    gone = torch.rand(n, generator=gen(32), device=DEV) < ignored
    t[gone] = -100
    h[gone] = float("nan")
    _, lse = mo.muon_head_loss(h, w, t)
    dh, _ = mo.muon_head_loss_backward(h, w, t, lse, dloss)
    _, vlse, p, valid, h64, at = ref.head(h, w, t, -100)
    assert torch.equal(valid, ~gone)
    _, blse, bl = ref.head_bounds(h64, w, vlse, valid)
    i = torch.arange(n, device=DEV)[valid]
    py, dl, wy = p[i, at[i]], dloss[i].double(), w.double()[at[i]]
    assert 0.05 < py.min() and py.max() < 0.5
    # the exponential, the scaling of dloss, the products with dloss and the
    # difference; then the product with w, the sum with what P's rounding took
    # off and the scaling back
    e = dl.abs() * (py * (torch.expm1((bl + blse)[i]) + 2.0 ** -20) + 6 * ref.U)
    g = dl * (py - 1)
    want, bound = g[:, None] * wy, e[:, None] * wy.abs() + 4 * ref.U * (g[:, None] * wy).abs()
    mine = wy != 0
    inside = rounded_between(dh[i], want - bound, want + bound)
    assert inside[mine].all()
    # the check tells a P that was rounded and not mended from one that was
    # (its factor, the largest |dloss|, is left out of the rounding)
    top = dl.abs().max()
    bare = ((g / top).float().to(BF).double() * top)[:, None] * wy
    assert (~rounded_between(bare.float().to(BF), want - bound, want + bound))[mine].float().mean() > 0.1
    assert (dh[gone] == 0).all()
    status_ok()


def test_head_loss_gradients_of_confident_rows():
    """Rows whose target leads by 8 to 40.  The target's entry of P is
    dloss (exp(l - lse) - 1) with l the same number in both passes, so that l's
    own error cancels and the entry is off by half a step of lse, by the
    exponential's error next to 1 and by the sum's, however small the loss is.
    Every other entry is off relative to itself."""
    n, vocab, dim = 300, 5003, 2048
    w = (torch.randn(vocab, dim, generator=gen(97), device=DEV) * 0.02).to(BF)
    t = torch.randint(0, vocab, (n,), generator=gen(98), device=DEV)
    lead = torch.linspace(8, 40, n, device=DEV)[:, None]
    wt = w[t].float()
    h = (torch.randn(n, dim, generator=gen(99), device=DEV) * 0.1 + wt * (lead / wt.square().sum(1, keepdim=True))).to(BF)
    dloss = torch.rand(n, generator=gen(100), device=DEV) + 0.5
    _, lse = mo.muon_head_loss(h, w, t)
    dh, dw = mo.muon_head_loss_backward(h, w, t, lse, dloss)
    _, vlse, p, valid, h64, at = ref.head(h, w, t, -100)
    _, _, el = ref.head_bounds(h64, w, vlse, valid)
    i, w64, dl = torch.arange(n, device=DEV), w.double(), dloss.double()[:, None]
    g = p.clone()
    g[i, at] = 0
    rest = g.sum(1, keepdim=True)  # 1 - p of the target with all its digits
    # another entry: two logits' errors, the exponential (2^-22 and |x| steps
    # of its argument, |x| < 64), dloss
    rel = torch.expm1(2 * el)[:, None] + 2.0 ** -22 + 70 * ref.U
    e = dl * g * rel
    # the target's: the others' sum, the additions to the sum that holds its 1
    # (128 columns, the pairs of a group, 32 groups), lse's half step and log,
    # the exponential next to 1, dloss and the difference
    additions = 128 + 2 * (vocab / 4096 + 1) + 2 * 32
    e[i, at] = (dl * (rest * rel + additions * ref.U + ref.U * vlse.abs()[:, None] + 2.0 ** -22 + 4 * ref.U))[:, 0]
    g[i, at] = -rest[:, 0]
    g = g * dl
    # P as the products take it, and their sums
    e = e + ref.half(BF) * (g.abs() + e)
    dh64, dw64 = g @ w64, g.T @ h64
    edh = e @ w64.abs() + vocab * 2.0 ** -23 * (g.abs() @ w64.abs())
    edw = e.T @ h64.abs() + n * 2.0 ** -23 * (g.abs().T @ h64.abs())
    ref.close(dh, dh64, edh + ref.half(BF) * (dh64.abs() + edh))
    ref.close(dw, dw64, edw + ref.half(BF) * (dw64.abs() + edw))
    status_ok()
