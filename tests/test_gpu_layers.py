"""The AdamW lane's layers as torch modules: gradients through autograd, a
training step through all of them and the hybrid optimizer, row-sparse
gradients, CUDA graphs, streams, and sizes past 2^31 elements."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import matrix_orthogonalizing_optimizer_step_b200 as mo
from matrix_orthogonalizing_optimizer_step_b200 import layers
from matrix_orthogonalizing_optimizer_step_b200.optim import MuonHybrid, split_params
from oracle import muon_oracle as orc
from tests import _lane_ref as ref
from tests._util import to64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(shape, seed, dtype=F32, scale=1.0):
    return (torch.randn(shape, generator=gen(seed), device=DEV) * scale).to(dtype)


def ids(shape, vocab, seed):
    return torch.randint(0, vocab, shape, generator=gen(seed), device=DEV)


def status_ok():
    st, bad = mo.muon_device_status(DEV)
    assert st == mo.MUON_OK, (st, bad)


# ---- single layers ---------------------------------------------------------------


def test_embedding_gradient():
    w = normal((50, 24), 1).requires_grad_()
    t = ids((3, 7), 50, 2)
    g = normal((3, 7, 24), 3)
    layers.embedding(t, w, scale=1.5, padding_idx=int(t[0, 0])).backward(g)
    want, bound = ref.embedding_grad(t, g, 50, 1.5, int(t[0, 0]))
    ref.close(w.grad, want, bound + ref.half(F32) * (want.abs() + bound))
    # a gradient that autograd expands, and transposed tokens
    w.grad = None
    layers.embedding(t.t(), w).sum().backward()
    assert torch.equal(w.grad.double(), torch.bincount(t.flatten(), minlength=50).double()[:, None].expand(50, 24))
    # bf16 weight, fp32 activations
    wb = normal((50, 24), 4, BF).requires_grad_()
    y = layers.embedding(t, wb, out_dtype=F32)
    assert y.dtype == F32
    y.backward(g)
    want, bound = ref.embedding_grad(t, g, 50, 1.0, None)
    assert wb.grad.dtype == BF
    ref.close(wb.grad, want, bound + ref.half(BF) * (want.abs() + bound))
    status_ok()


@pytest.mark.parametrize("affine", ["both", "weight", "bias", "none"])
def test_layer_norm_gradient(affine):
    x = normal((4, 9, 40), 5).requires_grad_()
    w = (normal((40,), 6) * 0.2 + 1).requires_grad_() if affine in ("both", "weight") else None
    b = normal((40,), 7).requires_grad_() if affine in ("both", "bias") else None
    g = normal((4, 9, 40), 8)
    layers.layer_norm(x, w, b).backward(g)
    _, mean, rstd = mo.muon_layer_norm(x.detach(), w, b)
    want, bound = ref.norm_grad(g, x.detach(), mean, rstd, w)
    for p, v, e in zip((x, w, b), want, bound):
        if p is not None:
            ref.close(p.grad, v, e + ref.half(F32) * (v.abs() + e))
    # columns of a wider tensor and an expanded gradient
    x2 = normal((40, 36), 9).requires_grad_()
    layers.layer_norm(x2.t()).sum().backward()
    assert x2.grad.shape == (40, 36) and x2.grad.abs().max() < 1e-5
    status_ok()


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
def test_head_loss_gradient(reduction):
    h = normal((2, 30, 64), 10).requires_grad_()
    w = normal((300, 64), 11, scale=0.1).requires_grad_()
    t = ids((2, 30), 300, 12)
    t[0, ::3] = -100
    loss = layers.head_loss(h, w, t, reduction=reduction)
    hb, wb = h.detach().to(BF), w.detach().to(BF)
    vloss, vlse, p, valid, h64, at = ref.head(hb, wb, t, -100)
    bloss, blse, bl = ref.head_bounds(h64, wb, vlse, valid)
    count = valid.sum()
    if reduction == "none":
        ref.close(loss.detach().reshape(-1), vloss, torch.where(valid, bloss, 0.0))
        dl = normal((2, 30), 13)
        loss.backward(dl)
    else:
        f = 1.0 if reduction == "sum" else 1.0 / count
        n = valid.numel()
        ref.close(loss.detach(), vloss.sum() * f, (bloss.sum() + n * ref.U * vloss.abs().sum()) * f)
        loss.backward()
        dl = torch.full((2, 30), 1.0 if reduction == "sum" else float(1.0 / count.float()), device=DEV)
    want, bound = ref.head_grad(h64, wb, p, valid, at, dl.reshape(-1), bl, blse)
    for got, v, e in zip((h.grad.reshape(-1, 64), w.grad), want, bound):
        assert got.dtype == F32
        ref.close(got, v, e + ref.half(BF) * (v.abs() + e))
    status_ok()


def test_head_loss_of_nothing_and_frozen_parts():
    h = normal((5, 16), 14, BF).requires_grad_()
    w = normal((9, 16), 15, BF).requires_grad_()
    t = torch.full((5,), -100, device=DEV)
    loss = layers.head_loss(h, w, t)
    loss.backward()
    assert loss == 0 and (h.grad == 0).all() and (w.grad == 0).all()
    t = ids((5,), 9, 16)
    layers.head_loss(h, w, t).backward()
    dh, dw = h.grad.clone(), w.grad.clone()
    h.grad = w.grad = None
    layers.head_loss(h.detach(), w, t).backward()
    assert torch.equal(w.grad, dw)
    w.grad = None
    layers.head_loss(h, w.detach(), t).backward()
    assert torch.equal(h.grad, dh) and w.grad is None
    # rows that do not start on 16 bytes are copied first
    flat = torch.zeros(5 * 16 + 1, device=DEV, dtype=BF)
    flat[1:] = h.detach().reshape(-1)
    assert torch.equal(layers.head_loss(flat[1:].view(5, 16), w.detach(), t), layers.head_loss(h.detach(), w.detach(), t))


# ---- differences -------------------------------------------------------------------


def test_layer_norm_gradient_against_differences():
    """<dx, v> against (f(x + h v) - f(x - h v)) / 2h for f = sum(c y) with the
    kernel's own y.  y varies with x / sd on a scale of one: the third
    derivative along a unit-variance v is below 64 per element's share, the
    rounding of y's sum is 2 U |c y| per element."""
    x, v, c = normal((3, 200), 20), normal((3, 200), 21), normal((3, 200), 22)
    w, b = normal((200,), 23), normal((200,), 24)
    v = v / v.norm()

    def f(x):
        y = mo.muon_layer_norm(x, w, b)[0].double()
        return (c.double() * y).sum(), (c.double() * y).abs().sum()

    x64 = x.double().requires_grad_()
    y64 = ref.norm(x64, w, b, 1e-5)[0]
    (c.double() * y64).sum().backward()
    h = 2.0 ** -6
    up, size = f((x + h * v))
    dn, _ = f((x - h * v))
    _, mean, rstd = mo.muon_layer_norm(x, w, b)
    dx, _, _ = mo.muon_layer_norm_backward(c, x, mean, rstd, w)
    slope = (dx.double() * v.double()).sum()
    # the truncation is that of the 64-bit function itself
    e64 = (ref.norm(x.double() + h * v.double(), w, b, 1e-5)[0] - ref.norm(x.double() - h * v.double(), w, b, 1e-5)[0])
    trunc = ((c.double() * e64).sum() / (2 * h) - (x64.grad * v.double()).sum()).abs()
    bound = norm_sum_bound(x, w, b, c, h, v)
    assert (slope - (up - dn) / (2 * h)).abs() <= trunc + bound / h


def norm_sum_bound(x, w, b, c, h, v):
    """Rounding of one evaluation of sum(c y) at x +- h v, the inputs' own included."""
    y, _, _ = ref.norm_bounds(x, w, b, 1e-5, F32)
    r = ref.norm(x, w, b, 1e-5)[2][..., None]
    moved = ref.U * (x.double().abs() + h * v.double().abs()) * r * w.double().abs() * 4
    return (c.double().abs() * (1.1 * y + moved)).sum()


def test_head_loss_gradient_against_differences():
    """Along directions of -1, 0, 1 on a grid of 1/8 with a step of 1/32 every
    perturbed value is exact in bf16.  The truncation of a central difference
    is h^2 / 6 of the third derivative, at most the cube of the range of the
    logits' slopes; the loss is off by its bound, dh by its own."""
    n, vocab, dim = 20, 200, 32
    h = torch.randint(-8, 9, (n, dim), generator=gen(30), device=DEV) / 8
    w = torch.randint(-8, 9, (vocab, dim), generator=gen(31), device=DEV) / 32
    t = ids((n,), vocab, 32)
    v = torch.randint(-1, 2, (n, dim), generator=gen(33), device=DEV).float() * (torch.arange(dim, device=DEV) < 4)
    step = 1 / 32
    hb, wb = h.to(BF), w.to(BF)
    up = mo.muon_head_loss((h + step * v).to(BF), wb, t)[0].double()
    dn = mo.muon_head_loss((h - step * v).to(BF), wb, t)[0].double()
    loss, lse = mo.muon_head_loss(hb, wb, t)
    dh, _ = mo.muon_head_loss_backward(hb, wb, t, lse, torch.ones(n, device=DEV))
    _, vlse, p, valid, h64, at = ref.head(hb, wb, t, -100)
    bloss, blse, bl = ref.head_bounds(h64, wb, vlse, valid)
    (want, _), (edh, _) = ref.head_grad(h64, wb, p, valid, at, torch.ones(n, device=DEV), bl, blse)
    edh = edh + ref.half(BF) * (want.abs() + edh)
    slopes = v.double() @ w.double().T
    third = (slopes.max(1).values - slopes.min(1).values) ** 3
    tol = (edh * v.double().abs()).sum(1) + step ** 2 / 6 * third + 1.1 * bloss / step
    assert ((dh.double() * v.double()).sum(1) - (up - dn) / (2 * step)).abs().sub(tol).max() <= 0


def test_embedding_gradient_against_differences():
    """The lookup is linear: with small integers the difference is the slope exactly."""
    w = torch.randint(-4, 5, (30, 8), generator=gen(34), device=DEV).float()
    d = torch.randint(-4, 5, (30, 8), generator=gen(35), device=DEV).float()
    g = torch.randint(-4, 5, (100, 8), generator=gen(36), device=DEV).float()
    t = ids((100,), 30, 37)
    dw = mo.muon_embedding_backward(t, g, 30, scale=2.0)
    diff = ((mo.muon_embedding(t, w + d, scale=2.0) - mo.muon_embedding(t, w - d, scale=2.0)) * g).sum() / 2
    assert (dw * d).sum() == diff


# ---- a training step -----------------------------------------------------------------


class TinyLM(torch.nn.Module):
    """Token and position embedding, one LayerNorm'd matrix block, final
    LayerNorm, output head: every kind of parameter that split_params knows."""

    def __init__(self, vocab=997, dim=64, length=40):
        super().__init__()
        self.wte = layers.Embedding(vocab, dim, scale=math.sqrt(dim))
        self.wpe = layers.Embedding(length, dim)
        self.ln_1 = layers.LayerNorm(dim)
        self.fc = torch.nn.Linear(dim, 4 * dim, bias=False)
        self.proj = torch.nn.Linear(4 * dim, dim, bias=False)
        self.ln_f = layers.LayerNorm(dim)
        self.lm_head = layers.HeadLoss(dim, vocab)

    def forward(self, tokens, targets):
        x = self.wte(tokens) + self.wpe(torch.arange(tokens.shape[1], device=tokens.device).expand_as(tokens))
        x = x + self.proj(torch.nn.functional.gelu(self.fc(self.ln_1(x))))
        return self.lm_head(self.ln_f(x), targets)


def test_training_step_through_all_layers():
    """Each layer's gradients, inside one model's backward pass, against the
    64-bit forms at the layer's own inputs, then the hybrid step on them."""
    mo.muon_reset_config()
    torch.manual_seed(0)
    model = TinyLM().to(DEV)
    tokens, targets = ids((6, 40), 997, 40), ids((6, 40), 997, 41)
    targets[:, :5] = -100
    seen = {}

    def watch(name):
        def hook(module, args, out):
            if torch.is_tensor(args[0]) and args[0].requires_grad:
                args[0].retain_grad()
            out.retain_grad()
            seen[name] = (args, out)
        return hook

    for name in ("wte", "wpe", "ln_1", "ln_f", "lm_head"):
        getattr(model, name).register_forward_hook(watch(name))
    loss = model(tokens, targets)
    loss.backward()
    muon_p, adamw_p = split_params(model.named_parameters())
    assert [n for n, _ in muon_p] == ["fc.weight", "proj.weight"] and len(adamw_p) == 7
    for name, scale, vocab in (("wte", 8.0, 997), ("wpe", 1.0, 40)):
        (t,), out = seen[name]
        want, bound = ref.embedding_grad(t, out.grad, vocab, scale, None)
        ref.close(getattr(model, name).weight.grad, want, bound + ref.half(F32) * (want.abs() + bound))
    for name in ("ln_1", "ln_f"):
        (x,), out = seen[name]
        m = getattr(model, name)
        _, mean, rstd = mo.muon_layer_norm(x.detach(), m.weight, m.bias)
        want, bound = ref.norm_grad(out.grad, x.detach(), mean, rstd, m.weight.detach())
        for got, v, e in zip((m.weight.grad, m.bias.grad), want[1:], bound[1:]):
            ref.close(got, v, e + ref.half(F32) * (v.abs() + e))
    (h, _), out = seen["lm_head"]
    hb, wb = h.detach().to(BF), model.lm_head.weight.detach().to(BF)
    _, vlse, p, valid, h64, at = ref.head(hb, wb, targets, -100)
    _, blse, bl = ref.head_bounds(h64, wb, vlse, valid)
    dl = torch.full((240,), float(1.0 / valid.sum().float()), device=DEV)
    want, bound = ref.head_grad(h64, wb, p, valid, at, dl, bl, blse)
    for got, v, e in zip((h.grad.reshape(-1, 64), model.lm_head.weight.grad), want, bound):
        ref.close(got, v, e + ref.half(BF) * (v.abs() + e))

    before = {n: to64(p) for n, p in model.named_parameters()}
    opt = MuonHybrid(muon_p, adamw_p, lr=0.02, adamw_lr=1e-3)
    opt.step()
    for name, p in adamw_p:
        p1, _, _ = orc.adamw_step(before[name].ravel(), to64(p.grad).ravel(), np.zeros(p.numel()), np.zeros(p.numel()),
                                  1, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
        assert np.max(np.abs(to64(p).ravel() - p1)) <= 1e-6 * 1e-3 + 2e-7 * np.max(np.abs(p1)), name
    for name, p in muon_p:
        assert torch.isfinite(p).all() and not np.array_equal(to64(p), before[name])
    # further steps run on the gradients of new batches
    for i in range(3):
        opt.zero_grad()
        model(ids((6, 40), 997, 50 + i), targets).backward()
        opt.step()
    assert all(torch.isfinite(p).all() for p in model.parameters())
    status_ok()


def test_tied_head_adds_both_gradients():
    torch.manual_seed(1)
    wte = layers.Embedding(50, 16, device=DEV)
    head = layers.HeadLoss(16, 50, weight=wte.weight)
    t, y = ids((30,), 50, 60), ids((30,), 50, 61)
    x = wte(t)
    x.retain_grad()
    head(x, y).backward()
    both = wte.weight.grad.clone()
    one = mo.muon_embedding_backward(t, x.grad, 50)
    wte.weight.grad = None
    head(x.detach(), y).backward()
    ref.close(both, one.double() + wte.weight.grad.double(), ref.U * (one.double() + wte.weight.grad.double()).abs())
    with pytest.raises(ValueError):
        layers.HeadLoss(16, 51, weight=wte.weight)


# ---- row-sparse gradients --------------------------------------------------------------


@pytest.mark.parametrize("dtype", [F32, BF])
def test_hybrid_step_takes_row_sparse_gradients(dtype):
    """torch.nn.Embedding(sparse=True) and its dense form give the same step.
    The gradient rows are small integers, so both sums are exact."""
    mo.muon_reset_config()
    t = ids((300,), 100, 70)
    g = torch.randint(-3, 4, (300, 24), generator=gen(71), device=DEV).to(dtype)
    start = normal((100, 24), 72, dtype)
    got = []
    for sparse in (True, False):
        emb = torch.nn.Embedding(100, 24, sparse=sparse, device=DEV, dtype=dtype)
        mat = torch.nn.Parameter(normal((64, 64), 73, dtype))
        with torch.no_grad():
            emb.weight.copy_(start)
        opt = MuonHybrid([mat], [emb.weight], lr=0.01, adamw_lr=1e-2)
        for step in range(3):
            opt.zero_grad()
            emb(t[:100 * (step + 1)]).backward(g[:100 * (step + 1)])
            mat.grad = normal((64, 64), 74 + step, dtype)
            assert emb.weight.grad.is_sparse == sparse
            opt.step()
        got.append((emb.weight.detach().clone(), mat.detach().clone()))
        assert set(opt.state_dict()["state"][1]) == {"exp_avg", "exp_avg_sq", "step"}
    for a, b in zip(*got):
        assert torch.equal(a, b)
    mo.muon_reset_config()
    status_ok()


def test_hybrid_step_refuses_other_sparse_gradients():
    mat = torch.nn.Parameter(normal((8, 8), 75))
    mat.grad = torch.eye(8, device=DEV).to_sparse()
    with pytest.raises(TypeError):
        MuonHybrid([mat], []).step()
    with pytest.raises(TypeError):
        MuonHybrid([], [mat]).step()


# ---- graphs and streams ----------------------------------------------------------------


def lane_calls(seed, n):
    """A closure that runs every call of the lane on one set of inputs and
    returns all outputs."""
    t = ids((n,), 700, seed)
    table, g = normal((700, 64), seed + 1), normal((n, 64), seed + 2, BF)
    w, b = normal((64,), seed + 3), normal((64,), seed + 4)
    hw = normal((700, 64), seed + 5, BF, 0.2)
    y = t.flip(0).clone()
    y[::7] = -100
    dl = torch.rand(n, generator=gen(seed + 6), device=DEV)

    def run():
        x = mo.muon_embedding(t, table, scale=2.0, out_dtype=BF)
        h, mean, rstd = mo.muon_layer_norm(x, w, b)
        loss, lse = mo.muon_head_loss(h, hw, y)
        dh, dw = mo.muon_head_loss_backward(h, hw, y, lse, dl)
        dx, dnw, dnb = mo.muon_layer_norm_backward(dh, x, mean, rstd, w)
        dt = mo.muon_embedding_backward(t, dx, 700, scale=2.0, grad_dtype=F32)
        dt2 = mo.muon_embedding_backward(t, g, 700)
        return x, h, mean, rstd, loss, lse, dh, dw, dx, dnw, dnb, dt, dt2

    return run, (t, table, g, y, dl)


@pytest.mark.parametrize("n", [50, 1000, 20000])
def test_captured_calls_replay_as_eager(n):
    run, (t, table, g, y, dl) = lane_calls(100, n)
    want = [o.clone() for o in run()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(2):
        for o in got:
            o.fill_(7)
        graph.replay()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    # new inputs in the same places
    t.copy_(t.roll(3))
    table.mul_(1.5)
    y.copy_(torch.where(y == -100, 5, -100))
    want = [o.clone() for o in run()]
    graph.replay()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    status_ok()


def test_first_call_under_capture_is_refused():
    """The first call of a process allocates the status word, which no capture
    allows: it is refused, and the same call works afterwards."""
    code = """
import torch, matrix_orthogonalizing_optimizer_step_b200 as mo
table, t = torch.ones(4, 8, device="cuda"), torch.zeros(3, dtype=torch.long, device="cuda")
torch.cuda.synchronize()
try:
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        mo.muon_embedding(t, table)
except mo.MuonError as e:
    assert e.code == mo.MUON_ERR_UNSUPPORTED, e
else:
    raise SystemExit("not refused")
assert torch.equal(mo.muon_embedding(t, table), table[t])
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = mo.muon_embedding(t, table)
g.replay()
assert torch.equal(out, table[t])
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0, r.stderr[-2000:]


def test_two_graphs_replay_at_once():
    """Two captured calls have workspaces of their own: replayed on two streams
    without any order between them, each gives its own results."""
    sets = [lane_calls(200, 3000), lane_calls(300, 3000)]
    want, graphs, outs = [], [], []
    for run, _ in sets:
        want.append([o.clone() for o in run()])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(run())
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for got, w in zip(outs, want):
        for a, b in zip(got, w):
            assert torch.equal(a, b)
    status_ok()


def test_eager_calls_on_two_streams():
    sets = [lane_calls(400, 3000), lane_calls(500, 3000)]
    want = [[o.clone() for o in run()] for run, _ in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for i, (run, _) in enumerate(sets):
            with torch.cuda.stream(streams[i]):
                got[i] = run()
    torch.cuda.synchronize()
    for a, w in zip(got, want):
        for x, y in zip(a, w):
            assert torch.equal(x, y)
    # and next to a Muon step of the library's own workspace
    mo.muon_reset_config()
    P, G, M = ([normal((128, 256), 600 + i, d)] for i, d in ((0, F32), (1, BF), (2, BF)))
    with torch.cuda.stream(streams[0]):
        mo.muon_step(P, G, M)
        a = sets[0][0]()
    with torch.cuda.stream(streams[1]):
        b = sets[1][0]()
    torch.cuda.synchronize()
    for x, y in zip((*a, *b), (*want[0], *want[1])):
        assert torch.equal(x, y)
    status_ok()


def test_backward_capture_of_a_model():
    """Forward, backward and the gradients in one capture."""
    torch.manual_seed(2)
    model = TinyLM().to(DEV)
    tokens, targets = ids((4, 40), 997, 80), ids((4, 40), 997, 81)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):  # warm up on the side stream, as torch asks
        for _ in range(2):
            model.zero_grad(set_to_none=True)
            model(tokens, targets).backward()
    torch.cuda.synchronize()
    want = [p.grad.clone() for p in model.parameters()]
    model.zero_grad(set_to_none=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        model(tokens, targets).backward()
    graph.replay()
    torch.cuda.synchronize()
    for p, w in zip(model.parameters(), want):
        ref.close(p.grad, w.double(), 1e-5 * w.double().abs().max())
    status_ok()


# ---- sizes past 2^31 elements --------------------------------------------------------------


def test_tables_past_2_31_elements():
    vocab, dim = 540_000, 4096  # 2.2e9 elements
    table = torch.zeros(vocab, dim, device=DEV, dtype=BF)
    last = normal((dim,), 90, BF)
    table[-1] = last
    t = torch.tensor([vocab - 1, 0, vocab - 1, vocab - 2], device=DEV)
    got = mo.muon_embedding(t, table)
    assert torch.equal(got[0], last) and torch.equal(got[2], last) and (got[[1, 3]] == 0).all()
    g = torch.randint(-3, 4, (4, dim), generator=gen(91), device=DEV).to(BF)
    d = mo.muon_embedding_backward(t, g, vocab)
    assert torch.equal(d[-1], g[0] + g[2]) and torch.equal(d[0], g[1]) and torch.equal(d[-2], g[3])
    assert (d[1:-2] == 0).all()
    del d, got
    # the head: a large logit in the last row decides alone
    table[-1] = 1.0
    h = torch.ones(3, dim, device=DEV, dtype=BF)
    y = torch.tensor([vocab - 1, 0, vocab - 2], device=DEV)
    loss, lse = mo.muon_head_loss(h, table, y)
    assert loss[0] == 0 and (loss[1:] == dim).all()
    dh, dw = mo.muon_head_loss_backward(h, table, y, lse, torch.ones(3, device=DEV))
    assert (dh[0] == 0).all() and (dh[1:] == 1).all()
    assert (dw[-1] == 2).all() and (dw[0] == -1).all() and (dw[-2] == -1).all() and (dw[1:-2] == 0).all()
    status_ok()


def test_rows_past_2_31_elements():
    rows, dim = 530_000, 4096
    x = torch.zeros(rows, dim, device=DEV, dtype=BF)
    last = normal((dim,), 92, BF)
    x[-1] = last
    w, b = normal((dim,), 93), normal((dim,), 94)
    y, mean, rstd = mo.muon_layer_norm(x, w, b)
    one = mo.muon_layer_norm(last[None], w, b)
    assert torch.equal(y[-1], one[0][0]) and mean[-1] == one[1][0] and rstd[-1] == one[2][0]
    assert torch.equal(y[0], b.to(BF)) and torch.equal(y[-2], y[0])
    dy = torch.zeros_like(x)
    dy[-1] = 1
    dx, dw, db = mo.muon_layer_norm_backward(dy, x, mean, rstd, w)
    for a, c in zip((dx[-1:], dw, db), mo.muon_layer_norm_backward(dy[-1:], last[None], *one[1:], w)):
        assert torch.equal(a, c)
    assert (dx[:-1] == 0).all()
    # rows of an embedding past 2^31 in the activations
    table = normal((5, dim), 95, BF)
    t = torch.zeros(rows, device=DEV, dtype=torch.int32)
    t[-1] = 4
    del x, y, dy, dx
    out = mo.muon_embedding(t, table)
    assert torch.equal(out[-1], table[4]) and torch.equal(out[-2], table[0])
    d = mo.muon_embedding_backward(t[-20000:], out[-20000:], 5, grad_dtype=F32)
    assert torch.equal(d[4], table[4].float()) and (d[1:4] == 0).all()
    status_ok()
