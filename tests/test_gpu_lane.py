"""The AdamW lane's layers on the GPU against their 64-bit forms: token
embedding, LayerNorm, output head with its loss, and their gradients."""
import math

import pytest
import torch

import matrix_orthogonalizing_optimizer_step_b200 as mo
from tests import _lane_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
BF, F32 = torch.bfloat16, torch.float32
TYPES = [F32, BF]


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(shape, seed, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen(seed), device=DEV) * scale).to(dtype)


def ids(n, vocab, seed, dtype=torch.int64):
    return torch.randint(0, vocab, (n,), generator=gen(seed), device=DEV).to(dtype)


def status_ok():
    st, bad = mo.muon_device_status(DEV)
    assert st == mo.MUON_OK, (st, bad)


# ---- embedding -----------------------------------------------------------------


@pytest.mark.parametrize("td", TYPES)
@pytest.mark.parametrize("od", TYPES)
@pytest.mark.parametrize("n,vocab,dim", [(1, 1, 1), (1, 50, 8), (5, 7, 333), (100, 1000, 768), (33, 257, 1025),
                                         (17, 100, 4096), (3, 10, 1032)])
def test_embedding(td, od, n, vocab, dim):
    table = normal((vocab, dim), 1, td)
    for it in (torch.int32, torch.int64):
        t = ids(n, vocab, 2, it)
        for scale in (1.0, 2.5):
            got = mo.muon_embedding(t, table, scale=scale, out_dtype=od)
            assert got.dtype == od and got.shape == (n, dim)
            want = ref.embedding(t.long(), table, scale)
            ref.close(got, want, ref.embedding_bound(want, od))
    status_ok()


def test_embedding_shapes_and_offsets():
    table = normal((11 * 24 + 1,), 3, BF)[1:].view(11, 24)  # 2-byte aligned
    t = ids(12, 11, 4).view(3, 2, 2)
    got = mo.muon_embedding(t, table)
    assert torch.equal(got, table[t])
    assert mo.muon_embedding(t[:0], table).shape == (0, 2, 2, 24)
    # the first and the last row, and the same token again
    t = torch.tensor([10, 0, 10, 10], device=DEV)
    assert torch.equal(mo.muon_embedding(t, table), table[t])
    status_ok()


@pytest.mark.parametrize("gd", TYPES)
@pytest.mark.parametrize("od", TYPES)
@pytest.mark.parametrize("n,vocab,dim", [(1, 1, 1), (1, 1000, 8), (16, 3, 40), (17, 1, 333), (300, 7, 264),
                                         (1000, 5003, 333), (4096, 300, 768), (777, 70000, 24),
                                         (16384, 2000, 40), (16385, 900, 72), (20000, 5003, 33),
                                         (600, 400000, 8), (70000, 3000, 8), (33000, 400000, 8)])
def test_embedding_backward(gd, od, n, vocab, dim):
    g = normal((n, dim), 5, gd)
    for it, padding, scale in ((torch.int64, None, 1.0), (torch.int32, vocab // 2, 2.5)):
        t = ids(n, vocab, 6, it)
        got = mo.muon_embedding_backward(t, g, vocab, scale=scale, padding_idx=padding, grad_dtype=od)
        assert got.dtype == od
        want, bound = ref.embedding_grad(t, g, vocab, scale, padding)
        ref.close(got, want, bound + ref.half(od) * (want.abs() + bound))
        # the same call again gives the same bits
        assert torch.equal(got, mo.muon_embedding_backward(t, g, vocab, scale=scale, padding_idx=padding, grad_dtype=od))
    status_ok()


@pytest.mark.parametrize("n", [1, 15, 16, 17, 32, 33, 127, 128, 129, 4095, 4096, 4097, 40000])
def test_embedding_backward_runs(n):
    """Integer gradients add without rounding, so every count must come out
    exactly: one token only, two that alternate, runs that end at, before and
    behind a chunk border, and all different."""
    vocab, dim = 40001, 16
    g = torch.randint(-3, 4, (n, dim), generator=gen(7), device=DEV).float()
    i = torch.arange(n, device=DEV)
    for t in (torch.full((n,), vocab - 1, device=DEV), i % 2, i // 16, i // 17, (i + 5) // 16, i, n - 1 - i,
              torch.where(i < n // 2, 3, i)):
        got = mo.muon_embedding_backward(t, g, vocab)
        want = torch.zeros(vocab, dim, device=DEV, dtype=torch.float64).index_add_(0, t, g.double())
        assert torch.equal(got.double(), want)
    status_ok()


@pytest.mark.parametrize("n", [100, 3000, 16384])
def test_embedding_backward_one_class(n):
    """Tokens that are all equal modulo the SM count, which the first launch
    gives to one CTA: few and many rows, long and short runs."""
    sms = torch.cuda.get_device_properties(DEV).multi_processor_count
    vocab, dim = 40001, 24
    rows = (vocab - 1) // sms
    g = torch.randint(-3, 4, (n, dim), generator=gen(8), device=DEV).float()
    i = torch.arange(n, device=DEV)
    for t in (i % rows * sms, i * 7 % 5 * sms + 3, torch.where(i % 3 == 0, sms, i % rows * sms)):
        got = mo.muon_embedding_backward(t, g, vocab)
        want = torch.zeros(vocab, dim, device=DEV, dtype=torch.float64).index_add_(0, t, g.double())
        assert torch.equal(got.double(), want)
    status_ok()


def test_embedding_backward_strides_and_out():
    vocab, n = 37, 50
    wide = normal((n, 80), 8, BF)
    t = ids(n, vocab, 9)
    for cut in (wide[:, 8:48], wide[:, 3:36]):  # aligned and not
        got = mo.muon_embedding_backward(t, cut, vocab)
        want, bound = ref.embedding_grad(t, cut, vocab, 1.0, None)
        ref.close(got, want, bound + ref.half(BF) * (want.abs() + bound))
    # a destination whose neighbours must stay, 2-byte aligned
    flat = torch.full((vocab * 40 + 9,), 5.0, device=DEV, dtype=BF)
    out = flat[1:1 + vocab * 40].view(vocab, 40)
    r = mo.muon_embedding_backward(t, wide[:, 8:48].contiguous(), vocab, out=out)
    assert r.data_ptr() == out.data_ptr()
    want, bound = ref.embedding_grad(t, wide[:, 8:48], vocab, 1.0, None)
    ref.close(out, want, bound + ref.half(BF) * (want.abs() + bound))
    assert flat[0] == 5 and (flat[1 + vocab * 40:] == 5).all()
    # no tokens, no gradient; and only padding
    assert (mo.muon_embedding_backward(t[:0], wide[:0, :40], vocab) == 0).all()
    pad = torch.full((n,), 4, device=DEV)
    nan = torch.full((n, 40), float("nan"), device=DEV)
    assert (mo.muon_embedding_backward(pad, nan, vocab, padding_idx=4) == 0).all()
    status_ok()


def test_bad_tokens_are_reported():
    table = normal((10, 16), 10, F32)
    t = torch.tensor([1, 2, 10, -1, 3], device=DEV)
    got = mo.muon_embedding(t, table)
    assert torch.isnan(got[2:4]).all() and torch.equal(got[[0, 1, 4]], table[[1, 2, 3]])
    assert mo.muon_device_status(DEV) == (mo.MUON_ERR_INDEX, 2)
    assert mo.muon_device_status(DEV) == (mo.MUON_OK, -1)
    g = normal((5, 16), 11, F32)
    got = mo.muon_embedding_backward(t, g, 10)
    want = torch.zeros(10, 16, device=DEV)
    want[[1, 2, 3]] = g[[0, 1, 4]]
    assert torch.equal(got, want)
    assert mo.muon_device_status(DEV) == (mo.MUON_ERR_INDEX, 2)


# ---- LayerNorm -----------------------------------------------------------------

NORM_DIMS = [1, 2, 7, 8, 31, 100, 256, 264, 333, 512, 768, 1000, 1024, 1025, 1600, 2048, 2056, 4096, 5000, 7168, 8192,
             8200, 12345, 16384, 16385, 20000]


@pytest.mark.parametrize("dim", NORM_DIMS)
@pytest.mark.parametrize("xd", TYPES)
@pytest.mark.parametrize("pd", TYPES)
def test_layer_norm(dim, xd, pd):
    for rows in (1, 5):
        x = (normal((rows, dim), 12, F32) * 2 + 0.7).to(xd)
        w, b = (normal((dim,), 13, F32) * 0.2 + 1).to(pd), normal((dim,), 14, pd, 0.3)
        for ww, bb in ((w, b), (w, None), (None, b), (None, None)):
            y, mean, rstd = mo.muon_layer_norm(x, ww, bb, eps=1e-5)
            assert y.dtype == xd and mean.dtype == rstd.dtype == F32 and mean.shape == (rows,)
            for got, want, bound in zip((y, mean, rstd), ref.norm(x, ww, bb, 1e-5),
                                        ref.norm_bounds(x, ww, bb, 1e-5, xd)):
                ref.close(got, want, bound)
    status_ok()


@pytest.mark.parametrize("dim", NORM_DIMS)
@pytest.mark.parametrize("xd", TYPES)
@pytest.mark.parametrize("pd", TYPES)
def test_layer_norm_backward(dim, xd, pd):
    for rows in (1, 7):
        x = (normal((rows, dim), 15, F32) * 2 + 0.7).to(xd)
        dy = normal((rows, dim), 16, xd)
        w = (normal((dim,), 17, F32) * 0.2 + 1).to(pd)
        _, mean, rstd = (t.float() for t in ref.norm(x, None, None, 1e-5))
        for ww, bias in ((w, True), (w, False), (None, True), (None, False)):
            dx, dw, db = mo.muon_layer_norm_backward(dy, x, mean, rstd, ww, bias=bias)
            assert (dw is None) == (ww is None) and (db is None) == (not bias)
            want, bound = ref.norm_grad(dy, x, mean, rstd, ww)
            for got, v, e in zip((dx, dw, db), want, bound):
                if got is not None:
                    ref.close(got, v, e + ref.half(got.dtype) * (v.abs() + e))
    status_ok()


@pytest.mark.parametrize("rows,dim", [(2, 256), (1000, 256), (4099, 1025), (3001, 768), (2500, 2048), (700, 4096),
                                      (600, 333), (450, 20000)])
@pytest.mark.parametrize("xd", TYPES)
def test_layer_norm_many_rows(rows, dim, xd):
    x = (normal((rows, dim), 18, F32) * 2 + 0.7).to(xd)
    dy = normal((rows, dim), 19, xd)
    w, b = normal((dim,), 20, F32, 0.2) + 1, normal((dim,), 21, F32)
    y, mean, rstd = mo.muon_layer_norm(x, w, b)
    for got, want, bound in zip((y, mean, rstd), ref.norm(x, w, b, 1e-5), ref.norm_bounds(x, w, b, 1e-5, xd)):
        ref.close(got, want, bound)
    got = mo.muon_layer_norm_backward(dy, x, mean, rstd, w)
    want, bound = ref.norm_grad(dy, x, mean, rstd, w)
    for g, v, e in zip(got, want, bound):
        ref.close(g, v, e + ref.half(g.dtype) * (v.abs() + e))
    for a, c in zip(got, mo.muon_layer_norm_backward(dy, x, mean, rstd, w)):
        assert torch.equal(a, c)
    status_ok()


def test_layer_norm_strides_shapes_and_special_rows():
    wide = normal((2, 3, 96), 22, F32)
    x = wide[..., 8:72]  # rows of stride 96
    w = normal((64,), 23, F32)
    y, mean, rstd = mo.muon_layer_norm(x, w)
    assert y.shape == x.shape and y.is_contiguous() and mean.shape == (2, 3)
    same = mo.muon_layer_norm(x.contiguous(), w)
    for a, c in zip((y, mean, rstd), same):
        assert torch.equal(a, c)
    dy = normal((2, 3, 80), 24, F32)[..., 4:68]
    got = mo.muon_layer_norm_backward(dy, x, mean, rstd, w)
    for a, c in zip(got, mo.muon_layer_norm_backward(dy.contiguous(), x.contiguous(), mean, rstd, w)):
        assert torch.equal(a, c)
    # rows that start on 2 bytes
    for dim in (64, 333):
        flat, gflat = normal((5 * dim + 1,), 28, BF), normal((5 * dim + 1,), 29, BF)
        xb, gb = flat[1:].view(5, dim), gflat[1:].view(5, dim)
        wb = normal((dim,), 30, F32)
        one = mo.muon_layer_norm(xb, wb)
        for a, c in zip(one, mo.muon_layer_norm(xb.clone(), wb)):
            assert a.shape == c.shape
        for a, v, e in zip(one, ref.norm(xb, wb, None, 1e-5), ref.norm_bounds(xb, wb, None, 1e-5, BF)):
            ref.close(a, v, e)
        got, want = (mo.muon_layer_norm_backward(q, v, one[1], one[2], wb) for q, v in ((gb, xb), (gb.clone(), xb.clone())))
        v64, e64 = ref.norm_grad(gb, xb, one[1], one[2], wb)
        for a, c, v, e in zip(got, want, v64, e64):
            for k in (a, c):
                ref.close(k, v, e + ref.half(k.dtype) * (v.abs() + e))
    # no rows: empty outputs and zero parameter gradients
    y, mean, rstd = mo.muon_layer_norm(x[:0], w)
    assert y.shape == (0, 3, 64) and mean.shape == (0, 3)
    dx, dw, db = mo.muon_layer_norm_backward(dy[:0], x[:0], mean, rstd, w)
    assert dx.shape == (0, 3, 64) and (dw == 0).all() and (db == 0).all()
    # a constant row has no variance: y is the bias; one NaN poisons its row only
    x = normal((4, 40), 25, F32)
    x[1] = 3.0
    x[2, 5] = float("nan")
    b = normal((40,), 26, F32)
    y, mean, rstd = mo.muon_layer_norm(x, None, b)
    assert torch.equal(y[1], b) and torch.isnan(y[2]).all() and torch.isfinite(y[[0, 1, 3]]).all()
    # a large common offset: the variance is taken about the mean
    x = normal((3, 768), 27, F32) + 4096.0
    y, mean, rstd = mo.muon_layer_norm(x)
    for got, want, bound in zip((y, mean, rstd), ref.norm(x, None, None, 1e-5),
                                ref.norm_bounds(x, None, None, 1e-5, F32)):
        ref.close(got, want, bound)
    status_ok()


# ---- output head ---------------------------------------------------------------


def head_case(n, vocab, dim, seed, ignored=0.0, lean=True):
    w = normal((vocab, dim), seed, BF, 0.5 / math.sqrt(dim))
    t = ids(n, vocab, seed + 1)
    h = normal((n, dim), seed + 2, F32)
    if lean:
        h = h + w[t].float() * 12
    if ignored:
        t[torch.rand(n, generator=gen(seed + 3), device=DEV) < ignored] = -100
    return h.to(BF), w, t, torch.rand(n, generator=gen(seed + 4), device=DEV) + 0.1


def check_head(h, w, t, dloss, ignore=-100):
    loss, lse = mo.muon_head_loss(h, w, t, ignore_index=ignore)
    vloss, vlse, p, valid, h64, at = ref.head(h, w, t, ignore)
    bloss, blse, bl = ref.head_bounds(h64, w, vlse, valid)
    ref.close(loss.reshape(-1), vloss, torch.where(valid, bloss, 0.0))
    ref.close(lse.reshape(-1), vlse, torch.where(valid, blse, 0.0))
    dh, dw = mo.muon_head_loss_backward(h, w, t, lse, dloss, ignore_index=ignore)
    assert dh.shape == h.shape and dw.shape == w.shape and dh.dtype == dw.dtype == BF
    want, bound = ref.head_grad(h64, w, p, valid, at, dloss.reshape(-1), bl, blse)
    for got, v, e in zip((dh.reshape(-1, h.shape[-1]), dw), want, bound):
        ref.close(got, v, e + ref.half(BF) * (v.abs() + e))
    return loss, lse, dh, dw


@pytest.mark.parametrize("n,vocab,dim", [
    (1, 1, 8), (1, 2, 8), (3, 5, 16), (1, 1000, 64), (61, 5003, 256), (255, 255, 72), (256, 256, 64), (257, 257, 256),
    (300, 1031, 768), (512, 2048, 264), (700, 3001, 128), (130, 10007, 512), (1024, 513, 1024)])
def test_head_loss(n, vocab, dim):
    check_head(*head_case(n, vocab, dim, 30 + n))
    status_ok()


@pytest.mark.parametrize("ignored", [0.01, 0.5, 0.98, 1.0])
def test_head_loss_ignored_tokens(ignored):
    """Ignored rows hold NaN and infinity, and their dloss too: nothing of
    them reaches a result."""
    h, w, t, dloss = head_case(600, 1500, 128, 50, ignored)
    if ignored == 1.0:
        t.fill_(-100)
    gone = t == -100
    h[gone] = float("nan")
    h[gone.nonzero()[::2, 0]] = float("inf")
    dloss[gone] = float("nan")
    loss, lse, dh, dw = check_head(h, w, t, dloss)
    assert (loss[gone] == 0).all() and (lse[gone] == 0).all() and (dh[gone] == 0).all()
    if ignored == 1.0:
        assert (dw == 0).all()
    status_ok()


def test_head_loss_types_strides_and_shapes():
    h, w, t, dloss = head_case(48, 700, 64, 60)
    base = check_head(h, w, t, dloss)
    wide = torch.full((48, 160), float("nan"), device=DEV, dtype=BF)
    wide[:, 32:96] = h
    cases = [(wide[:, 32:96], t, dloss), (h, t.int(), dloss),
             (h.view(4, 12, 64), t.view(4, 12), dloss.view(4, 12))]
    for hh, tt, dd in cases:
        loss, lse = mo.muon_head_loss(hh, w, tt)
        dh, dw = mo.muon_head_loss_backward(hh, w, tt, lse, dd)
        assert loss.shape == tt.shape and dh.shape == hh.shape
        for a, c in zip((loss, lse, dh, dw), base):
            assert torch.equal(a.reshape(c.shape), c)
    # another ignore_index, one that is a token
    check_head(h, w, t, dloss, ignore=int(t[3]))
    # one gradient only
    dh, none = mo.muon_head_loss_backward(h, w, t, base[1], dloss, weight_grad=False)
    assert none is None and torch.equal(dh, base[2])
    none, dw = mo.muon_head_loss_backward(h, w, t, base[1], dloss, hidden_grad=False)
    assert none is None and torch.equal(dw, base[3])
    # no tokens
    loss, lse = mo.muon_head_loss(h[:0], w, t[:0])
    assert loss.shape == (0,)
    dh, dw = mo.muon_head_loss_backward(h[:0], w, t[:0], lse, dloss[:0])
    assert dh.shape == (0, 64) and (dw == 0).all()
    status_ok()


def test_head_loss_exact_values():
    """A zero weight makes every probability 1 / vocab.  With a power of two
    for the vocabulary and small integers for the rest no product or sum
    rounds, so both gradients must come out exactly."""
    n, vocab, dim = 200, 1024, 64
    w = torch.zeros(vocab, dim, device=DEV, dtype=BF)
    h = torch.randint(-2, 3, (n, dim), generator=gen(70), device=DEV).to(BF)
    t = ids(n, 32, 71) * 31  # few distinct targets, each several times
    dloss = torch.full((n,), 1024.0, device=DEV)
    loss, lse = mo.muon_head_loss(h, w, t)
    assert (loss - math.log(vocab)).abs().max() < 1e-5
    # exp(0 - lse) is 1 / 1024 up to 2^-20, which bf16 rounds away
    dh, dw = mo.muon_head_loss_backward(h, w, t, lse, dloss)
    assert (dh == 0).all()
    onehot = torch.zeros(n, vocab, device=DEV, dtype=torch.float64)
    onehot[torch.arange(n, device=DEV), t] = 1024.0
    # 1 - 1024 = -1023 rounds to -1024 in bf16's 8 bits
    g = torch.where(onehot > 0, -1024.0, 1.0).double()
    want = g.T @ h.double()
    ref.close(dw, want, ref.half(BF) * want.abs())
    status_ok()


def test_head_loss_extreme_logits():
    """Logits of several thousand, and one that decides alone."""
    n, vocab, dim = 5, 300, 8
    w = torch.zeros(vocab, dim, device=DEV, dtype=BF)
    w[7, 0], w[299, 1] = 64.0, -64.0
    h = torch.zeros(n, dim, device=DEV, dtype=BF)
    h[0, 0], h[1, 1], h[2, 0], h[3, 1] = 64.0, 64.0, -64.0, -64.0
    t = torch.tensor([7, 299, 7, 299, 0], device=DEV)
    loss, lse = mo.muon_head_loss(h, w, t)
    want = torch.tensor([0.0, 4096 + math.log(299), 4096 + math.log(299), 0.0, math.log(300)], device=DEV)
    assert torch.allclose(loss, want, rtol=1e-6, atol=1e-6)
    dh, dw = mo.muon_head_loss_backward(h, w, t, lse, torch.ones(n, device=DEV))
    assert torch.isfinite(dh).all() and torch.isfinite(dw).all()
    assert (dh[0] == 0).all() and (dh[3] == 0).all() and dh[2, 0] == -64.0
    # a row that holds an infinity that counts is NaN, the others are not
    h[4, 0] = float("inf")
    loss, _ = mo.muon_head_loss(h, w, t)
    assert torch.isnan(loss[4]) and torch.isfinite(loss[:4]).all()
    status_ok()


def test_head_loss_bad_targets_are_reported():
    h, w, t, dloss = head_case(40, 100, 64, 80)
    t[5], t[9] = 100, -1
    loss, lse = mo.muon_head_loss(h, w, t)
    assert torch.isnan(loss[[5, 9]]).all() and torch.isfinite(loss).sum() == 38
    assert mo.muon_device_status(DEV) == (mo.MUON_ERR_INDEX, 5)
    dh, dw = mo.muon_head_loss_backward(h, w, t, lse, dloss)
    assert mo.muon_device_status(DEV) == (mo.MUON_ERR_INDEX, 5)
    t[5], t[9] = -100, -100
    lse2 = mo.muon_head_loss(h, w, t)[1]
    for a, c in zip((dh, dw), mo.muon_head_loss_backward(h, w, t, lse2, dloss)):
        assert torch.equal(a, c)
    status_ok()


def test_head_loss_pieces():
    """A batch whose probabilities exceed the piece size: several pieces of the
    vocabulary, the last one shorter, against the 64-bit form."""
    check_head(*head_case(8200, 33000, 64, 90, ignored=0.1))
    status_ok()


@pytest.mark.parametrize("n", [8200, 33000])
def test_head_loss_many_tokens(n):
    """More tokens than one step of the launch that finds the rows, half of them ignored."""
    check_head(*head_case(n, 300, 64, 92, ignored=0.5))
    check_head(*head_case(n, 300, 64, 93))
    status_ok()


def test_head_loss_repeats():
    h, w, t, dloss = head_case(1000, 5000, 256, 95, 0.2)
    loss, lse = mo.muon_head_loss(h, w, t)
    first = (loss, lse, *mo.muon_head_loss_backward(h, w, t, lse, dloss))
    loss, lse = mo.muon_head_loss(h, w, t)
    for a, c in zip(first, (loss, lse, *mo.muon_head_loss_backward(h, w, t, lse, dloss))):
        assert torch.equal(a, c)
    status_ok()


@pytest.mark.parametrize("ignored", [0.0, 0.3])
def test_head_loss_equal_targets(ignored):
    # one token is every row's target, then a few tokens of one 128-column stretch are
    h, w, t, dloss = head_case(300, 1500, 264, 96, ignored)
    counts = t != -100
    t[counts] = 777
    check_head(h, w, t, dloss)
    t[counts] = 640 + torch.arange(int(counts.sum()), device=DEV) % 5
    check_head(h, w, t, dloss)


def test_head_loss_of_confident_rows():
    # the target's logit leads by 8 to 40: losses from 0.5 down to 1e-14
    n, vocab, dim = 300, 5003, 2048
    g = torch.Generator(device=DEV).manual_seed(97)
    w = (torch.randn(vocab, dim, generator=g, device=DEV) * 0.02).bfloat16()
    t = torch.randint(0, vocab, (n,), generator=g, device=DEV)
    lead = torch.linspace(8, 40, n, device=DEV)[:, None]
    wt = w[t].float()
    h = (torch.randn(n, dim, generator=g, device=DEV) * 0.1 + wt * (lead / wt.square().sum(1, keepdim=True))).bfloat16()
    loss, lse = mo.muon_head_loss(h, w, t)
    vloss, vlse, p, valid, h64, at = ref.head(h, w, t, -100)
    assert (h64 @ w.double().T).argmax(1).eq(t).all()
    # log s of s = 1 + x: the maximum is the target's logit itself.  x is off by
    # the logits' differences' error and the exponential's, and s by half a step
    # for each addition to a sum that holds the 1: 128 columns, the pairs of a
    # group (each scaled), 32 groups; log by 2 steps
    _, _, el = ref.head_bounds(h64, w, vlse, valid)
    x = torch.expm1(vloss)
    additions = 128 + 2 * (vocab / 4096 + 1) + 2 * 32
    ref.close(loss, vloss, x * (torch.expm1(2 * el) + 2.0 ** -19) + additions * ref.U + 4 * ref.U * vloss)
    assert (loss >= 0).all()
    assert loss[-1] < 1e-6


@pytest.mark.parametrize("n,vocab,dim", [(1, 300, 64), (61, 20000, 72), (255, 20000, 256), (256, 40000, 64), (257, 20000, 64)])
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_head_loss_one_row_block(n, vocab, dim, index):
    # batches of one block of 256 rows: more vocabulary tiles than CTA pairs, ignored rows of NaN and infinities
    h, w, t, dloss = head_case(n, vocab, dim, 98 + n, 0.4)
    off = t == -100
    h[off] = float("nan")
    h[off & (torch.arange(n, device=DEV) % 2 == 0)] = float("inf")
    t = t.to(index)
    loss, lse, dh, _ = check_head(h, w, t, dloss)
    assert (loss[off] == 0).all() and (lse[off] == 0).all() and (dh[off] == 0).all()
    t[:] = -100
    loss, lse = mo.muon_head_loss(h, w, t)
    assert (loss == 0).all() and (lse == 0).all()
    status_ok()
