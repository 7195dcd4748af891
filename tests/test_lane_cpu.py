"""Host-side tests of the AdamW lane's layers (no GPU): refusals of the C
entry points and of the Python binding, and the reference forms' gradients
against differences."""
import ctypes

import pytest
import torch

import matrix_orthogonalizing_optimizer_step_b200 as mo
from tests import _lane_ref as ref

BAD, UNS = mo.MUON_ERR_INVALID_ARG, mo.MUON_ERR_UNSUPPORTED
P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10001)
I64, BF, F32 = mo.MUON_INDEX_I64, mo.MUON_DTYPE_BF16, mo.MUON_DTYPE_F32
BIG = 1 << 62


@pytest.fixture(scope="module")
def lib():
    return mo.lib()


def call(f, args, **changed):
    """f(*args) with named arguments changed; args is a list of (name, value)."""
    names = [n for n, _ in args]
    assert set(changed) <= set(names)
    return f(*[changed.get(n, v) for n, v in args])


def no_gpu(rc):
    if not torch.cuda.is_available():
        assert rc == mo.MUON_ERR_CUDA


EMB = [("tokens", P), ("it", I64), ("count", 5), ("table", P), ("td", F32), ("vocab", 10), ("dim", 8), ("scale", 1.0),
       ("out", P), ("od", BF)]


def test_embedding_refusals(lib):
    f = lib.muon_embedding
    for bad in (dict(count=-1), dict(count=1 << 31), dict(vocab=0), dict(vocab=1 << 31), dict(dim=0),
                dict(dim=(1 << 20) + 1), dict(tokens=None), dict(tokens=ODD), dict(table=None), dict(out=None),
                dict(table=ODD), dict(out=ODD), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(count=2_000_000_000, dim=1 << 20)):
        assert call(f, EMB, **bad) == BAD, bad
        assert lib.muon_last_error()
    for bad in (dict(it=2), dict(it=-1), dict(td=2), dict(od=7)):
        assert call(f, EMB, **bad) == UNS, bad
    assert call(f, EMB, count=0, tokens=None, table=None, out=None) == mo.MUON_OK
    no_gpu(call(f, EMB))


EMBB = [("tokens", P), ("it", I64), ("count", 5), ("grad", P), ("gd", BF), ("ld", 8), ("vocab", 10), ("dim", 8),
        ("scale", 1.0), ("pad", -1), ("out", P), ("od", BF), ("ws", P), ("nb", 1 << 20)]


def test_embedding_backward_refusals(lib):
    f = lib.muon_embedding_backward
    for bad in (dict(count=-1), dict(vocab=0), dict(dim=0), dict(tokens=None), dict(grad=None), dict(out=None),
                dict(out=ODD), dict(grad=ODD), dict(ld=7), dict(pad=-2), dict(pad=10), dict(scale=float("nan")),
                dict(ws=None), dict(ws=ctypes.c_void_p(0x10010)), dict(nb=16), dict(nb=-1)):
        assert call(f, EMBB, **bad) == BAD, bad
    for bad in (dict(it=3), dict(gd=2), dict(od=2)):
        assert call(f, EMBB, **bad) == UNS, bad
    no_gpu(call(f, EMBB))
    q = lib.muon_embedding_backward_workspace
    assert q(-1, 10, 8) == BAD and q(5, 0, 8) == BAD and q(5, 10, 0) == BAD and q(1 << 31, 10, 8) == BAD
    assert 0 <= q(0, 10, 8) <= q(5, 10, 8) <= q(5000, 10, 8)


NORM = [("x", P), ("xd", BF), ("ld", 8), ("rows", 5), ("dim", 8), ("w", P), ("b", P), ("pd", F32), ("eps", 1e-5),
        ("y", P), ("mean", P), ("rstd", P)]


def test_layer_norm_refusals(lib):
    f = lib.muon_layer_norm
    for bad in (dict(rows=-1), dict(rows=1 << 31), dict(dim=0), dict(dim=BIG), dict(ld=7), dict(eps=-1.0),
                dict(eps=float("nan")), dict(x=None), dict(y=None), dict(mean=None), dict(rstd=None), dict(x=ODD),
                dict(w=ODD), dict(b=ODD), dict(mean=ctypes.c_void_p(0x10002))):
        assert call(f, NORM, **bad) == BAD, bad
    for bad in (dict(xd=2), dict(pd=2)):
        assert call(f, NORM, **bad) == UNS, bad
    assert call(f, NORM, rows=0, x=None, y=None, mean=None, rstd=None) == mo.MUON_OK
    no_gpu(call(f, NORM, w=None, b=None))


NORMB = [("dy", P), ("ldg", 8), ("x", P), ("xd", BF), ("ldx", 8), ("rows", 5), ("dim", 8), ("mean", P), ("rstd", P),
         ("w", P), ("pd", F32), ("dx", P), ("dw", P), ("db", P), ("ws", P), ("nb", 1 << 20)]


def test_layer_norm_backward_refusals(lib):
    f = lib.muon_layer_norm_backward
    for bad in (dict(rows=-1), dict(dim=0), dict(ldg=7), dict(ldx=7), dict(dy=None), dict(x=None), dict(mean=None),
                dict(rstd=None), dict(dx=None), dict(dx=ODD), dict(dw=ODD), dict(ws=None), dict(nb=8)):
        assert call(f, NORMB, **bad) == BAD, bad
    for bad in (dict(xd=2), dict(pd=9)):
        assert call(f, NORMB, **bad) == UNS, bad
    no_gpu(call(f, NORMB, w=None, dw=None))
    q = lib.muon_layer_norm_backward_workspace
    assert q(-1, 8) == BAD and q(5, 0) == BAD and q(0, 8) == 0 and q(5, 8) > 0


HEAD = [("h", P), ("ld", 16), ("w", P), ("t", P), ("it", I64), ("tokens", 5), ("vocab", 10), ("dim", 16),
        ("ignore", -100), ("loss", P), ("lse", P), ("ws", P), ("nb", 1 << 24)]
HEADB = HEAD[:9] + [("lse", P), ("dl", P), ("dh", P), ("dw", P), ("ws", P), ("nb", 1 << 24)]


def test_head_loss_refusals(lib):
    shared = (dict(tokens=-1), dict(vocab=0), dict(dim=0), dict(ld=8), dict(ld=17), dict(h=None), dict(w=None),
              dict(t=None), dict(h=ctypes.c_void_p(0x10008)), dict(w=ctypes.c_void_p(0x10008)), dict(t=ODD),
              dict(ws=None), dict(nb=100), dict(tokens=1 << 30, vocab=1 << 30))
    for f, args, more in ((lib.muon_head_loss, HEAD, (dict(loss=None), dict(lse=None))),
                          (lib.muon_head_loss_backward, HEADB,
                           (dict(lse=None), dict(dl=None), dict(dh=None, dw=None), dict(dh=ODD), dict(dw=ODD)))):
        for bad in shared + more:
            assert call(f, args, **bad) == BAD, bad
        for bad in (dict(it=5), dict(dim=12)):
            assert call(f, args, **bad) == UNS, bad
        no_gpu(call(f, args))
    assert call(lib.muon_head_loss, HEAD, tokens=0, h=None, t=None) == mo.MUON_OK
    assert call(lib.muon_head_loss_backward, HEADB, tokens=0, h=None, t=None, dw=None) in (mo.MUON_OK, mo.MUON_ERR_CUDA)
    q = lib.muon_head_loss_workspace
    for b in (0, 1):
        assert q(-1, 10, 16, b) == BAD and q(5, 0, 16, b) == BAD and q(5, 10, 0, b) == BAD
        assert q(0, 10, 16, b) == 0 and q(5, 10, 16, b) > 0
    # the probabilities of a large batch stay within the piece size, whatever the vocabulary
    a, c = q(8192, 50257, 768, 1), q(8192, 5025700, 768, 1)
    assert c < 1.5 * a < 8192 * 50257 * 2


def test_binding_refusals():
    """The binding checks types, shapes and strides itself and raises ValueError."""
    t = torch.zeros(4, dtype=torch.int64)
    table = torch.zeros(10, 16)
    g = torch.zeros(4, 16)
    for args, kw in (((t.float(), table), {}), ((t, table.double()), {}), ((t, table[:, ::2]), {}), ((t, table[0]), {}),
                     ((t.expand(3, 4).t(), table), {}), ((t, table[:0]), {}), ((t, table), dict(out_dtype=torch.float16)),
                     ((t, table), {})):  # the last: not CUDA tensors
        with pytest.raises(ValueError):
            mo.muon_embedding(*args, **kw)
    for args, kw in (((t, g[:3], 10), {}), ((t, g.t(), 10), {}), ((t, g, 0), {}), ((t, g, 10), dict(padding_idx=10)),
                     ((t, g, 10), dict(padding_idx=-1)), ((t, g, 10), dict(grad_dtype=torch.float64)),
                     ((t, g, 10), dict(out=torch.zeros(10, 8))), ((t, g[:1].expand(4, 16), 10), {}), ((t, g, 10), {})):
        with pytest.raises(ValueError):
            mo.muon_embedding_backward(*args, **kw)
    x, w = torch.zeros(3, 16), torch.zeros(16)
    for args in ((x.half(), w), (x, w[:8]), (x, w.double()), (x, w, w.bfloat16()), (x.t(), torch.zeros(3)),
                 (torch.zeros(()), w), (torch.zeros(3, 0), w), (torch.zeros(4, 3, 16).transpose(0, 1), w), (x, w)):
        with pytest.raises(ValueError):
            mo.muon_layer_norm(*args)
    s = torch.zeros(3)
    for args, kw in (((x.bfloat16(), x, s, s, w), {}), ((x[:2], x, s, s, w), {}), ((x, x, s[:2], s, w), {}),
                     ((x, x, s.double(), s, w), {}), ((x, x, s, s, w), dict(param_dtype=torch.bfloat16)),
                     ((x, x, s, s, w), {})):
        with pytest.raises(ValueError):
            mo.muon_layer_norm_backward(*args, **kw)
    h, hw = torch.zeros(4, 16).bfloat16(), torch.zeros(10, 16).bfloat16()
    for args in ((h.float(), hw, t), (h, hw.float(), t), (h, hw, t[:3]), (h, hw[:, :8].contiguous(), t),
                 (h[:, :12].contiguous(), hw[:, :12].contiguous(), t), (h, hw, t.float()),
                 (torch.zeros(4, 20).bfloat16()[:, :16], hw, t), (h, hw, t)):
        with pytest.raises(ValueError):
            mo.muon_head_loss(*args)
    f = torch.zeros(4)
    for args, kw in (((h, hw, t, f[:3], f), {}), ((h, hw, t, f, f.bfloat16()), {}),
                     ((h, hw, t, f, f), dict(hidden_grad=False, weight_grad=False)), ((h, hw, t, f, f), {})):
        with pytest.raises(ValueError):
            mo.muon_head_loss_backward(*args, **kw)


# ---- the reference forms themselves -----------------------------------------------------


def differences(f, x, v, h=1e-5):
    return (f(x + h * v) - f(x - h * v)) / (2 * h)


def test_reference_norm_gradient_against_differences():
    g = torch.Generator().manual_seed(0)
    x, dy, v = (torch.randn(5, 12, generator=g, dtype=torch.float64) for _ in range(3))
    w, b, vw = (torch.randn(12, generator=g, dtype=torch.float64) for _ in range(3))
    _, mean, rstd = ref.norm(x, w, b, 1e-5)
    (dx, dw, db), _ = ref.norm_grad(dy, x, mean, rstd, w)
    for grad, at, along, f in ((dx, x, v, lambda q: (dy * ref.norm(q, w, b, 1e-5)[0]).sum()),
                               (dw, w, vw, lambda q: (dy * ref.norm(x, q, b, 1e-5)[0]).sum()),
                               (db, b, vw, lambda q: (dy * ref.norm(x, w, q, 1e-5)[0]).sum())):
        assert abs((grad * along).sum() - differences(f, at, along)) < 1e-7


def test_reference_head_gradient_against_differences():
    g = torch.Generator().manual_seed(1)
    h, v = (torch.randn(6, 8, generator=g, dtype=torch.float64) for _ in range(2))
    w, vw = (torch.randn(9, 8, generator=g, dtype=torch.float64) for _ in range(2))
    t = torch.tensor([0, 8, 3, -100, 3, 5])
    dl = torch.rand(6, generator=g, dtype=torch.float64)
    _, lse, p, valid, h64, at = ref.head(h, w, t, -100)
    zero = torch.zeros(6, dtype=torch.float64)
    (dh, dw), _ = ref.head_grad(h64, w, p, valid, at, dl, zero, zero)
    for grad, x, along, f in ((dh, h, v, lambda q: (dl * ref.head(q, w, t, -100)[0]).sum()),
                              (dw, w, vw, lambda q: (dl * ref.head(h, q, t, -100)[0]).sum())):
        assert abs((grad * along).sum() - differences(f, x, along)) < 1e-7


def test_reference_embedding_gradient_against_differences():
    g = torch.Generator().manual_seed(2)
    t = torch.tensor([1, 4, 1, 0, 4, 4])
    dy, w, v = torch.randn(6, 3, generator=g, dtype=torch.float64), *torch.randn(2, 5, 3, generator=g, dtype=torch.float64)
    d, _ = ref.embedding_grad(t, dy, 5, 2.0, None)
    assert abs((d * v).sum() - differences(lambda q: (dy * ref.embedding(t, q, 2.0)).sum(), w, v)) < 1e-7
    assert (ref.embedding_grad(t, dy, 5, 2.0, 4)[0][4] == 0).all()
