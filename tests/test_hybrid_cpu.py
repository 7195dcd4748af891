"""Bookkeeping of MuonHybrid.step (no GPU): the calls into the library are
replaced by records of what they were given."""
import pytest
import torch

import matrix_orthogonalizing_optimizer_step_b200 as mo
from matrix_orthogonalizing_optimizer_step_b200 import layers, optim


@pytest.fixture
def calls(monkeypatch):
    """The library's calls as a list of (name, step counts, gradients)."""
    seen = []

    def dense(tokens, rows, vocab, out=None):
        if out is None:
            out = torch.empty(vocab, rows.shape[1], dtype=rows.dtype, device=rows.device)
        seen.append(("embedding_backward", out))
        return out.zero_().index_add_(0, tokens, rows)

    monkeypatch.setattr(mo, "muon_embedding_backward", dense, raising=False)
    monkeypatch.setattr(optim, "muon_set_config", lambda **kw: None)
    monkeypatch.setattr(optim, "muon_step", lambda *a, **kw: seen.append(("step",)))
    monkeypatch.setattr(optim, "muon_adamw_step", lambda P, G, M, V, t, **kw: seen.append(("adamw", t, [g.clone() for g in G])))
    monkeypatch.setattr(optim, "muon_hybrid_step",
                        lambda W, G, M, P, AG, M1, M2, t, **kw: seen.append(("hybrid", t, [g.clone() for g in AG])))
    return seen


def row_sparse(p, rows):
    values = torch.ones(len(rows), p.shape[1])
    return torch.sparse_coo_tensor(torch.tensor([rows]), values, p.shape)


def parameters():
    torch.manual_seed(0)
    return [torch.nn.Parameter(torch.randn(*s)) for s in ((6, 4), (8, 4), (5,))]


def test_a_refused_step_leaves_the_counts(calls):
    """A gradient that the step refuses: no count moves, and the next valid step
    is the one of a fresh optimizer, both lanes in one call."""
    mat, emb, vec = parameters()
    opt = optim.MuonHybrid([mat], [vec, emb])
    mat.grad, vec.grad = torch.randn(6, 4), torch.randn(5)
    emb.grad = torch.randn(8, 4).to_sparse()  # single elements, not rows
    for _ in range(2):
        with pytest.raises(TypeError):
            opt.step()
    assert all(s.get("step", 0) == 0 for s in opt.state.values()) and calls == []
    emb.grad = row_sparse(emb, [1, 1, 3])
    opt.step()
    assert [c[:2] for c in calls if c[0] != "embedding_backward"] == [("hybrid", 1)]
    assert opt.state[vec]["step"] == opt.state[emb]["step"] == 1


def test_a_refused_group_leaves_the_other_groups_counts(calls):
    mat, emb, vec = parameters()
    opt = optim.MuonHybrid([], [vec])
    opt.add_param_group(dict(params=[mat], kind="muon", lr=0.1, momentum=0.9, nesterov=True))
    vec.grad, mat.grad = torch.randn(5), torch.eye(6, 4).to_sparse()
    with pytest.raises(TypeError):
        opt.step()
    assert opt.state.get(vec, {}).get("step", 0) == 0
    mat.grad = torch.randn(6, 4)
    opt.step()
    assert [c[:2] for c in calls] == [("hybrid", 1)]


def test_counts_of_parameters_that_skip_steps(calls):
    """Parameters without a gradient keep their count; each count is a call of its own."""
    _, emb, vec = parameters()
    opt = optim.MuonHybrid([], [vec, emb])
    vec.grad = torch.randn(5)
    opt.step()
    emb.grad = row_sparse(emb, [0])
    opt.step()
    assert [c[:2] for c in calls if c[0] == "adamw"] == [("adamw", 1), ("adamw", 1), ("adamw", 2)]


def test_buffer_of_row_sparse_gradients_follows_its_parameter(calls):
    """After model.to(other device) the buffer is a new one there."""
    _, emb, _ = parameters()
    opt = optim.MuonHybrid([], [emb])
    opt._row_grads[emb] = torch.empty(8, 4, device="meta")
    emb.grad = row_sparse(emb, [1, 2, 1])
    opt.step()
    assert opt._row_grads[emb].device == emb.device
    assert torch.equal(calls[-1][2][0], emb.grad.to_dense().view(-1))


def test_buffer_of_row_sparse_gradients_is_reused_and_dropped(calls):
    _, emb, _ = parameters()
    opt = optim.MuonHybrid([], [emb])
    emb.grad = row_sparse(emb, [1, 2, 1])
    opt.step()
    opt.step()
    first, second = (c[1] for c in calls if c[0] == "embedding_backward")
    assert first is second
    emb.grad = torch.randn(8, 4)  # dense from here on: nothing is kept
    opt.step()
    assert not opt._row_grads


def test_embedding_refuses_a_padding_index_outside_the_vocabulary():
    """In the forward pass, where torch's own layer would take a negative one,
    not in the backward pass of a step that has run."""
    w, t = torch.zeros(5, 8, requires_grad=True), torch.tensor([1, 2])
    for bad in (-1, 5):
        with pytest.raises(ValueError, match="padding_idx"):
            layers.embedding(t, w, padding_idx=bad)
        with pytest.raises(ValueError, match="padding_idx"):
            layers.Embedding(5, 8, padding_idx=bad)
