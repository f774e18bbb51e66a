"""CPU checks of the operators of a training step around the blocks: the 64-bit
forms that the GPU tests compare with (against torch autograd and against
differences), and what the entry points refuse before any work."""
import ctypes as C

import numpy as np
import pytest
import torch
import torch.nn.functional as F

import megatron_tensor_transformer_colwise_gb300 as tp
import training_refs as refs


def rng(seed):
    return np.random.default_rng(seed)


def test_layernorm_forms_equal_autograd():
    r = rng(1)
    x, dy, dres = (r.normal(size=(7, 24)) for _ in range(3))
    gain, bias = r.normal(size=24), r.normal(size=24)
    X, G, B = (torch.tensor(a, requires_grad=True) for a in (x, gain, bias))
    Y = F.layer_norm(X, (24,), G, B, 1e-3)
    (Y * torch.tensor(dy)).sum().backward()
    dx, dgain, dbias = refs.layernorm_backward(x, gain, 1e-3, dy, dres)[:3]
    np.testing.assert_allclose(refs.layernorm(x, gain, bias, 1e-3), Y.detach().numpy(), rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(dx, X.grad.numpy() + dres, rtol=1e-11, atol=1e-12)
    np.testing.assert_allclose(dgain, G.grad.numpy(), rtol=1e-11, atol=1e-12)
    np.testing.assert_allclose(dbias, B.grad.numpy(), rtol=1e-11, atol=1e-12)


def test_layernorm_gradient_against_differences():
    r = rng(2)
    x, dy, gain = r.normal(size=(3, 16)), r.normal(size=(3, 16)), r.normal(size=16)
    dx = refs.layernorm_backward(x, gain, 1e-5, dy)[0]
    e = 1e-5
    for at in [(0, 0), (1, 7), (2, 15)]:
        up, down = x.copy(), x.copy()
        up[at] += e
        down[at] -= e
        d = ((refs.layernorm(up, gain, 0, 1e-5) - refs.layernorm(down, gain, 0, 1e-5)) * dy).sum() / (2 * e)
        assert abs(d - dx[at]) < 1e-8


def test_embedding_forms_equal_autograd():
    r = rng(3)
    ids = np.array([3, 0, 3, 9, 3, 0])
    E = torch.tensor(r.normal(size=(10, 8)), requires_grad=True)
    d = r.normal(size=(6, 8))
    out = 2.5 * E[torch.tensor(ids)]
    (out * torch.tensor(d)).sum().backward()
    np.testing.assert_allclose(refs.embedding(ids, E.detach().numpy(), 2.5), out.detach().numpy())
    dE, _, count = refs.embedding_backward(ids, 10, d, 2.5)
    np.testing.assert_allclose(dE, E.grad.numpy(), rtol=1e-12)
    assert count.tolist() == [2, 0, 0, 3, 0, 0, 0, 0, 0, 1]
    assert not refs.embedding(np.array([-1, 10]), E.detach().numpy(), 2.0).any()


def test_loss_forms_equal_autograd_and_masks():
    r = rng(4)
    z = r.normal(size=(5, 12)) * 4
    z[2, 3:9] = -np.inf
    labels = np.array([1, -100, 2, 11, 0])
    w = r.uniform(size=5)
    Z = torch.tensor(z, requires_grad=True)
    L = F.cross_entropy(Z, torch.tensor(labels), reduction="none", ignore_index=-100)
    (L * torch.tensor(w)).sum().backward()
    out, grad = refs.loss(z, labels, w)
    np.testing.assert_allclose(out, L.detach().numpy(), rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(grad, Z.grad.numpy(), rtol=1e-10, atol=1e-15)
    # A label that is masked costs infinitely much, a row of nothing else has no answer.
    out, grad = refs.loss(np.array([[0.0, -np.inf], [-np.inf, -np.inf], [0, np.nan], [0, np.inf]]), np.array([1, 0, 0, 1]), np.ones(4))
    assert out[0] == np.inf and grad[0].tolist() == [1, -1] and np.isnan(out[1:]).all() and np.isnan(grad[1:]).all()


def test_loss_gradient_against_differences():
    r = rng(5)
    z, labels, w = r.normal(size=(2, 9)), np.array([4, 0]), np.array([0.7, 2.0])
    _, grad = refs.loss(z, labels, w)
    e = 1e-6
    for at in [(0, 4), (0, 1), (1, 0), (1, 8)]:
        up, down = z.copy(), z.copy()
        up[at] += e
        down[at] -= e
        d = ((refs.loss(up, labels, w)[0] - refs.loss(down, labels, w)[0]) * w).sum() / (2 * e)
        assert abs(d - grad[at]) < 1e-8


def test_clip_form():
    g = [torch.randn(5, dtype=torch.float64, requires_grad=True) for _ in range(3)]
    for x in g:
        x.grad = x.detach().clone()
    norm, out = refs.clip([x.detach().numpy() for x in g], 0.5)
    total = torch.nn.utils.clip_grad_norm_(g, 0.5)
    assert abs(norm - float(total)) < 1e-12
    for a, b in zip(out, g):
        np.testing.assert_allclose(a, b.grad.numpy(), rtol=1e-5)  # torch divides by norm + 1e-6


# ------------------------------------------------------------ refusals (no GPU work: any 16-byte multiple serves as an address)

P = 0x10000


def rc(name, *args):
    return getattr(tp.lib(), name)(*args)


def test_embedding_refusals():
    def fwd(ids=P, M=4, E=2 * P, v=64, h=16, t=4, out=3 * P):
        return rc("tp_vocab_embedding_scaled_forward", ids, M, E, v, h, t, 2.0, out, None)

    def bwd(ids=P, M=4, v=64, h=16, t=4, dOut=2 * P, dE=3 * P, ws=4 * P, n=1 << 20):
        return rc("tp_vocab_embedding_backward", ids, M, v, h, t, 2.0, dOut, dE, 0, ws, n, None)

    bad = tp.TP_ERR_INVALID_ARG
    for f in (fwd, bwd):
        assert f(ids=None) == bad and f(ids=P + 4) == bad and f(h=12) == bad and f(h=0) == bad and f(M=-1) == bad
        assert f(v=0) == bad and f(t=0) == bad and f(t=65) == bad and f(t=3) == tp.TP_ERR_NOT_DIVISIBLE
        assert f(M=1 << 31) == bad and f(v=1 << 31, t=1) == bad
    assert fwd(E=None) == bad and fwd(out=None) == bad and fwd(out=P + 2) == bad
    assert fwd(M=0, ids=None, E=None, out=None) == tp.TP_OK  # no tokens: nothing to do, no addresses
    assert bwd(dOut=None) == bad and bwd(dE=None) == bad and bwd(dE=P + 8) == bad
    need = tp.tp_vocab_embedding_backward_workspace_bytes(4, 64, 16)
    assert bwd(ws=None) == bwd(n=need - 1) == bwd(ws=P + 8) == tp.TP_ERR_WORKSPACE
    n = C.c_size_t()
    assert rc("tp_vocab_embedding_backward_workspace_bytes", 4, 64, 16, None) == bad
    assert rc("tp_vocab_embedding_backward_workspace_bytes", -1, 64, 16, C.byref(n)) == bad


def test_loss_refusals():
    def f(logits=P, M=4, v=64, t=4, labels=2 * P, dloss=None, loss=3 * P, d=4 * P):
        return rc("tp_vocab_parallel_cross_entropy_train", logits, M, v, t, labels, dloss, loss, d, None)

    bad = tp.TP_ERR_INVALID_ARG
    assert f(logits=None) == f(labels=None) == f(loss=None) == f(d=None) == bad
    assert f(logits=P + 2) == f(dloss=P + 4) == f(d=P + 8) == bad
    assert f(v=60, t=1) == bad and f(v=64, t=16) == bad and f(v=64, t=3) == tp.TP_ERR_NOT_DIVISIBLE
    assert f(M=-1) == f(M=1 << 31) == f(v=1 << 31, t=1) == bad
    assert f(M=0, logits=None, labels=None, loss=None, d=None) == tp.TP_OK


def test_output_gradient_refusals():
    def f(H=P, M=4, h=16, W=2 * P, v=64, t=4, d=3 * P, dH=4 * P, dW=5 * P, ws=6 * P, n=1 << 30):
        return rc("tp_vocab_logits_backward", H, M, h, W, v, t, d, dH, dW, 0, ws, n, None)

    bad = tp.TP_ERR_INVALID_ARG
    assert f(H=None) == f(W=None) == f(d=None) == f(H=P + 8) == f(dH=P + 8) == f(dW=P + 4) == bad
    assert f(h=12) == f(M=-1) == f(v=60, t=1) == bad and f(v=64, t=3) == tp.TP_ERR_NOT_DIVISIBLE
    assert f(M=0, H=None, W=None, d=None, dW=None) == tp.TP_OK
    assert f(dH=None, dW=None) == tp.TP_OK  # nothing wanted


def test_layernorm_refusals():
    def fwd(x=P, rows=4, h=64, gain=2 * P, bias=3 * P, eps=1e-5, y=4 * P, stats=None):
        return rc("tp_layernorm_forward", x, rows, h, gain, bias, eps, y, stats, None)

    def bwd(x=P, rows=4, h=64, gain=2 * P, eps=1e-5, stats=None, dy=3 * P, dres=None, dx=4 * P, dg=5 * P, db=6 * P, ws=7 * P,
            n=1 << 20):
        return rc("tp_layernorm_backward", x, rows, h, gain, eps, stats, dy, dres, dx, dg, db, 0, ws, n, None)

    bad = tp.TP_ERR_INVALID_ARG
    for f in (fwd, bwd):
        assert f(x=None) == f(x=P + 8) == f(gain=P + 2) == f(stats=P + 4) == bad
        assert f(h=0) == f(h=60) == f(h=16392) == f(rows=-1) == f(rows=(1 << 30) + 1) == bad
        assert f(eps=-1e-9) == f(eps=float("nan")) == bad
    assert fwd(y=None) == fwd(bias=P + 2) == bwd(dy=None) == bwd(dx=None) == bwd(dres=P + 2) == bwd(dg=P + 4) == bwd(db=P + 4) == bad
    need = tp.tp_layernorm_backward_workspace_bytes(4, 64)
    assert bwd(ws=None) == bwd(n=need - 1) == bwd(ws=P + 4) == tp.TP_ERR_WORKSPACE
    assert fwd(rows=0, x=None, y=None) == tp.TP_OK
    assert bwd(rows=0, x=None, dy=None, dx=None, dg=None, db=None, ws=None, n=0) == tp.TP_OK
    assert rc("tp_layernorm_backward_workspace_bytes", 4, 60, C.byref(C.c_size_t())) == bad
    assert rc("tp_layernorm_backward_workspace_bytes", 4, 64, None) == bad


def test_clip_refusals():
    T = tp.TPGradTensor

    def f(tensors, max_norm=1.0, norm=P, ws=2 * P, n=1 << 20, count=None):
        array = (T * max(len(tensors), 1))(*tensors)
        return rc("tp_grad_clip", array, len(tensors) if count is None else count, max_norm, norm, ws, n, None)

    a, bad = 1 << 24, tp.TP_ERR_INVALID_ARG
    assert f([T(None, a, 4, 0)]) == f([T(a + 4, a + 4, 4, 0)]) == f([T(a, a + 8, 4, 0)]) == bad
    assert f([T(a, a, -1, 0)]) == f([T(a, a, 4, 2)]) == f([T(a, a, (1 << 40) + 1, 0)]) == bad
    assert f([], count=-1) == f([], count=65537) == rc("tp_grad_clip", None, 1, 1.0, P, 2 * P, 1 << 20, None) == bad
    one = [T(a, a, 4, 0)]
    assert f(one, max_norm=-1.0) == f(one, max_norm=float("nan")) == f(one, norm=None) == f(one, norm=P + 4) == bad
    need = tp.tp_grad_clip_workspace_bytes(1)
    assert f(one, ws=None) == f(one, n=need - 1) == f(one, ws=P + 8) == tp.TP_ERR_WORKSPACE
    # What is written overlaps nothing else: the same tensor twice, a tail, another one's input or output.
    assert f([T(a, a, 100, 0), T(a, a, 100, 0)]) == bad
    assert f([T(a, a, 100, 0), T(a + 384, a + 384, 100, 0)]) == bad
    assert f([T(a, a + 4096, 100, 0), T(a + 8192, a + 4096 + 16, 4, 0)]) == bad
    assert f([T(a, None, 100, 0), T(a + 8192, a + 16, 4, 0)]) == bad
    assert f([T(a, a + 16, 100, 0)]) == bad
    assert f([T(a, a, 1 << 20, 0), T(a + 4096, None, 4, 1), T(a + 64, None, 4, 1)]) == bad


def test_grad_list_refuses_what_it_cannot_pass():
    x = torch.zeros(4, 4)
    with pytest.raises(ValueError):
        tp.make_grad_list([x.double()])
    with pytest.raises(ValueError):
        tp.make_grad_list([x.T[1:]])
    with pytest.raises(ValueError):
        tp.make_grad_list([x], [x.bfloat16()])
    with pytest.raises(ValueError):
        tp.make_grad_list([x], [x, x])
    assert len(tp.make_grad_list([x, x.bfloat16()], [None, None])) == 2
