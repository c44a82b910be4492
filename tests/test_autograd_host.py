"""Host test of the autograd forms, with the kernels' calls replaced by plain ones that autograd
does not see, as it does not see the kernels: a first derivative under create_graph is right,
a second one is refused instead of being taken for zero."""
import pytest
import torch

import invariant_token_logprob_gb300 as rlk


def logprobs(x, targets, *_, **__):
    x = x.detach()
    lse = torch.logsumexp(x, 1)
    logp = x - lse[:, None]
    T = x.shape[0]
    return rlk.TokenLogprobs(logp[torch.arange(T), targets.long()], lse, -(logp.exp() * logp).sum(1),
                             torch.zeros(T, 0, dtype=torch.int32), torch.zeros(T, 0))


def logprobs_grad(x, targets, lse, entropy, g_logp, *_, **__):
    d = -torch.exp(x.detach() - lse.detach()[:, None])
    d[torch.arange(x.shape[0]), targets.long()] += 1
    return d * g_logp.detach()[:, None]


def head_logprob(h, W, targets, inv_temp):
    r = logprobs(h @ W.t(), targets)
    return r.logp, r.lse, targets


def head_grad(h, W, targets, lse, g, inv_temp, need_h, need_W):
    with torch.no_grad():
        dz = logprobs_grad(h @ W.t(), targets, lse, None, g)
        return (dz @ W if need_h else None), (dz.t() @ h if need_W else None), None


def check(f, x, want):
    out = f(x)
    (g,) = torch.autograd.grad(out.sum(), x, create_graph=True)
    assert torch.allclose(g, want, atol=1e-6)
    with pytest.raises(RuntimeError, match="first derivatives only"):
        torch.autograd.grad((g * g).sum(), x)
    x.grad = None
    with pytest.raises(RuntimeError, match="first derivatives only"):
        (f(x).sum() + (g * g).sum()).backward()


def inputs():
    gen = torch.Generator().manual_seed(0)
    return torch.randn(3, 7, generator=gen), torch.tensor([1, 6, 0], dtype=torch.int32), torch.randn(11, 7, generator=gen)


def test_second_derivative_of_token_logprobs_is_refused(monkeypatch):
    monkeypatch.setattr(rlk, "token_logprobs", logprobs)
    monkeypatch.setattr(rlk, "token_logprobs_backward", logprobs_grad)
    x, tg, _ = inputs()
    want = logprobs_grad(x, tg, torch.logsumexp(x, 1), None, torch.ones(3))
    check(lambda y: rlk.differentiable_token_logprobs(y, tg).logp, x.requires_grad_(), want)


def test_second_derivative_of_selected_token_logprob_is_refused(monkeypatch):
    monkeypatch.setattr(rlk, "logprob", head_logprob)
    monkeypatch.setattr(rlk, "logprob_backward", head_grad)
    h, tg, W = inputs()
    want = logprobs_grad(h @ W.t(), tg, torch.logsumexp(h @ W.t(), 1), None, torch.ones(3)) @ W
    check(lambda y: rlk.selected_token_logprob(y, W, tg), h.requires_grad_(), want)
