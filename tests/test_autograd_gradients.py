"""Gradients as autograd hands them to the entry points of global_attention_b200.autograd: parts of a larger tensor that begin
anywhere (the backward of torch.cat), expanded numbers (of a sum).  The kernels take contiguous rows that begin at 16 bytes."""
import pytest
import torch

from global_attention_b200.autograd import zgcm_attention, zgcm_qk_norm_rope


def _seen(seen, *grads):
    seen.extend((d.is_contiguous(), d.data_ptr() % 16) for d in grads)


def _norm(seen, x):
    def bwd(q, k, gq, gk, pos, dqr, dkr, **kw):
        _seen(seen, dqr, dkr)
        return dict(dq=dqr * 2, dk=dkr * 2, dgamma_q=gq, dgamma_k=gk)

    y = zgcm_qk_norm_rope(x, x, torch.ones(8), torch.ones(8), ops=(lambda q, k, *a, **kw: (q * 2, k * 2), bwd))
    return torch.stack(y)


def _attention(seen, x):
    def bwd(q, k, v, g, gq, gk, out, lse, dout, **kw):
        _seen(seen, dout)
        z = torch.zeros_like(dout)
        return dict(dq=dout * 2, dk=z, dv=z, dg=z, dgamma_q=gq, dgamma_k=gk)

    ops = (lambda q, *a, **kw: (q * 2, torch.zeros(q.shape[0], q.shape[2], q.shape[1])), bwd, lambda *a: 0)
    return zgcm_attention(x, x, x, x, torch.ones(8), torch.ones(8), ops=ops)


@pytest.mark.parametrize("f", [_norm, _attention])
@pytest.mark.parametrize("before", [0, 1, 2, 3])
def test_gradients_of_concatenated_outputs(f, before):
    x = torch.randn(2, 3, 2, 8, requires_grad=True)
    seen = []
    y = f(seen, x)
    w = torch.randn(before + y.numel())
    (torch.cat([torch.ones(before), y.flatten()]) * w).sum().backward()
    assert seen and all(s == (True, 0) for s in seen)
    assert torch.equal(x.grad, 2 * w[before:].view(-1, *x.shape).sum(0))
    seen.clear()
    f(seen, x).sum().backward()
    assert seen and all(s == (True, 0) for s in seen)


@pytest.mark.gpu
def test_concatenated_outputs_on_the_gpu():
    """The same bits as from gradients of their own."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gen = torch.Generator().manual_seed(6)
    q, k, v, g = (torch.randn((1, 70, h, 128), generator=gen).to(torch.bfloat16).cuda() for h in (8, 2, 2, 8))
    gq, gk = (torch.rand(128, generator=gen).cuda() for _ in range(2))
    head = torch.zeros(3, dtype=torch.bfloat16, device="cuda")
    for f, xs in ((lambda q, k: torch.cat([t.flatten() for t in zgcm_qk_norm_rope(q, k, gq, gk)]), (q, k)),
                  (lambda q, k, v, g: zgcm_attention(q, k, v, g, gq, gk).flatten(), (q, k, v, g))):
        kept = []
        for skip in (0, 3):
            leaves = [t.clone().requires_grad_() for t in xs]
            y = f(*leaves)
            w = torch.randn(y.shape, generator=torch.Generator().manual_seed(7)).to(y).sign()
            kept.append(torch.autograd.grad(torch.cat([head[:skip], y]), leaves, torch.cat([head[:skip], w])))
        assert all(torch.equal(a, b) for a, b in zip(*kept))
