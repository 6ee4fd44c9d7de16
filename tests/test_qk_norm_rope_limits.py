"""The q/k normalisation and rotation operator (include/zgcm_qkrope.h): tensors that begin elsewhere than the allocator's
own, the length of dgamma's sums.  Helpers and tolerances are those of tests/test_qk_norm_rope.py.
"""
import numpy as np
import pytest
import torch

import global_attention_b200 as ga
from global_attention_b200.autograd import zgcm_qk_norm_rope
from oracle import qkrope
from test_qk_norm_rope import _inputs, _partner, cuda  # noqa: F401  (cuda: the fixture)

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("skip", [1, 2, 3])
def test_slices_of_positions(cuda, skip):  # noqa: F811
    """Positions that begin 4, 8 and 12 bytes past a 16-byte boundary: the same bits, in both directions and through autograd."""
    q, k, gq, gk, pos, dqr, dkr = (t.cuda() for t in _inputs(24, 4, 2, "bf16", "bf16", seed=5))
    part = torch.cat([pos[:skip], pos])[skip:]
    assert part.data_ptr() % 16 == 4 * skip
    args = [(q, k, gq, gk, p) for p in (pos, part)]
    for f in (lambda a: ga.zgcm_qk_norm_rope_fwd(*a), lambda a: [*ga.zgcm_qk_norm_rope_bwd(*a, dqr, dkr).values()]):
        assert all(torch.equal(x, y) for x, y in zip(*(f(a) for a in args)))
    kept = []
    for p in (pos, part):
        leaves = [t.clone().view(2, 12, *t.shape[1:]).requires_grad_() for t in (q, k)]
        y = zgcm_qk_norm_rope(*leaves, gq, gk, p.view(2, 12))
        kept.append([*y, *torch.autograd.grad(y, leaves, [d.view_as(x) for d, x in zip((dqr, dkr), y)])])
    assert all(torch.equal(x, y) for x, y in zip(*kept))


@gpu
@pytest.mark.parametrize("T,Hq,Hkv,R,xt,yt", [(1, 32, 8, 42, "bf16", "bf16"), (100, 32, 8, 42, "bf16", "fp16"),
                                              (2368, 9, 1, 64, "fp16", "bf16"), (2369, 32, 8, 42, "bf16", "bf16"),
                                              (20000, 5, 2, 42, "fp32", "fp32"), (40000, 4, 1, 42, "bf16", "bf16")])
def test_gamma_gradients_by_their_chains(cuda, T, Hq, Hkv, R, xt, yt):  # noqa: F811
    """dgamma's sums are no longer than the kernel makes them: a warp, one of 296 x 8, takes every 2368th token, four rows at
    a time, so a lane adds ceil(T / 2368) ceil(H / 4) terms; then 2 shuffles, 8 warps, 10 partials of 32 warps and these: 52
    more.  Each term is off by 2^-19 of its magnitude as the file of the helpers derives."""
    q, k, gq, gk, pos, dqr, dkr = _inputs(T, Hq, Hkv, xt, yt, seed=T)
    gr = ga.zgcm_qk_norm_rope_bwd(*(t.cuda() for t in (q, k, gq, gk, pos, dqr, dkr)), rope_dims=R)
    for x, gamma, dy, got in ((q, gq, dqr, gr["dgamma_q"]), (k, gk, dkr, gr["dgamma_k"])):
        _, ref = qkrope.backward(x, gamma, pos, dy, rope_dims=R)
        xd, dyd = (np.abs(t.double().numpy()) for t in (x, dy))
        mag = ((dyd + _partner(dyd, R)) * xd / np.sqrt((xd * xd).mean(-1, keepdims=True) + 1e-6)).sum((0, 1))
        chain = -(-T // 2368) * -(-x.shape[1] // 4) + 52
        err = np.abs(got.double().cpu().numpy() - ref) / mag
        assert (err <= 2.0 ** -19 + chain * 2.0 ** -24).all(), float(err.max())
