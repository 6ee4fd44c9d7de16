"""The q/k normalisation and rotation operator (include/zgcm_qkrope.h) on tensors that begin elsewhere than the
allocator's own.  Helpers and tolerances are those of tests/test_qk_norm_rope.py.
"""
import pytest
import torch

import global_attention_b200 as ga
from global_attention_b200.autograd import zgcm_qk_norm_rope
from test_qk_norm_rope import _inputs, cuda  # noqa: F401  (cuda: the fixture)

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
