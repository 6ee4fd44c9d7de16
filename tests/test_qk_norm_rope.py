"""The q/k normalisation and rotation operator (include/zgcm_qkrope.h): argument checks and autograd
plumbing on the CPU, numerics on the B200 against the fp64 oracle (oracle/qkrope.py).

Tolerances, from the arithmetic.  An output element is rounded once: half a step of its type,
finfo.eps / 2 relative (and half the smallest subnormal of fp16).  Before that, in fp32 with
u = 2^-24: the sum of 128 squares (8 serial + 4 tree additions) 13u, halved by the root, rsqrt
4u, the two products 2u, the cosine and sine 2^-22 absolute (angle reduced in fp64, held in
fp32), two products and a sum 3u: below 32u = 2^-19 of |y| + |partner|.  The backward adds a
second sum of 128 and its products: 2^-18 of the magnitudes summed.  dgamma is a sum of fp32
terms, each off by 2^-19 of its magnitude, in chains of at most n rows per lane group, 16
groups and 592 / 8 + 8 partials: (n + 98) u.
"""
import ctypes

import numpy as np
import pytest
import torch

import global_attention_b200 as ga
from global_attention_b200.autograd import zgcm_qk_norm_rope
from global_attention_b200.build import build
from oracle import qkrope

P = 0x7F0000000000
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------ CPU: refusals

@pytest.fixture(scope="module")
def lib():
    build()
    return ga.load()


def _c(lib, bwd=False, T=4, Hq=4, Hkv=2, D=128, xt=0, yt=0, R=42, base=1e4, eps=1e-6, bad=None, ptr=0, stride=512, ws=None):
    def rows(n):
        return ga._Rows(ptr if bad == n else P + 256 * n, stride if bad == n else 512, 128)

    vp = ctypes.c_void_p
    ptrs = [vp(ptr if bad == 10 + i else P + 8192 + 256 * i) for i in range(5)]
    if not bwd:
        return lib.zgcm_qk_norm_rope_fwd(rows(0), rows(1), *ptrs[:3], T, Hq, Hkv, D, xt, yt, R, base, eps, rows(2),
                                         rows(3), None)
    need = lib.zgcm_qk_norm_rope_bwd_workspace_size(T)
    wp, wb = (P + 2 ** 20, need) if ws is None else ws
    return lib.zgcm_qk_norm_rope_bwd(rows(0), rows(1), *ptrs[:3], rows(2), rows(3), T, Hq, Hkv, D, xt, yt, R, base, eps,
                                     rows(4), rows(5), *ptrs[3:], vp(wp), wb, None)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), -1), (dict(Hq=0), -1), (dict(Hkv=0), -1), (dict(xt=3), -1), (dict(yt=-1), -1), (dict(R=41), -1),
    (dict(R=130), -1), (dict(base=0.0), -1), (dict(base=float("inf")), -1), (dict(eps=-1.0), -1),
    (dict(eps=float("nan")), -1), (dict(D=64), -2), (dict(T=2 ** 31 - 1, Hq=64), -2),
])
def test_refuses_arguments(lib, bwd, kw, status):
    assert _c(lib, bwd, **kw) == status


@pytest.mark.parametrize("bwd", [False, True])
def test_refuses_pointers(lib, bwd):
    for n in (range(6) if bwd else range(4)):
        assert _c(lib, bwd, bad=n, ptr=0) == -1
        assert _c(lib, bwd, bad=n, ptr=P + 8) == -3
        assert _c(lib, bwd, bad=n, ptr=P, stride=12) == -3
        assert _c(lib, bwd, bad=n, ptr=P, stride=2 ** 32) == -2
        assert _c(lib, bwd, bad=n, ptr=P, stride=-512) == -2
    for n in (range(10, 15) if bwd else range(10, 13)):
        assert _c(lib, bwd, bad=n, ptr=0) == -1
        assert _c(lib, bwd, bad=n, ptr=P + 4) == -3


def test_workspace(lib):
    size = lib.zgcm_qk_norm_rope_bwd_workspace_size
    # 1 KB for each CTA: 2 for a token (16 warps share its rows), at most 296
    assert size(0) == 0 and size(-3) == 0 and size(1) == 2 * 1024
    assert size(10 ** 6) == 296 * 1024
    need = size(4)
    assert _c(lib, True, ws=(P, need - 1)) == -4
    assert _c(lib, True, ws=(0, need)) == -4
    assert _c(lib, True, ws=(P + 8, need)) == -3


def test_empty_forward_launches_nothing(lib):
    assert _c(lib, T=0) == 0


def test_binding_refuses(monkeypatch):
    class NoLib:
        def __getattr__(self, name):
            raise AssertionError(f"reached the library ({name})")

    monkeypatch.setattr(ga, "load", lambda: NoLib())
    q, k = torch.zeros(6, 4, 128, dtype=torch.bfloat16), torch.zeros(6, 2, 128, dtype=torch.bfloat16)
    g, pos = torch.ones(128), torch.zeros(6, dtype=torch.int32)
    ok = dict(q=q, k=k, gamma_q=g, gamma_k=g, pos=pos)
    for bad in (dict(k=k[:5]), dict(pos=pos[:5]), dict(pos=pos.long()), dict(gamma_q=g[:64]), dict(gamma_k=g.double()),
                dict(k=k.half()), dict(q=q.double()), dict(q=q.transpose(1, 2)), dict(q=q[0]), dict(k=None),
                dict(out_dtype=torch.float64), dict(qr=q, kr=k[:3]), dict(qr=q, out_dtype=torch.float16),
                dict(qr=q[:1].expand(6, 4, 128)), dict(kr=torch.zeros(400, dtype=torch.bfloat16).as_strided((6, 2, 128), (8, 4, 1)))):
        with pytest.raises(TypeError):
            ga.zgcm_qk_norm_rope_fwd(**dict(ok, **bad))
    with pytest.raises(TypeError, match="CUDA"):
        ga.zgcm_qk_norm_rope_fwd(**ok)
    okb = dict(ok, dqr=q, dkr=k)
    grads = dict(dq=q, dk=k, dgamma_q=g, dgamma_k=g)
    for bad in (dict(dkr=k.half()), dict(dqr=q[:, :2]), dict(dqr=None), dict(grads=dict(grads, dq=q.float())),
                dict(grads=dict(grads, dgamma_k=g[:2])), dict(workspace=torch.zeros(4))):
        with pytest.raises(TypeError):
            ga.zgcm_qk_norm_rope_bwd(**dict(okb, **bad))
    with pytest.raises(TypeError, match="CUDA"):
        ga.zgcm_qk_norm_rope_bwd(**okb, grads=grads)


def _oracle_ops():
    def fwd(q, k, gq, gk, pos, *, out_dtype, **kw):
        return tuple(torch.from_numpy(qkrope.forward(x, g, pos, **kw)).to(out_dtype) for x, g in ((q, gq), (k, gk)))

    def bwd(q, k, gq, gk, pos, dqr, dkr, **kw):
        dq, dgq = qkrope.backward(q, gq, pos, dqr, **kw)
        dk, dgk = qkrope.backward(k, gk, pos, dkr, **kw)
        return {n: torch.from_numpy(x) for n, x in dict(dq=dq, dk=dk, dgamma_q=dgq, dgamma_k=dgk).items()}

    return fwd, bwd


def test_autograd_gradients_by_differences():
    torch.manual_seed(1)
    x = [torch.randn(2, 3, h, 8, dtype=torch.float64, requires_grad=True) for h in (2, 1)]
    g = [(torch.rand(8, dtype=torch.float64) + 0.5).requires_grad_() for _ in range(2)]
    f = lambda *a: zgcm_qk_norm_rope(*a, rope_dims=6, rope_base=50.0, eps=1e-3, ops=_oracle_ops())  # noqa: E731
    assert torch.autograd.gradcheck(f, (*x, *g))
    qr, kr = f(*x, *g)
    assert qr.shape == x[0].shape and kr.shape == x[1].shape
    np.testing.assert_array_equal(qr[1].detach().numpy(), qkrope.forward(x[0][1], g[0], [0, 1, 2], 6, 50.0, 1e-3))
    with pytest.raises(TypeError):
        zgcm_qk_norm_rope(x[0][0], x[1][0], *g)
    with pytest.raises(TypeError):
        zgcm_qk_norm_rope(x[0], x[1][:1], *g)


# ---------------------------------------------------------------------------------- GPU

gpu = pytest.mark.gpu


@pytest.fixture()
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ga.load()


def _inputs(T, Hq, Hkv, xt, yt, seed=0, far=300000):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((T, Hq, 128), generator=g) * torch.exp(torch.randn((T, Hq, 1), generator=g))
    k = torch.randn((T, Hkv, 128), generator=g) * 0.1
    d = [torch.randn((T, h, 128), generator=g).to(DT[yt]) for h in (Hq, Hkv)]
    gam = [torch.rand(128, generator=g) * 2 - 0.5 for _ in range(2)]
    pos = torch.randint(-5, far, (T,), generator=g, dtype=torch.int32)
    return q.to(DT[xt]), k.to(DT[xt]), *gam, pos, *d


def _half(dtype):
    return torch.finfo(dtype).eps / 2, (2.0 ** -25 if dtype == torch.float16 else 0.0)


def _near(name, got, ref, mag, dtype, extra):
    rel, sub = _half(dtype)
    got = got.double().cpu().numpy()
    err = np.abs(got - ref) - (rel * np.abs(ref) * (1 + 2.0 ** -10) + sub + extra * mag)
    assert np.isfinite(got).all() and (err <= 0).all(), (name, float(err.max()))


def _partner(a, R):
    h, b = R // 2, a.copy()
    b[..., :h], b[..., h:2 * h] = a[..., h:2 * h], a[..., :h]
    return b


def _check_fwd(x, gamma, pos, R, got, dtype):
    ref = qkrope.forward(x, gamma, pos, rope_dims=R)
    flat = np.abs(qkrope.forward(x, gamma, pos, rope_dims=0))
    _near("y", got, ref, flat + _partner(flat, R), dtype, 2.0 ** -19)


def _check_bwd(x, gamma, pos, dy, R, dx, dgamma, dtype):
    rdx, rdg = qkrope.backward(x, gamma, pos, dy, rope_dims=R)
    xd, gd, dyd = (np.abs(t.double().numpy()) for t in (x, gamma, dy))
    rms = np.sqrt((xd * xd).mean(-1, keepdims=True) + 1e-6)
    u = (dyd + _partner(dyd, R))
    w = u * gd
    _near("dx", dx, rdx, w / rms + xd * (w * xd).mean(-1, keepdims=True) / rms ** 3, dtype, 2.0 ** -18)
    T, H = x.shape[:2]
    mag = (u * xd / rms).sum((0, 1))
    chain = -(-T // 592) * H + 98
    err = np.abs(dgamma.double().cpu().numpy() - rdg)
    assert (err <= (2.0 ** -19 + chain * 2.0 ** -24) * mag).all(), float((err / mag).max())


@gpu
@pytest.mark.parametrize("T,Hq,Hkv,R,xt,yt", [
    (1, 32, 8, 42, "bf16", "bf16"), (1, 1, 1, 42, "bf16", "fp16"), (5, 3, 1, 128, "fp16", "fp16"),
    (67, 32, 8, 42, "bf16", "fp16"), (700, 5, 2, 0, "bf16", "bf16"), (595, 12, 1, 2, "fp32", "fp32"),
    (1203, 16, 2, 42, "fp32", "bf16"), (2401, 4, 4, 64, "fp16", "fp32"), (130, 32, 8, 126, "fp16", "bf16"), (5003, 4, 2, 42, "bf16", "bf16"), (8001, 3, 1, 42, "fp16", "bf16"),
    (7500, 1, 2, 40, "fp32", "fp32"),
])
def test_against_oracle(cuda, T, Hq, Hkv, R, xt, yt):
    q, k, gq, gk, pos, dqr, dkr = _inputs(T, Hq, Hkv, xt, yt, seed=T)
    d = [t.cuda() for t in (q, k, gq, gk, pos)]
    qr, kr = ga.zgcm_qk_norm_rope_fwd(*d, rope_dims=R, out_dtype=DT[yt])
    assert qr.dtype == kr.dtype == DT[yt]
    _check_fwd(q, gq, pos, R, qr, DT[yt])
    _check_fwd(k, gk, pos, R, kr, DT[yt])
    gr = ga.zgcm_qk_norm_rope_bwd(*d, dqr.cuda(), dkr.cuda(), rope_dims=R)
    _check_bwd(q, gq, pos, dqr, R, gr["dq"], gr["dgamma_q"], DT[xt])
    _check_bwd(k, gk, pos, dkr, R, gr["dk"], gr["dgamma_k"], DT[xt])
    again = ga.zgcm_qk_norm_rope_bwd(*d, dqr.cuda(), dkr.cuda(), rope_dims=R)
    assert all(torch.equal(gr[n], again[n]) for n in gr)


@gpu
def test_packed_projection_in_place(cuda):
    """q and k as columns of one [T, (2 Hq + 2 Hkv) D] projection, outputs and gradients into
    another, a head order other than the natural one; the columns beside them stay as they were."""
    T, Hq, Hkv = 77, 4, 2
    q, k, gq, gk, pos, dqr, dkr = _inputs(T, Hq, Hkv, "bf16", "bf16", seed=9)
    buf = torch.full((T, 12, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    views = lambda b: (b[:, 0:8:2], b[:, 9:11])  # noqa: E731   (heads two apart, the others between)
    for v, t in zip(views(buf), (q, k)):
        v.copy_(t)
    dev = [gq.cuda(), gk.cuda(), pos.cuda()]
    out = torch.full_like(buf, 3.0)
    qr, kr = ga.zgcm_qk_norm_rope_fwd(*views(buf), *dev, qr=views(out)[0], kr=views(out)[1])
    plain = ga.zgcm_qk_norm_rope_fwd(q.cuda(), k.cuda(), *dev)
    assert torch.equal(qr, plain[0]) and torch.equal(kr, plain[1])
    keep = [1, 3, 5, 7, 8, 11]
    assert (out[:, keep] == 3.0).all()
    dy, gout = torch.full_like(buf, 5.0), torch.full_like(buf, 3.0)
    for v, t in zip(views(dy), (dqr, dkr)):
        v.copy_(t)
    ref = ga.zgcm_qk_norm_rope_bwd(q.cuda(), k.cuda(), *dev, dqr.cuda(), dkr.cuda())
    gr = dict(dq=views(gout)[0], dk=views(gout)[1], dgamma_q=torch.empty(128, device="cuda"),
              dgamma_k=torch.empty(128, device="cuda"))
    ga.zgcm_qk_norm_rope_bwd(*views(buf), *dev, *views(dy), grads=gr)
    assert all(torch.equal(gr[n], ref[n]) for n in gr) and (gout[:, keep] == 3.0).all()


@gpu
def test_non_finite_rows_stay_alone(cuda):
    q, k, gq, gk, pos, dqr, dkr = _inputs(9, 4, 2, "bf16", "bf16", seed=4)
    clean = ga.zgcm_qk_norm_rope_fwd(q.cuda(), k.cuda(), gq.cuda(), gk.cuda(), pos.cuda())
    q[3, 1, 5], q[7, 2, 100], k[0, 1, 0] = float("nan"), float("inf"), float("-inf")
    d = [t.cuda() for t in (q, k, gq, gk, pos)]
    qr, kr = ga.zgcm_qk_norm_rope_fwd(*d)
    gr = ga.zgcm_qk_norm_rope_bwd(*d, dqr.cuda(), dkr.cuda())
    for got, dx, ref, bad in ((qr, gr["dq"], clean[0], {(3, 1), (7, 2)}), (kr, gr["dk"], clean[1], {(0, 1)})):
        for t, h in np.ndindex(*got.shape[:2]):
            if (t, h) in bad:
                assert not torch.isfinite(got[t, h]).all()
            else:
                assert torch.equal(got[t, h], ref[t, h]) and torch.isfinite(dx[t, h]).all()


@gpu
def test_empty_and_zero_rows(cuda):
    d = [t.cuda() for t in _inputs(3, 2, 1, "bf16", "bf16")]
    q, k, gq, gk, pos, dqr, dkr = d
    qr, kr = ga.zgcm_qk_norm_rope_fwd(q[:0], k[:0], gq, gk, pos[:0])
    assert qr.shape == (0, 2, 128) and kr.shape == (0, 1, 128)
    gr = ga.zgcm_qk_norm_rope_bwd(q[:0], k[:0], gq, gk, pos[:0], dqr[:0], dkr[:0])
    assert not gr["dgamma_q"].any() and not gr["dgamma_k"].any()
    z = torch.zeros_like(q)
    qr, _ = ga.zgcm_qk_norm_rope_fwd(z, k, gq, gk, pos)     # a padded batch's rows: 0 / sqrt(eps)
    assert not qr.any()


@gpu
def test_autograd_on_the_gpu(cuda):
    q, k, gq, gk, pos, dqr, dkr = _inputs(24, 4, 2, "bf16", "bf16", seed=2)
    x = [t.cuda().view(2, 12, *t.shape[1:]).requires_grad_() for t in (q, k)]
    g = [t.cuda().requires_grad_() for t in (gq, gk)]
    qr, kr = zgcm_qk_norm_rope(*x, *g)
    seq = torch.arange(12, dtype=torch.int32).repeat(2)
    _check_fwd(q, gq, seq, 42, qr.detach().view(24, 4, 128), torch.bfloat16)
    torch.autograd.backward((qr, kr), (dqr.cuda().view_as(qr), dkr.cuda().view_as(kr)))
    _check_bwd(q, gq, seq, dqr, 42, x[0].grad.view(24, 4, 128), g[0].grad, torch.bfloat16)
    _check_bwd(k, gk, seq, dkr, 42, x[1].grad.view(24, 2, 128), g[1].grad, torch.bfloat16)
    # a gradient that is one expanded number, and one output that is not used
    qr, kr = zgcm_qk_norm_rope(*x, *g)
    x[0].grad = None
    qr.sum().backward()
    ones = torch.ones_like(q)
    _check_bwd(q, gq, seq, ones, 42, x[0].grad.view(24, 4, 128), qkrope_dgamma(q, gq, seq, ones), torch.bfloat16)


def qkrope_dgamma(q, gq, seq, dy):
    return torch.from_numpy(qkrope.backward(q, gq, seq, dy)[1])


@gpu
def test_autograd_shared_gamma_broadcast_input_and_capture(cuda):
    """One gamma for q and k, one sequence's q broadcast over the batch; then forward and backward in a graph, replayed
    on new inputs."""
    q, k, g, _, _, dqr, dkr = _inputs(24, 4, 2, "fp32", "fp32", seed=3)
    leaves = [q[:12].cuda().requires_grad_(), k.cuda().view(2, 12, 2, 128).requires_grad_(), g.cuda().requires_grad_()]
    dy = [dqr.cuda().view(2, 12, 4, 128), dkr.cuda().view(2, 12, 2, 128)]

    def step():
        y = zgcm_qk_norm_rope(leaves[0].expand(2, 12, 4, 128), leaves[1], leaves[2], leaves[2])
        return torch.autograd.grad(y, leaves, dy)

    got = step()
    seq = torch.arange(12, dtype=torch.int32).repeat(2)
    both = q[:12].repeat(2, 1, 1)
    dq, dgq = qkrope.backward(both, g, seq, dqr)
    dk, dgk = qkrope.backward(k, g, seq, dkr)
    # as in _check_bwd: 2^-18 of the magnitudes of each part, and one more rounding of their sum
    for n, ref, x, d, out in (("dq", dq, both, dqr, got[0]), ("dk", dk, k, dkr, got[1])):
        xd, dyd = np.abs(x.double().numpy()), np.abs(d.double().numpy())
        rms = np.sqrt((xd * xd).mean(-1, keepdims=True) + 1e-6)
        w = (dyd + _partner(dyd, 42)) * np.abs(g.double().numpy())
        mag = w / rms + xd * (w * xd).mean(-1, keepdims=True) / rms ** 3
        if n == "dq":
            ref, mag = ref[:12] + ref[12:], mag[:12] + mag[12:]
        _near(n, out.view(ref.shape), ref, mag, torch.float32, 2.0 ** -17)
    xd = [np.abs(t.double().numpy()) for t in (both, k, dqr, dkr)]
    mag = sum((x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6) * (d + _partner(d, 42))).sum((0, 1))
              for x, d in ((xd[0], xd[2]), (xd[1], xd[3])))
    err = np.abs(got[2].double().cpu().numpy() - dgq - dgk)
    assert (err <= (2.0 ** -19 + 110 * 2.0 ** -24) * mag).all()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    with torch.no_grad():
        leaves[0].mul_(0.5).add_(0.25)
        dy[1].neg_()
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(held, step()):
        assert torch.equal(x, y)


@gpu
def test_graph_replay_and_stream(cuda):
    """Forward and backward captured together, replayed on new inputs and another stream."""
    a, b = ([t.cuda() for t in _inputs(650, 8, 2, "bf16", "bf16", seed=s)] for s in (1, 2))
    st = [t.clone() for t in a]
    ws = torch.empty(ga.zgcm_qk_norm_rope_bwd_workspace_size(650), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ga.zgcm_qk_norm_rope_bwd(*st, workspace=ws)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ga.zgcm_qk_norm_rope_fwd(*st[:5])
        gr = ga.zgcm_qk_norm_rope_bwd(*st, workspace=ws)
    for src in (a, b):
        for t, x in zip(st, src):
            t.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        ref, rg = ga.zgcm_qk_norm_rope_fwd(*src[:5]), ga.zgcm_qk_norm_rope_bwd(*src)
        assert all(torch.equal(m, n) for m, n in zip(y, ref)) and all(torch.equal(gr[n], rg[n]) for n in rg)


@gpu
def test_keys_for_the_decode_cache(cuda):
    """What a prompt leaves in zgcm_attn_decode's 16-bit cache: this operator's fp16 keys.  The decode
    step over them gives the layer forward's row for the next token."""
    from global_attention_b200.synth import make_inputs
    t = {n: x.cuda() for n, x in make_inputs(2, 200, seed=11).items()}
    S = 199
    pos = torch.arange(S, dtype=torch.int32, device="cuda").repeat(2)
    kc = torch.zeros(2, 256, 8, 128, dtype=torch.float16, device="cuda")
    vc = torch.zeros(2, 256, 8, 128, dtype=torch.bfloat16, device="cuda")
    _, kr = ga.zgcm_qk_norm_rope_fwd(t["q"][:, :S].reshape(-1, 32, 128), t["k"][:, :S].reshape(-1, 8, 128), t["gamma_q"],
                                     t["gamma_k"], pos, out_dtype=torch.float16)
    kc[:, :S], vc[:, :S] = kr.view(2, S, 8, 128), t["v"][:, :S]
    at = torch.full((2,), S, dtype=torch.int32, device="cuda")
    out, lse = ga.zgcm_attn_decode(*(t[n][:, S].contiguous() for n in "qkvg"), t["gamma_q"], t["gamma_k"], at, kc, vc,
                                   window=1000)
    ref, ref_lse = ga.zgcm_attn_fwd(t["q"], t["k"], t["v"], t["g"], t["gamma_q"], t["gamma_k"], window=1000)
    from parity_util import assert_bf16_close, assert_lse_close
    assert_bf16_close("out", out, ref[:, S].double().cpu().numpy(), rrms=1e-2)   # two roundings apart
    assert_lse_close("lse", lse, ref_lse[:, :, S].double().cpu().numpy())
