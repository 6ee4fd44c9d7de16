"""Pins of the oracles of the 8-bit cache operators (oracle/qkrope.py, oracle/kv8.py): the layer's own
oracle, finite differences, torch's float8 type and softmax, small cases by hand."""
import numpy as np
import pytest
import torch

import oracle
from global_attention_b200.synth import make_inputs
from oracle import kv8, qkrope


def test_rotation_by_hand():
    """One pair of dims, theta_0 = 1: a quarter turn takes (1, 0) to (0, 1); the rest is untouched."""
    x = np.ones((1, 1, 4)) * np.array([1.0, 0.0, 1.0, 1.0])
    y = qkrope.forward(x, np.ones(4), [np.pi / 2], rope_dims=2, rope_base=10.0, eps=0.0)
    rms = np.sqrt(3 / 4)
    assert np.allclose(y[0, 0], np.array([0, 1, 1, 1]) / rms, atol=1e-15)


@pytest.mark.parametrize("R", [0, 2, 6, 8])
def test_norm_rope_gradients(R):
    rng = np.random.default_rng(R)
    x, g, dy = rng.normal(size=(3, 2, 8)), rng.uniform(0.5, 1.5, 8), rng.normal(size=(3, 2, 8))
    pos, kw = [0, 7, 100000], dict(rope_dims=R, rope_base=500.0, eps=1e-3)
    dx, dg = qkrope.backward(x, g, pos, dy, **kw)
    for at in np.ndindex(*x.shape):
        d = np.zeros_like(x)
        d[at] = 1e-6
        num = ((qkrope.forward(x + d, g, pos, **kw) - qkrope.forward(x - d, g, pos, **kw)) * dy).sum() / 2e-6
        assert abs(num - dx[at]) <= 1e-8 * (1 + abs(num))
    for i in range(8):
        d = np.zeros(8)
        d[i] = 1e-6
        num = ((qkrope.forward(x, g + d, pos, **kw) - qkrope.forward(x, g - d, pos, **kw)) * dy).sum() / 2e-6
        assert abs(num - dg[i]) <= 1e-8 * (1 + abs(num))


def test_norm_rope_is_the_layers_own():
    """With prepared keys and queries put through a plain softmax the layer's oracle comes out."""
    oracle.build()
    t = make_inputs(1, 9, Hq=4, Hkv=2, D=16, seed=3)
    kw = dict(rope_dims=6, rope_base=100.0, eps=1e-4)
    ref, ref_lse = oracle.Problem(t["q"], t["k"], t["v"], t["g"], t["gamma_q"], t["gamma_k"], window=5, **kw,
                                  scale=0.25).forward()
    pos = np.arange(9)
    q = qkrope.forward(t["q"][0], t["gamma_q"], pos, **kw)
    k = qkrope.forward(t["k"][0], t["gamma_k"], pos, **kw)
    for i in range(9):
        out, lse, *_ = kv8.attend(q[i], t["g"][0, i], k[:i + 1], t["v"][0, :i + 1], code="e4m3", window=5, scale=0.25)
        np.testing.assert_allclose(out, np.asarray(ref)[0, i], atol=1e-12)
        np.testing.assert_allclose(lse, np.asarray(ref_lse)[0, :, i], atol=1e-12)


def test_code_grid_is_torchs_float8():
    y = torch.cat([torch.linspace(-448, 448, 20001), torch.linspace(-0.05, 0.05, 20001),
                   torch.arange(0, 256).to(torch.uint8).view(torch.float8_e4m3fn).float().nan_to_num(0.0),
                   # midpoints of neighbours
                   torch.tensor([1.0625, 1.1875, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, -(2.0 ** -10)])])
    got = kv8.code_grid(y.numpy(), "e4m3")
    assert np.array_equal(got, y.to(torch.float8_e4m3fn).double().numpy())
    assert np.array_equal(kv8.code_grid([0.5, 1.5, -2.5, 126.6], "int8"), [0, 2, -2, 127])


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_quantise(code):
    x = np.zeros((64, 4))
    assert kv8.quantise(x, code)[1] == np.float32(2.0 ** -126)
    x[5, 1] = -3.5
    y, s = kv8.quantise(x, code)
    assert y[5, 1] == -kv8.TOP[code] and s == np.float32(3.5) * (np.float32(1) / np.float32(kv8.TOP[code]))
    x[6, 2] = np.inf
    y, s = kv8.quantise(x, code)
    assert np.isnan(s) and not y.any()


def test_attend_reads_codes_and_tail():
    rng = np.random.default_rng(0)
    k, v = rng.normal(size=(130, 1, 8)), rng.normal(size=(130, 1, 8))
    q = rng.normal(size=(2, 8))
    s = kv8.stored(k, "int8")
    assert np.array_equal(s[128:], k[128:]) and not np.array_equal(s[:128], k[:128])
    assert np.abs(s - k).max() <= np.abs(k).max() / 127 * 0.5001
    out, lse, *_ = kv8.attend(q, None, k, v, code="int8", window=10 ** 6)
    x = torch.from_numpy(s[:, 0]) @ torch.from_numpy(q).T * 8 ** -0.5
    np.testing.assert_allclose(lse, torch.logsumexp(x, 0).numpy(), atol=1e-12)
    np.testing.assert_allclose(out, (torch.softmax(x, 0).T @ torch.from_numpy(kv8.stored(v, "int8")[:, 0])).numpy(),
                               atol=1e-12)
    # a list: block 1 and the own block
    one, *_ = kv8.attend(q, None, k, v, code="int8", window=10 ** 6, blocks=[[1, -1]])
    x = x[64:]
    np.testing.assert_allclose(one, (torch.softmax(x, 0).T @ torch.from_numpy(kv8.stored(v, "int8")[64:, 0])).numpy(),
                               atol=1e-12)


def test_select_by_hand():
    mean = np.array([3.0, 1, 5, 1, 4, np.nan, 1])[:, None, None]
    q = np.array([[1.0], [0.5]])
    sel = lambda **kw: kv8.select(q, mean, first_block=10, **kw).tolist()  # noqa: E731
    assert sel(n_select=3, n_first=0, n_last=0) == [[10, 12, 14]]
    assert sel(n_select=4, n_first=0, n_last=0) == [[10, 11, 12, 14]]         # a tie: the lowest block
    assert sel(n_select=3, n_first=1, n_last=1) == [[10, 12, 16]]
    assert sel(n_select=9, n_first=0, n_last=1) == [[10, 11, 12, 13, 14, 15, 16, -1, -1]]
