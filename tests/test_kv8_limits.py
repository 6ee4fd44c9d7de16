"""The 8-bit block cache (include/zgcm_kv8.h) where its arithmetic and its calls are strained.  Against the
oracle of the definition, as tests/test_kv8.py, whose helpers these tests use; tolerances beyond those of that file are
derived at each test.
"""
import ctypes
import threading

import numpy as np
import pytest
import torch

import global_attention_b200 as ga
from oracle import kv8
from test_kv8 import (ALL, KEY, _check_decode, _check_select, _feed, _i32, _means, _new, _queries, _tokens,  # noqa: F401
                      cuda)  # (the fixture)

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("code,key", [("e4m3", "bf16"), ("int8", "fp16")])
@pytest.mark.parametrize("Hq,Hkv,S", [(4, 1, 64), (3, 1, 40), (8, 1, 64), (4, 4, 320), (32, 8, 320), (8, 1, 320), (12, 1, 640),
                                      (4, 1, 33280), (12, 1, 33280)])
def test_outputs_that_cancel(cuda, code, key, Hq, Hkv, S):  # noqa: F811
    """Every other token's score is d higher and its value the other's negative: out = -v tanh(d / 2), a 2^-11th of
    sum p |v| and less, which probabilities of 11 or 16 bits do not give.

    Bound relative to sum p |v|, with p exact to 2^-22 (exp2; its two fp16 halves, or three bf16 parts in the newest
    block): sums on the tensor cores, 2^-23 a step, of a block's 32 keys and 16-key steps, 4 warps and 16 CTAs: within
    2^-19 for the newest block alone, within 2^-17 for the sums of many blocks.  An error of the normaliser is
    one of out itself: 2^-17 of it.  Scores are at most d, their errors 2^-16 d: e below 2^-25."""
    g = torch.Generator().manual_seed(S + Hq)
    k = torch.zeros(1, S, Hkv, 128)
    k[:, 1::2, :, 0] = 1.0
    v = torch.randn(1, 1, Hkv, 128, generator=g).repeat(1, S, 1, 1)
    v[:, 1::2] *= -1
    d = 2.0 ** (-14 + 4 * torch.rand(Hq, generator=g))
    q = torch.zeros(1, Hq, 128)
    q[0, :, 0] = d * 128 ** 0.5
    k, v, q = k.to(KEY[key]), v.to(torch.bfloat16), q.to(KEY[key])
    c = _new(1, -(-S // 64), Hkv, code, key)
    _feed(c, k, v, [S])
    out, lse = ga.zgcm_attn_decode_kv8(c, q.cuda(), None, _i32(S - 1), window=ALL)
    ref, ref_lse, mag, _ = kv8.attend(q[0], None, k[0], v[0], code=code, window=ALL)
    assert (np.abs(ref) <= 2.0 ** -10.9 * mag).all()
    err = np.abs(out[0].double().cpu().numpy() - ref) / (2.0 ** -8 * 1.001 * np.abs(ref) + 2.0 ** (-19 if S <= 64 else -17) * mag)
    assert err.max() <= 1, float(err.max())
    assert (np.abs(lse[0].double().cpu().numpy() - ref_lse) <= 2.0 ** -17 + 2.0 ** -22 * np.abs(ref_lse)).all()


@gpu
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("key", ["bf16", "fp16"])
@pytest.mark.parametrize("S", [400, 33400])
def test_scores_beyond_2_25(cuda, code, key, S):  # noqa: F811
    """Finite keys and queries whose scores pass 2^25 in base 2, where fp32 counts in steps of 4 and more: one key takes
    all, and out is its value as its code stands for it (p is exactly 1: one rounding to bf16, and 2^-20 for the scale and
    the normaliser), lse its score (128 products in fp32: 2^-17, and 2^-22 for scale, base and rounding)."""
    heads, at = 16, [5, 64 + 17, 300, 310]
    g = torch.Generator().manual_seed(S)
    k = torch.full((1, S, 4, 128), -2000.0)
    v = torch.randn(1, S, 4, 128, generator=g).to(torch.bfloat16)
    for h, t in enumerate(at):
        k[0, t, h] = 2000.0
    k = k.to(KEY[key])
    amp = 2.0 ** torch.linspace(25.01, 28, heads) / (128 * 2000.0 * 128 ** -0.5 * np.log2(np.e))
    q = amp.view(1, heads, 1).expand(1, heads, 128).contiguous().to(KEY[key])
    c = _new(1, S // 64 + 1, 4, code, key)
    _feed(c, k, v, [S])
    out, lse = ga.zgcm_attn_decode_kv8(c, q.cuda(), None, _i32(S - 1), window=ALL)
    held_k, held_v = kv8.stored(k[0], code), kv8.stored(v[0], code)
    for h in range(heads):
        t = at[h // 4]
        s = (held_k[t, h // 4] * q[0, h].double().numpy()).sum() * 128 ** -0.5
        assert s * np.log2(np.e) > 2.0 ** 25
        ref, got = held_v[t, h // 4], out[0, h].double().cpu().numpy()
        assert (np.abs(got - ref) <= (2.0 ** -8 * 1.001 + 2.0 ** -20) * np.abs(ref)).all(), (h, got[:4], ref[:4])
        assert abs(float(lse[0, h]) - s) <= (2.0 ** -17 + 2.0 ** -22) * s


@gpu
def test_select_from_two_threads(cuda):  # noqa: F811
    """Contexts of different sizes from two threads at once, each on its own stream: no call may depend on what another one
    has set for the kernel they share."""
    jobs = []
    for blocks in (1100, 16384):
        c = _new(1, blocks, 1, "e4m3", "bf16", garbage=False)
        _means(c, seed=blocks)
        q, pos = _queries(1, 4, "bf16")[0].cuda(), _i32(64 * blocks - 1)
        ref = ga.zgcm_kv8_select(c, q, pos, 8, window=ALL)
        jobs.append((c, q, pos, ref, torch.empty_like(ref), torch.cuda.Stream()))
    torch.cuda.synchronize()
    lib, got = ga.load(), [set(), set()]

    def work(i):
        c, q, pos, _, out, stream = jobs[i]
        q, pos, out = (ctypes.c_void_p(t.data_ptr()) for t in (q, pos, out))
        for _ in range(3000):
            got[i].add(lib.zgcm_kv8_select(ctypes.byref(c._c), q, pos, 4, 2 ** 31 - 1, 8, 1, 1, out,
                                           ctypes.c_void_p(stream.cuda_stream)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert got == [{0}, {0}]
    for _, _, _, ref, out, _ in jobs:
        assert torch.equal(ref, out)


@gpu
def test_slices_of_positions_and_lists(cuda):  # noqa: F811
    """Positions, counts and lists as rows of longer tensors, 4, 8 and 12 bytes past a 16-byte boundary: the same bits as
    tensors of their own, eagerly and in a graph that follows what is written into them; select's out in place."""
    k, v = _tokens(3, 300, 2, "bf16", seed=31)
    q, g = (x.cuda() for x in _queries(3, 4, "bf16"))
    steps = _i32(*[-9] * 3, 0, 0, 0, 299, 280, 299, 299, 299, 299).view(4, 3)
    count = _i32(-9, 300, 281, 300, -9)
    kept = []
    for cut in (lambda t: t, torch.clone):
        c = _new(3, 5, 2, "e4m3", "bf16")
        start, pos, n = cut(steps[1]), cut(steps[2]), cut(count[1:4])
        assert cut is torch.clone or all(x.data_ptr() % 16 for x in (start, pos, n))
        ga.zgcm_kv8_append(c, k.cuda(), v.cuda(), start, count=n)
        lists = torch.full((20,), -9, dtype=torch.int32, device="cuda")
        sel = ga.zgcm_kv8_select(c, q, pos, 3, window=ALL, out=lists[1:19].view(3, 2, 3) if cut is not torch.clone else None)
        if cut is not torch.clone:
            assert sel.data_ptr() == lists.data_ptr() + 4 and lists[0] == lists[-1] == -9
        out = ga.zgcm_attn_decode_kv8(c, q, g, pos, window=ALL, blocks=sel)
        kept.append([sel, *out, c.k_tail.nan_to_num(7.0), c.v_tail.nan_to_num(7.0), c.k_codes.view(torch.uint8)])
        if cut is not torch.clone:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                held = ga.zgcm_attn_decode_kv8(c, q, g, pos, window=ALL)
            for p in (299, 290):
                steps[2] = p
                graph.replay()
                alone = ga.zgcm_attn_decode_kv8(c, q, g, _i32(p, p, p), window=ALL)
                # (as bits: sequence 1 holds 281 tokens, what it reads past them is NaN on both sides)
                assert all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip(held, alone))
            steps[2] = _i32(299, 280, 299)
    assert all(torch.equal(x, y) for x, y in zip(*kept))


@gpu
@pytest.mark.parametrize("n_blocks,window", [(6, ALL), (5, 130)])
def test_rewinding(cuda, n_blocks, window):  # noqa: F811
    """Back to a position of the newest block, and to the first position of earlier ones, other tokens from there on: the cache
    and the attention are those of the sequence as it is then.  (A table of 5 blocks is one more than a window of 130
    touches: it goes back by one.)"""
    k, v = _tokens(2, 330, 2, "bf16", seed=33)
    others = _tokens(2, 330, 2, "bf16", seed=34)
    c = _new(2, n_blocks, 2, "e4m3", "bf16")
    _feed(c, k[:, :270], v[:, :270], [70, 199, 1])
    q, g = _queries(2, 4, "bf16")
    # 270 tokens -> 257 .. 275 (newest block 4), 256 .. 260 (its first position), 192 .. 240 (a block earlier), 200 .. 310
    for start, end in ((257, 275), (256, 260), (192, 240), (200, 310)):
        k[:, start:end], v[:, start:end] = others[0][:, start:end], others[1][:, start:end]
        _feed(c, k[:, start:end], v[:, start:end], [end - start], start=start)
        _check_decode(c, k[:, :end], v[:, :end], q, g, "e4m3", window=window)


@gpu
@pytest.mark.parametrize("key", ["bf16", "fp16"])
@pytest.mark.parametrize("blocks,near", [(700, 200), (700, 500), (2500, 256), (2500, 1000)])
@pytest.mark.parametrize("G", [1, 12])
def test_select_by_less_than_a_rounding(cuda, key, blocks, near, G):  # noqa: F811
    """`near` blocks whose scores are 2^15 - 2^15 + i 2^-20, which fp32 sums cannot tell apart, the cut in their middle: as
    few as are ranked one by one (256 at most) and more; one of G heads has these scores, the others' are lower."""
    gen = torch.Generator().manual_seed(blocks + near)
    c = _new(1, blocks, 1, "e4m3", key, garbage=False)
    at = torch.randperm(blocks - 1, generator=gen)
    mean = torch.zeros(blocks, 128)
    mean[:, :2] = 2.0 ** 15
    i = torch.arange(near)
    mean[at[:near], 2], mean[at[:near], 3] = (i >> 6) * 2.0 ** -6, (i & 63) * 2.0 ** -6
    mean[at[near:near + 100], 4], mean[at[near + 100:], 4] = 64.0, -64.0
    mean[:, 5] = 1000.0
    c.k_mean[c.table[0].long(), 0] = mean.to(KEY[key]).cuda()
    q = torch.zeros(1, G, 128)
    q[0, :, 5] = -1.0
    q[0, -1, :6] = torch.tensor([1.0, -1.0, 2.0 ** -8, 2.0 ** -14, 1.0, 0.0])
    assert (np.float32(2 ** 15) + (i * 2.0 ** -20).float().numpy() == np.float32(2 ** 15)).all()
    got = _check_select(c, q.to(KEY[key]), [64 * blocks], 100 + near // 2, 0, 0)
    # by hand: the 100 above and the upper half of the near ones
    assert sorted(at[near // 2 + near % 2:near + 100].tolist()) == got[0, 0].tolist()


@gpu
@pytest.mark.parametrize("key", ["bf16", "fp16"])
@pytest.mark.parametrize("blocks", [2048, 5000])
def test_select_of_many_heads_and_blocks(cuda, key, blocks):  # noqa: F811
    """More heads than one round of the scores takes, and more blocks than one CTA does."""
    c = _new(1, blocks, 2, "e4m3", key, garbage=False)
    _means(c, seed=blocks)
    for Hq in (18, 24, 34):
        q, _ = _queries(1, Hq, key, seed=Hq)
        for n, first, last in ((3, 0, 0), (64, 1, 1), (700, 2, 3)):
            _check_select(c, q, [64 * blocks], n, first, last)


@gpu
@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (12, 2)])
@pytest.mark.parametrize("S", [40, 200, 33000])
def test_non_finite_values_of_the_newest_block(cuda, Hq, Hkv, S):  # noqa: F811
    """An infinity or NaN among the values in 16 bits: out is not finite in its dim, for the heads that read it, and as ever
    elsewhere; out of the window, or behind the newest token, it does not matter."""
    k, v = _tokens(1, S, Hkv, "bf16", seed=S)
    q, g = _queries(1, Hq, "bf16")
    clean = v.clone()
    v[0, S - 5, 0, 7], v[0, S - 2, 0, 100], v[0, S - 3, 1, 50] = float("inf"), float("nan"), float("-inf")
    c = _new(1, S // 64 + 1, Hkv, "e4m3", "bf16")
    _feed(c, k, v, [S])
    same = _new(1, S // 64 + 1, Hkv, "e4m3", "bf16")
    _feed(same, k, clean, [S])
    args = q.cuda(), g.cuda(), _i32(S - 1)
    out, lse = ga.zgcm_attn_decode_kv8(c, *args, window=ALL)
    ref, ref_lse = ga.zgcm_attn_decode_kv8(same, *args, window=ALL)
    bad = torch.zeros(1, Hq, 128, dtype=torch.bool, device="cuda")
    bad[:, :Hq // 2, 7] = bad[:, :Hq // 2, 100] = bad[:, Hq // 2:, 50] = True
    assert torch.equal(torch.isfinite(out), ~bad) and torch.equal(out[~bad], ref[~bad]) and torch.equal(lse, ref_lse)
    out, lse = ga.zgcm_attn_decode_kv8(c, *args, window=1)
    ref, ref_lse = ga.zgcm_attn_decode_kv8(same, *args, window=1)
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)


@gpu
def test_slices_on_another_stream(cuda):  # noqa: F811
    """A slice of positions is copied on the call's stream, behind what that stream writes into it."""
    k, v = _tokens(3, 6400, 2, "bf16", seed=35)
    q, g = (x.cuda() for x in _queries(3, 4, "bf16"))
    c = _new(3, 100, 2, "int8", "bf16")
    _feed(c, k, v, [6400])
    ref = ga.zgcm_attn_decode_kv8(c, q, g, _i32(6399, 6399, 6399), window=ALL)
    steps, side = _i32(*[-1] * 7), torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(4):
            busy = busy @ busy * 1e-3
        steps.fill_(6399)
    out = ga.zgcm_attn_decode_kv8(c, q, g, steps[3:6], window=ALL, stream=side)
    sel = ga.zgcm_kv8_select(c, q, steps[3:6], 5, window=ALL, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(out, ref)) and (sel >= 0).all()
