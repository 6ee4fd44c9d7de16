"""The 8-bit block cache (include/zgcm_kv8.h): append, decode attention, block selection.  Argument
checks on the CPU, results on the B200 against the oracle of the definition (oracle/kv8.py).

Tolerances, from the arithmetic.  Codes, scales and tails: none (the definition's fp32 steps
are the kernel's).  Block means: fp32 sums of 64 (20 additions deep, 2^-24 each) and one
rounding to the keys' type.  Attention, u = 2^-24:
a score is an fp32 sum of 128 products, 128u of the sum of their magnitudes at most, times fp32 scales (4u), so each
probability is off by a factor within e = 2^-16 sum |q k| scale at most (its own error and the normaliser's), exp2 by
2^-22; a score's rounding in base 2 adds 2^-24 |s|, covered by the same bound; sums of up to 2^16 keys in tiles and partial
records 2^-17.  A block's p enters the second product as fp16, 2^-11 of it off, or, below fp16's normal numbers, half their
step: p 2^14 is relative to its block's largest, so 2^-25 / 2^14 = 2^-39 of that for each of 64 keys, 2^-33 of the block's p
times its largest |v|.  The output is rounded once to bf16 (2^-8 of the value).  Together
2^-8 |ref| + (2 e + 2^-11 + 2^-15) sum p |v| + 2^-33 sum of blocks' p max |v|.  lse: e + 2^-17 + 2^-22 |lse|.
Selected blocks: equal.
"""
import ctypes
import types

import numpy as np
import pytest
import torch

import global_attention_b200 as ga
from global_attention_b200.build import build
from oracle import kv8

P0 = 0x7F0000000000
CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
KEY = {"bf16": torch.bfloat16, "fp16": torch.float16}
ALL = 2 ** 40


# ------------------------------------------------------------------------------ CPU: refusals

@pytest.fixture(scope="module")
def lib():
    build()
    return ga.load()


def _cache(bad=None, ptr=0, **kw):
    names = ga.ZgcmKv8Cache._NAMES
    a = dict({n: P0 + 4096 * i for i, n in enumerate(names)}, n_seq=2, n_blocks=4, n_pages=8, Hkv=2, D=128, code_type=0,
             key_type=0)
    a.update(kw)
    if bad is not None:
        a[bad] = ptr
    return ctypes.byref(ga._Kv8Struct(*(a[n] for n, _ in ga._Kv8Struct._fields_)))


vp = ctypes.c_void_p


def _append(lib, cache=None, ptrs=None, strides=(256,) * 6, N=3):
    k, v, pos, count = (P0 + 2 ** 20 + 4096 * i for i in range(4)) if ptrs is None else ptrs
    return lib.zgcm_kv8_append(_cache() if cache is None else cache, vp(k), *strides[:3], vp(v), *strides[3:], vp(pos), vp(count), N, None)


def _decode(lib, cache=None, bad=None, ptr=0, n_list=0, Hq=8, window=128, scale=0.1, ws=None):
    p = [P0 + 2 ** 20 + 4096 * i for i in range(6)]   # q, g, pos, blocks, out, lse
    if bad is not None:
        p[bad] = ptr
    w, wb = (P0 + 2 ** 24, 2 ** 30) if ws is None else ws
    return lib.zgcm_attn_decode_kv8(_cache() if cache is None else cache, *(vp(x) for x in p[:4]), n_list, Hq, window, scale,
                                    *(vp(x) for x in p[4:]), vp(w), wb, None)


def _select(lib, cache=None, bad=None, ptr=0, Hq=8, window=128, n=4, first=1, last=1):
    p = [P0 + 2 ** 20 + 4096 * i for i in range(3)]
    if bad is not None:
        p[bad] = ptr
    return lib.zgcm_kv8_select(_cache() if cache is None else cache, vp(p[0]), vp(p[1]), Hq, window, n, first, last, vp(p[2]), None)


@pytest.mark.parametrize("call", [_append, _decode, _select])
def test_refuses_caches(lib, call):
    for kw, st in ((dict(n_seq=-1), -1), (dict(n_blocks=0), -1), (dict(n_pages=0), -1), (dict(Hkv=0), -1),
                   (dict(code_type=2), -1), (dict(key_type=2), -1), (dict(D=64), -2), (dict(D=0), -1),
                   (dict(n_pages=2 ** 24, Hkv=2), -2), (dict(n_seq=65536), -2)):
        assert call(lib, _cache(**kw)) == st, kw
    for n in ga.ZgcmKv8Cache._NAMES:
        assert call(lib, _cache(bad=n, ptr=0)) == -1
        assert call(lib, _cache(bad=n, ptr=P0 + 8)) == -3
    assert call(lib, ctypes.POINTER(ga._Kv8Struct)()) == -1


def test_refuses_append(lib):
    good = [P0 + 2 ** 20 + 4096 * i for i in range(4)]
    for i in range(4):
        p = list(good)
        p[i] = 0
        if i < 3:
            assert _append(lib, ptrs=p) == -1
        p[i] = good[i] + 8
        assert _append(lib, ptrs=p) == -3
    for i in range(6):
        s = [256] * 6
        s[i] = 260
        assert _append(lib, strides=s) == -3
    assert _append(lib, N=-1) == -1
    assert _append(lib, N=0) == 0 and _append(lib, _cache(n_seq=0)) == 0   # nothing to do, nothing launched


def test_refuses_decode(lib):
    for i in range(6):
        if i not in (1, 3):
            assert _decode(lib, bad=i, ptr=0) == -1
        assert _decode(lib, bad=i, ptr=P0 + 4) == -3
    for kw in (dict(Hq=0), dict(Hq=7), dict(window=0), dict(scale=0.0), dict(scale=float("nan")), dict(n_list=-1)):
        assert _decode(lib, ws=(P0, 2 ** 40), **kw) == -1, kw
    # many blocks (150000 tokens of two sequences, or a list of that many): records of 2 x 2 items and 592 CTAs, 4 heads
    size = lib.zgcm_attn_decode_kv8_workspace_size
    big, need = dict(n_blocks=2400), (2 * 2 + 592) * 4 * 132 * 4
    assert size(_cache(**big), 8, 10 ** 6, -1) == size(_cache(), 8, 128, 2400) == need
    for kw in (dict(cache=_cache(**big), window=10 ** 6), dict(n_list=2400)):
        if "n_list" not in kw:
            kw.update(bad=3, ptr=0)   # no list
        assert _decode(lib, ws=(P0, need - 1), **kw) == -4 and _decode(lib, ws=(0, need), **kw) == -4
        assert _decode(lib, ws=(P0 + 8, need), **kw) == -3
    # few blocks by the window, by the list or by the table: none
    assert size(_cache(**big), 8, 128, -1) == size(_cache(**big), 8, 10 ** 6, 32) == size(_cache(), 8, 10 ** 6, -1) == 0
    assert size(_cache(**big), 7, 10 ** 6, -1) == size(_cache(n_seq=0, **big), 8, 10 ** 6, -1) == 0
    assert _decode(lib, _cache(n_seq=0)) == 0


def test_refuses_select(lib):
    for i in range(3):
        assert _select(lib, bad=i, ptr=0) == -1
        assert _select(lib, bad=i, ptr=P0 + 4) == -3
    for kw in (dict(Hq=0), dict(Hq=7), dict(window=0), dict(n=0), dict(first=-1), dict(last=-1), dict(first=3, last=2),
               dict(first=2 ** 31 - 1, last=2 ** 31 - 1)):
        assert _select(lib, **kw) == -1, kw
    assert _select(lib, _cache(n_blocks=16385)) == -2
    assert _select(lib, _cache(n_seq=0)) == 0


def _cpu_tensors(code="e4m3", key="bf16", P=8, Hkv=2, B=2, NB=4):
    z = lambda t, *s: torch.zeros(s, dtype=t)  # noqa: E731
    codes = [z(torch.uint8, P, Hkv, 64, 128).view(CODE[code]) for _ in range(2)]
    return dict(k_codes=codes[0], v_codes=codes[1], k_scale=z(torch.float32, P, Hkv), v_scale=z(torch.float32, P, Hkv),
                k_mean=z(KEY[key], P, Hkv, 128), k_tail=z(KEY[key], B, Hkv, 64, 128),
                v_tail=z(torch.bfloat16, B, Hkv, 64, 128), table=z(torch.int32, B, NB))


def test_binding_refuses(monkeypatch):
    class NoLib:
        def __getattr__(self, name):
            raise AssertionError(f"reached the library ({name})")

    monkeypatch.setattr(ga, "load", lambda: NoLib())
    t = _cpu_tensors()
    for n, x in t.items():
        for bad in (x[..., :1], x[:-1] if n != "table" else x.long(), x.double() if x.dtype != torch.float8_e4m3fn else x.float(), None):
            with pytest.raises(TypeError):
                ga.ZgcmKv8Cache(**dict(t, **{n: bad}))
    with pytest.raises(TypeError, match="CUDA"):
        ga.ZgcmKv8Cache(**t)
    with pytest.raises(TypeError):
        ga.zgcm_kv8_alloc(1, 1, 1, code_dtype=torch.uint8, device="cpu")
    with pytest.raises(TypeError):
        ga.zgcm_kv8_alloc(1, 1, 1, key_dtype=torch.float32, device="cpu")
    # the calls, with a cache whose tensors pass for CUDA ones
    monkeypatch.setattr(ga, "_one_device", lambda *a: None)
    c = ga.ZgcmKv8Cache(**t)
    with pytest.raises(AttributeError):
        c.table = t["table"].clone()
    with pytest.raises(AttributeError):
        c.no_such_tensor
    bf = dict(dtype=torch.bfloat16)
    k, pos = torch.zeros(2, 3, 2, 128, **bf), torch.zeros(2, dtype=torch.int32)
    ok = dict(cache=c, k=k, v=k, pos=pos)
    for bad in (dict(cache=None), dict(k=k.half()), dict(v=k.half()), dict(v=k[:, :2]), dict(k=k[:, :, :1]), dict(k=k[0]),
                dict(k=k.transpose(2, 3)), dict(pos=pos[:1]), dict(pos=pos.long()), dict(count=pos[:1]), dict(k=None)):
        with pytest.raises(TypeError):
            ga.zgcm_kv8_append(**dict(ok, **bad))
    with pytest.raises(TypeError, match="CUDA"):
        ga.zgcm_kv8_append(**ok)
    q = torch.zeros(2, 8, 128, **bf)
    bl = torch.zeros(2, 2, 5, dtype=torch.int32)
    ok = dict(cache=c, q=q, g=q, pos=pos, blocks=bl)
    for bad in (dict(cache=t), dict(q=q.half()), dict(q=q[:1]), dict(q=q[0]), dict(g=q[:, :4]), dict(pos=pos.float()),
                dict(blocks=bl[0]), dict(blocks=bl.long()), dict(blocks=bl[:, :1]), dict(out=q.float()), dict(lse=q)):
        with pytest.raises(TypeError):
            ga.zgcm_attn_decode_kv8(**dict(ok, **bad))
    with pytest.raises(TypeError, match="CUDA"):
        ga.zgcm_attn_decode_kv8(**ok)
    for bad in (dict(cache=t), dict(q=q.half()), dict(q=q[0]), dict(pos=pos[:1]), dict(out=bl)):
        with pytest.raises(TypeError):
            ga.zgcm_kv8_select(**dict(dict(cache=c, q=q, pos=pos, n_select=4), **bad))
    with pytest.raises(TypeError, match="CUDA"):
        ga.zgcm_kv8_select(c, q, pos, 4)


# ---------------------------------------------------------------------------------- GPU

gpu = pytest.mark.gpu


@pytest.fixture()
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ga.load()


def _tokens(B, S, Hkv, key, seed=0):
    g = torch.Generator().manual_seed(seed)
    k = torch.randn((B, S, Hkv, 128), generator=g) * torch.exp(0.5 * torch.randn((1, 1, Hkv, 128), generator=g))
    v = torch.randn((B, S, Hkv, 128), generator=g) * torch.exp(torch.randn((B, S, Hkv, 1), generator=g))
    return k.to(KEY[key]), v.to(torch.bfloat16)


def _new(B, NB, Hkv, code, key, spare=2, seed=0, garbage=True):
    """A cache with its pages in random order and, everywhere a call may not look, garbage."""
    n = B * NB + spare
    c = ga.zgcm_kv8_alloc(B, NB, Hkv, n_pages=n, code_dtype=CODE[code], key_dtype=KEY[key])
    perm = torch.randperm(n, generator=torch.Generator().manual_seed(seed))[:B * NB]
    c.table.copy_(perm.view(B, NB).to(torch.int32))
    if garbage:
        for t in (c.k_codes, c.v_codes):
            t.view(torch.uint8).fill_(0x7F)     # a NaN as e4m3
        for t in (c.k_scale, c.v_scale, c.k_mean, c.k_tail, c.v_tail):
            t.fill_(float("nan"))
    return c


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _feed(c, k, v, steps, start=0):
    """Append k, v [B, S, Hkv, D] in calls of the given lengths."""
    k, v = k.cuda(), v.cuda()
    at = 0
    for n in steps:
        ga.zgcm_kv8_append(c, k[:, at:at + n], v[:, at:at + n], _i32(*[start + at] * k.shape[0]))
        at += n
    assert at == k.shape[1]


def _check_held(c, k, v, code, lens=None, upto=None):
    """Codes, scales, means and tails of every sequence against the definition.  upto: blocks still in the ring."""
    B, _, Hkv, _ = k.shape
    table = c.table.cpu()
    cpu = {n: getattr(c, n).cpu() for n in ga.ZgcmKv8Cache._NAMES}
    for b in range(B):
        S = k.shape[1] if lens is None else lens[b]
        if S == 0:
            continue
        last = (S - 1) // 64
        for j in range(max(0, last - c.n_blocks + 1), S // 64):
            page = int(table[b, j % c.n_blocks])
            for side, x in (("k", k), ("v", v)):
                for h in range(Hkv):
                    blk = x[b, j * 64:(j + 1) * 64, h]
                    y, s = kv8.quantise(blk, code)
                    got = cpu[side + "_codes"][page, h].float().numpy()
                    assert np.array_equal(got, y), (b, j, side, h)
                    assert np.array_equal(cpu[side + "_scale"][page, h].numpy(), s, equal_nan=True)
                    if side == "k" and np.isfinite(s):
                        x64 = blk.double()
                        m = cpu["k_mean"][page, h].double()
                        tol = torch.finfo(k.dtype).eps / 2 * x64.mean(0).abs() * 1.001 + 20 * 2.0 ** -24 * x64.abs().mean(0)
                        # below the type's normal numbers: half its smallest step
                        tol += 2.0 ** -25 if k.dtype == torch.float16 else 2.0 ** -134
                        assert ((m - x64.mean(0)).abs() <= tol).all()
        n = S - last * 64
        for side, x in (("k", k), ("v", v)):
            assert torch.equal(cpu[side + "_tail"][b, :, :n], x[b, last * 64:S].transpose(0, 1))
            assert n == 64 or torch.isnan(cpu[side + "_tail"][b, :, n:]).all() or last > 0


def _close(name, out, lse, ref, ref_lse, mag, top, q, k, scale):
    """One sequence's rows against the oracle."""
    # sum |q k| by row: |q| . max_j |k_j| element by element over the finite keys (a row that sees another is
    # not compared), with what coding may add to a key (1/16)
    G = len(q) // k.shape[1]
    km = k.double().abs().nan_to_num(0.0, posinf=0.0).amax(0).numpy()
    qk = np.array([(np.abs(q[h].double().numpy()) * km[h // G]).sum() for h in range(len(q))]) * scale * 1.0625
    e = (2.0 ** -16 * qk)[:, None]
    got = out.double().cpu().numpy()
    err = np.abs(got - ref) - (2.0 ** -8 * np.abs(ref) * 1.001 + (2 * e + 2.0 ** -11 + 2.0 ** -15) * mag + 2.0 ** -33 * top[:, None] + 1e-37)
    assert np.isfinite(got).all() and (err <= 0).all(), (name, float(err.max()))
    err = np.abs(lse.double().cpu().numpy() - ref_lse) - (e[:, 0] + 2.0 ** -17 + 2.0 ** -22 * np.abs(ref_lse))
    assert (err <= 0).all(), (name, "lse", float(err.max()))


def _queries(B, Hq, key, seed=5, amp=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((B, Hq, 128), generator=g) * amp).to(KEY[key]), torch.randn((B, Hq, 128), generator=g).to(torch.bfloat16) * 2


def _check_decode(c, k, v, q, g, code, window=ALL, lens=None, blocks=None, scale=None, **kw):
    B, S = k.shape[:2]
    lens = [S] * B if lens is None else lens
    pos = _i32(*[n - 1 for n in lens])
    out, lse = ga.zgcm_attn_decode_kv8(c, q.cuda(), None if g is None else g.cuda(), pos, window=window, scale=scale,
                                       blocks=blocks, **kw)
    for b, n in enumerate(lens):
        if n == 0:
            assert not out[b].any() and torch.isneginf(lse[b]).all()
            continue
        ref = kv8.attend(q[b], None if g is None else g[b], k[b, :n], v[b, :n], code=code, window=window, scale=scale,
                         blocks=None if blocks is None else blocks[b].cpu().numpy())
        _close((b, n), out[b], lse[b], *ref, q[b], k[b, :n], 128 ** -0.5 if scale is None else scale)
    return out, lse


@gpu
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("key", ["bf16", "fp16"])
def test_append_holds_the_definition(cuda, code, key):
    """The same tokens in one call, in uneven prompts, one by one: the same bits, those of the definition."""
    k, v = _tokens(2, 200, 3, key, seed=1)
    k[0, 70, 1] *= 50.0      # a far larger token in one block of one head
    v[1, :64, 2] = 0.0       # a block of zeros
    v[1, 64:128, 0] *= 1e-38
    kept = None
    for steps in ([200], [1] * 200, [70, 1, 57, 64, 8], [64, 64, 64, 8], [3, 130, 67]):
        c = _new(2, 4, 3, code, key)
        _feed(c, k, v, steps)
        _check_held(c, k, v, code)
        for b in range(2):
            pages = c.table[b, :3].long()
            now = [getattr(c, n)[pages] for n in ("k_codes", "v_codes", "k_scale", "v_scale", "k_mean")]
            now = [x.view(torch.uint8) if x.element_size() == 1 else x for x in now] + [c.k_tail[b, :, :8], c.v_tail[b, :, :8]]
            kept = kept or {}
            assert all(torch.equal(x, y) for x, y in zip(now, kept.setdefault(b, now)))
        # pages that no block went to keep their bits
        free = [p for p in range(10) if p not in set(c.table[:, :3].flatten().tolist())]
        assert (c.k_codes.view(torch.uint8)[free] == 0x7F).all() and torch.isnan(c.k_scale[free]).all()


@gpu
def test_append_ragged_idle_and_strided(cuda):
    """A padded batch: counts of 0, 1, 63 .. 130, an idle sequence, rows past the count NaN; k and v as
    columns of one packed tensor."""
    lens = [0, 1, 63, 64, 65, 128, 130, 7]
    k, v = _tokens(8, 130, 2, "bf16", seed=2)
    packed = torch.full((8, 130, 7, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    for b, n in enumerate(lens):
        packed[b, :n, 1:3], packed[b, :n, 3:7:2] = k[b, :n].cuda(), v[b, :n].cuda()
    c = _new(8, 3, 2, "e4m3", "bf16")
    ga.zgcm_kv8_append(c, packed[:, :, 1:3], packed[:, :, 3:7:2], _i32(*[0] * 7, -1), count=_i32(*lens))
    lens[7] = 0              # idle
    _check_held(c, k, v, "e4m3", lens)
    assert torch.isnan(c.k_tail[7]).all() and torch.isnan(c.k_tail[0]).all()
    q, g = _queries(8, 4, "bf16")
    _check_decode(c, k, v, q, g, "e4m3", lens=lens)
    # counts out of range are the nearer bound
    c2 = _new(8, 3, 2, "e4m3", "bf16")
    ga.zgcm_kv8_append(c2, k.cuda(), v.cuda(), _i32(*[0] * 8), count=_i32(500, -3, *[130] * 6))
    _check_held(c2, k, v, "e4m3", [130, 0] + [130] * 6)
    assert torch.isnan(c2.k_tail[1]).all()


@gpu
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (4, 2), (6, 2), (32, 8), (5, 1), (8, 1), (12, 1), (16, 1), (33, 3)])
@pytest.mark.parametrize("code,key", [("e4m3", "fp16"), ("int8", "bf16")])
def test_decode_head_layouts(cuda, Hq, Hkv, code, key):
    k, v = _tokens(2, 331, Hkv, key, seed=Hq)
    c = _new(2, 6, Hkv, code, key)
    _feed(c, k, v, [331])
    q, g = _queries(2, Hq, key)
    _check_decode(c, k, v, q, g, code)
    _check_decode(c, k, v, q, None, code, window=100, scale=0.3)


@gpu
@pytest.mark.parametrize("code,key", [("e4m3", "bf16"), ("int8", "fp16")])
def test_decode_lengths(cuda, code, key):
    """One token to thousands, around every block border, in one ragged batch; an idle sequence."""
    lens = [1, 2, 17, 63, 64, 65, 127, 128, 129, 191, 192, 193, 640, 0, 1000, 4097]
    k, v = _tokens(len(lens), max(lens), 2, key, seed=3)
    c = _new(len(lens), 65, 2, code, key)
    ga.zgcm_kv8_append(c, k.cuda(), v.cuda(), _i32(*[0] * len(lens)), count=_i32(*lens))
    q, g = _queries(len(lens), 8, key)
    _check_decode(c, k, v, q, g, code, lens=lens)
    for window in (1, 64, 65, 128, 700):
        _check_decode(c, k, v, q, g, code, lens=lens, window=window)


@gpu
@pytest.mark.parametrize("code,key", [("e4m3", "fp16"), ("int8", "bf16")])
@pytest.mark.parametrize("B,Hq,Hkv,longest", [(1, 4, 1, 40000), (1, 4, 1, 30000), (2, 8, 2, 9000), (3, 12, 1, 36000), (90, 8, 2, 4700), (300, 1, 1, 4500)])
def test_decode_long_and_many(cuda, code, key, B, Hq, Hkv, longest):
    """Contexts of hundreds of blocks, and more sequences than an SM count: runs that begin and end inside
    sequences, short ones among long ones, idle ones."""
    g0 = torch.Generator().manual_seed(B)
    lens = torch.randint(0, longest + 1, (B,), generator=g0).tolist()
    lens[0] = longest
    for b in range(3, B, 7):
        lens[b] = (0, 1, 64, 65, 130)[b % 5]
    k, v = _tokens(min(B, 4), longest, Hkv, key, seed=B)
    src = [b % 4 for b in range(B)]
    c = _new(B, longest // 64 + 1, Hkv, code, key)
    ga.zgcm_kv8_append(c, k.cuda()[src], v.cuda()[src], _i32(*[0] * B), count=_i32(*lens))
    q, g = _queries(B, Hq, key)
    pos = _i32(*[n - 1 for n in lens])
    out, lse = ga.zgcm_attn_decode_kv8(c, q.cuda(), g.cuda(), pos, window=ALL)
    again = ga.zgcm_attn_decode_kv8(c, q.cuda(), g.cuda(), pos, window=ALL)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    for b in sorted({0, 1, 2, 3, 10, 17, B // 2, B - 2, B - 1} & set(range(B))):
        if lens[b] == 0:
            assert not out[b].any() and torch.isneginf(lse[b]).all()
            continue
        x, y = k[src[b], :lens[b]], v[src[b], :lens[b]]
        _close((b, lens[b]), out[b], lse[b], *kv8.attend(q[b], g[b], x, y, code=code, window=ALL), q[b], x, 128 ** -0.5)
    assert torch.isfinite(out).all()
    assert ga.zgcm_attn_device_error() == 0


@gpu
def test_decode_every_step_of_a_ring(cuda):
    """A sliding layer: three blocks for each sequence, 300 single tokens after a prompt longer than the
    ring, sequences a block border apart; every step against the definition."""
    B, S, W, first = 2, 560, 128, [250, 231]
    k, v = _tokens(B, S, 2, "fp16", seed=8)
    c = _new(B, 3, 2, "e4m3", "fp16", garbage=True)
    kd, vd = k.cuda(), v.cuda()
    ga.zgcm_kv8_append(c, kd[:, :250], vd[:, :250], _i32(0, 0), count=_i32(*first))
    q, g = _queries(B, 8, "fp16")
    for i in range(300):
        at = [f + i for f in first]
        ga.zgcm_kv8_append(c, torch.stack([kd[b, p:p + 1] for b, p in enumerate(at)]),
                           torch.stack([vd[b, p:p + 1] for b, p in enumerate(at)]), _i32(*at))
        if i % 7 == 0 or any(p % 64 in (0, 62, 63) for p in at):
            _check_decode(c, k, v, q, g, "e4m3", window=W, lens=[p + 1 for p in at])
    # a window the ring cannot hold: NaN, for the rows it concerns alone
    out, lse = ga.zgcm_attn_decode_kv8(c, q.cuda(), g.cuda(), _i32(at[0], -1), window=200)
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all() and not out[1].any()
    sel = ga.zgcm_kv8_select(c, q.cuda(), _i32(at[0], -1), 4, window=200)
    assert (sel == -1).all()


@gpu
def test_prompt_longer_than_the_ring(cuda):
    """Blocks that the same call would overwrite are not stored (two blocks, one page, no order)."""
    for n in (63, 64, 192, 256, 1000, 1024):
        k, v = _tokens(1, n, 2, "bf16", seed=n)
        c = _new(1, 3, 2, "int8", "bf16")
        _feed(c, k, v, [n])
        _check_held(c, k, v, "int8")
        q, g = _queries(1, 4, "bf16")
        _check_decode(c, k, v, q, g, "int8", window=129)


@gpu
@pytest.mark.parametrize("Hq", [8, 16])
def test_decode_block_lists(cuda, Hq):
    k, v = _tokens(3, 700, 2, "bf16", seed=6)
    lens = [700, 641, 100]
    c = _new(3, 11, 2, "e4m3", "bf16")
    ga.zgcm_kv8_append(c, k.cuda(), v.cuda(), _i32(0, 0, 0), count=_i32(*lens))
    q, g = _queries(3, Hq, "bf16")
    lists = [[[0, 3, 9, -1], [-1, -1, -1, -1]], [[1, 2, 3, 4], [9, -1, -1, -1]], [[0, -1, -1, -1], [-1, -1, -1, -1]]]
    _check_decode(c, k, v, q, g, "e4m3", lens=lens, blocks=_i32(*np.ravel(lists)).view(3, 2, 4))
    _check_decode(c, k, v, q, g, "e4m3", lens=lens, blocks=torch.zeros(3, 2, 0, dtype=torch.int32, device="cuda"))
    # passed over: the own block and later ones, negative ones, what is not above the entry before, blocks
    # wholly before the window
    odd = [[[3, 3, 10, 99], [5, 4, 4, 6]], [[-7, 2, 2 ** 31 - 1, 2], [0, 10, 9, 9]], [[0, 0, 1, 2], [1, 1, 1, 1]]]
    same = [[[3, -1, -1, -1], [5, 6, -1, -1]], [[2, -1, -1, -1], [0, -1, -1, -1]], [[0, -1, -1, -1], [-1, -1, -1, -1]]]
    a = ga.zgcm_attn_decode_kv8(c, q.cuda(), g.cuda(), _i32(*[n - 1 for n in lens]), window=ALL,
                                blocks=_i32(*np.ravel(odd)).view(3, 2, 4))
    _check_decode(c, k, v, q, g, "e4m3", lens=lens, blocks=_i32(*np.ravel(same)).view(3, 2, 4))
    for b in range(3):
        ref = kv8.attend(q[b], g[b], k[b, :lens[b]], v[b, :lens[b]], code="e4m3", window=ALL, blocks=same[b])
        _close(b, a[0][b], a[1][b], *ref, q[b], k[b, :lens[b]], 128 ** -0.5)
    # with a window the list's block 3 (rows up to 255) is out of reach, block 9 is read in part
    few = _i32(*np.ravel([[[3, 9], [9, -1]]] * 3)).view(3, 2, 2)
    _check_decode(c, k, v, q, g, "e4m3", lens=lens, blocks=few, window=90)


@gpu
def test_bad_pages(cuda):
    """Page numbers outside the cache: no access, NaN for the rows whose blocks they are."""
    k, v = _tokens(3, 300, 2, "bf16", seed=7)
    c = _new(3, 5, 2, "int8", "bf16")
    good = c.table.clone()
    c.table[1, 2], c.table[2, 0] = -1, c.n_pages
    _feed(c, k, v, [300])
    q, g = _queries(3, 4, "bf16")
    pos = _i32(299, 299, 299)
    out, lse = ga.zgcm_attn_decode_kv8(c, q.cuda(), g.cuda(), pos, window=ALL)
    assert torch.isnan(out[1:]).all() and torch.isnan(lse[1:]).all()
    ref = kv8.attend(q[0], g[0], k[0], v[0], code="int8", window=ALL)
    _close(0, out[0], lse[0], *ref, q[0], k[0], 128 ** -0.5)
    # out of the window's reach they do not matter
    _check_decode(c, k, v, q, g, "int8", window=100)
    c.table[0] = 2 ** 31 - 1
    c.table[2] = -2 ** 31
    out, _ = ga.zgcm_attn_decode_kv8(c, q.cuda(), g.cuda(), pos, window=ALL)
    assert torch.isnan(out).all()
    # a bad page's score is the lowest
    c.table.copy_(good)
    c.table[1, 2] = -1
    sel = ga.zgcm_kv8_select(c, q.cuda(), pos, 3, n_first=0, n_last=0, window=ALL)
    assert not (sel[1] == 2).any()


@gpu
@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_non_finite_tokens(cuda, code):
    """A block with a NaN or infinity reads as NaN for its head; heads beside it, later windows and a tail's
    rows past the newest token are not touched by it."""
    k, v = _tokens(1, 290, 3, "bf16", seed=9)
    k[0, 70, 0, 3], v[0, 80, 1, 127] = float("nan"), float("inf")
    c = _new(1, 5, 3, code, "bf16")
    _feed(c, k, v, [290])
    _check_held(c, k, v, code)
    q, g = _queries(1, 6, "bf16")
    out, lse = ga.zgcm_attn_decode_kv8(c, q.cuda(), g.cuda(), _i32(289), window=ALL)
    assert torch.isnan(out[0, :4]).all() and torch.isnan(lse[0, :2]).all()
    assert torch.isfinite(out[0, 4:]).all() and torch.isfinite(lse[0, 4:]).all()
    _check_decode(c, k, v, q, g, code, window=290 - 128)
    # the other blocks by list
    bl = _i32(0, 2, 3).repeat(3).view(1, 3, 3)
    _check_decode(c, k, v, q, g, code, blocks=bl)


@gpu
def test_extreme_scores_and_values(cuda):
    """Scores far apart (one key takes all), all equal, magnitudes at the ends of the keys' and values' ranges."""
    k, v = _tokens(1, 333, 1, "bf16", seed=10)
    c = _new(1, 6, 1, "int8", "bf16")
    v[0, :64] *= 1e30
    v[0, 64:128] *= 1e-30
    _feed(c, k, v, [333])
    for amp in (0.0, 1e-30, 1.0, 60.0, 1e4):
        q, g = _queries(1, 4, "bf16", amp=amp)
        _check_decode(c, k, v, q, g, "int8")
    k2, v2 = _tokens(1, 333, 1, "bf16", seed=11)
    k2 = k2 * 1e15
    c2 = _new(1, 6, 1, "e4m3", "bf16")
    _feed(c2, k2, v2, [333])
    q, g = _queries(1, 4, "bf16", amp=1e-15)
    _check_decode(c2, k2, v2, q, g, "e4m3")
    g[:] = float("inf")      # an open and a shut gate
    g[:, 1] = float("-inf")
    out, _ = ga.zgcm_attn_decode_kv8(c2, q.cuda(), g.cuda(), _i32(332), window=ALL)
    ref, *_ = kv8.attend(q[0], None, k2[0], v2[0], code="e4m3", window=ALL)
    assert not out[0, 1].any() and np.abs(out[0, 0].double().cpu().numpy() - ref[0]).max() < 0.05


# ------------------------------------------------------------------------------- selection

def _means(c, seed=0):
    g = torch.Generator().manual_seed(seed)
    c.k_mean.copy_(torch.randn(c.k_mean.shape, generator=g) * 0.2)


def _check_select(c, q, lens, n, first, last, window=ALL):
    sel = ga.zgcm_kv8_select(c, q.cuda(), _i32(*[x - 1 for x in lens]), n, n_first=first, n_last=last, window=window).cpu()
    mean, table = c.k_mean.cpu(), c.table.cpu().long()
    for b, S in enumerate(lens):
        p = S - 1
        lo, own = max(0, p - min(window, S) + 1) // 64, max(p, 0) // 64
        m = mean[table[b, [j % c.n_blocks for j in range(lo, own)]]] if own > lo else mean[:0]
        ref = kv8.select(q[b], m, first_block=lo, n_select=n, n_first=first, n_last=last)
        assert np.array_equal(sel[b].numpy(), ref), (b, S)
    return sel


@gpu
@pytest.mark.parametrize("key", ["bf16", "fp16"])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (32, 8), (12, 1), (5, 1)])
def test_select(cuda, key, Hq, Hkv):
    lens = [0, 1, 64, 65, 640, 1000, 4097, 6400]
    c = _new(len(lens), 101, Hkv, "e4m3", key, garbage=False)
    _means(c)
    q, _ = _queries(len(lens), Hq, key)
    for n, first, last in ((1, 0, 0), (5, 1, 1), (16, 0, 3), (31, 31, 0), (64, 2, 2), (150, 1, 1)):
        _check_select(c, q, lens, n, first, last)
    _check_select(c, q, lens, 7, 1, 2, window=2000)


@gpu
@pytest.mark.parametrize("blocks", [1023, 4096, 16384])
def test_select_long_contexts(cuda, blocks):
    """Up to a million tokens: slices of a cluster, the last digit's ties, few rows."""
    c = _new(1, blocks, 1, "e4m3", "bf16", garbage=False)
    _means(c, seed=blocks)
    q, _ = _queries(1, 4, "bf16")
    for n in (2, 64, 512):
        _check_select(c, q, [blocks * 64], n, 1, 1)


@gpu
@pytest.mark.parametrize("blocks", [700, 1500])
def test_select_ties_and_specials(cuda, blocks):
    c = _new(1, blocks, 2, "e4m3", "bf16", garbage=False)
    q, _ = _queries(1, 4, "bf16")
    c.k_mean.zero_()                                   # every score 0 (and -0)
    _check_select(c, q, [64 * blocks], 9, 1, 1)
    _means(c, seed=3)
    page = c.table[0].long()
    c.k_mean[page[100:400:3]] = c.k_mean[page[5]].clone()      # ties across slices
    c.k_mean[page[17]] = float("nan")
    c.k_mean[page[18], 0, 0] = float("inf")
    c.k_mean[page[19], :, 5] = float("-inf")
    for n in (3, 40, 90, 200, 699):
        _check_select(c, q, [64 * blocks], n, 0, 0)
        _check_select(c, q, [64 * blocks], n, 1, 1)


# ------------------------------------------------------------------- together, streams, graphs

def _step(c, t, s, pos, window, n_select):
    """One token of a layer as a user's program runs it."""
    qr, kr = ga.zgcm_qk_norm_rope_fwd(s["q"], s["k"], t["gamma_q"], t["gamma_k"], pos, out_dtype=c.key_dtype)
    ga.zgcm_kv8_append(c, kr[:, None], s["v"][:, None], pos)
    blocks = ga.zgcm_kv8_select(c, qr, pos, n_select, window=window) if n_select else None
    out, lse = ga.zgcm_attn_decode_kv8(c, qr, s["g"], pos, window=window, blocks=blocks)
    return qr, kr, out, lse, blocks


def _layer(B, S, Hq, Hkv, seed):
    from global_attention_b200.synth import make_inputs
    return make_inputs(B, S, Hq=Hq, Hkv=Hkv, D=128, seed=seed)


@gpu
@pytest.mark.parametrize("n_select", [0, 3])
def test_prompt_then_tokens(cuda, n_select):
    """A prompt through the layer's forward and into the cache, then tokens: every step against the
    definition on the step's own prepared rows, and (nothing left out) near the 16-bit layer."""
    B, S, n0, Hq, Hkv = 2, 460, 390, 8, 2
    t = _layer(B, S, Hq, Hkv, seed=12)
    d = {n: x.cuda() for n, x in t.items()}
    pos = torch.arange(n0, dtype=torch.int32, device="cuda").repeat(B)
    _, kr = ga.zgcm_qk_norm_rope_fwd(d["q"][:, :n0].reshape(-1, Hq, 128), d["k"][:, :n0].reshape(-1, Hkv, 128),
                                     d["gamma_q"], d["gamma_k"], pos, out_dtype=torch.float16)
    c = _new(B, 8, Hkv, "int8", "fp16")
    ga.zgcm_kv8_append(c, kr.view(B, n0, Hkv, 128), d["v"][:, :n0], _i32(0, 0))
    keys = torch.zeros(B, S, Hkv, 128, dtype=torch.float16)
    keys[:, :n0] = kr.view(B, n0, Hkv, 128).cpu()
    dense, _ = ga.zgcm_attn_fwd(d["q"], d["k"], d["v"], d["g"], d["gamma_q"], d["gamma_k"], window=S)
    for p in range(n0, S):
        at = _i32(p, p)
        qr, kr, out, lse, bl = _step(c, d, {n: d[n][:, p].contiguous() for n in "qkvg"}, at, ALL, n_select)
        keys[:, p] = kr.cpu()
        if p % 5 == 0 or p % 64 in (0, 63):
            for b in range(B):
                ref = kv8.attend(qr[b].cpu(), t["g"][b, p], keys[b, :p + 1], t["v"][b, :p + 1], code="int8", window=ALL,
                                 blocks=None if bl is None else bl[b].cpu().numpy())
                _close((p, b), out[b], lse[b], *ref, qr[b].cpu(), keys[b, :p + 1], 128 ** -0.5)
                if not n_select:
                    # int8: a value within amax / 254, a key within amax / 254 in each of 128 products
                    a = t["v"][b].double().abs().max().item() / 254
                    x = qr[b].double().abs().sum(-1).max().item() * keys[b].double().abs().max().item() / 254 * 128 ** -0.5
                    vmax = t["v"][b].double().abs().max().item()
                    assert (out[b].double() - dense[b, p].double()).abs().max() <= a + 2 * np.expm1(2 * x) * vmax + 0.05
    _check_held(c, keys, t["v"], "int8")


@gpu
def test_graphs_follow_positions(cuda):
    """A captured step (append, select, attention) follows positions and inputs written into its buffers; two
    graphs with one workspace, replayed in turn, do not disturb each other."""
    B, Hq, Hkv = 2, 8, 2
    k, v = _tokens(B, 300, Hkv, "bf16", seed=13)
    caches = [_new(B, 6, Hkv, "e4m3", "bf16", seed=s) for s in (0, 1)]
    for c in caches:
        _feed(c, k[:, :190], v[:, :190], [190])
    q, g = _queries(B, Hq, "bf16")
    ws = torch.empty(2 ** 20, dtype=torch.uint8, device="cuda")
    qd, gd, kd, vd = q.cuda(), g.cuda(), k.cuda(), v.cuda()
    st = dict(k=kd[:, 190:191].clone(), v=vd[:, 190:191].clone(), pos=_i32(190, 190))

    def step(c, windowed):
        ga.zgcm_kv8_append(c, st["k"], st["v"], st["pos"])
        bl = None if windowed else ga.zgcm_kv8_select(c, qd, st["pos"], 3, window=ALL)
        return ga.zgcm_attn_decode_kv8(c, qd, gd, st["pos"], window=100 if windowed else ALL, blocks=bl, workspace=ws), bl

    for i, c in enumerate(caches):
        step(c, i == 1)
    torch.cuda.synchronize()
    graphs, got = [], []
    for i, c in enumerate(caches):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(step(c, i == 1))
        graphs.append(graph)
    for p in range(190, 262):
        st["k"].copy_(kd[:, p:p + 1])
        st["v"].copy_(vd[:, p:p + 1])
        st["pos"].fill_(p)
        for graph in graphs:
            graph.replay()
        if p % 16 == 0 or p % 64 in (63, 0):
            for ((out, lse), bl), windowed in zip(got, (False, True)):
                for b in range(B):
                    ref = kv8.attend(q[b], g[b], k[b, :p + 1], v[b, :p + 1], code="e4m3", window=100 if windowed else ALL,
                                     blocks=None if bl is None else bl[b].cpu().numpy())
                    _close((p, b), out[b], lse[b], *ref, q[b], k[b, :p + 1], 128 ** -0.5)


def _one_history(B, S, seed):
    """A cache of B sequences whose tables name the same pages: one history of S tokens, read by all."""
    k, v = _tokens(1, S, 1, "bf16", seed=seed)
    c = _new(B, S // 64 + 1, 1, "e4m3", "bf16", seed=seed)
    ga.zgcm_kv8_append(c, k.cuda().expand(B, -1, -1, -1), v.cuda().expand(B, -1, -1, -1), _i32(0, *[-1] * (B - 1)))
    c.table.copy_(c.table[:1].clone().expand(B, -1))
    c.k_tail.copy_(c.k_tail[:1].clone().expand(B, -1, -1, -1))
    c.v_tail.copy_(c.v_tail[:1].clone().expand(B, -1, -1, -1))
    return c, k[0], v[0]


@gpu
def test_graphs_share_a_records_workspace(cuda):
    """Enough long sequences that the work is split over a workspace of records: two graphs that hold the same
    one, replayed in turn, and calls on a stream of their own with a workspace that nobody keeps."""
    B, S = 150, 4300
    histories = [_one_history(B, S, seed) for seed in (21, 22)]
    q, g = _queries(B, 8, "bf16")
    qd, gd, pos = q.cuda(), g.cuda(), _i32(*[S - 1] * B)
    need = ga.zgcm_attn_decode_kv8_workspace_size(histories[0][0], 8, window=ALL)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    alone = [ga.zgcm_attn_decode_kv8(c, qd, gd, pos, window=ALL, workspace=ws) for c, _, _ in histories]
    for (out, lse), (c, k, v) in zip(alone, histories):
        for b in (0, 77, B - 1):
            ref = kv8.attend(q[b], g[b], k, v, code="e4m3", window=ALL)
            _close(b, out[b], lse[b], *ref, q[b], k, 128 ** -0.5)
    graphs, got = [], []
    for c, _, _ in histories:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(ga.zgcm_attn_decode_kv8(c, qd, gd, pos, window=ALL, workspace=ws))
        graphs.append(graph)
    for _ in range(5):
        for x in got:
            x[0].zero_()
        for graph in graphs:
            graph.replay()
        for x, y in zip(got, alone):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kept = []
    for i in range(10):
        kept.append(ga.zgcm_attn_decode_kv8(histories[i % 2][0], qd, gd, pos, window=ALL, stream=side))
        torch.empty(need, dtype=torch.uint8, device="cuda").fill_(255)   # on the current stream, meanwhile
    torch.cuda.synchronize()
    for i, x in enumerate(kept):
        assert torch.equal(x[0], alone[i % 2][0]) and torch.equal(x[1], alone[i % 2][1])
    other = types.SimpleNamespace(device_index=1 + torch.cuda.current_device(), cuda_stream=0)
    for call in (lambda: ga.zgcm_attn_decode_kv8(histories[0][0], qd, gd, pos, window=ALL, stream=other),
                 lambda: ga.zgcm_kv8_select(histories[0][0], qd, pos, 4, stream=other)):
        with pytest.raises(TypeError, match="stream"):
            call()
    assert ga.zgcm_attn_device_error() == 0


@gpu
def test_two_streams_and_repeats(cuda):
    """Two caches worked on from two streams at once, many times: the same bits as alone."""
    k, v = _tokens(2, 2000, 2, "fp16", seed=14)
    caches = [_new(2, 32, 2, code, "fp16") for code in ("e4m3", "int8")]
    for c in caches:
        _feed(c, k, v, [2000])
    q, g = (x.cuda() for x in _queries(2, 8, "fp16"))
    pos = _i32(1999, 1999)
    alone = [ga.zgcm_attn_decode_kv8(c, q, g, pos, window=ALL) for c in caches]
    sel = [ga.zgcm_kv8_select(c, q, pos, 8, window=ALL) for c in caches]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in caches]
    kept = []
    for _ in range(20):
        for c, s in zip(caches, streams):
            with torch.cuda.stream(s):
                kept.append((ga.zgcm_attn_decode_kv8(c, q, g, pos, window=ALL), ga.zgcm_kv8_select(c, q, pos, 8, window=ALL)))
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(kept):
        assert torch.equal(a[0], alone[i % 2][0]) and torch.equal(a[1], alone[i % 2][1]) and torch.equal(b, sel[i % 2])
    assert ga.zgcm_attn_device_error() == 0


@gpu
def test_shared_prefix_pages(cuda):
    """Two sequences whose first blocks are the same pages."""
    k, v = _tokens(2, 200, 2, "bf16", seed=15)
    k[1, :128], v[1, :128] = k[0, :128], v[0, :128]
    c = _new(2, 4, 2, "e4m3", "bf16")
    _feed(c, k[:, :128], v[:, :128], [128])
    c.table[1, :2] = c.table[0, :2]
    _feed(c, k[:, 128:], v[:, 128:], [72], start=128)
    q, g = _queries(2, 4, "bf16")
    _check_decode(c, k, v, q, g, "e4m3")


@gpu
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("key", ["bf16", "fp16"])
def test_codes_of_every_mantissa(cuda, code, key):
    """Quotients at and next to the middle between two codes: every significand of three binades against largest
    magnitudes of many kinds (those that put ties exactly on 16-bit values among them), down to where the scale is its
    smallest."""
    bits = 7 if key == "bf16" else 10
    g = torch.Generator().manual_seed(4)
    # a head's 64 x 128 values; heads 0 .. 39: largest magnitudes 1 .. 2, 448 / 256 and 127 / 64 among them
    tops = torch.cat([1 + torch.arange(0, 32) / 32, torch.tensor([1.75, 127 / 64, 448 / 256 * 0.875, 1.0625]),
                      1 + torch.rand(4, generator=g)])
    shift = 2.0 ** (1 - torch.randint(0, 9, (64, 128), generator=g).double())
    sig = 1 + (torch.arange(64 * 128) % 2 ** bits).view(64, 128).double() / 2 ** bits
    sign = torch.where(torch.rand(64, 128, generator=g) < 0.5, -1.0, 1.0)
    x = (sig * shift * sign).unsqueeze(1).repeat(1, 40, 1)
    for down in (1.0, 2.0 ** -10, 2.0 ** -100, 2.0 ** -118, 2.0 ** -124) if key == "bf16" else (1.0, 2.0 ** -8, 2.0 ** 12):
        t = (tops.to(KEY[key]).double() * 2).view(1, 40, 1)
        y = torch.where(x.abs() > t, x / 4, x)
        y[0, :, 0] = t[0, :, 0]
        k = (y * down).to(KEY[key]).unsqueeze(0)
        v = (y.flip(0) * (down if key == "bf16" else 1.0)).to(torch.bfloat16).unsqueeze(0)
        c = _new(1, 2, 40, code, key)
        _feed(c, k, v, [64])
        _check_held(c, k, v, code)
