"""Cases of the operators around the 8-bit block cache: normalisation and rotation of queries and
keys (both directions), filling the cache, attention of single tokens over it, block selection.

A block is 64 tokens of a sequence; its codes, one scale for each KV head and the mean of its keys
live in a page, and the block of a sequence's newest token is held in 16 bits as well.  Head counts
are the layer's own (32 query / 8 KV heads of 128) and other groupings; lengths go from one token
to the 16K, 64K and 256K contexts; 64 sequences at 16K are the benchmark's decode workload.
"""
import math

import torch

own = False

D = 128
BLOCK = 64
SMALLEST_SCALE = 2.0 ** -126
ROPE_DIMS, ROPE_BASE, EPS = 42, 10000.0, 1e-6
SCALE = D ** -0.5
EVERY = 1 << 30          # a window that reaches every earlier token
HEADS = ((32, 8), (16, 8), (24, 8), (8, 8), (32, 4), (32, 2), (12, 1))
T16 = {"bf16": torch.bfloat16, "fp16": torch.float16}
CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
TOP = {"e4m3": 448.0, "int8": 127.0}


# ------------------------------------------------------------------------------------- cases

def listed():
    return [
        # the new tokens of 64 sequences on their way into a decode step
        _norm("norm_rope 64", "fwd", 64, out="fp16"),
        # queries and keys of a training batch of 4 x 16K tokens
        _norm("norm_rope 64K", "fwd", 65536),
        # gradients of an odd-sized packed batch with far positions
        _norm("norm_rope grad 1000", "bwd", 1000, far=262144),
        # gradients of the training batch
        _norm("norm_rope grad 64K", "bwd", 65536),
        # one new token of each of 64 sequences, some completing their block
        _append("append 64x1", 64, 1, 16300, "e4m3", "fp16"),
        # a padded batch of prompts of up to 16K tokens
        _append("append 4x16K", 4, 16384, 0, "e4m3", "bf16"),
        # one conversation of a thousand tokens: latency
        _decode("decode 1x1000", 1, 1000, EVERY, "e4m3", "fp16", ragged=False),
        # a sliding layer of 64 sequences at 16K: three blocks resident for each
        _decode("decode 64x16K window 128", 64, 16384, 128, "e4m3", "fp16"),
        # a global layer of 64 sequences of 8K to 16K, integer codes
        _decode("decode 64x16K int8", 64, 16384, EVERY, "int8", "bf16"),
        # 16 contexts of up to 64K of which 32 selected blocks are read
        _decode("decode 16x64K 32 blocks", 16, 65536, EVERY, "e4m3", "bf16", n_sel=32),
        # choosing 32 of the up to 256 blocks of 64 sequences
        _select("select 64x16K", 64, 16384, 32, "fp16"),
        # choosing 64 of the 4096 blocks of two 256K contexts
        _select("select 2x256K", 2, 262144, 64, "bf16", ragged=False),
    ]


def _norm(name, way, T, Hq=32, Hkv=8, out="bf16", far=16384):
    return dict(name=name, op="norm_" + way, T=T, Hq=Hq, Hkv=Hkv, out=out, far=far)


def _append(name, B, N, start, code, key, Hkv=8, ragged=True):
    return dict(name=name, op="append", B=B, N=N, start=start, Hkv=Hkv, code=code, key=key, ragged=ragged)


def _decode(name, B, ctx, window, code, key, Hq=32, Hkv=8, n_sel=0, ragged=True):
    return dict(name=name, op="decode", B=B, ctx=ctx, window=window, Hq=Hq, Hkv=Hkv, code=code, key=key, n_sel=n_sel,
                ragged=ragged)


def _select(name, B, ctx, n_sel, key, Hq=32, Hkv=8, ragged=True):
    return dict(name=name, op="select", B=B, ctx=ctx, Hq=Hq, Hkv=Hkv, key=key, n_sel=n_sel, ragged=ragged)


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))

    Hq, Hkv = rng.choice(HEADS)
    code, key, ragged = rng.choice(("e4m3", "int8")), rng.choice(("bf16", "fp16")), rng.random() < 0.7
    kind = rng.choice(("norm", "norm", "append", "append", "decode", "decode", "window", "sparse", "select", "select"))
    if kind == "norm":
        case = _norm("", rng.choice(("fwd", "bwd")), spread(1, 65536), Hq, Hkv, rng.choice(("bf16", "fp16")),
                     spread(64, 262144))
    elif kind == "append":
        if rng.random() < 0.4:
            case = _append("", spread(1, 256), 1, spread(1, 65536) - 1, code, key, Hkv, ragged)
        else:
            N = spread(2, 16384)
            case = _append("", spread(1, max(1, 65536 // N)), N, BLOCK * rng.choice((0, 0, 1, 37)), code, key, Hkv, ragged)
    else:
        ctx = spread(1, 131072)
        B = spread(1, max(1, min(64, (1 << 20) // ctx)))
        if kind == "select":   # always more blocks than are chosen: the shortest context has 32
            ctx = spread(4096, 262144)
            B = spread(1, max(1, min(64, (1 << 20) // ctx)))
            case = _select("", B, ctx, rng.choice([n for n in (8, 16, 31, 64) if n < ctx // 128]), key, Hq, Hkv, ragged)
        else:
            case = _decode("", B, ctx, spread(1, 4096) if kind == "window" else EVERY, code, key, Hq, Hkv,
                           rng.choice((8, 16, 31, 64)) if kind == "sparse" else 0, ragged)
    del case["name"]
    return case


# ------------------------------------------------------------------------------------ inputs

def _table_width(ctx, window):
    """Blocks a sequence keeps: all of its context, or those a window can touch."""
    return min(-(-ctx // BLOCK), -(-(min(window, ctx) - 1) // BLOCK) + 1)


def _positions(c, g):
    """The newest token's position in each sequence."""
    if not c["ragged"]:
        return torch.full((c["B"],), c["ctx"] - 1, dtype=torch.int32, device="cuda")
    return torch.randint(c["ctx"] // 2, c["ctx"], (c["B"],), generator=g, device="cuda", dtype=torch.int32)


def _paged(B, width, Hkv, code, key, g, fill):
    """A cache of B sequences: pages in random order, a few of them unused."""
    pages = B * width + 3
    s = {"table": torch.randperm(pages, generator=g, device="cuda")[:B * width].to(torch.int32).view(B, width)}
    shape = (pages, Hkv, BLOCK, D)
    if fill:
        gain = torch.exp(0.5 * torch.randn(Hkv, 1, D, generator=g, device="cuda"))
        k = torch.randn(shape, generator=g, device="cuda") * gain
        s["k_mean"] = k.mean(2).to(T16[key])
        s["k_codes"], s["k_scale"] = _quantise(k, code)
        del k
        v = torch.randn(shape, generator=g, device="cuda")
        v *= torch.exp(torch.randn(pages, Hkv, 1, 1, generator=g, device="cuda"))
        s["v_codes"], s["v_scale"] = _quantise(v, code)
    else:
        for n in ("k", "v"):
            s[n + "_codes"] = torch.zeros(shape, dtype=torch.uint8, device="cuda").view(CODE[code])
            s[n + "_scale"] = torch.zeros(pages, Hkv, device="cuda")
        s["k_mean"] = torch.randn(pages, Hkv, D, generator=g, device="cuda").to(T16[key]) * 0.125
    s["k_tail"] = torch.randn(B, Hkv, BLOCK, D, generator=g, device="cuda").to(T16[key])
    s["v_tail"] = torch.randn(B, Hkv, BLOCK, D, generator=g, device="cuda").to(torch.bfloat16)
    return s


def _handle(s):
    import global_attention_b200 as ga
    return ga.ZgcmKv8Cache(*(s[n] for n in ("k_codes", "v_codes", "k_scale", "v_scale", "k_mean", "k_tail", "v_tail",
                                            "table")))


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, t=torch.bfloat16):
        return torch.randn(shape, generator=g, device="cuda").to(t)

    s = {"case": c}
    if c["op"].startswith("norm"):
        T, Hq, Hkv = c["T"], c["Hq"], c["Hkv"]
        s.update(q=randn(T, Hq, D) * 3, k=randn(T, Hkv, D) * torch.exp(randn(T, 1, 1)),
                 gamma_q=torch.rand(D, generator=g, device="cuda") + 0.5,
                 gamma_k=torch.rand(D, generator=g, device="cuda") + 0.5,
                 # packed sequences: positions count up from a few starts
                 pos=((torch.arange(T, device="cuda") + torch.randint(0, c["far"], (1,), generator=g, device="cuda"))
                      % c["far"]).to(torch.int32))
        if c["op"] == "norm_bwd":
            s.update(dqr=randn(T, Hq, D), dkr=randn(T, Hkv, D))
        return s
    B, Hkv = c["B"], c["Hkv"]
    if c["op"] == "append":
        N, far = c["N"], c["start"] + c["N"]
        start = torch.full((B,), c["start"], dtype=torch.int32, device="cuda")
        count = torch.full((B,), N, dtype=torch.int32, device="cuda")
        if c["ragged"] and N == 1:
            start += torch.randint(0, 2 * BLOCK, (B,), generator=g, device="cuda", dtype=torch.int32)
            far += 2 * BLOCK
        elif c["ragged"]:
            count = torch.randint(N // 2, N + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        s.update(_paged(B, min(-(-far // BLOCK), 1024), Hkv, c["code"], c["key"], g, False))
        s.update(k=randn(B, N, Hkv, D, t=T16[c["key"]]), v=randn(B, N, Hkv, D), start=start, count=count)
    else:
        s["pos"] = _positions(c, g)
        window = c.get("window", EVERY)
        s.update(_paged(B, _table_width(c["ctx"], window), Hkv, c.get("code", "e4m3"), c["key"], g, c["op"] == "decode"))
        s["q"] = randn(B, c["Hq"], D, t=T16[c["key"]])
        s["g"] = randn(B, c["Hq"], D)
        s["blocks"] = None
        if c["op"] == "decode" and c["n_sel"]:
            # distinct blocks before the newest token's, ascending, -1 behind the last
            n, width = c["n_sel"], s["table"].shape[1]
            have = (s["pos"] // BLOCK).view(B, 1, 1)
            rank = torch.rand(B, Hkv, max(width, n), generator=g, device="cuda")
            rank = rank.masked_fill(torch.arange(max(width, n), device="cuda") >= have, 2.0)
            val, idx = rank.sort(-1)
            idx = idx[..., :n].masked_fill(val[..., :n] > 1.5, 1 << 30).sort(-1).values
            s["blocks"] = idx.masked_fill(idx == 1 << 30, -1).to(torch.int32)
    if own:
        s["cache"] = _handle(s)
    return s


# -------------------------------------------------------------------------------- plain forms

def _quantise(x, code):
    """[..., 64, D] -> codes and the scale of each block; 32 bits, one division each."""
    amax = x.float().abs().amax((-2, -1))
    scale = (amax / TOP[code]).clamp_min(SMALLEST_SCALE)
    scale = torch.where(amax.isfinite(), scale, math.nan)
    y = (x.float() / scale[..., None, None]).masked_fill(~amax.isfinite()[..., None, None], 0.0)
    return (y.to(torch.float8_e4m3fn) if code == "e4m3" else torch.round(y).to(torch.int8)), scale


def _angles(pos):
    t = torch.arange(ROPE_DIMS // 2, device=pos.device, dtype=torch.float64)
    a = pos.double()[:, None, None] * ROPE_BASE ** (-2.0 * t / ROPE_DIMS)
    return a.cos().float(), a.sin().float()


def _rotate(x, cos, sin):
    h = ROPE_DIMS // 2
    a, b = x[..., :h], x[..., h:2 * h]
    return torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., 2 * h:]), -1)


def _norm_fwd(x, gamma, cos, sin, out):
    x = x.float()
    xh = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
    return _rotate(xh * gamma, cos, sin).to(out)


def _norm_bwd(x, gamma, cos, sin, dy):
    t, x = x.dtype, x.float()
    r = 1.0 / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
    xh = x * r
    u = _rotate(dy.float(), cos, -sin)
    dgamma = (u * xh).sum((0, 1), dtype=torch.float64).float()
    u = u * gamma
    return (r * (u - xh * (u * xh).mean(-1, keepdim=True))).to(t), dgamma


def _plain_append(s):
    c, NB = s["case"], s["table"].shape[1]
    B, N, Hkv = c["B"], c["N"], c["Hkv"]
    start, count = s["start"].long(), s["count"].long()
    n = -(-N // BLOCK) + (N == 1)
    first = start // BLOCK
    row = torch.arange(n * BLOCK, device="cuda")
    new = row - (start - first * BLOCK)[:, None]                       # the new token that goes to this row
    old = new < 0
    take = new.clamp(0, N - 1)[:, :, None, None].expand(-1, -1, Hkv, D)
    block = first[:, None] + torch.arange(n, device="cuda")
    last = (start + count - 1) // BLOCK
    whole = ((block + 1) * BLOCK <= (start + count)[:, None]) & (block > last[:, None] - NB) & (count > 0)[:, None]
    page = s["table"].gather(1, block % NB).long()[whole]
    rows = row.view(n, BLOCK)
    tail_at = (last - first).clamp_min(0)
    for x, codes, scale, tail, mean in ((s["k"], "k_codes", "k_scale", "k_tail", "k_mean"),
                                        (s["v"], "v_codes", "v_scale", "v_tail", None)):
        full = x.gather(1, take)
        was = s[tail].transpose(1, 2)                                  # [B, 64, Hkv, D]
        full = torch.where(old[:, :, None, None], was.repeat(1, n, 1, 1), full)
        full = full.view(B, n, BLOCK, Hkv, D).transpose(2, 3)          # [B, n, Hkv, 64, D]
        done = full[whole]
        y, z = _quantise(done, c["code"])
        s[codes].view(torch.uint8)[page] = y.view(torch.uint8)
        s[scale][page] = z
        if mean:
            s[mean][page] = done.float().mean(2).to(s[mean].dtype)
        end = full[torch.arange(B, device="cuda"), tail_at]            # [B, Hkv, 64, D]
        there = (rows[tail_at] < (start + count - first * BLOCK)[:, None]) & (count > 0)[:, None]
        s[tail].copy_(torch.where(there[:, None, :, None], end, s[tail]))


def _plain_decode(s):
    c, NB = s["case"], s["table"].shape[1]
    B, Hq, Hkv = c["B"], c["Hq"], c["Hkv"]
    pos = s["pos"].long()
    own_block, lo = pos // BLOCK, (pos - c["window"] + 1).clamp_min(0)
    if s["blocks"] is None:
        block = (own_block[:, None] - torch.arange(NB - 1, 0, -1, device="cuda"))[:, None].expand(-1, Hkv, -1)
    else:
        block = s["blocks"].long()
    n = block.shape[2]
    page = s["table"].long()[torch.arange(B, device="cuda")[:, None, None], block.clamp_min(0) % NB]
    head = torch.arange(Hkv, device="cuda")[None, :, None]

    def values(side):
        x = s[side + "_codes"].view(torch.uint8)[page, head].view(CODE[c["code"]]).float()
        x = x * s[side + "_scale"][page, head][..., None, None]
        return torch.cat((x.view(B, Hkv, n * BLOCK, D), s[side + "_tail"].float()), 2)

    r = torch.arange(BLOCK, device="cuda")
    j = (block[..., None] * BLOCK + r).masked_fill(block[..., None] < 0, -1).reshape(B, Hkv, n * BLOCK)
    j = torch.cat((j, (own_block[:, None] * BLOCK + r)[:, None].expand(-1, Hkv, -1)), 2)
    seen = (j >= lo[:, None, None]) & (j <= pos[:, None, None]) & (j >= 0)
    q = s["q"].float().view(B, Hkv, Hq // Hkv, D)
    x = (q @ values("k").transpose(2, 3)) * SCALE
    x = x.masked_fill(~seen[:, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    o = ((p @ values("v")) / total).view(B, Hq, D)
    lse = (m + torch.log(total)).view(B, Hq)
    return (o / (1 + torch.exp(-s["g"].float()))).to(torch.bfloat16), lse


def _plain_select(s):
    c, NB = s["case"], s["table"].shape[1]
    B, Hq, Hkv, n = c["B"], c["Hq"], c["Hkv"], c["n_sel"]
    have = (s["pos"].long() // BLOCK)[:, None, None]
    block = torch.arange(NB, device="cuda")
    mean = s["k_mean"][s["table"].long()].double()                     # [B, NB, Hkv, D], block j in column j
    q = s["q"].double().view(B, Hkv, Hq // Hkv, D)
    score = (q @ mean.permute(0, 2, 3, 1)).amax(2)                     # [B, Hkv, NB]
    score = score.masked_fill((block < 1) | (block >= have - 1), math.inf)
    score = score.masked_fill(block >= have, -math.inf).nan_to_num(nan=-math.inf, posinf=math.inf, neginf=-math.inf)
    idx = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :n]
    idx = torch.where(idx < have, idx, EVERY).sort(-1).values
    idx = torch.cat((idx, idx.new_full((B, Hkv, max(0, n - NB)), EVERY)), -1)
    return idx.masked_fill(idx == EVERY, -1).to(torch.int32)


# ---------------------------------------------------------------------------------------- run

CACHE = ("k_codes", "v_codes", "k_scale", "v_scale", "k_mean", "k_tail", "v_tail")


def run(state):
    s, c = state, state["case"]
    if own:
        import global_attention_b200 as ga
        if c["op"] == "norm_fwd":
            return ga.zgcm_qk_norm_rope_fwd(s["q"], s["k"], s["gamma_q"], s["gamma_k"], s["pos"], out_dtype=T16[c["out"]])
        if c["op"] == "norm_bwd":
            return ga.zgcm_qk_norm_rope_bwd(s["q"], s["k"], s["gamma_q"], s["gamma_k"], s["pos"], s["dqr"], s["dkr"])
        if c["op"] == "append":
            ga.zgcm_kv8_append(s["cache"], s["k"], s["v"], s["start"], count=s["count"])
            return {n: s[n] for n in CACHE}
        if c["op"] == "decode":
            return ga.zgcm_attn_decode_kv8(s["cache"], s["q"], s["g"], s["pos"], window=c["window"], blocks=s["blocks"])
        return ga.zgcm_kv8_select(s["cache"], s["q"], s["pos"], c["n_sel"], n_first=1, n_last=1, window=EVERY)
    if c["op"].startswith("norm"):
        cos, sin = _angles(s["pos"])
        if c["op"] == "norm_fwd":
            t = T16[c["out"]]
            return _norm_fwd(s["q"], s["gamma_q"], cos, sin, t), _norm_fwd(s["k"], s["gamma_k"], cos, sin, t)
        dq, dgq = _norm_bwd(s["q"], s["gamma_q"], cos, sin, s["dqr"])
        dk, dgk = _norm_bwd(s["k"], s["gamma_k"], cos, sin, s["dkr"])
        return {"dq": dq, "dk": dk, "dgamma_q": dgq, "dgamma_k": dgk}
    if c["op"] == "append":
        _plain_append(s)
        return {n: s[n] for n in CACHE}
    return _plain_decode(s) if c["op"] == "decode" else _plain_select(s)


# --------------------------------------------------------------------------------------- work

def _mean_length(c):
    return c["ctx"] * (0.75 if c["ragged"] else 1.0)


def work(case):
    c = case
    if c["op"].startswith("norm"):
        rows = c["T"] * (c["Hq"] + c["Hkv"])
        passes = 2 if c["op"] == "norm_fwd" else 3
        return {"bytes": rows * D * 2 * passes + c["T"] * 4 + 4 * D * (2 if passes == 2 else 4),
                "flops": rows * D * (8 if passes == 2 else 16)}
    if c["op"] == "append":
        tokens = c["B"] * c["N"] * (0.75 if c["ragged"] and c["N"] > 1 else 1.0)
        values = tokens * c["Hkv"] * D * 2
        if c["N"] == 1:   # the 16-bit row, and every 64th token its block: read, its codes written
            return {"bytes": values * (2 + 2 + 2 + 1), "flops": values * 4}
        return {"bytes": values * 3 + c["B"] * c["Hkv"] * BLOCK * D * 4, "flops": values * 4}
    near = _mean_length(c)
    if c["op"] == "select":
        read = c["B"] * c["Hkv"] * (near / BLOCK) * D
        return {"bytes": read * 2 + c["B"] * (c["Hq"] * D * 2 + c["Hkv"] * c["n_sel"] * 4),
                "flops": 2 * read * c["Hq"] / c["Hkv"]}
    keys = min(near, c["window"])
    if c["n_sel"]:
        keys = min(keys, (c["n_sel"] + 0.5) * BLOCK)
    tail = min(keys, BLOCK / 2)                # 16 bits for the newest block, 8 for those before it
    kv = c["B"] * c["Hkv"] * D * 2
    return {"bytes": kv * (keys - tail) + kv * 2 * tail + c["B"] * c["Hq"] * (D * 6 + 4),
            "flops": 4 * c["B"] * c["Hq"] * D * keys}


# -------------------------------------------------------------------------- 64-bit definitions

def _exact_norm(x, gamma, pos, dy=None):
    """Row by row from the definition: a rotation matrix's two entries for every dimension."""
    x = x.double()
    half = ROPE_DIMS // 2
    d = torch.arange(D, device="cuda")
    theta = torch.where(d < ROPE_DIMS, ROPE_BASE ** (-2.0 * (d % half).double() / ROPE_DIMS), 0.0)
    angle = pos.double()[:, None] * theta
    cos, sin = angle.cos()[:, None], (angle.sin() * torch.where(d < half, -1.0, 1.0))[:, None]
    partner = torch.where(d < half, d + half, torch.where(d < ROPE_DIMS, d - half, d))
    rms = (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt()
    if dy is None:
        y = x / rms * gamma.double()
        return y * cos + y[..., partner] * sin
    dy = dy.double()
    u = dy * cos - dy[..., partner] * sin
    dgamma = (u * x / rms).sum((0, 1))
    w = u * gamma.double()
    return w / rms - x * (w * x).sum(-1, keepdim=True) / (D * rms ** 3), dgamma


def _exact_codes(x, code):
    """The 8-bit values nearest to x / scale (ties to even) and the scale of one block."""
    scale = x.abs().max() / TOP[code]
    scale = torch.maximum(scale.float(), torch.tensor(SMALLEST_SCALE, device="cuda"))
    y = x / scale.double()
    if code == "int8":
        return torch.round(y).to(torch.int8), scale
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(y / step) * step, scale


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "norm_fwd":
        return _exact_norm(s["q"], s["gamma_q"], s["pos"]), _exact_norm(s["k"], s["gamma_k"], s["pos"])
    if c["op"] == "norm_bwd":
        dq, dgq = _exact_norm(s["q"], s["gamma_q"], s["pos"], s["dqr"])
        dk, dgk = _exact_norm(s["k"], s["gamma_k"], s["pos"], s["dkr"])
        return {"dq": dq, "dk": dk, "dgamma_q": dgq, "dgamma_k": dgk}
    if c["op"] == "append":
        if c["B"] * c["N"] * c["Hkv"] > 600000:
            return None
        got = {n: s[n].clone() if s[n].dtype == torch.int8 else s[n].double() for n in CACHE}
        NB = s["table"].shape[1]
        for b, (start, count) in enumerate(zip(s["start"].tolist(), s["count"].tolist())):
            if count < 1:
                continue
            last = (start + count - 1) // BLOCK
            for j in range(start // BLOCK, last + 1):
                lo, hi = max(start, j * BLOCK), min(start + count, (j + 1) * BLOCK)
                page = int(s["table"][b, j % NB])
                for side in "kv":
                    x = s[side + "_tail"][b].double().clone()
                    x[:, lo - j * BLOCK:hi - j * BLOCK] = s[side][b, lo - start:hi - start].double().transpose(0, 1)
                    if j == last:
                        n = hi - j * BLOCK
                        got[side + "_tail"][b, :, :n] = x[:, :n]
                    if hi == (j + 1) * BLOCK and j > last - NB:
                        for h in range(c["Hkv"]):
                            got[side + "_codes"][page, h], got[side + "_scale"][page, h] = _exact_codes(x[h], c["code"])
                        if side == "k":
                            got["k_mean"][page] = x.mean(1)
        return got
    if c["op"] == "select":
        return None
    G, NB = c["Hq"] // c["Hkv"], s["table"].shape[1]
    out = torch.empty(c["B"], c["Hq"], D, dtype=torch.float64, device="cuda")
    lse = torch.empty(c["B"], c["Hq"], dtype=torch.float64, device="cuda")
    for b, p in enumerate(s["pos"].tolist()):
        first = max(0, p - c["window"] + 1)
        for h in range(c["Hkv"]):
            blocks = list(range(first // BLOCK, p // BLOCK))
            if s["blocks"] is not None:
                blocks = [j for j in s["blocks"][b, h].tolist() if j >= 0]
            page = s["table"][b].long()[torch.tensor([j % NB for j in blocks], dtype=torch.int64, device="cuda")]
            at = [torch.arange(j * BLOCK, (j + 1) * BLOCK, device="cuda") for j in blocks]
            keep = torch.cat(at + [torch.arange(p // BLOCK * BLOCK, p + 1, device="cuda")]) >= first
            kv = []
            for side in "kv":
                old = s[side + "_codes"].view(torch.uint8)[page, h].view(CODE[c["code"]]).double()
                old = (old * s[side + "_scale"][page, h].double()[:, None, None]).reshape(-1, D)
                kv.append(torch.cat((old, s[side + "_tail"][b, h, :p % BLOCK + 1].double()))[keep])
            for i in range(h * G, (h + 1) * G):
                x = kv[0] @ s["q"][b, i].double() * SCALE
                lse[b, i] = torch.logsumexp(x, 0)
                out[b, i] = torch.sigmoid(s["g"][b, i].double()) * (torch.softmax(x, 0) @ kv[1])
    return out, lse
