"""PyTorch autograd entry point of the layer: out = zgcm_attention(q, k, v, g, gamma_q,
gamma_k, window=...) in a training graph, backward included.

The forward runs the training pair that keeps activations where it applies (the normalised,
rotated q~, k~ and every row's inverse RMS stay in a store that the backward reads instead of
converting q and k again; bit-identical to the plain pair), and the plain pair elsewhere.
Argument marshalling only: both passes are the library's kernels.  Gradients flow to q, k,
v, g, gamma_q and gamma_k; lse is kept for the backward and not returned.

zgcm_qk_norm_rope is the query/key preparation as an operator of its own: the normalised, rotated
q and k with gradients to q, k, gamma_q and gamma_k.

`ops` (tests only) replaces the three calls (forward, backward, store size) with others of the
same signatures, so that the plumbing can be checked on the CPU.
"""
from __future__ import annotations

import math

import torch


def _placed(grad):
    """A gradient as the kernels take it: an expanded one (of a sum, say) has rows that are not contiguous, a part of a larger
    one (of a concatenation) need not begin at 16 bytes."""
    grad = grad.contiguous()
    return grad if grad.data_ptr() % 16 == 0 else grad.clone()


def _default_ops():
    import global_attention_b200 as ga
    return ga.zgcm_attn_fwd, ga.zgcm_attn_bwd, ga.zgcm_attn_saved_size


class ZgcmAttentionFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, gamma_q, gamma_k, window, rope_dims, rope_base, eps, scale, ops):
        fwd, bwd, saved_size = ops
        B, S, Hq, D = q.shape
        Hkv = k.shape[2]
        kw = dict(rope_dims=rope_dims, rope_base=rope_base, window=window, eps=eps, scale=scale)
        n = saved_size(B, S, Hq, Hkv, D, rope_dims, window)
        store = torch.empty(n, dtype=torch.uint8, device=q.device) if n > 0 else None
        if store is not None:
            out, lse = fwd(q, k, v, g, gamma_q, gamma_k, saved=store, **kw)
        else:
            out, lse = fwd(q, k, v, g, gamma_q, gamma_k, **kw)
        ctx.save_for_backward(q, k, v, g, gamma_q, gamma_k, out, lse,
                              store if store is not None else torch.empty(0, dtype=torch.uint8))
        ctx.has_store, ctx.kw, ctx.bwd = store is not None, kw, bwd
        ctx.mark_non_differentiable(lse)
        return out, lse

    @staticmethod
    def backward(ctx, dout, _dlse):
        q, k, v, g, gamma_q, gamma_k, out, lse, store = ctx.saved_tensors
        extra = dict(saved=store) if ctx.has_store else {}
        gr = ctx.bwd(q, k, v, g, gamma_q, gamma_k, out, lse, _placed(dout), **ctx.kw, **extra)
        return (gr["dq"], gr["dk"], gr["dv"], gr["dg"], gr["dgamma_q"], gr["dgamma_k"],
                None, None, None, None, None, None)


def zgcm_attention(q, k, v, g, gamma_q, gamma_k, *, window=128, rope_dims=42, rope_base=10000.0, eps=1e-6,
                   scale=None, return_lse=False, ops=None):
    """Gated window attention with autograd: q, g [B,S,Hq,D], k, v [B,S,Hkv,D] (bf16, CUDA),
    gamma_q, gamma_k [D] fp32.  Returns out [B,S,Hq,D] (and lse [B,Hq,S] with return_lse)."""
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    out, lse = ZgcmAttentionFunction.apply(q, k, v, g, gamma_q, gamma_k, int(window), int(rope_dims),
                                           float(rope_base), float(eps), float(scale), ops or _default_ops())
    return (out, lse) if return_lse else out


def _default_norm_ops():
    import global_attention_b200 as ga
    return ga.zgcm_qk_norm_rope_fwd, ga.zgcm_qk_norm_rope_bwd


class ZgcmQkNormRopeFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, gamma_q, gamma_k, pos, out_dtype, rope_dims, rope_base, eps, ops):
        ctx.kw, ctx.ops = dict(rope_dims=rope_dims, rope_base=rope_base, eps=eps), ops
        ctx.save_for_backward(q, k, gamma_q, gamma_k, pos)
        return ops[0](q, k, gamma_q, gamma_k, pos, out_dtype=out_dtype, **ctx.kw)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dqr, dkr):
        q, k, gamma_q, gamma_k, pos = ctx.saved_tensors
        gr = ctx.ops[1](q, k, gamma_q, gamma_k, pos, _placed(dqr), _placed(dkr), **ctx.kw)
        return gr["dq"], gr["dk"], gr["dgamma_q"], gr["dgamma_k"], None, None, None, None, None, None


def zgcm_qk_norm_rope(q, k, gamma_q, gamma_k, pos=None, *, rope_dims=42, rope_base=10000.0, eps=1e-6, out_dtype=None,
                      ops=None):
    """Per-head RMSNorm and rotation of q [..., Hq, D] and k [..., Hkv, D] (bf16, fp16 or fp32, CUDA) with
    autograd; gamma_q, gamma_k [D] fp32.  pos: int32, the leading shape (default: q is [B, S, Hq, D] and every
    sequence counts from 0).  Returns (qr, kr) of out_dtype (default: q's)."""
    lead = q.shape[:-2]
    if k.shape[:-2] != lead:
        raise TypeError(f"q and k must have the same leading shape, not {tuple(lead)} and {tuple(k.shape[:-2])}")
    if pos is None:
        if len(lead) != 2:
            raise TypeError("pos is needed unless q is [B, S, Hq, D]")
        pos = torch.arange(lead[1], dtype=torch.int32, device=q.device).expand(lead)
    if pos.shape != lead:
        raise TypeError(f"pos must have shape {tuple(lead)}, not {tuple(pos.shape)}")
    qr, kr = ZgcmQkNormRopeFunction.apply(q.reshape(-1, *q.shape[-2:]), k.reshape(-1, *k.shape[-2:]), gamma_q, gamma_k,
                                          pos.reshape(-1), out_dtype or q.dtype, int(rope_dims), float(rope_base),
                                          float(eps), ops or _default_norm_ops())
    return qr.view(q.shape), kr.view(k.shape)
