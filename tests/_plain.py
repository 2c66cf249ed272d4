"""Attention with a mask in plain float64 torch, and error bounds for the bf16 kernels.

The bounds count roundings: a value stored in bf16 is off by at most U = 2^-8
of itself (half a step). The kernels round the unnormalised weights P (to
compute O and dV) and dS (to compute dQ and dK) to bf16, keep every sum and
softmax statistic in fp32, and round each output once. SLACK covers the fp32
arithmetic (exp2 and sums of a few thousand terms: below 2^-13 relative).
"""
import math

import torch

U = 2.0 ** -8
SLACK = 2.0 ** -12


def visible(lq, lk, causal, window, sinks):
    """bool [lq, lk]: bottom-right aligned causal mask or window, with sinks left of the window."""
    i = torch.arange(lq)[:, None] + (lk - lq)
    j = torch.arange(lk)[None, :]
    left, right = window
    if causal:
        right = 0
    ok = torch.ones((lq, lk), dtype=torch.bool)
    if right >= 0:
        ok &= j <= i + right
    if left >= 0:
        ok &= (j >= i - left) | (j < sinks)
    return ok


def attention(q, k, v, ok, scale):
    """One sequence, float64: q [lq, H, d], k [lk, Hkv, d], v [lk, Hkv, dv] -> dict of o [lq, H, dv],
    lse [H, lq], p [H, lq, lk] and bound (of o)."""
    H, Hkv = q.shape[1], k.shape[1]
    kx, vx = k.repeat_interleave(H // Hkv, 1), v.repeat_interleave(H // Hkv, 1)
    s = torch.einsum("ihd,jhd->hij", q, kx) * scale
    s = s.masked_fill(~ok, -math.inf)
    lse = torch.logsumexp(s, -1) if s.shape[-1] else torch.full(s.shape[:2], -math.inf, dtype=s.dtype)
    p = torch.where(ok, torch.exp(s - torch.where(torch.isfinite(lse), lse, 0.0)[..., None]), 0.0)
    o = torch.einsum("hij,jhd->ihd", p, vx)
    spread = torch.einsum("hij,jhd->ihd", p, vx.abs())
    return {"o": o, "lse": lse, "p": p, "bound": (U + SLACK) * (spread + o.abs())}


def gradients(q, k, v, do, ok, scale):
    """dq, dk, dv of sum(o * do) and their bounds, from the formulas."""
    H, Hkv = q.shape[1], k.shape[1]
    r = H // Hkv
    kx, vx = k.repeat_interleave(r, 1), v.repeat_interleave(r, 1)
    f = attention(q, k, v, ok, scale)
    p, o = f["p"], f["o"]
    dp = torch.einsum("ihd,jhd->hij", do, vx)
    D = (do * o).sum(-1).t()[..., None]
    ds = p * (dp - D) * scale
    # the kernels' D comes from the rounded O
    D_err = (do.abs() * f["bound"]).sum(-1).t()[..., None]
    ds_err = (U + SLACK) * ds.abs() + scale * p * (D_err + SLACK * torch.einsum("ihd,jhd->hij", do.abs(), vx.abs()))

    def back(x):   # sum the query heads that read a key/value head
        return x.reshape(x.shape[0], Hkv, r, x.shape[-1]).sum(2)

    dq, dq_b = torch.einsum("hij,jhd->ihd", ds, kx), torch.einsum("hij,jhd->ihd", ds_err, kx.abs())
    dk, dk_b = back(torch.einsum("hij,ihd->jhd", ds, q)), back(torch.einsum("hij,ihd->jhd", ds_err, q.abs()))
    dv = back(torch.einsum("hij,ihd->jhd", p, do))
    dv_b = back(torch.einsum("hij,ihd->jhd", p, do.abs())) * (U + SLACK)
    return {"dq": dq, "dk": dk, "dv": dv, "dq_bound": dq_b + U * (dq.abs() + dq_b),
            "dk_bound": dk_b + U * (dk.abs() + dk_b), "dv_bound": dv_b + U * (dv.abs() + dv_b)}


def assert_within(got, ref, bound, what, floor=1e-6):
    got = got.detach().double().cpu()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - ref).abs() - bound - floor
    assert over.max().item() <= 0 if over.numel() else True, \
        f"{what}: {over.max().item():.3e} past the bound at {int(over.argmax())}"


def assert_lse(got, ref, what, scores=30.0):
    """LSE in fp32: off by a few 2^-24 of the largest score it sums (|s| <= scores), -inf alike."""
    got = got.detach().double().cpu()
    assert torch.equal(torch.isneginf(got), torch.isneginf(ref)), f"{what}: rows without a key"
    fin = torch.isfinite(ref)
    if fin.any():
        err = (got[fin] - ref[fin]).abs().max().item()
        assert err <= scores * 2.0 ** -20, f"{what}: lse off by {err:.3e}"
