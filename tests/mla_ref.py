"""Latent attention in 64 bits, written from its formulas for the tests: packed sequences in the
expanded form with gradients, the absorbed form over a paged cache, and the cache's append.

Besides each result the functions return the sum of the magnitudes that its roundings scale
with, from which the tests' tolerances follow:
  * a bfloat16 rounding is off by at most 2^-8 of the value (half a step), so a softmax weight
    or a dS rounded before a matrix product moves a result by at most 2^-8 of the sum of
    |weight| |operand|, and the result's own rounding by 2^-8 of it;
  * float32 sums and exponentials stay under SLACK of the same magnitudes at these sizes: a
    score of 192 (or 576) products is off by at most 576 * 2^-24 = 2^-14.8 of its sum of
    magnitudes, which is below 2^4 here, so e^s is off by less than 2^-10.8 of itself.
"""
from __future__ import annotations

import math

import torch

DN, DR, DV, DL, DC = 128, 64, 128, 512, 576
HALF_STEP = 2.0 ** -8
SLACK = 2.0 ** -10


def visible(lq, lk, causal, device="cpu"):
    m = torch.ones(lq, lk, dtype=torch.bool, device=device)
    return torch.tril(m, diagonal=lk - lq) if causal else m


def softmax(x, vis):
    """Weights and lse over the last axis where `vis`; weights 0 and lse -inf in an empty row."""
    x = x.masked_fill(~vis, -math.inf)
    m = x.amax(-1, keepdim=True) if x.shape[-1] else torch.full((*x.shape[:-1], 1), -math.inf, dtype=x.dtype, device=x.device)
    m0 = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = torch.exp(x - m0)
    l = e.sum(-1, keepdim=True)
    return e / torch.where(l > 0, l, torch.ones_like(l)), (m0 + torch.log(l))[..., 0]


def attention(q, k, v, scale, vis):
    """One head: o, lse, and sum_j p_ij |v_j|."""
    p, lse = softmax(q @ k.T * scale, vis)
    return p @ v, lse, p @ v.abs()


def head_kv(kv, kr, h):
    return torch.cat([kv[:, h, :DN], kr], 1), kv[:, h, DN:]


def fwd(q, kv, kr, cu_q, cu_k, scale, causal):
    """o, lse and the magnitude of o's weighted sum; rows behind the last sequence are NaN."""
    q, kv, kr = q.double(), kv.double(), kr.double()
    o = torch.full((*q.shape[:2], DV), math.nan, dtype=torch.float64, device=q.device)
    mag, lse = o.clone(), torch.full(q.shape[:2], math.nan, dtype=torch.float64, device=q.device)
    for a, b, c, d in zip(cu_q, cu_q[1:], cu_k, cu_k[1:]):
        vis = visible(b - a, d - c, causal, q.device)
        for h in range(q.shape[1]):
            k, v = head_kv(kv[c:d], kr[c:d], h)
            o[a:b, h], lse[a:b, h], mag[a:b, h] = attention(q[a:b, h], k, v, scale, vis)
    return o, lse, mag


def bwd(q, kv, kr, o, lse, dO, cu_q, cu_k, scale, causal):
    """{name: (gradient, magnitude)}; the magnitude counts the rounding of p and dS and, times
    2^-6, the float32 error of dS = p (dP - D), which scales with its two terms."""
    q, kv, kr, o, lse, dO = (t.double() for t in (q, kv, kr, o, lse, dO))
    dq, dkv, dkr = (torch.full_like(t, math.nan) for t in (q, kv, kr))
    mq, mkv, mkr = (torch.full_like(t, math.nan) for t in (q, kv, kr))
    dkr[cu_k[0]:cu_k[-1]], mkr[cu_k[0]:cu_k[-1]] = 0.0, 0.0
    for a, b, c, d in zip(cu_q, cu_q[1:], cu_k, cu_k[1:]):
        vis = visible(b - a, d - c, causal, q.device)
        for h in range(q.shape[1]):
            k, v = head_kv(kv[c:d], kr[c:d], h)
            g = dO[a:b, h]
            x = (q[a:b, h] @ k.T * scale - lse[a:b, h][:, None]).masked_fill(~vis, -math.inf)
            p = torch.exp(x)
            D = (g * o[a:b, h]).sum(1, keepdim=True)
            ds = scale * p * (g @ v.T - D)
            two = scale * p * (g.abs() @ v.abs().T + (g * o[a:b, h]).abs().sum(1, keepdim=True))
            w = ds.abs() + two * 2.0 ** -6
            dq[a:b, h], mq[a:b, h] = ds @ k, w @ k.abs()
            dk, mk = ds.T @ q[a:b, h], w.T @ q[a:b, h].abs()
            dkv[c:d, h], mkv[c:d, h] = torch.cat([dk[:, :DN], p.T @ g], 1), torch.cat([mk[:, :DN], p.T @ g.abs()], 1)
            dkr[c:d] += dk[:, DN:]
            mkr[c:d] += mk[:, DN:]
    return {"dq": (dq, mq), "dkv": (dkv, mkv), "dk_rope": (dkr, mkr)}


def rows_of(cache, scale, table_row, length):
    """The first `length` rows [length, G, 576] of a sequence, as the values they stand for."""
    ps = cache.shape[1]
    ids = table_row[:-(-length // ps)].long()
    c = cache[ids].double()
    if scale is not None:
        c = c * scale[ids].double()[:, None, :, None]
    return c.reshape(-1, *cache.shape[2:])[:length]


def decode(q, cache, scale_of, table, lens, scale):
    N, Sq, H, _ = q.shape
    G = cache.shape[2]
    o = torch.zeros(N, Sq, H, DL, dtype=torch.float64, device=q.device)
    mag, lse = o.clone(), torch.full((N, Sq, H), -math.inf, dtype=torch.float64, device=q.device)
    for n in range(N):
        L = int(lens[n])
        c = rows_of(cache, scale_of, table[n], L)
        vis = visible(Sq, L, True, q.device)
        for h in range(H):
            k = c[:, h // (H // G)]
            o[n, :, h], lse[n, :, h], mag[n, :, h] = attention(q[n, :, h].double(), k, k[:, :DL], scale, vis)
    return o, lse, mag


def power_for(amax: float) -> float:
    if not math.isfinite(amax):
        return math.nan
    s = 2.0 ** -100
    while amax > 448.0 * s:
        s *= 2.0
    return s


def append(new, cu, lens, table, cache, scale):
    """In place on CPU tensors, row by row."""
    ps, G = cache.shape[1], cache.shape[2]
    for n in range(len(lens)):
        rows, at = new[cu[n]:cu[n + 1]], int(lens[n])
        done = 0
        while done < len(rows):
            p, slot = int(table[n, (at + done) // ps]), (at + done) % ps
            m = min(ps - slot, len(rows) - done)
            part = rows[done:done + m]
            if scale is None:
                cache[p, slot:slot + m] = part
            else:
                for g in range(G):
                    s = power_for(float(part[:, g].float().abs().max()))
                    if slot and not math.isnan(s):
                        old = float(scale[p, g])
                        s = max(s, old) if not math.isnan(old) else math.nan
                    if slot:
                        cache[p, :slot, g] = (cache[p, :slot, g].double() * (float(scale[p, g]) / s)).float().to(cache.dtype)
                    scale[p, g] = s
                    cache[p, slot:slot + m, g] = (part[:, g].double() / s).float().to(cache.dtype)
            done += m


def close(got, ref, mag, what=""):
    """got (bfloat16) within half a step of the result and of the rounded weights."""
    got = got.double()
    tol = HALF_STEP * ref.abs() + (HALF_STEP + SLACK) * mag + 1e-30
    worst = float(((got - ref).abs() / tol).max()) if got.numel() else 0.0
    assert not math.isnan(worst) and worst <= 1.0, (what, worst)


def lse_close(got, ref, q_abs):
    """Natural log of a float32 sum of exponentials: the scores' float32 sums (of magnitude below
    q_abs) and the logarithm's own rounding."""
    empty = torch.isinf(ref)
    assert torch.equal(torch.isinf(got) & (got < 0), empty)
    if empty.all():
        return
    err = (got.double() - ref)[~empty].abs()
    assert float((err / (576 * 2.0 ** -24 * q_abs + 2.0 ** -20 * (1 + ref[~empty].abs()))).max()) <= 1.0
