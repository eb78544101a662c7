"""64-bit forms of packed and paged attention with error bounds for their 16-bit kernels (CPU).

Every bound counts roundings.  u is half a step of the 16-bit type (torch.finfo(t).eps / 2).  A
score is a sum of d products accumulated in float32, each addition off by at most one step of
2^-23 of the terms' absolute sum: delta = (d + 4) 2^-23 max_j scale sum_c |q_c k_jc|, to which
2^-21 is added for the exponential of its scaled value; a softmax weight is then off by a factor
within 1 +- 2 delta (its own score and the normalisation).
"""
from __future__ import annotations

import math

import torch

SLACK = 1.05      # products of two roundings


def offsets(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def _score_error(q, k, scale):
    d = q.shape[-1]
    return (d + 4) * 2.0 ** -23 * (scale * (q.abs() @ k.abs().T)).amax(1, keepdim=True) + 2.0 ** -21


def attend(q, k, v, last, scale, u):
    """One head: row i of q over keys 0 .. last[i].  (p, out, its bound, lse, its bound, score error).
    A row with last[i] < 0 is zero and its lse -inf."""
    z = scale * (q @ k.T)
    seen = torch.arange(k.shape[0])[None] <= last[:, None]
    z = z.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(z, 1) if k.shape[0] else torch.full((q.shape[0],), -math.inf, dtype=q.dtype)
    some = seen.any(1, keepdim=True) if k.shape[0] else torch.zeros(q.shape[0], 1, dtype=torch.bool)
    p = torch.where(seen & some, torch.exp(z - lse[:, None]), torch.zeros_like(z))
    vv = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
    out = p @ vv
    delta = _score_error(q, k, scale) if k.shape[0] else torch.zeros(q.shape[0], 1, dtype=q.dtype)
    # each weight: its rounding (u; 2 u where the sum takes rounded weights) and 2 delta; then out's rounding
    bound = SLACK * ((2 * u + 2 * delta) * (p @ vv.abs()) + u * out.abs()) + 1e-7
    # lse: the largest relative change of a sum of weights, and of float32 itself
    lse_bound = SLACK * delta[:, 0] + 4e-7 * (1 + lse.abs().nan_to_num(0, 0, 0)) + 1e-6
    return p, out, bound, lse, lse_bound, delta


def varlen(q, k, v, lens, causal, scale, dtype):
    """[H, T, d] float64 tensors; dict of out, lse and bounds (zeros / 0 behind the last sequence)."""
    G, u = q.shape[0] // k.shape[0], half_step(dtype)
    out, bound = torch.zeros_like(q), torch.zeros_like(q)
    lse, lse_bound = torch.zeros(q.shape[:2]).double(), torch.zeros(q.shape[:2]).double()
    for a, n in zip(offsets(lens), lens):
        r = slice(a, a + n)
        last = torch.arange(n) if causal else torch.full((n,), n - 1)
        for h in range(q.shape[0] if n else 0):
            _, out[h, r], bound[h, r], lse[h, r], lse_bound[h, r], _ = attend(
                q[h, r], k[h // G, r], v[h // G, r], last, scale, u)
    return dict(out=out, bound=bound, lse=lse, lse_bound=lse_bound)


def varlen_grads(q, k, v, dout, lens, causal, scale, dtype):
    """dq, dk, dv in float64, and their bounds."""
    G, u = q.shape[0] // k.shape[0], half_step(dtype)
    g = {x: torch.zeros_like(y) for x, y in (("dq", q), ("dk", k), ("dv", v))}
    b = {x: torch.zeros_like(y) for x, y in g.items()}
    d = q.shape[-1]
    for a, n in zip(offsets(lens), lens):
        r = slice(a, a + n)
        last = torch.arange(n) if causal else torch.full((n,), n - 1)
        for h in range(q.shape[0] if n else 0):
            j = h // G
            qh, kh, vh, oh = q[h, r], k[j, r], v[j, r], dout[h, r]
            p, _, _, _, _, delta = attend(qh, kh, vh, last, scale, u)
            dp = oh @ vh.T
            mean = (p * dp).sum(1, keepdim=True)
            dz = p * (dp - mean)
            # dP and Delta: float32 sums of d products
            edp = (d + 4) * 2.0 ** -23 * (oh.abs() @ vh.abs().T).amax(1, keepdim=True)
            # the forward's weights are off by up to u + 2 delta each, and its sum takes them as they
            # are rounded: Delta moves by at most their P-weighted deviations |dP - Delta|
            emean = (2 * u + 2 * delta) * (p * (dp - mean).abs()).sum(1, keepdim=True) + edp
            # P from the forward's lse (rounded weights: u), its scores (2 delta); dz's own rounding (u)
            ez = (2 * u + 2 * delta) * dz.abs() + p * (emean + edp)
            g["dq"][h, r] = scale * (dz @ kh)
            b["dq"][h, r] = scale * (ez @ kh.abs())
            g["dk"][j, r] += scale * (dz.T @ qh)
            b["dk"][j, r] += scale * (ez.T @ qh.abs())
            g["dv"][j, r] += p.T @ oh
            b["dv"][j, r] += ((2 * u + 2 * delta) * p).T @ oh.abs()
    for x in g:
        b[x] = SLACK * (b[x] + u * g[x].abs()) + 1e-7
    return g, b


def paged(q, k_cache, v_cache, table, new, kv, scale, dtype):
    """q [Hq, T, d], caches [P, Hkv, ps, d] float64, table a list of lists."""
    Hkv, ps, d = k_cache.shape[1:]
    G, u = q.shape[0] // Hkv, half_step(dtype)
    out, bound = torch.zeros_like(q), torch.zeros_like(q)
    lse, lse_bound = torch.zeros(q.shape[:2]).double(), torch.zeros(q.shape[:2]).double()
    for b, (a, n, m) in enumerate(zip(offsets(new), new, kv)):
        ids = [int(x) for x in table[b][: -(-m // ps)]]
        r = slice(a, a + n)
        for h in range(q.shape[0] if n else 0):
            k, v = (c[ids, h // G].reshape(-1, d)[:m] for c in (k_cache, v_cache))
            _, out[h, r], bound[h, r], lse[h, r], lse_bound[h, r], _ = attend(
                q[h, r], k, v, torch.arange(m - n, m), scale, u)
    return dict(out=out, bound=bound, lse=lse, lse_bound=lse_bound)


def plan(past, new, table, free, num_free, page_size, T):
    """The page plan in plain Python; table is a list of lists, changed in place."""
    width = len(table[0])
    need = [-(-(p + n) // page_size) - -(-p // page_size) if p >= 0 and n >= 0 else 0
            for p, n in zip(past, new)]
    fits = (all(p >= 0 and n >= 0 and -(-(p + n) // page_size) <= width for p, n in zip(past, new))
            and sum(new) <= T and sum(need) <= num_free)
    if not fits:
        return dict(slots=[-1] * T, cu=[0] * (len(past) + 1), kv_lens=list(past), num_free=num_free, ok=False)
    slots = []
    for b, (p, n) in enumerate(zip(past, new)):
        for i in range(-(-p // page_size), -(-(p + n) // page_size)):
            num_free -= 1
            table[b][i] = free[num_free]
        slots += [table[b][x // page_size] * page_size + x % page_size for x in range(p, p + n)]
    return dict(slots=slots + [-1] * (T - len(slots)), cu=offsets(new),
                kv_lens=[p + n for p, n in zip(past, new)], num_free=num_free, ok=True)


def check(got, want, bound, what):
    got = got.detach().double().cpu()
    err = (got - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} values outside their bound, "
                           f"worst {float((err / bound).nan_to_num(1e9).max()):.3g} of it, first at "
                           f"{[int(x) for x in bad.nonzero()[0]]}: {float(got[bad][0])} want {float(want[bad][0])}")
