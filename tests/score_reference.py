"""Plain 64-bit definitions of attention with shaped scores, for the tests: every score is
formed, nothing is blocked, and the visible pairs are listed one rule at a time."""
import math

import torch


def visible(B, N, causal=False, window=(-1, -1), documents=None, prefix=None):
    """[B, N, N] bool: does query i see key j?"""
    i, j = torch.arange(N)[:, None], torch.arange(N)[None]
    out = torch.zeros(B, N, N, dtype=torch.bool)
    left, right = window
    for b in range(B):
        cuts = [0, N] if documents is None else [int(x) for x in documents[b]]
        for m in range(len(cuts) - 1):
            s, e = cuts[m], cuts[m + 1]
            if e <= s:
                continue
            ahead = s if prefix is None else s + max(0, int(prefix.reshape(B, -1)[b][m]))
            inside = (i >= s) & (i < e) & (j >= s) & (j < e)
            r = 0 if causal else right
            if r >= 0:
                inside = inside & ((j <= i + r) | (j < ahead))
            if left >= 0:
                inside = inside & (j >= i - left)
            out[b] |= inside
    return out


def attention(q, k, v, mask, scale, softcap=None, slopes=None):
    """(o, lse) in 64 bits; differentiable. mask: [B, N, N]."""
    q, k, v = q.double(), k.double(), v.double()
    H, Hkv, N = q.shape[1], k.shape[1], q.shape[2]
    of = torch.arange(H, device=q.device) // (H // Hkv)  # the K/V head of each query head
    s = torch.einsum("bhid,bhjd->bhij", q, k[:, of]) * scale
    if softcap is not None:
        s = softcap * torch.tanh(s / softcap)
    if slopes is not None:
        at = torch.arange(N, dtype=torch.float64, device=q.device)
        s = s - slopes.double()[None, :, None, None] * (at[:, None] - at[None]).abs()
    s = s.masked_fill(~mask[:, None], -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[..., None])
    return torch.einsum("bhij,bhjd->bhid", p, v[:, of]), lse


def unit(dtype):
    """Largest relative error of one rounding to the type, and the absolute one near zero."""
    return torch.finfo(dtype).eps / 2, torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2


def gradients(q, k, v, do, mask, scale, softcap=None, slopes=None):
    """(values, bounds), each (o, lse, dq, dk, dv), in 64 bits; the gradients by the formulas
    dS = P o (dP - rowsum(dO o O)) * (1 - tanh^2) * scale, summed over shared heads.

    The bounds follow the roundings that the method makes, with u the type's unit roundoff:
      logits: d products summed in 32 bits, then the cap (3e-7 of its result, or 4e-7 of the
        cap) and the bias, each rounded once: err_t <= 2^-23 (d sum|q k| scale + 8 (|t| + cap
        + 1)) per score, and LSE as much, plus its own rounding;
      P: err_t twice (score and LSE) and one rounding to the type: e_p = u + 2 max err_t;
      O: e_p on every weight, u again for the sum of the rounded weights that O is divided
        by, and u for O itself;
      D: dO times the error of the rounded O;
      dS: P times the error of D, and e_p + u of itself; dQ, dK, dV: those through |K|, |Q|,
        |dO|, and u for the output itself.
    A twentieth is added for the products of these small terms and the sums in 32 bits."""
    dtype, d = q.dtype, q.shape[-1]
    u, tiny = unit(dtype)
    q, k, v, do = q.double(), k.double(), v.double(), do.double()
    B, H, N, _ = q.shape
    Hkv = k.shape[1]
    of = torch.arange(H, device=q.device) // (H // Hkv)
    kx, vx = k[:, of], v[:, of]
    o, lse = attention(q, k, v, mask, scale, softcap, slopes)
    dot = lambda a, b: torch.einsum("bhid,bhjd->bhij", a, b)  # noqa: E731
    x = dot(q, kx) * scale
    th = torch.tanh(x / softcap) if softcap is not None else torch.zeros_like(x)
    t = softcap * th if softcap is not None else x
    if slopes is not None:
        at = torch.arange(N, dtype=torch.float64, device=q.device)
        t = t - slopes.double()[None, :, None, None] * (at[:, None] - at[None]).abs()
    seen = mask[:, None] & (lse > -math.inf)[..., None]
    zero = torch.zeros_like(t)
    p = torch.where(seen, torch.exp(torch.where(seen, t - lse[..., None], zero)), zero)
    dp = dot(do, vx)
    shape = (1.0 - th * th) * scale
    ds = p * (dp - (do * o).sum(-1, keepdim=True)) * shape
    cap = 0.0 if softcap is None else softcap
    err_t = torch.where(seen, 2.0 ** -23 * (d * dot(q.abs(), kx.abs()) * scale
                                            + 8 * (t.abs() + cap + 1)), zero)
    b_lse = err_t.amax(-1) + 2.0 ** -23 * torch.where(lse > -math.inf, lse.abs(), lse * 0 + 1) + 1e-6
    b_lse = torch.where(lse > -math.inf, b_lse, torch.zeros_like(b_lse))
    e_p = u + 2 * err_t.amax(-1, keepdim=True)
    err_p = e_p * p + tiny * seen
    b_o = torch.einsum("bhij,bhjd->bhid", err_p + u * p, vx.abs()) + u * o.abs() + tiny
    b_d = (do.abs() * b_o).sum(-1, keepdim=True) + d * 2.0 ** -23 * dot(do.abs(), vx.abs()).amax(
        -1, keepdim=True)
    err_s = p * b_d * shape + (e_p + u) * ds.abs() + tiny * seen * scale
    if softcap is not None:
        # 1 - tanh^2 from tanh in 32 bits. With r = 1 / (1 + e^2x): the exponential is off by
        # 2^-22 of itself and by its argument's rounding (|2x| 2^-24), which r (1 - r) and
        # r (1 - r) |2x| <= 0.45 bring down to 0.25 * 2^-22 + 0.45 * 2^-24; the reciprocal adds
        # 2^-23 + 2^-24 at most: r is off by 3e-7 and tanh = 1 - 2r by 6.3e-7. So its square
        # is off by 2 * 6.3e-7 and the difference's own rounding: 1.5e-6, absolute, which
        # counts where tanh is near 1.
        err_s = err_s + p * (dp - (do * o).sum(-1, keepdim=True)).abs() * scale * 1.5e-6
    values, bounds = [o, lse], [b_o, b_lse]

    def keep(value, bound):
        values.append(value)
        bounds.append(1.05 * bound + u * value.abs() + tiny)

    keep(torch.einsum("bhij,bhjd->bhid", ds, kx), torch.einsum("bhij,bhjd->bhid", err_s, kx.abs()))
    share = (B, Hkv, H // Hkv, N, d)
    turn = lambda a, b: torch.einsum("bhij,bhid->bhjd", a, b).reshape(share).sum(2)  # noqa: E731
    keep(turn(ds, q), turn(err_s, q.abs()))
    keep(turn(p, do), turn(err_p, do.abs()))
    return values, bounds
