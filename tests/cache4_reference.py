"""Plain definitions of the 4-bit cache for the tests: quantised rows, their values, and the
attention over them in 64 bits, one sequence and head at a time."""
import math

import torch

import score_reference as ref


def quantise(x):
    """(code, scale, zero) of rows of the last axis; every step in 32 bits, as specified."""
    f = x.float()
    low, high = f.amin(-1, keepdim=True), f.amax(-1, keepdim=True)
    fifteenth = torch.tensor(1.0 / 15.0, dtype=torch.float32, device=x.device)
    scale = (high * fifteenth - low * fifteenth).to(x.dtype)
    code = torch.round((f - low) / scale.float()).clamp(0, 15)
    code = torch.where(scale > 0, code, torch.zeros_like(code))
    return code.to(torch.uint8), scale, low.to(x.dtype)


def rows(codes, params, table_row, length):
    """(code, scale, zero) [2, Hkv, length, ...] of one sequence, in 64 bits."""
    page = codes.shape[3]
    pages = table_row[:-(-length // page)].long()
    c = torch.stack([codes[pages] & 15, codes[pages] >> 4], -1).flatten(-2).double()
    w = params[pages].double()
    turn = lambda x: x.permute(1, 2, 0, 3, 4).flatten(2, 3)[:, :, :length]  # noqa: E731
    c, w = turn(c), turn(w)
    return c, w[..., :1], w[..., 1:]


def attend(q, codes, params, table, lengths, scale, window_left=-1, softcap=None, slopes=None, gone=()):
    """((o, lse), bounds) in 64 bits. gone: pairs (sequence, page index) that hold nothing.

    The bounds: a score is d products q * (code - 8) summed in 32 bits, times the scale, plus
    sum q times zero + 8 scale: off by at most 2^-23 (d + 8) sum|q| (16 scale + |zero|), and
    31 for 16 leaves room for codes that are not centred; and, as any shaped score,
    8 * 2^-23 (|t| + cap + 1). The weights times the value's scale are rounded to bf16 (2^-8)
    before they meet code - 8, the sums over L tokens are in 32 bits (L * 2^-23 of what is
    summed), and the output is rounded to its type."""
    B, H, n, d = q.shape
    Hkv = codes.shape[2]
    u = ref.unit(q.dtype)[0]
    o = torch.zeros(B, H, n, d, dtype=torch.float64, device=q.device)
    lse = torch.full((B, H, n), -math.inf, dtype=torch.float64, device=q.device)
    b_o, b_lse = torch.zeros_like(o), torch.zeros_like(lse)
    for b in range(B):
        L = int(lengths[b])
        if L == 0:
            continue
        c, s, z = rows(codes, params, table[b].clamp(0, codes.shape[0] - 1), L)
        key = torch.arange(L, device=q.device)
        there = torch.ones(L, dtype=torch.bool, device=q.device)
        for seq, page in gone:
            if seq == b:
                there &= key // codes.shape[3] != page
        for h in range(H):
            hk = h // (H // Hkv)
            kc, ks, kz = c[0, hk], s[0, hk], z[0, hk]
            vc, vs, vz = c[1, hk], s[1, hk], z[1, hk]
            for i in range(n):
                at = L - n + i
                seen = there & (key <= at)
                if window_left >= 0:
                    seen &= key >= at - window_left
                if not seen.any():
                    continue
                x = q[b, h, i].double()
                t = ((ks * kc + kz) @ x * scale)[seen]
                size = (x.abs().sum() * (31 * ks + kz.abs()) * scale).squeeze(-1)[seen]
                if softcap is not None:
                    t = softcap * torch.tanh(t / softcap)
                if slopes is not None:
                    t = t - slopes[h].double() * (at - key[seen])
                err = float((2.0 ** -23 * ((d + 8) * size + 8 * (t.abs() + (softcap or 0) + 1))).max())
                lse[b, h, i] = torch.logsumexp(t, 0)
                p = torch.softmax(t, 0)
                v = (vs * vc + vz)[seen]
                o[b, h, i] = p @ v
                part = p @ (vs * (vc - 8).abs())[seen]
                every = p @ (vs * (vc - 8).abs() + 8 * vs + vz.abs())[seen]
                b_o[b, h, i] = 1.05 * (2.0 ** -8 * part + (2 * err + (L + 8) * 2.0 ** -23) * every) + u * o[b, h, i].abs() + 1e-7
                b_lse[b, h, i] = 1.05 * err + (L + 8) * 2.0 ** -23 + 2.0 ** -22 * abs(float(lse[b, h, i]))
    return (o, lse), (b_o, b_lse)
