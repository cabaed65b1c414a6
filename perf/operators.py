"""Cases of attention with shaped scores (training and prompts) and of attention over a
key/value cache held in 4 bits (append, read back, single tokens and short drafts).

Shaped scores: t = softcap * tanh(scale * q.k / softcap) - slope_h * |i - j|, over the keys
that the window, the causal mask with its prefix, and the documents of a packed row leave.

The cache: pages of `page` tokens. codes [n_pages, 2 (K, V), kv heads, page, d / 2] uint8, the
even channel of a pair in the low four bits; params [n_pages, 2, kv heads, page, 2] (scale,
zero) in the model's type. A value is scale * code + zero. page_table [B, pages per sequence]
int32, -1 where a sequence has no page.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one prompt of a chat turn: the smallest forward, where latency counts
        dict(name="prompt_small", op="forward", type="bf16", B=1, H=8, Hkv=8, N=77, d=128, left=-1,
             causal=True, cap=50.0, bias=False, docs=0, pad=0, prefix=0),
        # a long prompt through a layer with a sliding window and capped scores
        dict(name="prompt_window", op="forward", type="bf16", B=2, H=16, Hkv=8, N=8192, d=128, left=1024,
             causal=True, cap=30.0, bias=False, docs=0, pad=0, prefix=0),
        # pretraining at GPT-2's shape with a linear distance bias
        dict(name="train_bias", op="train", type="f16", B=8, H=12, Hkv=12, N=1024, d=64, left=-1,
             causal=True, cap=0.0, bias=True, docs=0, pad=0, prefix=0),
        # packed pretraining rows: ragged documents, a padded tail, shared key/value heads
        dict(name="train_documents", op="train", type="bf16", B=2, H=16, Hkv=4, N=4096, d=128, left=-1,
             causal=True, cap=0.0, bias=False, docs=11, pad=190, prefix=0),
        # fine-tuning on pairs whose first part sees itself both ways; odd length, all score terms
        dict(name="train_prefix", op="train", type="bf16", B=3, H=8, Hkv=2, N=1531, d=64, left=-1,
             causal=True, cap=20.0, bias=True, docs=5, pad=64, prefix=3),
        # long-context training with capped scores: the largest
        dict(name="train_long", op="train", type="bf16", B=1, H=8, Hkv=8, N=16384, d=128, left=-1,
             causal=True, cap=50.0, bias=False, docs=0, pad=0, prefix=0),
        # one decoded token for each of a few sequences goes into the cache
        dict(name="append_token", op="append", type="bf16", B=4, Hkv=8, d=128, n=1, L=1000, page=64),
        # prompts of a serving batch go into the cache
        dict(name="append_prompts", op="append", type="bf16", B=16, Hkv=8, d=128, n=2048, L=5000, page=64),
        # the first tokens of a single answer: latency
        dict(name="decode_small", op="attend", type="bf16", B=1, H=8, Hkv=8, d=64, q=1, L=127, page=16,
             left=-1, cap=0.0, bias=False),
        # a full serving batch, ragged lengths, capped scores
        dict(name="decode_batch", op="attend", type="bf16", B=64, H=32, Hkv=8, d=128, q=1, L=8192, page=64,
             left=-1, cap=50.0, bias=False),
        # one very long document
        dict(name="decode_long", op="attend", type="f16", B=1, H=32, Hkv=4, d=128, q=1, L=131071, page=128,
             left=-1, cap=0.0, bias=True),
        # drafts of five tokens checked at once, in a layer with a sliding window
        dict(name="decode_draft", op="attend", type="bf16", B=8, H=16, Hkv=4, d=128, q=5, L=4099, page=32,
             left=2047, cap=0.0, bias=False),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["forward", "train", "train", "append", "attend", "attend"])
    kind = rng.choice(["bf16", "bf16", "f16"])
    d = rng.choice([64, 128])
    if op in ("forward", "train"):
        Hkv = rng.choice([1, 2, 4, 8])
        H = Hkv * rng.choice([1, 1, 2, 4])
        N = _spread(rng, 1, 16384)
        most = (1 << 29) // (H * N * N)
        B = max(1, min(_spread(rng, 1, 16), most))
        while B * H * N * N > 1 << 30:
            N = N // 2 + 1
        docs = rng.choice([0, 0, rng.randint(1, 16)])
        return dict(op=op, type=kind, B=B, H=H, Hkv=Hkv, N=N, d=d, left=rng.choice([-1, -1, _spread(rng, 1, N)]),
                    causal=rng.random() < 0.8, cap=rng.choice([0.0, 20.0, 30.0, 50.0]), bias=rng.random() < 0.4,
                    docs=docs, pad=rng.randint(0, N // 4) if docs else 0, prefix=rng.choice([0, 0, rng.randint(1, 8)]))
    Hkv = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128, 256])
    B = _spread(rng, 1, 64)
    if op == "append":
        n = min(_spread(rng, 1, 4096), max(1, (1 << 18) // (B * Hkv)))
        return dict(op=op, type=kind, B=B, Hkv=Hkv, d=d, n=n, L=n + _spread(rng, 1, 4096), page=page)
    L = min(_spread(rng, 1, 131072), max(1, (1 << 22) // (B * Hkv)))
    return dict(op=op, type=kind, B=B, H=Hkv * rng.choice([1, 2, 4, 8]), Hkv=Hkv, d=d, q=rng.choice([1, 1, 2, 5, 8]), L=L,
                page=page, left=rng.choice([-1, -1, _spread(rng, 1, L)]), cap=rng.choice([0.0, 0.0, 50.0]),
                bias=rng.random() < 0.3)


# ------------------------------------------------------------------ what a case's ragged parts are


def _documents(case):
    """Offsets [B][docs + 1] of the documents of each row (the tail behind the last is padding)
    and how many of each document's first tokens see each other both ways [B][docs]."""
    B, N, M = case["B"], case["N"], max(1, case["docs"])
    rows, pre = [], []
    for b in range(B):
        used = N - case["pad"] * (b + 1) // B
        inner = sorted(int((((i + 1) * 0.618034 + 0.37 * b) % 1.0) * used) for i in range(M - 1))
        cuts = [0] + inner + [used]
        rows.append(cuts)
        pre.append([(cuts[m + 1] - cuts[m]) * case["prefix"] // 8 for m in range(M)])
    return rows, pre


def _lengths(case):
    """Tokens of each sequence, from a quarter of the longest to the longest."""
    B, L = case["B"], case["L"]
    return [max(1, L - (L * 3 // 4) * ((b * 5) % B) // B) for b in range(B)]


def _counts(case):
    """New tokens of each sequence: the longest prompt and shorter ones."""
    B, n = case["B"], case["n"]
    return [max(1, n - (n // 2) * ((b * 3) % B) // B) for b in range(B)]


def _slopes(H, device):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=torch.float32, device=device)


def _visible(case):
    """Keys that each row sees, summed over the rows and the batch."""
    rows, pre = _documents(case)
    total = 0
    for cuts, p in zip(rows, pre):
        for m in range(len(p)):
            s, e = cuts[m], cuts[m + 1]
            if e <= s:
                continue
            i = torch.arange(s, e)
            lo = torch.clamp(i - case["left"], min=s) if case["left"] >= 0 else torch.full_like(i, s)
            hi = torch.clamp(i + 1, min=s + p[m], max=e) if case["causal"] else torch.full_like(i, e)
            total += int((hi - lo).sum())
    return total


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["type"]]
    d, B, Hkv = case["d"], case["B"], case["Hkv"]

    def normal(*shape, gain=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * gain).to(dt)

    st = dict(case=case, scale=1.0 / math.sqrt(d))
    if case["op"] in ("forward", "train"):
        H, N = case["H"], case["N"]
        # capped models are those whose scores grow large
        st["q"] = normal(B, H, N, d, gain=4.0 if case["cap"] else 1.0)
        st["k"], st["v"] = normal(B, Hkv, N, d), normal(B, Hkv, N, d)
        if case["op"] == "train":
            st["do"] = normal(B, H, N, d)
        rows, pre = _documents(case)
        st["documents"] = torch.tensor(rows, dtype=torch.int32, device=dev) if case["docs"] else None
        st["prefix"] = torch.tensor(pre, dtype=torch.int32, device=dev) if case["prefix"] else None
        st["slopes"] = _slopes(H, dev) if case["bias"] else None
        return st
    page, L = case["page"], case["L"]
    per = -(-L // page)
    n_pages = B * per + 3
    order = torch.randperm(n_pages, generator=gen, device=dev)[:B * per].reshape(B, per).to(torch.int32)
    # keys and values with means of their own in each channel, as projections give them
    mean = torch.randn(2, Hkv, 1, d, generator=gen, device=dev) * 0.5
    st["codes"] = torch.empty(n_pages, 2, Hkv, page, d // 2, dtype=torch.uint8, device=dev)
    st["params"] = torch.empty(n_pages, 2, Hkv, page, 2, dtype=dt, device=dev)
    step = max(1, (1 << 26) // (2 * Hkv * page * d))
    for a in range(0, n_pages, step):
        x = torch.randn(min(step, n_pages - a), 2, Hkv, page, d, generator=gen, device=dev) + mean
        st["codes"][a:a + step], st["params"][a:a + step] = _quantise(x.to(dt))
    if case["op"] == "append":
        count = _counts(case)
        tokens = torch.tensor(count, dtype=torch.int32, device=dev)
        st["counts"] = tokens
        st["positions"] = torch.tensor([(L - case["n"]) * (b + 1) // B for b in range(B)], dtype=torch.int32, device=dev)
        st["table"] = order.contiguous()
        st["k"] = (torch.randn(B, Hkv, case["n"], d, generator=gen, device=dev) + mean[0]).to(dt)
        st["v"] = (torch.randn(B, Hkv, case["n"], d, generator=gen, device=dev) + mean[1]).to(dt)
        return st
    lengths = torch.tensor(_lengths(case), dtype=torch.int32, device=dev)
    need = (lengths + page - 1) // page
    st["table"] = torch.where(torch.arange(per, device=dev)[None] < need[:, None], order, torch.full_like(order, -1))
    st["lengths"] = lengths
    st["slopes"] = _slopes(case["H"], dev) if case["bias"] else None
    st["q"] = normal(B, case["H"], case["q"], d, gain=4.0 if case["cap"] else 1.0)
    return st


# ------------------------------------------------------------------ plain forms, 32 bits


def _quantise(x):
    """codes and (scale, zero) of rows of the last axis."""
    f = x.float()
    low, high = f.amin(-1, keepdim=True), f.amax(-1, keepdim=True)
    scale = (high / 15.0 - low / 15.0).to(x.dtype)
    c = torch.round((f - low) / scale.float()).clamp(0.0, 15.0)
    c = torch.where(scale > 0, c, torch.zeros_like(c)).to(torch.uint8)
    codes = c[..., 0::2] | (c[..., 1::2] << 4)
    return codes, torch.cat([scale, low.to(x.dtype)], -1)


def _values(codes, params):
    """What codes and params stand for, in 32 bits."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    return c * params[..., :1].float() + params[..., 1:].float()


def _scores(case, st, q, k, distance, mask):
    """softmax weights, tanh of the capped scores (or None) and the log-sum-exp."""
    s = (q @ k.transpose(-1, -2)) * st["scale"]
    th = None
    if case["cap"]:
        th = torch.tanh(s / case["cap"])
        s = case["cap"] * th
    if st["slopes"] is not None:
        s = s - st["slopes"][..., None, None] * distance
    s = torch.where(mask, s, torch.full_like(s, -math.inf))
    top = s.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total)).squeeze(-1)
    return p / torch.where(total > 0, total, torch.ones_like(total)), th, lse


def _plain_shaped(case, st):
    q, k, v = st["q"].float(), st["k"].float(), st["v"].float()
    dt, B, N, H, Hkv = st["q"].dtype, case["B"], case["N"], case["H"], case["Hkv"]
    pos = torch.arange(N, device=q.device)
    cuts = st["documents"]
    if cuts is None:
        cuts = torch.tensor([[0, N]], dtype=torch.int32, device=q.device).expand(B, 2)
    of = (pos[None, :, None] >= cuts[:, None, :]).sum(-1) - 1  # [B, N]: the token's document
    real = (of >= 0) & (of < cuts.shape[1] - 1)
    of = of.clamp(0, cuts.shape[1] - 2)
    start = cuts.long().gather(1, of)
    ahead = start + (st["prefix"].long().gather(1, of) if st["prefix"] is not None else 0)
    mask = real[:, :, None] & real[:, None, :] & (of[:, :, None] == of[:, None, :])
    if case["causal"]:
        mask = mask & ((pos[None, None, :] <= pos[None, :, None]) | (pos[None, None, :] < ahead[:, None, :]))
    if case["left"] >= 0:
        mask = mask & (pos[None, :] >= pos[:, None] - case["left"])
    g = H // Hkv
    ke, ve = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
    p, th, lse = _scores(case, st, q, ke, (pos[:, None] - pos[None, :]).abs().float(), mask[:, None])
    o = p @ ve
    if case["op"] == "forward":
        return o.to(dt), lse
    do = st["do"].float()
    dp = do @ ve.transpose(-1, -2)
    dv = p.transpose(-1, -2) @ do
    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * st["scale"]
    if th is not None:
        ds = ds * (1.0 - th * th)
    dq = ds @ ke
    dk = ds.transpose(-1, -2) @ q
    shared = (B, Hkv, g, N, case["d"])
    return o.to(dt), lse, dq.to(dt), dk.reshape(shared).sum(2).to(dt), dv.reshape(shared).sum(2).to(dt)


def _plain_append(case, st):
    n, page = case["n"], case["page"]
    at = st["positions"].long()[:, None] + torch.arange(n, device=st["k"].device)  # [B, n]
    there = torch.arange(n, device=at.device)[None] < st["counts"][:, None]
    where = at.clamp(max=st["table"].shape[1] * page - 1)
    pages = st["table"].long().gather(1, where // page)[there]
    slots = (where % page)[there]
    kv = torch.stack([st["k"], st["v"]], 1).permute(0, 3, 1, 2, 4)[there]  # [rows, 2, Hkv, d]
    codes, params = _quantise(kv)
    st["codes"][pages, :, :, slots] = codes
    st["params"][pages, :, :, slots] = params
    back = _values(st["codes"][pages, :, :, slots], st["params"][pages, :, :, slots]).to(st["k"].dtype)
    out = torch.zeros(case["B"], n, 2, case["Hkv"], case["d"], dtype=st["k"].dtype, device=at.device)
    out[there] = back
    return out[:, :, 0].transpose(1, 2).contiguous(), out[:, :, 1].transpose(1, 2).contiguous()


def _plain_attend(case, st):
    B, Hkv, page, d, n = case["B"], case["Hkv"], case["page"], case["d"], case["q"]
    table = st["table"].long().clamp(min=0)
    all_rows = table.shape[1] * page
    kv = _values(st["codes"][table], st["params"][table])  # [B, pages, 2, Hkv, page, d]
    kv = kv.permute(2, 0, 3, 1, 4, 5).reshape(2, B, Hkv, 1, all_rows, d)
    length = st["lengths"].long()[:, None, None]
    at = torch.arange(n, device=table.device)[None, :, None] + length - n  # [B, q, 1]
    key = torch.arange(all_rows, device=table.device)
    mask = key <= at
    if case["left"] >= 0:
        mask = mask & (key >= at - case["left"])
    g = case["H"] // Hkv
    q = st["q"].float().reshape(B, Hkv, g, n, d)
    part = dict(st, slopes=None if st["slopes"] is None else st["slopes"].reshape(Hkv, g))
    distance = (at - key).float()[:, None, None]
    p, _, lse = _scores(case, part, q, kv[0], distance, mask[:, None, None])
    o = p @ kv[1]
    return o.reshape(B, case["H"], n, d).to(st["q"].dtype), lse.reshape(B, case["H"], n)


def run(st):
    case = st["case"]
    if not own:
        plain = {"append": _plain_append, "attend": _plain_attend}.get(case["op"], _plain_shaped)
        return plain(case, st)
    from io_aware_attention_flashattention_b200 import api

    cap = case.get("cap") or None
    if case["op"] == "append":
        api.cache4_append(st["codes"], st["params"], st["k"], st["v"], st["table"], st["positions"], counts=st["counts"])
        return api.cache4_read(st["codes"], st["params"], st["table"], st["positions"], case["n"], counts=st["counts"])
    if case["op"] == "attend":
        return api.cache4_attend(st["q"], st["codes"], st["params"], st["table"], st["lengths"], scale=st["scale"],
                                 window_left=case["left"], softcap=cap, slopes=st["slopes"], max_len=case["L"])
    how = dict(causal=case["causal"], scale=st["scale"], window=(case["left"], -1), softcap=cap, slopes=st["slopes"],
               documents=st["documents"], prefix=st["prefix"])
    o, lse = api.forward(st["q"], st["k"], st["v"], **how)
    if case["op"] == "forward":
        return o, lse
    return (o, lse) + tuple(api.backward(st["q"], st["k"], st["v"], o, lse, st["do"], **how))


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    d = case["d"]
    if case["op"] in ("forward", "train"):
        pairs = _visible(case) * case["H"]
        rows = case["B"] * case["N"]
        fwd = rows * (case["H"] * (4 * d + 4) + case["Hkv"] * 4 * d)  # q, o, lse; k, v
        if case["op"] == "forward":
            return {"bytes": fwd, "flops": 4 * d * pairs}
        return {"bytes": fwd + rows * (case["H"] * 4 * d + case["Hkv"] * 4 * d), "flops": 14 * d * pairs}
    row = d // 2 + 4
    if case["op"] == "append":
        rows = sum(_counts(case)) * case["Hkv"] * 2
        return {"bytes": rows * (2 * d + row) * 2, "flops": rows * d * 6}
    left = case["left"]
    seen = [n if left < 0 else min(n, left + case["q"]) for n in _lengths(case)]
    new = case["B"] * case["H"] * case["q"]
    return {"bytes": sum(seen) * case["Hkv"] * 2 * row + new * (4 * d + 4),
            "flops": 4 * d * sum(seen) * case["H"] * case["q"]}


# ------------------------------------------------------------------ the definitions in 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend}.get(case["op"], _exact_shaped)(case, st)


def _exact_shaped(case, st):
    B, H, N, d, g = case["B"], case["H"], case["N"], case["d"], case["H"] // case["Hkv"]
    rows, pre = _documents(case)
    q, k, v = st["q"], st["k"], st["v"]
    o = torch.zeros(B, H, N, d, dtype=torch.float64, device=q.device)
    lse = torch.full((B, H, N), -math.inf, dtype=torch.float64, device=q.device)
    dq = torch.zeros_like(o)
    dk = torch.zeros(B, case["Hkv"], N, d, dtype=torch.float64, device=q.device)
    dv = torch.zeros_like(dk)
    for b in range(B):
        for m in range(len(pre[b])):
            s, e = rows[b][m], rows[b][m + 1]
            for a in range(s, e, 4096):  # rows [a, z) of one document against all its keys
                z = min(e, a + 4096)
                i = torch.arange(a, z, device=q.device)[:, None]
                j = torch.arange(s, e, device=q.device)[None]
                hidden = torch.zeros(z - a, e - s, dtype=torch.bool, device=q.device)
                if case["causal"]:
                    hidden |= (j > i) & (j - s >= pre[b][m])
                if case["left"] >= 0:
                    hidden |= i - j > case["left"]
                for h in range(H):
                    kk, vv, qq = k[b, h // g, s:e].double(), v[b, h // g, s:e].double(), q[b, h, a:z].double()
                    x = torch.einsum("id,jd->ij", qq, kk).mul_(st["scale"])
                    slope = 1.0
                    if case["cap"]:
                        y = torch.exp(2.0 * x / case["cap"])
                        y = 1.0 - 2.0 / (1.0 + y)
                        x, slope = case["cap"] * y, 1.0 - y * y
                    if case["bias"]:
                        x = x - st["slopes"][h].double() * (i - j).abs()
                    x = x.masked_fill(hidden, -math.inf)
                    lse[b, h, a:z] = torch.logsumexp(x, -1)
                    w = torch.exp(x - lse[b, h, a:z, None])
                    o[b, h, a:z] = torch.einsum("ij,jd->id", w, vv)
                    if case["op"] == "train":
                        do = st["do"][b, h, a:z].double()
                        dv[b, h // g, s:e] += torch.einsum("ij,id->jd", w, do)
                        back = torch.einsum("id,jd->ij", do, vv) - (do * o[b, h, a:z]).sum(-1, keepdim=True)
                        back = back.mul_(w).mul_(slope).mul_(st["scale"])
                        dq[b, h, a:z] = torch.einsum("ij,jd->id", back, kk)
                        dk[b, h // g, s:e] += torch.einsum("ij,id->jd", back, qq)
    return (o, lse) if case["op"] == "forward" else (o, lse, dq, dk, dv)


def _exact_append(case, st):
    out = []
    for x in (st["k"], st["v"]):
        w = x.double()
        low = w.min(-1, keepdim=True).values
        unit = ((w.max(-1, keepdim=True).values - low) / 15).to(x.dtype).double()
        code = torch.where(unit > 0, ((w - low) / unit).round().clamp(0, 15), torch.zeros_like(w))
        value = low + code * unit
        for b, n in enumerate(_counts(case)):
            value[b, :, n:] = 0
        out.append(value)
    return tuple(out)


def _exact_attend(case, st):
    B, H, n, d, page, g = case["B"], case["H"], case["q"], case["d"], case["page"], case["H"] // case["Hkv"]
    o = torch.zeros(B, H, n, d, dtype=torch.float64, device=st["q"].device)
    lse = torch.full((B, H, n), -math.inf, dtype=torch.float64, device=o.device)
    for b, length in enumerate(_lengths(case)):
        pages = st["table"][b, :-(-length // page)].long()
        for h in range(H):
            rows = []
            for which in (0, 1):
                c, w = st["codes"][pages, which, h // g].reshape(-1, d // 2), st["params"][pages, which, h // g].reshape(-1, 2).double()
                x = torch.empty(c.shape[0], d, dtype=torch.float64, device=o.device)
                x[:, 0::2], x[:, 1::2] = (c % 16).double(), (c // 16).double()
                rows.append((x * w[:, :1] + w[:, 1:])[:length])
            for t in range(n):
                i = length - n + t
                lo = max(0, i - case["left"]) if case["left"] >= 0 else 0
                if i < 0:
                    continue
                x = rows[0][lo:i + 1] @ st["q"][b, h, t].double() * st["scale"]
                if case["cap"]:
                    x = case["cap"] * torch.tanh(x / case["cap"])
                if case["bias"]:
                    x = x - st["slopes"][h].double() * (i - torch.arange(lo, i + 1, device=o.device))
                lse[b, h, t] = torch.logsumexp(x, 0)
                o[b, h, t] = torch.exp(x - lse[b, h, t]) @ rows[1][lo:i + 1]
    return o, lse
