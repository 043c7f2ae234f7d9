"""Cases and plain forms of the paged-serving operators: block tables and slot maps from request lengths, the write
of new keys and values into the paged cache, attention with a sliding window and sink tokens (decode and prefill), and
decode for a batch that shares a long prefix.

A step of a server runs them in this order: the lengths of the step's requests are on the GPU; the block tables grow
and every new token gets its slot; the new keys and values go to their slots; attention reads the cache through the
tables.  Sizes follow this repository's workloads: 32 query heads over 8 key/value heads, head dim 128 (64 for the
small prefill), lengths up to a few thousand tokens, contexts up to 32768, pages of 16 to 256 tokens.
"""
import math
import random

import numpy as np
import torch

own = False   # True: run() calls this repository's operators; False: their plain form

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a small batch: one new token each
        dict(name="tables_decode_16", op="tables", B=16, ctx_lo=1, ctx_hi=4095, new_lo=1, new_hi=1, bs=128),
        # prompts of a large batch, chunked and not, admitted at once
        dict(name="tables_prompts_512", op="tables", B=512, ctx_lo=0, ctx_hi=8191, new_lo=1, new_hi=2047, bs=16),
        # the new tokens of one decode step, every layer of the model calls it
        dict(name="write_decode_16", op="write", T=16, N2=8, D=128, bs=128, pool="BNBD", dt="bf16", fused=True),
        # the prompts of a step, keys and values being slices of one fused projection's output
        dict(name="write_prompts_32k", op="write", T=32771, N2=8, D=128, bs=128, pool="BBH", dt="bf16", fused=True),
        # one conversation, far past its window
        dict(name="window_decode_1", op="wdecode", B=1, N1=32, N2=8, D=128, Q=1, lo=20001, hi=20001, pre=1023, sink=4,
             bs=16, dt="bf16"),
        # the paged decode workload's batch with a window
        dict(name="window_decode_16", op="wdecode", B=16, N1=32, N2=8, D=128, Q=1, lo=1, hi=4096, pre=1023, sink=4,
             bs=128, dt="bf16"),
        # a large batch of long contexts, four new tokens each (drafted tokens being checked)
        dict(name="window_decode_64_q4", op="wdecode", B=64, N1=32, N2=8, D=128, Q=4, lo=900, hi=32768, pre=4095,
             sink=16, bs=128, dt="bf16"),
        # the small prefill workload with a window
        dict(name="window_prefill_small", op="wprefill", B=1, N1=2, N2=2, D=64, lo=128, hi=128, ctx_lo=0, ctx_hi=0,
             pre=31, sink=4, layout="BNSD", bs=0, dt="f16"),
        # ragged prompts packed together
        dict(name="window_prefill_tnd", op="wprefill", B=8, N1=32, N2=8, D=128, lo=256, hi=4096, ctx_lo=0, ctx_hi=0,
             pre=1023, sink=4, layout="TND", bs=0, dt="bf16"),
        # chunks of long prompts against what the cache holds of them
        dict(name="window_prefill_chunks", op="wprefill", B=8, N1=32, N2=8, D=128, lo=2048, hi=2048, ctx_lo=0,
             ctx_hi=14336, pre=4095, sink=4, layout="BNSD", bs=256, dt="bf16"),
        # a few answers drawn from one prompt
        dict(name="prefix_decode_8", op="prefix", B=8, N1=32, N2=8, D=128, Q=1, P=2048, lo=1, hi=256, bs=128,
             dt="bf16"),
        # a large batch behind one long system prompt with documents
        dict(name="prefix_decode_64", op="prefix", B=64, N1=32, N2=8, D=128, Q=1, P=32768, lo=1, hi=1024, bs=128,
             dt="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    return rng.choice([(32, 8), (32, 8), (8, 2), (16, 16), (24, 8), (28, 4), (8, 1), (40, 8)])


def draw(rng):
    op = rng.choice(["tables", "write", "wdecode", "wdecode", "wprefill", "wprefill", "prefix", "prefix"])
    dt = rng.choice(["bf16", "bf16", "f16"])
    D = rng.choice([128, 128, 64])
    if op == "tables":
        B = _log(rng, 1, 512)
        hi = rng.choice([1, 4, _log(rng, 2, 2047)])
        return dict(op=op, B=B, ctx_lo=0, ctx_hi=_log(rng, 64, 8191), new_lo=rng.choice([0, 1]), new_hi=hi,
                    bs=rng.choice([16, 32, 64, 128, 256]))
    if op == "write":
        n2 = rng.choice([1, 2, 4, 8, 16])
        return dict(op=op, T=max(1, _log(rng, 1, 32768) // max(1, n2 // 8)), N2=n2, D=D, bs=rng.choice([16, 64, 128, 256]),
                    pool=rng.choice(["BNBD", "BBH"]), dt=dt, fused=rng.choice([True, False]))
    n1, n2 = _heads(rng)
    sink = rng.choice([0, 1, 4, 16, _log(rng, 1, 300)])
    if op == "wdecode":
        q = rng.choice([1, 1, 2, 4, _log(rng, 1, 8)])
        q = q if q * (n1 // n2) <= 64 else 1
        pre = _log(rng, 16, 4095) - 1
        hi = _log(rng, 16, 32768)
        most = 64 * 8 * 4112 * 4 // (n2 * (pre + 1 + sink) * q)
        return dict(op=op, B=max(1, min(most, _log(rng, 1, 64))), N1=n1, N2=n2, D=D, Q=q, lo=rng.choice([1, hi // 2 + 1]),
                    hi=hi, pre=pre, sink=sink, bs=rng.choice([16, 32, 64, 128, 256]), dt=dt)
    if op == "wprefill":
        layout = rng.choice(["TND", "TND", "BNSD", "BSND"])
        paged = layout != "TND" and rng.random() < 0.5
        hi = _log(rng, 16, 2048)
        return dict(op=op, B=_log(rng, 1, 8), N1=n1, N2=n2, D=D, lo=rng.choice([1, hi // 2 + 1, hi]), hi=hi, ctx_lo=0,
                    ctx_hi=_log(rng, 16, 8192) if paged else 0, pre=_log(rng, 16, 2048) - 1, sink=sink, layout=layout,
                    bs=rng.choice([128, 256, 512]) if paged else 0, dt=dt)
    q = rng.choice([1, 1, 1, 2, 4])
    bs = rng.choice([16, 64, 128, 256])
    return dict(op=op, B=_log(rng, 2, 64) // q + 1, N1=n1, N2=n2, D=D, Q=q, P=_log(rng, 256, 16384) // bs * bs + bs, lo=1,
                hi=_log(rng, 4, 1024), bs=bs, dt=dt)


# ------------------------------------------------------------------ inputs
def _spread(lo, hi, n):
    """n lengths spread evenly over [lo, hi]: a case's work does not depend on the seed."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _shuffled(lo, hi, n, rng):
    x = _spread(lo, hi, n)
    rng.shuffle(x)
    return x


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _pages(lengths, bs, rng, spare):
    """Block tables that give every sequence its own blocks, in random order: ([B, columns], blocks in the pool)."""
    need = [-(-n // bs) for n in lengths]
    pool = sum(need) + spare
    ids = np.random.default_rng(rng.randrange(1 << 30)).permutation(pool).astype(np.int32)
    table = np.zeros((len(lengths), max(max(need), 1)), dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return torch.from_numpy(table).cuda(), pool, ids[at:]


def _normal(shape, dt, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(DTYPES[dt])


def prepare(case, seed):
    c = dict(case)
    rng = random.Random("%d" % seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "tables":
        ctx = _shuffled(c["ctx_lo"], c["ctx_hi"], c["B"], rng)
        new = _shuffled(c["new_lo"], c["new_hi"], c["B"], rng)
        total = [a + b for a, b in zip(ctx, new)]
        _, pool, _ = _pages(total, c["bs"], rng, 0)
        held, _, free = _pages(ctx, c["bs"], rng, pool - sum(-(-n // c["bs"]) for n in ctx) + 7)
        table = torch.zeros((c["B"], -(-(c["ctx_hi"] + c["new_hi"]) // c["bs"]) + 2), dtype=torch.int32, device="cuda")
        table[:, :held.shape[1]] = held[:, :table.shape[1]]
        s.update(ctx=_i32(ctx), new=_i32(new), free=torch.from_numpy(free).cuda(), table=table,
                 tokens=sum(new) + (sum(new) % 3))
    elif c["op"] == "write":
        t, n2, d, bs = c["T"], c["N2"], c["D"], c["bs"]
        nb = -(-t // bs) * 2 + 1
        shape = (nb, n2, bs, d) if c["pool"] == "BNBD" else (nb, bs, n2 * d)
        s.update(kc=_normal(shape, c["dt"], g), vc=_normal(shape, c["dt"], g))
        if c["fused"]:   # the projection's output: the queries' columns (4 a key head), then keys, then values
            x = _normal((t, 6 * n2, d), c["dt"], g)
            s.update(k=x[:, 4 * n2:5 * n2], v=x[:, 5 * n2:])
        else:
            s.update(k=_normal((t, n2, d), c["dt"], g), v=_normal((t, n2, d), c["dt"], g))
        # runs of consecutive slots, as sequences have them: whole blocks in random order; a few padded tokens
        blocks = np.random.default_rng(seed).permutation(nb)[:-(-t // bs)]
        slots = (blocks[:, None] * bs + np.arange(bs)).reshape(-1)[:t].astype(np.int32)
        slots[t - t // 16:] = -1
        s["slots"] = torch.from_numpy(slots).cuda()
    elif c["op"] == "wprefill":
        new = _shuffled(c["lo"], c["hi"], c["B"], rng)
        ctx = _shuffled(c["ctx_lo"], c["ctx_hi"], c["B"], rng)
        kv = [a + b for a, b in zip(ctx, new)]
        n1, n2, d, smax = c["N1"], c["N2"], c["D"], c["hi"]
        if c["layout"] == "TND":
            t = sum(new)
            s.update(q=_normal((t, n1, d), c["dt"], g), k=_normal((t, n2, d), c["dt"], g),
                     v=_normal((t, n2, d), c["dt"], g))
            cu = _i32(list(np.cumsum(new)))
            s.update(ql=cu, kl=cu, table=None)
        else:
            swap = (lambda b, n, m, e: (b, n, m, e)) if c["layout"] == "BNSD" else (lambda b, n, m, e: (b, m, n, e))
            s["q"] = _normal(swap(c["B"], n1, smax, d), c["dt"], g)
            s.update(ql=_i32(new), kl=_i32(kv))
            if c["bs"]:
                s["table"], pool, _ = _pages(kv, c["bs"], rng, 3)
                shape = (pool, n2, c["bs"], d)
            else:
                s["table"] = None
                shape = swap(c["B"], n2, smax, d)
            s.update(k=_normal(shape, c["dt"], g), v=_normal(shape, c["dt"], g))
    else:
        n1, n2, d, q, bs = c["N1"], c["N2"], c["D"], c["Q"], c["bs"]
        lens = _shuffled(c["lo"], c["hi"], c["B"], rng)
        lens = [max(n, q) for n in lens]
        table, pool, _ = _pages(lens, bs, rng, 5)
        if c["op"] == "prefix":   # every table starts with the prefix's blocks
            pages = c["P"] // bs
            first = np.random.default_rng(seed).permutation(pages).astype(np.int32)
            table = torch.cat([torch.from_numpy(first).cuda().expand(c["B"], pages), table + pages], dim=1).contiguous()
            pool += pages
            lens = [c["P"] + n for n in lens]
        s.update(q=_normal((c["B"], n1, q, d), c["dt"], g), k=_normal((pool, n2, bs, d), c["dt"], g),
                 v=_normal((pool, n2, bs, d), c["dt"], g), table=table, kl=_i32(lens))
    return s


# ------------------------------------------------------------------ the framework's operators
def _run_own(s):
    import attention_fia_prefill_gb300 as fia
    c = s["case"]
    if c["op"] == "tables":
        return (s["table"],) + tuple(fia.fia_block_table_append(s["ctx"], s["new"], s["free"], s["table"],
                                                               block_size=c["bs"], num_tokens=s["tokens"]))
    if c["op"] == "write":
        return fia.fia_cache_write(s["k"], s["v"], s["kc"], s["vc"], s["slots"])
    kw = dict(num_heads=c["N1"], num_key_value_heads=c["N2"], scale_value=c["D"] ** -0.5, softmax_lse_flag=True,
              actual_seq_kvlen=s["kl"])
    if c["op"] == "wdecode":
        return fia.fia_decode_window(s["q"], s["k"], s["v"], block_table=s["table"], block_size=c["bs"],
                                     input_layout="BNSD", pre_tokens=c["pre"], sink_tokens=c["sink"], **kw)
    if c["op"] == "wprefill":
        return fia.fia_prefill_window(s["q"], s["k"], s["v"], actual_seq_qlen=s["ql"], block_table=s["table"],
                                      block_size=c["bs"], input_layout=c["layout"], pre_tokens=c["pre"],
                                      sink_tokens=c["sink"], **kw)
    return fia.fia_decode_shared_prefix(s["q"], s["k"], s["v"], block_table=s["table"], block_size=c["bs"],
                                        shared_prefix_len=c["P"], input_layout="BNSD", **kw)


# ------------------------------------------------------------------ the plain form
def _tables(s):
    c, table = s["case"], s["table"]
    bs, t = c["bs"], s["tokens"]
    ctx, new = s["ctx"].long(), s["new"].long()
    total = ctx + new
    have, need = (ctx + bs - 1) // bs, (total + bs - 1) // bs
    cu = new.cumsum(0)
    ends = (need - have).cumsum(0)
    col = torch.arange(table.shape[1], device=table.device)
    fresh = (col >= have[:, None]) & (col < need[:, None])
    at = (ends - (need - have))[:, None] + col - have[:, None]
    table.copy_(torch.where(fresh, s["free"][at.clamp(0, s["free"].shape[0] - 1)], table))
    i = torch.arange(t, device=table.device)
    b = torch.searchsorted(cu, i, right=True).clamp(max=c["B"] - 1)
    pos = ctx[b] + i - (cu - new)[b]
    slot = table[b, (pos // bs).clamp(max=table.shape[1] - 1)].long() * bs + pos % bs
    slot = torch.where(i < cu[-1], slot, -1)
    return table, slot.int(), total.int(), cu.int(), ends[-1:].int()


def _write(s):
    bs, n2 = s["case"]["bs"], s["case"]["N2"]
    keep = s["slots"] >= 0
    slot = s["slots"][keep].long()
    for x, cache in ((s["k"], s["kc"]), (s["v"], s["vc"])):
        rows = cache.transpose(1, 2) if cache.dim() == 4 else cache.view(cache.shape[0], bs, n2, -1)
        rows[slot // bs, slot % bs] = x[keep]
    return s["kc"], s["vc"]


def _attend(q, k, v, see, scale):
    """q (B, N1, Q, D), k / v (B, N2, M, D), see (B, Q, M): softmax attention in 32 bits; rows that see nothing give
    0 and an lse of +inf.  Returns out (B, N1, Q, D) and lse (B, N1, Q, 1)."""
    b, n1, nq, d = q.shape
    n2, m = k.shape[1:3]
    live = see.any(1)[:, None, :, None]
    k, v = torch.where(live, k.float(), 0.0), torch.where(live, v.float(), 0.0)
    x = torch.matmul(q.float().reshape(b, n2, (n1 // n2) * nq, d), k.transpose(2, 3)).view(b, n2, n1 // n2, nq, m)
    x.mul_(scale).masked_fill_(~see[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    out = torch.matmul(x.view(b, n2, (n1 // n2) * nq, m), v).view(b, n2, n1 // n2, nq, d)
    out = torch.where(total > 0, out / total, 0.0).reshape(b, n1, nq, d)
    lse = torch.where(total > 0, top + total.log(), math.inf).reshape(b, n1, nq, 1)
    return out, lse


def _gather(cache, table, pos, bs):
    """Rows `pos` (B, M) of every sequence from a (blocks, N2, bs, D) cache: (B, N2, M, D)."""
    pos = pos.clamp(0, table.shape[1] * bs - 1)
    block = torch.gather(table.long(), 1, pos // bs)
    return cache.transpose(1, 2)[block, pos % bs].transpose(1, 2)


def _window_see(pos, p, pre, sink):
    """Key positions (B, M) against query positions (B, Q): what each query sees."""
    j, p = pos[:, None, :], p[:, :, None]
    return (j >= 0) & (j <= p) & ((j >= p - pre) | (j < sink))


def _plain_decode(s):
    c, q = s["case"], s["q"]
    dev, n = q.device, s["kl"].long()
    p = n[:, None] - c["Q"] + torch.arange(c["Q"], device=dev)
    if c["op"] == "wdecode":
        # the sinks, and the positions that the window of some new token holds and that are no sinks
        span = min(c["hi"], c["pre"] + c["Q"])
        tail = n[:, None] - span + torch.arange(span, device=dev)
        first = torch.arange(c["sink"], device=dev).expand(c["B"], -1)
        pos = torch.cat([first, torch.where(tail >= c["sink"], tail, -1)], 1)
        see = _window_see(pos, p, c["pre"], c["sink"])
    else:
        pos = torch.arange(c["P"] + max(c["hi"], c["Q"]), device=dev).expand(c["B"], -1)
        see = pos[:, None, :] <= p[:, :, None]
    k, v = (_gather(s[x], s["table"], pos, c["bs"]) for x in ("k", "v"))
    out, lse = _attend(q, k, v, see, c["D"] ** -0.5)
    return out.to(q.dtype), lse


def _plain_prefill(s):
    c, q = s["case"], s["q"]
    dev, span, layout = q.device, torch.arange(c["hi"], device=q.device), c["layout"]
    if layout == "TND":
        cu = s["ql"].long()
        start = torch.cat([cu.new_zeros(1), cu[:-1]])
        ql = kl = cu - start
        rows = (start[:, None] + span).clamp(max=q.shape[0] - 1)
        qb, k, v = (s[x][rows].transpose(1, 2) for x in ("q", "k", "v"))
        pos = span.expand(c["B"], -1)
    else:
        ql, kl = s["ql"].long(), s["kl"].long()
        qb = q if layout == "BNSD" else q.transpose(1, 2)
        if c["bs"]:
            # the sinks, and the positions from the first row's window to the chunk's end
            m = min(c["ctx_hi"] + c["hi"], c["pre"] + c["hi"])
            tail = kl[:, None] - m + torch.arange(m, device=dev)
            first = torch.arange(c["sink"], device=dev).expand(c["B"], -1)
            pos = torch.cat([first, torch.where(tail >= c["sink"], tail, -1)], 1)
            k, v = (_gather(s[x], s["table"], pos, c["bs"]) for x in ("k", "v"))
        else:
            k, v = (s[x] if layout == "BNSD" else s[x].transpose(1, 2) for x in ("k", "v"))
            pos = span.expand(c["B"], -1)
    p = torch.where(span < ql[:, None], span + (kl - ql)[:, None], -1)   # rows past a length see nothing
    out, lse = _attend(qb.reshape(c["B"], c["N1"], c["hi"], c["D"]), k, v, _window_see(pos, p, c["pre"], c["sink"]),
                       c["D"] ** -0.5)
    out = out.to(q.dtype)
    if layout == "TND":
        live = span < ql[:, None]
        return out.transpose(1, 2)[live], lse.transpose(1, 2)[live]
    return (out if layout == "BNSD" else out.transpose(1, 2).contiguous()), lse


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "tables":
        return _tables(state)
    if op == "write":
        return _write(state)
    return _plain_prefill(state) if op == "wprefill" else _plain_decode(state)


# ------------------------------------------------------------------ work
def _seen(n, q, pre, sink):
    """(query, key) pairs and keys that the last q of n tokens see."""
    p = np.arange(n - q, n)
    lo = np.maximum(p - pre, 0)
    first = np.minimum(sink, lo)
    return int((p - lo + 1 + first).sum()), int(n - lo[0] + first[0]) if q else 0


def work(case):
    c = case
    if c["op"] == "tables":
        new = sum(_spread(c["new_lo"], c["new_hi"], c["B"]))
        blocks = -(-new // c["bs"])
        # lengths in and out, a slot for each token, a table and a free entry for each new block
        return {"bytes": 4.0 * (4 * c["B"] + new + 2 * blocks), "flops": 0.0}
    if c["op"] == "write":
        live = c["T"] - c["T"] // 16
        return {"bytes": 4.0 * c["T"] + 2 * 2 * 2.0 * live * c["N2"] * c["D"], "flops": 0.0}
    d, n1, n2 = c["D"], c["N1"], c["N2"]
    if c["op"] == "wprefill":
        new, ctx = _spread(c["lo"], c["hi"], c["B"]), _spread(c["ctx_lo"], c["ctx_hi"], c["B"])
        seen = [_seen(a + b, a, c["pre"], c["sink"]) for a, b in zip(new, ctx)]
        rows = sum(new)
    else:
        pre, sink = (c["pre"], c["sink"]) if c["op"] == "wdecode" else (1 << 40, 0)
        lens = [max(n, c["Q"]) + c.get("P", 0) for n in _spread(c["lo"], c["hi"], c["B"])]
        seen = [_seen(n, c["Q"], pre, sink) for n in lens]
        rows = c["B"] * c["Q"]
    pairs, keys = sum(x[0] for x in seen), sum(x[1] for x in seen)
    keys -= (c["B"] - 1) * c["P"] if c["op"] == "prefix" else 0
    return {"bytes": 2.0 * 2 * keys * n2 * d + 2.0 * 2 * rows * n1 * d + 4.0 * rows * n1, "flops": 4.0 * pairs * n1 * d}


# ------------------------------------------------------------------ the definition in 64 bits
def _softmax_rows(q, k, v, see, scale):
    """q (R, N1, D), k / v (M, N2, D) in 64 bits, see (R, M): out (R, N1, D), lse (R, N1, 1), from the definition."""
    g = q.shape[1] // k.shape[1]
    x = torch.einsum("rngd,mnd->ngrm", q.reshape(q.shape[0], k.shape[1], g, -1), k) * scale
    x = torch.where(see, x, -math.inf)
    lse = torch.logsumexp(x, -1)
    none = ~see.any(-1)
    w = torch.exp(x - torch.where(none, 0.0, lse)[..., None])
    out = torch.einsum("ngrm,mnd->rngd", w, v).reshape(q.shape)
    lse = torch.where(none, math.inf, lse).permute(2, 0, 1).reshape(q.shape[0], -1, 1)
    return out, lse


def exact(case, seed):
    c = dict(case)
    if c["op"] == "tables":
        return None   # whole numbers only
    s = prepare(case, seed)
    if c["op"] == "write":
        out = []
        slots = s["slots"].tolist()
        token = {slot: t for t, slot in enumerate(slots) if slot >= 0}
        at = torch.tensor(sorted(token), device="cuda")
        src = torch.tensor([token[i] for i in sorted(token)], device="cuda")
        for x, cache in ((s["k"], s["kc"]), (s["v"], s["vc"])):
            y = cache.double()
            flat = y.permute(0, 2, 1, 3).reshape(-1, c["N2"], c["D"]) if y.dim() == 4 else y.view(-1, c["N2"], c["D"])
            flat = flat.index_copy(0, at, x.double()[src])
            if y.dim() == 4:
                flat = flat.view(y.shape[0], c["bs"], c["N2"], c["D"]).permute(0, 2, 1, 3)
            out.append(flat.reshape(y.shape))
        return tuple(out)
    scale = c["D"] ** -0.5
    pre, sink = (c["pre"], c["sink"]) if c["op"] != "prefix" else (1 << 40, 0)
    tnd, bsnd = c.get("layout") == "TND", c.get("layout") == "BSND"
    q = s["q"].double()
    outs, lses = [], []
    kl = s["kl"].tolist()
    ql = s["ql"].tolist() if c["op"] == "wprefill" else [c["Q"]] * c["B"]
    if tnd:
        kl = ql = [b - a for a, b in zip([0] + ql, ql)]
    at = 0
    for b in range(c["B"]):
        n, m = ql[b], kl[b]
        if s["table"] is not None:
            ids = s["table"][b].long()
            k, v = (s[x][ids].transpose(1, 2).reshape(-1, c["N2"], c["D"]) for x in ("k", "v"))
        elif tnd:
            k, v = s["k"][at:at + m], s["v"][at:at + m]
        else:
            k, v = (s[x][b] if bsnd else s[x][b].transpose(0, 1) for x in ("k", "v"))
        rows = q[at:at + n] if tnd else q[b] if bsnd else q[b].transpose(0, 1)
        at += n
        o, l = torch.zeros_like(rows), torch.full(rows.shape[:2] + (1,), math.inf, dtype=torch.float64, device="cuda")
        for r in range(0, n, 512):
            e = min(n, r + 512)
            p = torch.arange(m - n + r, m - n + e, device="cuda")[:, None]
            lo = max(0, m - n + r - pre)
            j = torch.cat([torch.arange(min(sink, lo), device="cuda"), torch.arange(lo, max(lo, m - n + e), device="cuda")])
            see = (j <= p) & ((j >= p - pre) | (j < sink))
            o[r:e], l[r:e] = _softmax_rows(rows[r:e], k[j].double(), v[j].double(), see, scale)
        outs.append(o)
        lses.append(l)
    if tnd:
        return torch.cat(outs), torch.cat(lses)
    out, lse = torch.stack(outs), torch.stack(lses).transpose(1, 2)
    return (out if bsnd else out.transpose(1, 2)), lse
