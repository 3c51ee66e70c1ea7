"""Cases of the streaming operators: attention with a sliding window and sinks (forward, forward and
backward), the 4-bit paged K/V cache (append with read-back, attention over it) and the pages of
such a cache (forking and freeing, compaction).

`run` is one pass through an operator: with `own` true the library's calls, else the same
mathematics in elementary torch operations. `exact` is the definition in 64 bits.

Visibility (i of nq queries, j of nk keys, off = nk - nq): j <= i + off + right and
(j >= i + off - left or j < sinks); a negative bound is none.

4-bit cache: a group is 32 channels of one token and K/V head: lo = min, s = bf16((max - lo) / 15),
q = rint((x - lo) / s) in 0..15, value lo + s q. A block holds 16 tokens of one head in 20 d
bytes (K nibbles, V nibbles, K parameters, V parameters); a page is page_size / 16 blocks per head."""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # a short prompt under a window: latency
        dict(name="sink_fwd_small", op="sink_fwd", dtype="bf16", B=1, H=2, Hkv=2, nq=300, nk=300,
             d=64, left=64, right=0, sinks=4),
        # float32, the row-tiling example's length and width, a two-sided window, odd sinks
        dict(name="sink_fwd_fp32", op="sink_fwd", dtype="fp32", B=1, H=1, Hkv=1, nq=4096, nk=4096,
             d=64, left=511, right=128, sinks=5),
        # prefill of a long prompt, grouped-query heads
        dict(name="sink_fwd_large", op="sink_fwd", dtype="bf16", B=1, H=32, Hkv=8, nq=8192, nk=8192,
             d=128, left=1024, right=0, sinks=4),
        # a training step on ragged sizes: more keys than queries, sinks past a tile
        dict(name="sink_train_odd", op="sink_train", dtype="bf16", B=2, H=6, Hkv=2, nq=777,
             nk=1031, d=64, left=200, right=0, sinks=130),
        # a training step at the benchmark's sequence length
        dict(name="sink_train_large", op="sink_train", dtype="bf16", B=1, H=32, Hkv=8, nq=8192,
             nk=8192, d=128, left=1024, right=0, sinks=4),
        # one decoded token of each sequence goes into the cache
        dict(name="kv4_append_decode", op="kv4_append", B=64, Hkv=8, t=1, ragged=False, d=128, page=64,
             prefix=4096),
        # chunks of prompts, of different lengths, each from where its sequence stands
        dict(name="kv4_append_chunk", op="kv4_append", B=8, Hkv=8, t=2048, ragged=True, d=128,
             page=64, prefix=1000),
        # four drafted tokens per sequence under a window with sinks; the pages between are gone
        dict(name="kv4_attend_window", op="kv4_attend", B=16, H=8, Hkv=8, nq=4, d=64, page=16,
             n=16384, ragged=True, left=1024, sinks=4),
        # a decode step of a batch whose sequences have different lengths
        dict(name="kv4_attend_batch", op="kv4_attend", B=64, H=32, Hkv=8, nq=1, d=128, page=32,
             n=8192, ragged=True, left=-1, sinks=0),
        # a decode step of one long sequence
        dict(name="kv4_attend_long", op="kv4_attend", B=1, H=32, Hkv=8, nq=1, d=128, page=64,
             n=131072, ragged=False, left=-1, sinks=0),
        # a step of beam search: the losing beams leave, the winners are forked
        dict(name="pages_beam", op="pages_fork", parents=4, children=12, n=500, Hkv=8, d=128, page=16),
        # a batch ends, the pool is compacted, the next batch is admitted; twice
        dict(name="pages_compact", op="pages_compact", B=64, n=2048, Hkv=8, d=128, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sink_fwd", "sink_train", "kv4_append", "kv4_attend", "kv4_attend", "pages_fork",
                     "pages_compact"])
    d = rng.choice([32, 64, 128])
    g = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    if op in ("sink_fwd", "sink_train"):
        dtype = rng.choice(["bf16", "bf16", "fp32"]) if op == "sink_fwd" else "bf16"
        least = 1 if op == "sink_fwd" else 16        # one key alone has no gradient to measure
        nq = _log(rng, least, 4096)
        nk = max(least, min(4096, nq + rng.choice([0, 0, rng.randrange(-200, 1500)])))
        return dict(op=op, dtype=dtype, B=rng.randrange(1, 3), H=2 * g, Hkv=2, nq=nq, nk=nk, d=d,
                    left=_log(rng, 1, 2000), right=rng.choice([0, 0, rng.randrange(0, 300)]),
                    sinks=_log(rng, 1, 300))
    if op == "kv4_append":
        t = _log(rng, 1, 2000)
        return dict(op=op, B=max(1, min(64, _log(rng, 1, 64), 16384 // t)), Hkv=rng.randrange(1, 9), t=t,
                    ragged=rng.random() < 0.5, d=d, page=page, prefix=rng.randrange(0, 3000))
    if op == "kv4_attend":
        n = _log(rng, 1, 60000)
        hkv = rng.randrange(1, 9)
        windowed = rng.random() < 0.5
        return dict(op=op, B=max(1, min(48, _log(rng, 1, 48), 120000 // n)), H=hkv * g, Hkv=hkv,
                    nq=rng.choice([1, 1, 1, 2, 5]), d=d, page=page, n=n, ragged=rng.random() < 0.5,
                    left=_log(rng, 1, 4096) if windowed else -1,
                    sinks=rng.randrange(0, 70) if windowed else 0)
    if op == "pages_fork":
        return dict(op=op, parents=rng.randrange(1, 33), children=rng.randrange(1, 65),
                    n=_log(rng, 1, 4000), Hkv=rng.randrange(1, 5), d=d, page=page)
    return dict(op=op, B=_log(rng, 1, 64), n=_log(rng, 1, 1500), Hkv=rng.randrange(1, 5), d=d, page=page)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _keys_values(g, shape):
    """K and V as a model makes them: a few channels of K far larger than the rest."""
    d = shape[-1]
    big = 1 + 7 * (torch.rand(d, generator=g, device=DEV) < 0.04).float()
    k = _randn(g, shape) * big
    v = _randn(g, shape) * (0.2 + torch.rand(shape[:-1] + (1,), generator=g, device=DEV))
    return k.bfloat16(), v.bfloat16()


def _ints(x):
    return torch.as_tensor(x, dtype=torch.int32, device=DEV)


def _table(g, counts, width, pages):
    """Rows of page numbers (counts[i] of them, then -1), the pages in a random order."""
    order = torch.randperm(pages, generator=g, device=DEV).int()
    first = torch.cumsum(counts, 0) - counts
    m = torch.arange(width, device=DEV)
    at = (first[:, None] + m).clamp(max=pages - 1)
    return torch.where(m < counts[:, None], order[at], -1).int().contiguous()


def _lens(g, case, n):
    if not case["ragged"]:
        return torch.full((case["B"],), n, dtype=torch.int32, device=DEV)
    r = torch.rand(case["B"], generator=g, device=DEV)
    return (1 + r * (n - 1)).int()


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    st = dict(case)
    if op in ("sink_fwd", "sink_train"):
        B, H, Hkv, nq, nk, d = (case[x] for x in ("B", "H", "Hkv", "nq", "nk", "d"))
        dt = TYPES[case["dtype"]]
        st.update(q=_randn(g, (B, H, nq, d), dt), k=_randn(g, (B, Hkv, nk, d), dt),
                  v=_randn(g, (B, Hkv, nk, d), dt), do=_randn(g, (B, H, nq, d), dt))
        return st
    d, page, Hkv = case["d"], case["page"], case["Hkv"]
    slab = page // 16 * 20 * d                       # bytes of one page and K/V head
    if op == "kv4_append":
        B, t = case["B"], case["t"]
        counts = _lens(g, case, t)
        start = (case["prefix"] * (0.5 + 0.5 * torch.rand(B, generator=g, device=DEV))).int()
        held = (start + counts + page - 1) // page
        width = -(-(case["prefix"] + t) // page)
        pages = int(held.sum())
        k, v = _keys_values(g, (B, Hkv, t, d))
        pool = torch.zeros((pages, Hkv, slab), dtype=torch.uint8, device=DEV)
        st.update(k=k, v=v, start=start, counts=counts, table=_table(g, held, width, pages), pool=pool)
        return st
    if op == "kv4_attend":
        B, n = case["B"], case["n"]
        lens = _lens(g, case, n)
        held = (lens + page - 1) // page
        width, pages = -(-n // page), int(held.sum())
        table = _table(g, held, width, pages)
        if case["left"] >= 0:                        # what no query sees any more has been freed
            m = torch.arange(width, device=DEV)
            seen = lens[:, None] - case["nq"] - case["left"]
            gone = (m * page >= case["sinks"]) & ((m + 1) * page <= seen)
            table = torch.where(gone, -1, table).int().contiguous()
        k, v = _keys_values(g, (pages, Hkv, page, d))
        pool = _pack(*_quantise(k), *_quantise(v))
        q = _randn(g, (B, case["H"], case["nq"], d), torch.bfloat16)
        st.update(q=q, pool=pool, table=table, lens=lens)
        return st
    n = case["n"]
    width = -(-n // page)
    if op == "pages_fork":
        # parents 0 .. p-1; children p .. p+c-1, forked a step ago from other parents
        p, c = case["parents"], case["children"]
        plens = _ints([1 + (n - 1) * (i + 1) // p for i in range(p)])
        held = (plens + page - 1) // page
        pages = int(held.sum()) + 2 * c
        table = _table(g, torch.cat([held, torch.zeros(c, dtype=held.dtype, device=DEV)]), width, pages)
        lens = torch.cat([plens, torch.zeros(c, dtype=torch.int32, device=DEV)])
        refs = torch.bincount(table[table >= 0].long(), minlength=pages).int()
        parent = torch.randint(0, p, (c,), generator=g, device=DEV).int()
        child = torch.arange(p, p + c, device=DEV).int()
        before = torch.randint(0, p, (c,), generator=g, device=DEV).int()
        pool = torch.randint(0, 256, (pages, Hkv, slab), generator=g, device=DEV, dtype=torch.uint8)
        st.update(table=table, lens=lens, refs=refs, pool=pool, src=parent, dst=child)
        _fork(st, before, child)
        return st
    # batches A (sequences 0 .. B-1) and B (B .. 2B-1), their pages mixed
    B = case["B"]
    lens = torch.randint((n + 1) // 2, n + 1, (B,), generator=g, device=DEV).int().repeat(2)
    held = (lens + page - 1) // page
    pages = 2 * B * width + B * width // 4
    table = _table(g, held, width, pages)
    refs = torch.bincount(table[table >= 0].long(), minlength=pages).int()
    pool = torch.randint(0, 256, (pages, Hkv, slab), generator=g, device=DEV, dtype=torch.uint8)
    st.update(table=table, lens=lens, refs=refs, pool=pool, counts=lens[:B].clone(),
              a=torch.arange(B, device=DEV).int(), b=torch.arange(B, 2 * B, device=DEV).int())
    return st


# ------------------------------------------------------------------ the calls
def run(st):
    if own:
        return _own(st)
    return {"sink_fwd": _sink_forward, "sink_train": _sink_train, "kv4_append": _append_read,
            "kv4_attend": _attend, "pages_fork": _fork_step, "pages_compact": _two_batches}[st["op"]](st)


def _own(st):
    import exact_attention_138_b200 as ea
    op = st["op"]
    if op == "sink_fwd":
        return ea.forward(st["q"], st["k"], st["v"], window=(st["left"], st["right"]),
                          sinks=st["sinks"])
    if op == "sink_train":
        w = (st["left"], st["right"])
        o, lse = ea.forward(st["q"], st["k"], st["v"], window=w, sinks=st["sinks"])
        return (o, lse) + ea.backward(st["q"], st["k"], st["v"], o, st["do"], lse, window=w,
                                      sinks=st["sinks"])
    if op == "kv4_append":
        ea.kv4_append(st["pool"], st["table"], st["start"], st["k"], st["v"], counts=st["counts"])
        return ea.kv4_gather(st["pool"], st["table"], st["start"], st["t"], st["d"],
                             counts=st["counts"])
    if op == "kv4_attend":
        return ea.kv4_attend(st["q"], st["pool"], st["table"], st["lens"], window=(st["left"], 0),
                             sinks=st["sinks"])
    tab = (st["table"], st["lens"], st["refs"], st["page"])
    if op == "pages_fork":
        ea.pages_free(*tab, st["dst"])
        frm, to = ea.pages_fork(*tab, st["src"], st["dst"])
        ea.pages_copy(st["pool"], frm, to)
        return st["table"], st["lens"], st["refs"], frm, to, st["pool"]
    ea.pages_free(*tab, st["a"])
    ea.pages_copy(st["pool"], *ea.pages_compact(st["table"], st["refs"]))
    start_a = ea.pages_reserve(*tab, st["a"], st["counts"])
    ea.pages_free(*tab, st["b"])
    ea.pages_copy(st["pool"], *ea.pages_compact(st["table"], st["refs"]))
    start_b = ea.pages_reserve(*tab, st["b"], st["counts"])
    return st["table"], st["lens"], st["refs"], start_a, start_b, st["pool"]


# ------------------------------------------------------------------ plain forms: windows with sinks
def _visible(nq, nk, left, right, sinks):
    i = torch.arange(nq, device=DEV)[:, None] + (nk - nq)
    j = torch.arange(nk, device=DEV)
    vis = torch.ones((nq, nk), dtype=torch.bool, device=DEV)
    if right >= 0:
        vis &= j <= i + right
    if left >= 0:
        vis &= (j >= i - left) | (j < sinks)
    return vis


def _probabilities(st):
    """(P, LSE) with query heads grouped by their K/V head: P (B, Hkv, G, nq, nk) in 32 bits."""
    q, k = st["q"].float(), st["k"].float()
    B, H, nq, d = q.shape
    Hkv, nk = k.shape[1], k.shape[2]
    s = torch.matmul(q.view(B, Hkv, H // Hkv, nq, d) * (1 / math.sqrt(d)), k[:, :, None].transpose(-1, -2))
    s.masked_fill_(~_visible(nq, nk, st["left"], st["right"], st["sinks"]), -math.inf)
    m = s.amax(-1, keepdim=True)
    base = torch.where(torch.isinf(m), 0.0, m)
    p = s.sub_(base).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (base + total.log()).view(B, H, nq)
    return p.div_(torch.where(total > 0, total, 1.0)), lse


def _sink_forward(st):
    p, lse = _probabilities(st)
    o = torch.matmul(p, st["v"].float()[:, :, None])
    return o.reshape(st["q"].shape).to(st["q"].dtype), lse


def _sink_train(st):
    p, lse = _probabilities(st)
    q, k, v, do = (st[x].float() for x in ("q", "k", "v", "do"))
    B, H, nq, d = q.shape
    Hkv, scale = k.shape[1], 1 / math.sqrt(d)
    qg, dog = q.view(B, Hkv, H // Hkv, nq, d), do.view(B, Hkv, H // Hkv, nq, d)
    o = torch.matmul(p, v[:, :, None])
    dv = torch.matmul(p.transpose(-1, -2), dog).sum(2)
    ds = torch.matmul(dog, v[:, :, None].transpose(-1, -2))
    ds.sub_((dog * o).sum(-1, keepdim=True)).mul_(p)
    dq = torch.matmul(ds, k[:, :, None]).view(q.shape) * scale
    dk = torch.matmul(ds.transpose(-1, -2), qg).sum(2) * scale
    t = st["q"].dtype
    return o.reshape(q.shape).to(t), lse, dq.to(t), dk.to(t), dv.to(t)


# ------------------------------------------------------------------ plain forms: the 4-bit cache
def _quantise(x):
    """x (..., d) -> q (..., d) whole numbers 0..15, s and lo (..., d / 32) in bf16."""
    g = x.float().unflatten(-1, (-1, 32))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    s = ((hi - lo) / 15).bfloat16().double()
    s = torch.where(s < 2.0 ** -100, 0.0, s)
    q = torch.round((g.double() - lo.double()) / torch.where(s > 0, s, 1.0)).clamp_(0, 15)
    q = torch.where(s > 0, q, 0.0)
    return q.flatten(-2).to(torch.uint8), s.squeeze(-1).bfloat16(), lo.squeeze(-1).bfloat16()


def _nibbles(q, k):
    """q (..., tokens, d) in the order of the cache: (..., blocks, 8 d) bytes."""
    d = q.shape[-1]
    lead = q.shape[:-2]
    if k:      # token = half, row; channel = group, c, j, h -> half, row, c, group, h, j
        x = q.view(*lead, -1, 2, 8, d // 32, 4, 4, 2)
        x = x.movedim((-3, -1, -2), (-4, -2, -1))
    else:      # token = half, c, e; channel = group, row, j -> half, row, c, group, e, j
        x = q.view(*lead, -1, 2, 4, 2, d // 32, 8, 4)
        x = x.movedim((-2, -5, -3, -4), (-5, -4, -3, -2))
    x = x.reshape(*lead, q.shape[-2] // 16, -1, 2)
    return x[..., 0] | (x[..., 1] << 4)


def _pack(kq, ks, klo, vq, vs, vlo):
    """(pages, Hkv, page, ...) -> pool (pages, Hkv, page / 16 * 20 d) of bytes."""
    def params(s, lo):
        x = torch.stack((s, lo), -1).contiguous().view(torch.uint8)
        return x.reshape(*x.shape[:2], x.shape[2] // 16, -1)
    parts = (_nibbles(kq, True), _nibbles(vq, False), params(ks, klo), params(vs, vlo))
    return torch.cat(parts, -1).flatten(-2).contiguous()


def _unpack(slabs, d):
    """slabs (..., blocks * 20 d) -> K, V (..., blocks * 16, d) in 32 bits."""
    b = slabs.unflatten(-1, (-1, 20 * d))

    def values(nib, par, k):
        x = torch.stack((nib & 15, nib >> 4), -1).flatten(-2)
        lead = x.shape[:-1]
        if k:
            x = x.view(*lead, 2, 8, 4, d // 32, 2, 4)
            x = x.movedim((-4, -2, -1), (-3, -1, -2))
        else:
            x = x.view(*lead, 2, 8, 4, d // 32, 2, 4)
            x = x.movedim((-5, -4, -3, -2), (-2, -5, -3, -4))
        x = x.reshape(*lead, 16, d // 32, 32).float()
        sl = par.contiguous().view(torch.bfloat16).view(*lead, 16, d // 32, 2).float()
        return (sl[..., 1:] + sl[..., :1] * x).flatten(-2).flatten(-3, -2)
    return (values(b[..., :8 * d], b[..., 16 * d:18 * d], True),
            values(b[..., 8 * d:16 * d], b[..., 18 * d:], False))


def _append_read(st):
    """Quantises the new rows into the blocks of their pages, then reads them back."""
    k, v, start, counts, table, pool, page = (st[x] for x in ("k", "v", "start", "counts", "table",
                                                              "pool", "page"))
    B, Hkv, t, d = k.shape
    pos = start[:, None] + torch.arange(t, device=DEV)                     # (B, t)
    live = torch.arange(t, device=DEV) < counts[:, None]
    pg = torch.gather(table, 1, (pos // page).clamp(max=table.shape[1] - 1).long())
    # each row is packed as a block of its own; its bytes in the block go where its token stands
    tok = (pos % 16).long()
    base = (pos % page // 16).long() * (20 * d)
    kq, ks, klo = _quantise(k)
    vq, vs, vlo = _quantise(v)
    word = torch.arange(d // 8, device=DEV)
    c, grp = word // (d // 32), word % (d // 32)
    # K: word (half, row, c, group) of four bytes, nibble j + 4 h of channel 32 group + 8 c + 2 j + h
    kw = kq.view(B, Hkv, t, d // 32, 4, 4, 2).permute(0, 1, 2, 4, 3, 6, 5).reshape(B, Hkv, t, d // 8, 4, 2)
    kb = kw[..., 0] | (kw[..., 1] << 4)
    kat = ((tok // 8)[..., None] * 32 + (tok % 8)[..., None] * 4 + c) * (d // 32) + grp
    kat = (base[..., None] + kat * 4)[..., None] + torch.arange(4, device=DEV)
    # V: two bytes (half, row, c, group, e), nibble j of channel 32 group + 4 row + j
    vw = vq.view(B, Hkv, t, d // 32, 8, 2, 2).permute(0, 1, 2, 4, 3, 5, 6)
    vb = (vw[..., 0] | (vw[..., 1] << 4)).reshape(B, Hkv, t, d // 4, 2)
    unit = torch.arange(d // 4, device=DEV)
    row, vgrp = unit // (d // 32), unit % (d // 32)
    vat = ((tok // 8)[..., None] * 32 + row * 4 + (tok % 8 // 2)[..., None]) * (d // 32) + vgrp
    vat = (base[..., None] + 8 * d + vat * 4 + (tok % 2)[..., None] * 2)[..., None] + torch.arange(2, device=DEV)
    par = torch.arange(d // 8, device=DEV)
    pat = (base + 16 * d + tok * (d // 8))[..., None] + par
    kp = torch.stack((ks, klo), -1).contiguous().view(torch.uint8).reshape(B, Hkv, t, d // 8)
    vp = torch.stack((vs, vlo), -1).contiguous().view(torch.uint8).reshape(B, Hkv, t, d // 8)
    at = torch.cat((kat.flatten(-2), vat.flatten(-2), pat, pat + 2 * d), -1)      # (B, t, 1.25 d)
    new = torch.cat((kb.flatten(-2), vb.flatten(-2), kp, vp), -1)                 # (B, Hkv, t, 1.25 d)
    b, i = live.nonzero(as_tuple=True)
    head = torch.arange(Hkv, device=DEV)
    pool[pg[b, i].long()[:, None, None], head[None, :, None], at[b, i][:, None, :]] = new[b, :, i]
    # read back
    got = pool[pg[b, i].long()[:, None, None], head[None, :, None], at[b, i][:, None, :]]
    x = got[..., :d].reshape(-1, Hkv, d)
    kn = torch.stack((x[..., :d // 2] & 15, x[..., :d // 2] >> 4), -1).view(-1, Hkv, 4, d // 32, 2, 4)
    kn = kn.permute(0, 1, 3, 2, 5, 4).reshape(-1, Hkv, d // 32, 32).float()
    vn = torch.stack((x[..., d // 2:] & 15, x[..., d // 2:] >> 4), -1).view(-1, Hkv, 8, d // 32, 4)
    vn = vn.permute(0, 1, 3, 2, 4).reshape(-1, Hkv, d // 32, 32).float()
    sl = got[..., d:].contiguous().view(torch.bfloat16).view(-1, Hkv, 2, d // 32, 2).float()
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    ko[b, :, i] = (sl[:, :, 0, :, 1:] + sl[:, :, 0, :, :1] * kn).flatten(-2).bfloat16()
    vo[b, :, i] = (sl[:, :, 1, :, 1:] + sl[:, :, 1, :, :1] * vn).flatten(-2).bfloat16()
    return ko, vo


def _attend(st):
    q, pool, table, lens, page, d = (st[x] for x in ("q", "pool", "table", "lens", "page", "d"))
    B, H, nq, _ = q.shape
    Hkv = pool.shape[1]
    k, v = _unpack(pool[table.clamp(min=0).long()], d)                   # (B, M, Hkv, page, d)
    k = k.transpose(1, 2).reshape(B, Hkv, -1, d)
    v = v.transpose(1, 2).reshape(B, Hkv, -1, d)
    j = torch.arange(k.shape[2], device=DEV)
    pos = (lens[:, None] - nq + torch.arange(nq, device=DEV))[..., None]            # (B, nq, 1)
    vis = (j <= pos) & (table >= 0).repeat_interleave(page, 1)[:, None]
    if st["left"] >= 0:
        vis &= (j >= pos - st["left"]) | (j < st["sinks"])
    qg = q.float().view(B, Hkv, H // Hkv, nq, d) * (1 / math.sqrt(d))
    s = torch.matmul(qg, k[:, :, None].transpose(-1, -2)).masked_fill_(~vis[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    base = torch.where(torch.isinf(m), 0.0, m)
    p = s.sub_(base).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v[:, :, None]) / torch.where(total > 0, total, 1.0)
    return o.reshape(q.shape).bfloat16(), (base + total.log()).view(B, H, nq)


# ------------------------------------------------------------------ plain forms: pages
def _held(st, rows):
    m = torch.arange(st["table"].shape[1], device=DEV)
    return m < ((st["lens"][rows] + st["page"] - 1) // st["page"])[:, None]


def _free(st, seqs):
    rows = st["table"][seqs.long()]
    gone = rows[_held(st, seqs.long()) & (rows >= 0)].long()
    st["refs"].index_add_(0, gone, torch.full_like(gone, -1, dtype=torch.int32))
    st["table"][seqs.long()] = -1
    st["lens"][seqs.long()] = 0


def _fork(st, src, dst):
    table, lens, refs, page = (st[x] for x in ("table", "lens", "refs", "page"))
    src, dst = src.long(), dst.long()
    n = lens[src]
    full = n // page
    m = torch.arange(table.shape[1], device=DEV)
    rows = torch.where(m < full[:, None], table[src], -1)
    shared = rows[rows >= 0].long()
    part = (n % page > 0).nonzero().squeeze(1)
    new = (refs == 0).nonzero().squeeze(1)[:part.numel()].int()
    frm, to = torch.full_like(n, -1), torch.full_like(n, -1)
    frm[part] = table[src[part], full[part].long()]
    to[part] = new
    rows[part, full[part].long()] = new
    refs.index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    refs[new.long()] = 1
    table[dst] = rows
    lens[dst] = n
    return frm, to


def _copy(pool, frm, to):
    k = (frm >= 0).nonzero().squeeze(1)
    pool[to[k].long()] = pool[frm[k].long()]


def _fork_step(st):
    _free(st, st["dst"])
    frm, to = _fork(st, st["src"], st["dst"])
    _copy(st["pool"], frm, to)
    return st["table"], st["lens"], st["refs"], frm, to, st["pool"]


def _compact(st):
    table, refs, pool = st["table"], st["refs"], st["pool"]
    live = refs > 0
    page = torch.arange(refs.numel(), device=DEV)
    low = page < live.sum()
    frm, to = (live & ~low).nonzero().squeeze(1), (~live & low).nonzero().squeeze(1)
    pool[to] = pool[frm]
    refs[to] = refs[frm]
    refs[frm] = 0
    now = page.clone()
    now[frm] = to
    table.copy_(torch.where(table >= 0, now[table.clamp(min=0).long()], -1))


def _reserve(st, seqs, counts):
    table, lens, refs, page = (st[x] for x in ("table", "lens", "refs", "page"))
    start = lens[seqs.long()]
    have, want = (start + page - 1) // page, (start + counts + page - 1) // page
    m = torch.arange(table.shape[1], device=DEV)
    rows = table[seqs.long()]
    need = (m >= have[:, None]) & (m < want[:, None])
    new = (refs == 0).nonzero().squeeze(1)
    rank = torch.cumsum(need.flatten().long(), 0) - 1
    picked = new[rank.clamp(min=0, max=new.numel() - 1)].view(need.shape).int()
    rows = torch.where(need, picked, rows)
    table[seqs.long()] = rows
    refs[rows[need].long()] = 1
    lens[seqs.long()] = start + counts
    return start


def _two_batches(st):
    _free(st, st["a"])
    _compact(st)
    start_a = _reserve(st, st["a"], st["counts"])
    _free(st, st["b"])
    _compact(st)
    start_b = _reserve(st, st["b"], st["counts"])
    return st["table"], st["lens"], st["refs"], start_a, start_b, st["pool"]


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("sink_fwd", "sink_train"):
        return _exact_sink(st, op == "sink_train")
    if op == "kv4_append":
        return _exact_append(st)
    if op == "kv4_attend":
        return _exact_attend(st)
    return None                       # whole numbers: there is nothing to round


def _softmax_rows(s, hidden):
    """Rows of P and their log-sum-exp; a row that sees nothing has P = 0 and -inf."""
    s = torch.where(hidden, -math.inf, s)
    lse = torch.logsumexp(s, -1, keepdim=True)
    return torch.where(hidden, 0.0, torch.exp(s - torch.where(torch.isinf(lse), 0.0, lse))), lse[..., 0]


def _exact_sink(st, train):
    B, H, nq, d = st["q"].shape
    Hkv, nk = st["k"].shape[1:3]
    a = torch.arange(nk - nq, nk, device=DEV).unsqueeze(1)
    b = torch.arange(nk, device=DEV).unsqueeze(0)
    hidden = torch.zeros((nq, nk), dtype=torch.bool, device=DEV)
    if st["right"] >= 0:
        hidden = hidden | (b > a + st["right"])
    if st["left"] >= 0:
        hidden = hidden | ((b < a - st["left"]) & (b >= st["sinks"]))
    o = torch.zeros((B, H, nq, d), dtype=torch.float64, device=DEV)
    lse = torch.zeros((B, H, nq), dtype=torch.float64, device=DEV)
    dq = torch.zeros_like(o)
    dk = torch.zeros((B, Hkv, nk, d), dtype=torch.float64, device=DEV)
    dv = torch.zeros_like(dk)
    for x in range(B):
        for h in range(H):
            y = h * Hkv // H
            q, k, v, do = (st[n][x, z].double() for n, z in (("q", h), ("k", y), ("v", y), ("do", h)))
            p, lse[x, h] = _softmax_rows(q @ k.T / math.sqrt(d), hidden)
            o[x, h] = p @ v
            if train:
                ds = p * (do @ v.T - (do * o[x, h]).sum(1, keepdim=True)) / math.sqrt(d)
                dq[x, h] = ds @ k
                dk[x, y] += ds.T @ q
                dv[x, y] += p.T @ do
    return (o, lse, dq, dk, dv) if train else (o, lse)


def _exact_append(st):
    out = []
    for x in (st["k"], st["v"]):
        r = x.double().cpu().numpy()
        r = r.reshape(r.shape[:-1] + (-1, 32))
        lo, hi = r.min(-1, keepdims=True), r.max(-1, keepdims=True)
        s = torch.from_numpy((hi - lo) / 15).bfloat16().double().numpy()
        safe = np.where(s >= 2.0 ** -100, s, 1.0)
        y = np.where(s >= 2.0 ** -100, lo + safe * np.clip(np.rint((r - lo) / safe), 0, 15), lo)
        y = y.reshape(x.shape)
        dead = np.arange(x.shape[2])[None, :] >= st["counts"].cpu().numpy()[:, None]
        y[np.broadcast_to(dead[:, None, :], x.shape[:3])] = 0
        out.append(torch.from_numpy(y).to(DEV))
    return tuple(out)


def _exact_attend(st):
    """Sequence by sequence, its K and V read nibble by nibble from the bytes of its pages."""
    q, d, page = st["q"].double(), st["d"], st["page"]
    B, H, nq, _ = q.shape
    Hkv, G = st["pool"].shape[1], d // 32
    o = torch.zeros((B, H, nq, d), dtype=torch.float64, device=DEV)
    lse = torch.zeros((B, H, nq), dtype=torch.float64, device=DEV)
    lens = st["lens"].tolist()
    ch = torch.arange(d, device=DEV)
    grp, in32 = ch // 32, ch % 32
    for x in range(B):
        n = lens[x]
        j = torch.arange(n, device=DEV)
        pg = st["table"][x].long()[j // page]
        slab = st["pool"][pg.clamp(min=0)]                     # (n, Hkv, bytes)
        tok = (j % 16)[:, None]
        base = (j % page // 16 * (20 * d))[:, None]
        knib = (((tok // 8 * 8 + tok % 8) * 4 + in32 // 8) * G + grp) * 8 + in32 % 8 // 2 + 4 * (in32 % 2)
        vnib = ((tok // 8 * 32 + in32 // 4 * 4 + tok % 8 // 2) * G + grp) * 8 + 4 * (tok % 2) + in32 % 4

        def value(nib, data, par):
            byte = torch.gather(slab, 2, (base + data + nib // 2)[:, None].expand(-1, Hkv, -1))
            w = (byte.int() >> (4 * (nib % 2))[:, None]) & 15
            at = base + par + tok * (4 * G) + 4 * grp
            b = [torch.gather(slab, 2, (at + z)[:, None].expand(-1, Hkv, -1)).int() for z in range(4)]
            s = ((b[0] << 16) | (b[1] << 24)).view(torch.float32).double()
            lo = ((b[2] << 16) | (b[3] << 24)).view(torch.float32).double()
            return (lo + s * w).transpose(0, 1)
        k, v = value(knib, 0, 16 * d), value(vnib, 8 * d, 18 * d)
        a = torch.arange(n - nq, n, device=DEV).unsqueeze(1)
        hidden = (j > a) | (pg < 0)
        if st["left"] >= 0:
            hidden = hidden | ((j < a - st["left"]) & (j >= st["sinks"]))
        qx = q[x].view(Hkv, H // Hkv * nq, d)
        s = qx @ k.transpose(1, 2) / math.sqrt(d)
        p, r = _softmax_rows(s, hidden.repeat(H // Hkv, 1))
        o[x], lse[x] = (p @ v).view(H, nq, d), r.view(H, nq)
    return o, lse


# ------------------------------------------------------------------ what a pass cannot do without
def _pairs(nq, nk, left, right, sinks):
    """Visible pairs, and how many keys some query sees."""
    i = np.arange(nq, dtype=np.int64) + (nk - nq)
    hi = np.minimum(i + right, nk - 1) if right >= 0 else np.full(nq, nk - 1)
    lo = np.maximum(i - left, 0) if left >= 0 else np.zeros(nq, dtype=np.int64)
    lo = np.maximum(lo, 0)
    seen = np.maximum(hi - lo + 1, 0) + np.maximum(np.minimum(np.minimum(lo, sinks), hi + 1), 0)
    some = hi >= 0
    first = int(lo[some].min()) if some.any() else nk
    last = int(hi.max()) if some.any() else -1
    return int(seen.sum()), max(0, last + 1 - first) + min(first, sinks if some.any() else 0)


def work(case):
    op, d = case["op"], case["d"]
    if op in ("sink_fwd", "sink_train"):
        B, H, Hkv, nq, nk = (case[x] for x in ("B", "H", "Hkv", "nq", "nk"))
        e = TYPES[case["dtype"]].itemsize
        pairs, keys = _pairs(nq, nk, case["left"], case["right"], case["sinks"])
        qrows, krows = B * H * nq, B * Hkv
        if op == "sink_fwd":
            return {"bytes": e * d * 2 * (qrows + krows * keys) + 4 * qrows, "flops": 4 * d * B * H * pairs}
        return {"bytes": e * d * (4 * qrows + 2 * krows * (keys + nk)) + 4 * qrows,
                "flops": 14 * d * B * H * pairs}
    Hkv, page = case["Hkv"], case["page"]
    slab = page // 16 * 20 * d
    if op == "kv4_append":
        rows = case["B"] * Hkv * case["t"] * (0.5 if case["ragged"] and case["t"] > 1 else 1)
        padded = case["B"] * Hkv * case["t"]
        # new rows read, cache written, cache read, rows written (the padding too)
        return {"bytes": rows * (4 * d + 1.25 * d) + 1.25 * d * rows + padded * 4 * d, "flops": 0}
    if op == "kv4_attend":
        B, H, nq, n = (case[x] for x in ("B", "H", "nq", "n"))
        lens = [n] * B if not case["ragged"] else [1 + (n - 1) * (i + 0.5) / B for i in range(B)]
        counts = [_pairs(nq, int(x), case["left"], 0, case["sinks"]) for x in lens]
        return {"bytes": sum(c[1] for c in counts) * Hkv * 1.25 * d + B * H * nq * (4 * d + 4),
                "flops": 4 * d * H * sum(c[0] for c in counts)}
    n = case["n"]
    if op == "pages_fork":
        p, c = case["parents"], case["children"]
        lens = [1 + (n - 1) * (i + 1) // p for i in range(p)]
        part = c * sum(x % page > 0 for x in lens) / p
        entries = c * sum(-(-x // page) for x in lens) / p
        # pages read and written; entries and counts of the children's pages freed and set again
        return {"bytes": part * 2 * Hkv * slab + entries * 4 * 8, "flops": 0}
    moved = 2 * case["B"] * -(-int(0.75 * n) // page)
    return {"bytes": moved * 2 * Hkv * slab + 2 * 2 * 2 * case["B"] * -(-n // page) * 4, "flops": 0}
