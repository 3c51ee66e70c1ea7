"""fp64 references of the streaming operators in plain numpy, written from the formulas: attention
with a sliding window and sinks, its gradients, and how far rounding may take the bf16 kernels from
them. Test infrastructure only; it shares no code with the library."""
import math

import numpy as np

BF16 = 2.0 ** -8            # half a step of bf16, relative to the value


def visible(nq, nk, wl, wr, ns=0):
    """Key j is visible to query i iff j <= i+off+wr and (j >= i+off-wl or j < ns)."""
    i = np.arange(nq)[:, None] + (nk - nq)
    j = np.arange(nk)[None, :]
    vis = np.ones((nq, nk), bool)
    if wr >= 0:
        vis &= j <= i + wr
    if wl >= 0:
        vis &= (j >= i - wl) | (j < ns)
    return vis


def f64(t):
    return t.detach().double().cpu().numpy()


def _expand(x, H):
    return np.repeat(x, H // x.shape[1], axis=1)


def probabilities(q, k, vis, scale):
    """(P, LSE) of (B, H, n, d) arrays, k with its own head count; empty rows: 0 and -inf."""
    s = np.einsum("bhid,bhjd->bhij", q, _expand(k, q.shape[1])) * scale
    s = np.where(vis, s, -np.inf)
    m = s.max(-1, keepdims=True)
    base = np.where(np.isinf(m), 0.0, m)
    e = np.exp(s - base)
    l = e.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (base + np.log(l))[..., 0]
    return e / np.where(l > 0, l, 1.0), lse


def attention(q, k, v, vis, scale):
    """(O, LSE, bound): the bound on |O - exact| of a kernel that rounds P and O to bf16."""
    p, lse = probabilities(q, k, vis, scale)
    ve = _expand(v, q.shape[1])
    o = p @ ve
    return o, lse, BF16 * (p @ np.abs(ve) + np.abs(o)) * 1.02 + 1e-6


def gradients(q, k, v, do, vis, scale):
    """((dq, dk, dv), bounds): P, dS, O and the results are rounded to bf16 by the kernels, and
    D = rowsum(dO * O) is taken from the rounded O, so with e = 2^-8
        |err dS| <= e |dS| + P * sum_c |dO_c| |err O_c|,     |err dV| <= e P^T |dO| + e |dV|."""
    H, Hkv = q.shape[1], k.shape[1]
    p, _ = probabilities(q, k, vis, scale)
    ke, ve = _expand(k, H), _expand(v, H)
    o, _, eo = attention(q, k, v, vis, scale)
    ds = p * (do @ ve.swapaxes(-1, -2) - (do * o).sum(-1, keepdims=True))
    eds = BF16 * np.abs(ds) + p * (np.abs(do) * eo).sum(-1, keepdims=True)
    t = lambda x: x.swapaxes(-1, -2)                                   # noqa: E731

    def group(x):
        return x.reshape(x.shape[0], Hkv, H // Hkv, *x.shape[2:]).sum(2)
    dq, eq = scale * ds @ ke, scale * eds @ np.abs(ke)
    dk, ek = group(scale * t(ds) @ q), group(scale * t(eds) @ np.abs(q))
    dv, ev = group(t(p) @ do), group(BF16 * t(p) @ np.abs(do))
    out = (dq, dk, dv)
    return out, tuple((e + BF16 * np.abs(x)) * 1.02 + 1e-6 for x, e in zip(out, (eq, ek, ev)))


def default_scale(d):
    return 1.0 / math.sqrt(d)


# ---------------------------------------------------------------- the 4-bit cache
def bf16(x):
    """fp64 -> the nearest bf16 (ties to even), as fp64."""
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, np.float64)).to(torch.bfloat16).double().numpy()


def quantise(x):
    """x (..., d) -> q whole numbers, s, lo (..., d / 32), from the definition in exact arithmetic: fp64
    holds x - lo and (n + 1/2) s of bf16 values within 40 bits of each other exactly."""
    g = x.reshape(*x.shape[:-1], -1, 32)
    lo, hi = g.min(-1), g.max(-1)
    s = bf16((hi - lo) / 15)
    s = np.where(s < 2.0 ** -100, 0.0, s)
    t, s1 = g - lo[..., None], np.where(s > 0, s, 1.0)[..., None]
    n = np.floor(t / s1)
    n += t - (n + 1) * s1 >= 0                             # floor, whatever the division's rounding
    border = (n + 0.5) * s1
    q = n + ((t > border) | ((t == border) & (n % 2 == 1)))
    q = np.where(s[..., None] > 0, np.clip(q, 0, 15), 0)
    return q.astype(np.int64).reshape(x.shape), s, lo


def value(q, s, lo):
    return (lo[..., None] + s[..., None] * q.reshape(*s.shape, 32)).reshape(q.shape)


def nibble_at(tok, d, k):
    """Offset in nibbles, inside K's or V's part of a block, of every channel of token `tok` (0..15)."""
    ch = np.arange(d)
    g, i, G = ch // 32, ch % 32, d // 32
    if k:
        word = ((tok // 8) * 32 + (tok % 8) * 4 + i // 8) * G + g
        return word * 8 + i % 8 // 2 + 4 * (i % 2)
    word = ((tok // 8) * 32 + (i // 4) * 4 + tok % 8 // 2) * G + g
    return word * 8 + 4 * (tok % 2) + i % 4


def bf16_bits(x):
    return (np.asarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def store(pool, page, head, pos_in_page, k, v):
    """Writes one token's k, v (d,) into pool (pages, Hkv, bytes) uint8, in place."""
    d = k.shape[0]
    tok = pos_in_page % 16
    blk = pool[page, head, pos_in_page // 16 * 20 * d:][:20 * d]
    for x, data, par, isk in ((k, 0, 16 * d, True), (v, 8 * d, 18 * d, False)):
        q, s, lo = quantise(x)
        for n, w in zip(nibble_at(tok, d, isk), q):
            b = data + n // 2
            blk[b] = (blk[b] & (0xF0 if n % 2 == 0 else 0x0F)) | (int(w) << (4 * (n % 2)))
        words = np.stack((bf16_bits(s), bf16_bits(lo)), -1).reshape(-1)
        blk[par + tok * d // 8: par + (tok + 1) * d // 8] = words.view(np.uint8)


def load(pool, table_row, n, page_size, d):
    """K, V (Hkv, n, d) that tokens 0 .. n-1 stand for, and which lie on a page (n,)."""
    Hkv = pool.shape[1]
    k, v = np.zeros((Hkv, n, d)), np.zeros((Hkv, n, d))
    held = np.zeros(n, bool)
    ch = np.arange(d) // 32
    for j in range(n):
        pg = table_row[j // page_size]
        if pg < 0 or pg >= pool.shape[0]:
            continue
        held[j] = True
        blk = pool[pg][:, j % page_size // 16 * 20 * d:][:, :20 * d]
        for out, data, par, isk in ((k, 0, 16 * d, True), (v, 8 * d, 18 * d, False)):
            n4 = nibble_at(j % 16, d, isk)
            q = blk[:, data + n4 // 2] >> (4 * (n4 % 2)) & 15
            w = np.ascontiguousarray(blk[:, par + j % 16 * d // 8:][:, :d // 8]).view(np.uint16).astype(np.uint32)
            f = (w << 16).view(np.float32).astype(np.float64).reshape(Hkv, -1, 2)
            with np.errstate(invalid="ignore"):
                out[:, j] = f[:, ch, 1] + f[:, ch, 0] * q
    return k, v, held


def attend(q, pool, table, lens, seqs, page_size, wl, wr, ns):
    """(O, LSE, bounds of both) of q (B, H, nq, d) over the cache. The kernel rounds P s to fp16 (2^-11,
    and 2^-28 of the largest weight at the least), O to bf16; scores are fp32 sums of d products."""
    B, H, nq, d = q.shape
    o, lse = np.zeros(q.shape), np.full((B, H, nq), -np.inf)
    eo, el = np.zeros(q.shape), np.zeros((B, H, nq))
    for b in range(B):
        r = int(seqs[b])
        n = int(lens[r]) if 0 <= r < len(lens) else 0
        if n == 0:
            continue
        k, v, held = load(pool, table[r], n, page_size, d)
        vis = visible(nq, n, wl, wr, ns) & held
        any_ = vis.any(0)
        k, v, vis = k[:, any_], v[:, any_], vis[:, any_]
        if not any_.any():
            continue
        scale = default_scale(d)
        p, l = probabilities(q[b:b + 1], k[None], vis, scale)
        ve, ke = _expand(v[None], H), _expand(k[None], H)
        o[b], lse[b] = (p @ ve)[0], l[0]
        size = scale * np.einsum("bhid,bhjd->bhij", np.abs(q[b:b + 1]), np.abs(ke)).max(-1)[0]
        el[b] = 2.0 ** -20 * size + 4e-6
        spread = np.abs(ve) + np.abs(ve).max(-1, keepdims=True)       # s q <= |value| + |lo|
        eo[b] = (BF16 * np.abs(o[b]) + (p @ spread)[0] * (2.0 ** -11 + 2 * el[b][..., None]) +
                 2.0 ** -27 * vis.sum(1)[None, :, None] * np.abs(ve).max() * p.max(-1)[0][..., None]) * 1.02 + 1e-38
    return o, lse, eo, el
