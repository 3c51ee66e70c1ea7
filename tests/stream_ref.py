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
