"""Plain float64 CPU attention with shaped scores, cache decode and eviction: the
oracle for those entry points. TEST INFRASTRUCTURE, as oracle/attention.py is.

    x = scale q.k,  z = cap tanh(x / cap) - slope |i - j|,  -inf where hidden,
    O = softmax(z) V,  LSE = logsumexp(z),
    dV = P^T dO,  dZ = P (dO V^T - D),  D_i = dO_i . O_i,
    dX = dZ (1 - tanh^2),  dQ = scale dX K,  dK = scale dX^T Q.

Beside each result stands the bound that one relative error per rounded
operand puts on it (for instance |O| <= sum_j P_ij |V_j|), from which the tests
derive their tolerances.
"""
from __future__ import annotations

import dataclasses

import numpy as np

from .attention import _f64


def visible(n: int, causal: bool, begin=None, end=None) -> np.ndarray:
    """[n, n] mask of one sequence: key j (column) is seen by query i (row)."""
    j = np.arange(n)
    see = np.ones((n, n), dtype=bool)
    if causal:
        see &= j[None, :] <= j[:, None]
    if begin is not None:
        see &= j[None, :] >= np.asarray(begin)[:, None]
    if end is not None:
        see &= j[None, :] < np.asarray(end)[:, None]
    return see


def logits(q, k, scale, cap, slope, dist, see):
    """z, and the derivative of the cap, of one head."""
    x = scale * (q @ k.T)
    grad = np.ones_like(x)
    if cap:
        t = np.tanh(x / cap)
        x, grad = cap * t, 1.0 - t * t
    z = x - slope * np.abs(dist)
    return np.where(see, z, -np.inf), grad


def softmax(z):
    """P and LSE by rows; a row of -inf gives zeros and -inf."""
    if z.shape[1] == 0:
        return z, np.full(z.shape[0], -np.inf)
    m = z.max(axis=1, keepdims=True)
    m = np.where(np.isneginf(m), 0.0, m)
    e = np.exp(z - m)
    l = e.sum(axis=1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (m + np.log(l))[:, 0]
    return e / np.where(l > 0, l, 1.0), lse


@dataclasses.dataclass
class Forward:
    o: np.ndarray        # [T, H, D]
    lse: np.ndarray      # [H, T]
    o_abs: np.ndarray    # P |V|


@dataclasses.dataclass
class Backward:
    dq: np.ndarray
    dk: np.ndarray
    dv: np.ndarray
    dq_abs: np.ndarray   # scale |dX| |K|
    dk_abs: np.ndarray
    dv_abs: np.ndarray   # P^T |dO|
    dq_del: np.ndarray   # scale (P grad (|dO|.|O| + |dO|.(P|V|))) |K|: what D_i's rounding moves
    dk_del: np.ndarray
    dq_raw: np.ndarray   # scale |dZ| |K|: what an error of the cap's derivative moves
    dk_raw: np.ndarray
    dq_one: np.ndarray   # scale |dO V^T - D| |K| over the visible keys: what an absolute
    dk_one: np.ndarray   # error of P moves


def _heads(q, k, v, cu, causal, scale, cap, slopes, begin, end):
    """Yields per (sequence, head): its rows, kv head, and P, LSE, grad, q, k, v."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    H, H_kv = q.shape[1], k.shape[1]
    sl = None if slopes is None else _f64(slopes)
    for s0, s1 in zip(cu[:-1], cu[1:]):
        n = int(s1 - s0)
        if n == 0:
            continue
        rows = slice(int(s0), int(s1))
        see = visible(n, causal, None if begin is None else np.asarray(begin)[rows],
                      None if end is None else np.asarray(end)[rows])
        i = np.arange(n)
        for h in range(H):
            hk = h // (H // H_kv)
            z, grad = logits(q[rows, h], k[rows, hk], scale, cap, 0.0 if sl is None else sl[h],
                             i[:, None] - i[None, :], see)
            p, lse = softmax(z)
            yield rows, h, hk, p, lse, grad, q[rows, h], k[rows, hk], v[rows, hk]


def forward(q, k, v, cu, causal, scale, cap=0.0, slopes=None, begin=None, end=None) -> Forward:
    o = np.zeros(_f64(q).shape)
    o_abs = np.zeros_like(o)
    lse = np.full((o.shape[1], o.shape[0]), -np.inf)
    for rows, h, _, p, ls, _, _, _, vv in _heads(q, k, v, cu, causal, scale, cap, slopes, begin, end):
        o[rows, h], o_abs[rows, h], lse[h, rows] = p @ vv, p @ np.abs(vv), ls
    return Forward(o, lse, o_abs)


def backward(q, k, v, do, cu, causal, scale, cap=0.0, slopes=None, begin=None,
             end=None) -> Backward:
    g = _f64(do)
    r = Backward(*(np.zeros(_f64(x).shape) for x in (q, k, k, q, k, k, q, k, q, k, q, k)))
    for rows, h, hk, p, _, grad, qq, kk, vv in _heads(q, k, v, cu, causal, scale, cap, slopes,
                                                      begin, end):
        d = g[rows, h]
        o = p @ vv
        dp = d @ vv.T - (d * o).sum(1, keepdims=True)
        dz = p * dp
        dp = np.abs(dp) * (p > 0)
        dx = dz * grad
        r.dq[rows, h] += scale * dx @ kk
        r.dk[rows, hk] += scale * dx.T @ qq
        r.dv[rows, hk] += p.T @ d
        r.dq_abs[rows, h] += scale * np.abs(dx) @ np.abs(kk)
        r.dk_abs[rows, hk] += scale * np.abs(dx).T @ np.abs(qq)
        r.dv_abs[rows, hk] += p.T @ np.abs(d)
        de = p * grad * ((np.abs(d) * np.abs(o)).sum(1) + (np.abs(d) * (p @ np.abs(vv))).sum(1))[:, None]
        r.dq_del[rows, h] += scale * de @ np.abs(kk)
        r.dk_del[rows, hk] += scale * de.T @ np.abs(qq)
        r.dq_raw[rows, h] += scale * np.abs(dz) @ np.abs(kk)
        r.dk_raw[rows, hk] += scale * np.abs(dz).T @ np.abs(qq)
        r.dq_one[rows, h] += scale * dp @ np.abs(kk)
        r.dk_one[rows, hk] += scale * dp.T @ np.abs(qq)
    return r


def key_ranges(lengths, causal, doc_ids=None, prefix_lens=None, window=0):
    """begin, end of every token, sequence after sequence, one token at a time."""
    begin, end, start = [], [], 0
    for b, n in enumerate(lengths):
        for i in range(n):
            lo, hi = 0, n
            if doc_ids is not None:
                d = [int(x) for x in doc_ids[start:start + n]]
                lo = hi = i
                while lo > 0 and d[lo - 1] == d[i]:
                    lo -= 1
                while hi < n and d[hi] == d[i]:
                    hi += 1
            if causal:
                hi = min(hi, max(i + 1, int(prefix_lens[b]) if prefix_lens is not None else 0))
            if window:
                lo = max(lo, i - window + 1)
            begin.append(lo)
            end.append(hi)
        start += n
    return np.array(begin, dtype=np.int32), np.array(end, dtype=np.int32)


def cache_rows(b, n, page_size, block_table=None):
    """Cache rows of slots 0 .. n - 1 of sequence b."""
    j = np.arange(n)
    if block_table is None:
        return b * page_size + j
    return np.asarray(block_table)[b, j // page_size] * page_size + j % page_size


def decode(q, k_cache, v_cache, lens, *, q_len, scale, causal=True, page_size, block_table=None,
           cap=0.0, slopes=None, window=0, positions=None, slots=None):
    """O, LSE, P|V| [B q_len, H, ...] and the weights [B, H_kv, slots] that one call adds."""
    q = _f64(q)
    k_cache, v_cache = _f64(k_cache), _f64(v_cache)
    H, H_kv = q.shape[1], k_cache.shape[1]
    o, o_abs = np.zeros_like(q), np.zeros_like(q)
    lse = np.full(q.shape[:2], -np.inf)
    weights = np.zeros((len(lens), H_kv, int(slots if slots is not None else max(lens))))
    for b, n in enumerate(int(x) for x in lens):
        at = cache_rows(b, n, page_size, block_table)
        j = np.arange(n)
        for hk in range(H_kv):
            pj = j if positions is None else np.asarray(positions)[b, hk, :n].astype(np.int64)
            for t in range(q_len):
                s = n - q_len + t
                ps = s if s < 0 else int(pj[s])
                see = (j <= s) if causal else np.ones(n, dtype=bool)
                if window:
                    see = see & (ps - pj < window)
                for h in range(hk * (H // H_kv), (hk + 1) * (H // H_kv)):
                    z, _ = logits(q[b * q_len + t, h][None], k_cache[at, hk], scale, cap,
                                  0.0 if slopes is None else float(slopes[h]), (ps - pj)[None],
                                  see[None])
                    p, ls = softmax(z)
                    vis = np.where(see[:, None], v_cache[at, hk], 0.0)
                    o[b * q_len + t, h] = (p @ vis)[0]
                    o_abs[b * q_len + t, h] = (p @ np.abs(vis))[0]
                    lse[b * q_len + t, h] = ls[0]
                    weights[b, hk, :n] += p[0]
    return o, lse, o_abs, weights


def kept_slots(w, n, keep, recent):
    """Slots that stay of one head's n, ascending."""
    m = min(n, keep)
    last = min(recent, m)
    old = np.where(np.isnan(w[:n - last]), -np.inf, w[:n - last].astype(np.float64))
    # NaN after every number, -inf among them; equal weights by slot
    order = sorted(range(n - last), key=lambda j: (-old[j], np.isnan(w[j]), j))
    return np.array(sorted(order[:m - last]) + list(range(n - last, n)), dtype=np.int64)
