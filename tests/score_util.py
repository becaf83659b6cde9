"""Plain 64-bit forms of scored attention, of the cached tokens' shares and of eviction, in numpy."""
from __future__ import annotations

import numpy as np

from quant_util import B


def visible(pos, L, window=0, first=None, prefix=0):
    """Positions that the row at pos attends to, of a sequence of L tokens."""
    t = np.arange(L)
    ok = (t <= pos) | (t < min(prefix, L))
    if window > 0:
        ok &= t > pos - window
    if first is not None:
        ok &= t >= first
    return t[ok]


def rows_of(pools, table, t, h):
    """Held keys and values [len(t), D] of positions t, KV head h."""
    blk = np.asarray(table)[t // B]
    return pools.kh[blk, h, t % B], pools.vh[blk, h, t % B]


def ref_scored(q, where, pools, tables, lens, scale, cap=0.0, window=0, slopes=None, first=None, prefix=None):
    """q [T, Hq, D]; where[r] = (sequence, position) of row r; first per row.  Outputs [T, Hq, D], and for every row
    its visible positions and their shares [Hq, n]."""
    q = q.double().numpy()
    T, Hq, D = q.shape
    G = Hq // pools.Hkv
    out, shares = np.zeros_like(q), []
    for r, (s, pos) in enumerate(where):
        t = visible(pos, lens[s], window, None if first is None else first[r], 0 if prefix is None else prefix[s])
        p_all = np.zeros((Hq, len(t)))
        if len(t):
            for h in range(pools.Hkv):
                k, v = rows_of(pools, tables[s], t, h)
                x = q[r, h * G:(h + 1) * G] @ k.T * scale
                if cap > 0:
                    x = cap * np.tanh(x / cap)
                if slopes is not None:
                    x = x - slopes[h * G:(h + 1) * G, None].astype(np.float64) * np.abs(pos - t)
                p = np.exp(x - x.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                p_all[h * G:(h + 1) * G] = p
                out[r, h * G:(h + 1) * G] = p @ v
        shares.append((t, p_all))
    return out, shares


def share_bound(q, pools, scale, cap, slopes, L):
    """Bound on the relative error of a share: twice that of a score in natural units, plus the exponentials', sums'
    and products' own (2^-18).  A score's products are exact and its sum runs through at most 16 additions of tensor-core
    partial sums (8 MMAs of 17 terms, or D / 16 dependent terms and 4 shuffles on the CUDA cores), each within 17 * 2^-23
    of the sum of the absolute products; a coded key's, of |q|_1 (|zero| + scale * top) <= 3 |q|_1 max|k|.  The cap's tanh
    is within 2^-21 of 1, the distance term within 2^-22 of itself."""
    q1 = np.abs(q.double().numpy()).sum(-1).max()
    kmax = np.abs(pools.kh[np.isfinite(pools.kh)]).max()
    d = 16 * 17 * 2.0 ** -23 * 3 * q1 * kmax * scale + cap * 2.0 ** -21
    if slopes is not None:
        d += float(np.abs(slopes).max()) * L * 2.0 ** -22
    return 2 * d + 2.0 ** -18


def ref_weights(w0, shares, tables, lens, new, Hkv):
    """w0 float32 [NB, Hkv, 16] after the step: (exact weights, share of this step in each)."""
    w, step = w0.astype(np.float64).copy(), np.zeros_like(w0, dtype=np.float64)
    for s, (t, p) in enumerate(shares):
        L = lens[s]
        fresh = np.arange(L - (L if new is None else new[s]), L)
        for f in fresh:
            w[tables[s][f // B], :, f % B] = 0.0
        G = p.shape[0] // Hkv
        for h in range(Hkv):
            blk = np.asarray(tables[s])[t // B]
            add = p[h * G:(h + 1) * G].sum(0)
            np.add.at(w, (blk, h, t % B), add)
            np.add.at(step, (blk, h, t % B), add)
    return w, step


def ref_select_tokens(weights, tables, lens, n, sink, recent):
    """weights float32 [NB, Hkv, 16] -> kept int32 [S, Hkv, n]."""
    Hkv = weights.shape[1]
    kept = np.full((len(lens), Hkv, n), -1, np.int32)
    for s, L in enumerate(lens):
        t = np.arange(L)
        for h in range(Hkv):
            w = weights[np.asarray(tables[s])[t // B], h, t % B].astype(np.float64)
            nan = np.isnan(w)  # below every number, -inf too
            forced = (t < sink) | (t >= L - recent)
            order = np.lexsort((t, np.where(nan, 0.0, -w), nan, ~forced))[:n]
            kept[s, h, :len(order)] = np.sort(order)
    return kept
