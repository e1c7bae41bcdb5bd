"""The paged cache's operators in binary64 numpy, written from their definition.

Positions go through the page table one by one; codes are values on the e4m3
grid (4 significant bits, spacing never below 2^-9, halves to even, at most 448).
"""
import numpy as np

BLOCK = 16


def grid(x):
    """x rounded to the e4m3 grid; infinities to 448, NaN stays."""
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore"):
        _, e = np.frexp(np.where(np.isfinite(x), x, 1.0))
        step = np.exp2(np.maximum(e - 4, -9).astype(np.float64))
        return np.clip(np.round(x / step) * step, -448.0, 448.0)


def half_step(x):
    """Half the grid's spacing at x."""
    _, e = np.frexp(np.abs(x))
    return np.exp2(np.maximum(e - 4, -9).astype(np.float64)) / 2


def block_scale(amax):
    """Smallest 2^k, k >= -64, with amax <= 448 * 2^k."""
    k = -64
    while amax > 448.0 * 2.0 ** k:
        k += 1
    return 2.0 ** k


def rotate(x, t, inv_freq, inter):
    """One head's row at position t in binary64."""
    x = np.asarray(x, np.float64).copy()
    r = 2 * len(inv_freq)
    a = float(t) * np.asarray(inv_freq, np.float64)
    i = np.arange(r // 2)
    p, q = (2 * i, 2 * i + 1) if inter else (i, i + r // 2)
    c, s = np.cos(a), np.sin(a)
    y = x.copy()
    y[..., p] = x[..., p] * c - x[..., q] * s
    y[..., q] = x[..., q] * c + x[..., p] * s
    return y


def append(state, k, v, start, n_new, inv_freq, inter, q=None):
    """Appends to state = dict(K, V [n_pages][page][Hkv][d], scales or None, table) in place:
    K and V hold the values of bf16 pages unrounded, or codes.  Returns the rotated queries."""
    B, Nq = k.shape[:2]
    n_pages, page = state["K"].shape[:2]
    table, scales = state["table"], state["scales"]
    q_out = None if q is None else np.full(q.shape, np.nan)
    for b in range(B):
        n, t0 = min(n_new[b], Nq), int(start[b])
        if n <= 0 or t0 < 0:
            continue
        kr = np.stack([rotate(k[b, i], t0 + i, inv_freq, inter) for i in range(n)])
        if q is not None:
            for i in range(n):
                q_out[b, i] = rotate(q[b, i], t0 + i, inv_freq, inter)
        for blk in range(t0 // BLOCK, (t0 + n - 1) // BLOCK + 1):
            lo, hi = max(blk * BLOCK, t0), min((blk + 1) * BLOCK, t0 + n)
            if blk * BLOCK >= table.shape[1] * page:
                continue
            pg = table[b, blk * BLOCK // page]
            if pg < 0 or pg >= n_pages:
                continue
            s0 = blk * BLOCK % page
            for which, name, x in ((0, "K", kr), (1, "V", np.asarray(v[b], np.float64))):
                new = x[lo - t0:hi - t0]
                dst = state[name][pg, s0:s0 + BLOCK]
                at = slice(lo - blk * BLOCK, hi - blk * BLOCK)
                if scales is None:
                    dst[at] = new
                    continue
                for h in range(k.shape[2]):
                    fin = np.abs(new[:, h][np.isfinite(new[:, h])])
                    s = block_scale(fin.max() if fin.size else 0.0)
                    if at.start > 0:
                        was = float(scales[pg, s0 // BLOCK, which, h])
                        if s > was:
                            dst[:at.start, h] = grid(dst[:at.start, h] * (was / s))
                        else:
                            s = was
                    dst[at, h] = grid(new[:, h] / s)
                    scales[pg, s0 // BLOCK, which, h] = s
    return q_out


def attend(Kv, Vv, table, Q, idx, cnt, scale, sV=None):
    """Values Kv, Vv [n_pages][page][Hkv][d] (codes times scales): per row and head the output,
    its sum of p |v| (what errors of p scale with), the largest sum of |q k| and lse; with V's
    scales sV [n_pages][page][Hkv] the second is (that, max p sV * sum |codes|), what an
    absolute error of every p sV relative to the largest scales with."""
    n_pages, page, Hkv, d = Kv.shape
    B, Nq, Hq, _ = Q.shape
    O, A = np.zeros((B, Nq, Hq, d)), np.zeros((B, Nq, Hq, d))
    Z, L = np.zeros((B, Nq, Hq)), np.full((B, Nq, Hq), -np.inf)
    F = np.zeros((B, Nq, Hq, d))
    for b in range(B):
        for i in range(Nq):
            t = np.asarray(idx[b, i, :max(0, cnt[b, i])], np.int64)
            t = t[(t >= 0) & (t < table.shape[1] * page)]
            pg = table[b, t // page]
            ok = (pg >= 0) & (pg < n_pages)
            t, pg = t[ok], pg[ok]
            if len(t) == 0:
                continue
            for h in range(Hq):
                g = h // (Hq // Hkv)
                ks, vs = Kv[pg, t % page, g], Vv[pg, t % page, g]
                z = scale * (ks @ Q[b, i, h])
                m = z.max()
                p = np.exp(z - m)
                L[b, i, h] = m + np.log(p.sum())
                p /= p.sum()
                O[b, i, h], A[b, i, h] = p @ vs, p @ np.abs(vs)
                Z[b, i, h] = scale * (np.abs(ks) @ np.abs(Q[b, i, h])).max()
                if sV is not None:
                    sv = sV[pg, t % page, g]
                    F[b, i, h] = (p * sv).max() * (np.abs(vs) / sv[:, None]).sum(0)
    return O, (A if sV is None else (A, F)), Z, L
