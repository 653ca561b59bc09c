"""64-bit form of attention of many q rows over a paged cache, and the bounds of its errors.

As in paged_reference.py (u = 2^-24): a score is off by ds = (hd + 8) 2 u scale sum |q_d k_d| + 4 u |s| at most, a softmax
weight by a factor e^(2 ds) and the sums over n slots by (n / 8 + 64) 2 u.  That holds where q, the weights and an f32 cache's
rows keep 22 bits.  With out bf16 and an f16 cache q and the weights may be rounded to f16 (2^-11 of themselves: half a
step): ds grows by 2^-11 scale sum |q_d k_d|, each weight is off by another 2^-11 (2^-11 of the normalised weights' sum), and
the output is rounded to bf16 (2^-8 of it).
"""
import numpy as np

U = 2.0 ** -24


def rows_ref(k, v, q, places, scale, nh, nkv, hd, bf16_f16):
    """places[i]: the (page, row in page) index arrays that row i of q sees.  out [rows, nh * hd], lse [rows, nh] and bounds."""
    rows, G = q.shape[0], nh // nkv
    out, lse = np.zeros((rows, nh * hd)), np.full((rows, nh), -np.inf)
    b_out, b_lse = np.zeros_like(out), np.zeros_like(lse)
    cast = {}
    for i in range(rows):
        pages, at = places[i]
        n = len(pages)
        if n == 0:
            continue
        key = (tuple(pages[:1]), n, tuple(at[-1:]), tuple(pages[-1:]))
        if key not in cast:
            cast = {key: (k[pages, at].astype(np.float64).reshape(n, nkv, hd), v[pages, at].astype(np.float64).reshape(n, nkv, hd))}
        K, V = cast[key]
        for h in range(nh):
            x, kk, vv = q[i, h * hd:(h + 1) * hd].astype(np.float64), K[:, h // G], V[:, h // G]
            cols = slice(h * hd, (h + 1) * hd)
            with np.errstate(invalid="ignore", over="ignore"):
                s = scale * (kk @ x)
                m = s.max()
                p = np.exp(s - m)
                l = p.sum()
                p /= l
                out[i, cols] = p @ vv
                lse[i, h] = m + np.log(l) if m > -np.inf or m != m else -np.inf
                size = abs(scale) * (np.abs(kk) @ np.abs(x)).max()
                ds = (hd + 8) * 2 * U * size + 4 * U * np.abs(s).max() + (2.0 ** -11 * size if bf16_f16 else 0)
                rel = np.expm1(2 * ds) + (n / 8 + 64) * 2 * U + (2.0 ** -11 if bf16_f16 else 0)
                b_out[i, cols] = rel * (p @ np.abs(vv)) + 1e-37
                b_lse[i, h] = rel + 4 * U * abs(lse[i, h])
    return out, lse, b_out, b_lse


def prompt_places(c, first, lens, nt, window):
    """What each row of q sees; None for rows that belong to no sequence."""
    places = [None] * nt
    for b in range(c.B):
        a, e, n = int(first[b]), int(first[b + 1]), int(lens[b])
        for i in range(e - a):
            hi = max(0, n - (e - a) + i + 1)
            lo = max(0, n - (e - a) + i + 1 - window) if window else 0
            s = np.arange(min(lo, hi), hi)
            places[a + i] = (c.table[b, s // c.page], s % c.page)
    return places


def prefix_places(c, lens, share, prefix):
    places = []
    for b in range(c.B):
        s = np.arange(int(lens[b]))
        by = np.where(s < prefix[b], share[b], b)
        places.append((c.table[by, s // c.page], s % c.page))
    return places
