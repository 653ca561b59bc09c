"""Plain 64-bit forms of the paged-cache operators, and seeded caches for their tests.

The reference works on numpy arrays in float64 and addresses the cache slot by slot through
its page table.  Error bounds (u = 2^-24, the unit roundoff of f32):

  store, no norm: z = y + b rounds once (u); cos and sin are off by at most 2 ulp (4 u); each
    product and the sum round once: |r - exact| <= 7 u (|x0| + |x1|), taken as 8 u.
  store, norm: the sum of squares is a chain of at most hd/32 + 8 + 5 additions of values that
    are off by 2 u each: relative 24 u at hd = 256; the root halves it; division, + eps, root,
    reciprocal and the two products add 6 u: 18 u on each normed value, then the rotation: 32 u.
  attention: a score is a sum of hd products of values rounded (or split) to at least 22 bits,
    added in f32 (which the tensor cores may truncate: 2 u an addition):
    ds = (hd + 8) 2 u * sum |q_d k_d| * scale, plus 4 u |s| of the change to log2 terms.
    A softmax weight is then off by a factor e^(2 ds) (its own score, and the common sum), and
    the sums over n slots are chains of at most n/8 + 64 additions of 2 u each.
"""
import numpy as np

U = 2.0 ** -24


def f16_half_step(v):
    """Largest error of rounding v to f16: half a step, 2^-25 in the subnormal range."""
    return np.maximum(np.abs(v) * 2.0 ** -11, 2.0 ** -25)


class Cache:
    """Host copy of a paged cache with scattered pages; rows that nothing assigned hold `fill`."""

    def __init__(self, rng, B, nkv, hd, kv, page, max_pages, spare=2, fill=np.nan, table_fill=-1, lens=None):
        self.B, self.nkv, self.hd, self.kv, self.page, self.max_pages = B, nkv, hd, kv, page, max_pages
        self.cap = page * max_pages
        self.lens = np.asarray(lens if lens is not None else [self.cap] * B, np.int32)
        used = [-(-int(n) // page) for n in self.lens]
        self.n_pages = sum(used) + spare
        ids = iter(rng.permutation(self.n_pages))
        self.table = np.full((B, max_pages), table_fill, np.int32)
        for b, u in enumerate(used):
            for i in range(u):
                self.table[b, i] = next(ids)
        dt = np.float16 if kv == "f16" else np.float32
        self.k = np.full((self.n_pages, page, nkv * hd), fill, dt)
        self.v = np.full_like(self.k, fill)
        for b in range(B):
            for s in range(int(self.lens[b])):
                at = self.row(b, s)
                self.k[at] = rng.standard_normal(nkv * hd).astype(dt)
                self.v[at] = rng.standard_normal(nkv * hd).astype(dt)

    def row(self, b, s):
        return self.table[b, s // self.page], s % self.page

    def rows(self, pool, b, slots):
        slots = np.asarray(slots, np.int64)
        return pool[self.table[b, slots // self.page], slots % self.page]


def store_ref(Y, bias, qw, kw, eps, pos, nh, nkv, hd, inv_freq):
    """q, k, v of the tokens in 64 bits, and the bound of q's and k's errors."""
    z = Y.astype(np.float64) + (0.0 if bias is None else bias.astype(np.float64))
    nt = z.shape[0]
    z = z.reshape(nt, nh + 2 * nkv, hd)
    x, v = z[:, :nh + nkv], z[:, nh + nkv:]
    if qw is not None:
        w = np.concatenate([np.tile(qw, (nh, 1)), np.tile(kw, (nkv, 1))]).astype(np.float64)
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    angle = (pos.astype(np.float32)[:, None] * inv_freq[None]).astype(np.float64)[:, None]  # one f32 product
    c, s = np.cos(angle), np.sin(angle)
    x0, x1 = x[..., :hd // 2], x[..., hd // 2:]
    r = np.concatenate([x0 * c - x1 * s, x0 * s + x1 * c], -1)
    size = np.abs(x0) + np.abs(x1)
    bound = (8 if qw is None else 32) * U * np.concatenate([size, size], -1) + 1e-37
    flat = lambda t, a, b: t[:, a:b].reshape(nt, -1)  # noqa: E731
    return (flat(r, 0, nh), flat(r, nh, nh + nkv), v.reshape(nt, -1), flat(bound, 0, nh), flat(bound, nh, nh + nkv))


def attn_ref(cache, q, lens, scale, window, nh):
    """out, lse, weight (added) in 64 bits, and the bounds of their errors."""
    B, hd, nkv, G = cache.B, cache.hd, cache.nkv, nh // cache.nkv
    out, lse = np.zeros((B, nh * hd)), np.full((B, nh), -np.inf)
    weight = np.zeros((B, nkv, cache.cap))
    b_out, b_lse, b_weight = np.zeros_like(out), np.zeros((B, nh)), np.zeros_like(weight)
    for b in range(B):
        n = int(lens[b])
        j0 = max(0, n - window) if window else 0
        if n == j0:
            continue
        K = cache.rows(cache.k, b, range(j0, n)).astype(np.float64).reshape(-1, nkv, hd)
        V = cache.rows(cache.v, b, range(j0, n)).astype(np.float64).reshape(-1, nkv, hd)
        for h in range(nh):
            x, k, v = q[b, h * hd:(h + 1) * hd].astype(np.float64), K[:, h // G], V[:, h // G]
            with np.errstate(invalid="ignore", over="ignore"):
                s = scale * (k @ x)
                m = s.max()
                p = np.exp(s - m)
                l = p.sum()
                p /= l
                out[b, h * hd:(h + 1) * hd] = p @ v
                lse[b, h] = m + np.log(l) if m > -np.inf or m != m else -np.inf  # log 0 where every exp(s) is 0
                ds = (hd + 8) * 2 * U * abs(scale) * (np.abs(k) @ np.abs(x)).max() + 4 * U * np.abs(s).max()
                rel = 2 * ds + ((n - j0) / 8 + 64) * 2 * U
                b_out[b, h * hd:(h + 1) * hd] = rel * (p @ np.abs(v)) + 1e-37
                b_lse[b, h] = rel + 4 * U * abs(lse[b, h])
                weight[b, h // G, j0:n] += p
                b_weight[b, h // G, j0:n] += rel * p + 2 * U * p + 1e-37
    return out, lse, weight, b_out, b_lse, b_weight


def evict_ref(cache, lens, next_pos, weight, pos, budget, recent):
    """New k, v, lens, weight, pos (copies; slots at or above the new length as they were)."""
    k, v, w, t = cache.k.copy(), cache.v.copy(), weight.copy(), pos.copy()
    hd = cache.hd
    for b in range(cache.B):
        n = int(lens[b])
        if n <= budget:
            continue
        for h in range(cache.nkv):
            def rank(s):
                x = float(weight[b, h, s])
                if int(pos[b, h, s]) >= int(next_pos[b]) - recent:
                    return 0, 0.0, s
                return (1, 0.0, s) if x != x else (2, -x, s)
            kept = set(sorted(range(n), key=rank)[:budget])
            holes = [s for s in range(budget) if s not in kept]
            movers = [s for s in range(budget, n) if s in kept]
            assert len(holes) == len(movers)
            for i, j in zip(holes, movers):
                for pool in (k, v):
                    pool[cache.row(b, i)][h * hd:(h + 1) * hd] = pool[cache.row(b, j)][h * hd:(h + 1) * hd]
                w[b, h, i], t[b, h, i] = weight[b, h, j], pos[b, h, j]
    return k, v, np.minimum(lens, budget), w, t
