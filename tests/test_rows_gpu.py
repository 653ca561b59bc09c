"""Attention with many q rows over the paged cache (prompts, shared prefixes) on the GPU against its 64-bit form
(rows_reference.py, which derives the bounds)."""
import numpy as np
import pytest

import paged_reference
import qkv_rope_kv_gb300 as Q
import rows_reference as ref
from test_paged_gpu import close, dev, make_plan, short

pytestmark = pytest.mark.gpu


def pools_of(c, pool_off=0, page_gap=0):
    import torch
    step = c.page * c.nkv * c.hd + page_gap
    dt = torch.float16 if c.kv == "f16" else torch.float32
    pools = []
    for a in (c.k, c.v):
        flat = torch.full((c.n_pages * step + pool_off,), float("nan"), dtype=dt, device="cuda")
        view = flat[pool_off:].as_strided(a.shape, (step, c.nkv * c.hd, 1))
        view.copy_(dev(a))
        pools.append(view)
    return pools


def buffers(rows, nqt, x, out, stride):
    import torch
    q = torch.zeros(rows, nqt + stride, device="cuda")[:, :nqt]
    q.copy_(dev(x))
    o = torch.full((rows, nqt + stride), 77.0, dtype=torch.bfloat16 if out == "bf16" else torch.float32, device="cuda")
    return q, o


def check(c, x, places, nh, scale, out, o, lse, nqt):
    """Rows that belong to no sequence keep what they held."""
    rows = [i for i, p in enumerate(places) if p is not None]
    single = out == "bf16" and c.kv == "f16"
    want, wl, bo, bl = ref.rows_ref(c.k, c.v, x[rows], [places[i] for i in rows], scale, nh, c.nkv, c.hd, single)
    got = o.float().cpu().numpy()
    bound = bo + (2.0 ** -8 * (np.abs(want) + bo) if out == "bf16" else 0)
    close(got[rows][:, :nqt], want, bound, "out")
    close(lse.cpu().numpy()[rows], wl, bl, "lse")
    others = [i for i in range(len(places)) if places[i] is None]
    assert (got[others] == 77.0).all() and (got[:, nqt:] == 77.0).all()
    assert (lse.cpu().numpy()[others] == 55.0).all()


def run_prompt(nh, nkv, hd, kv, page, new, cached, window=0, out="f32", seed=0, q_scale=1.5, change=None, stride=0,
               pool_off=0, page_gap=0, behind=0, ahead=0, lens=None, plan=None, workspace=None, twice=True, scale=None):
    import torch
    rng = np.random.default_rng(seed)
    B = len(new)
    lens = np.array([n + c for n, c in zip(new, cached)] if lens is None else lens, np.int32)
    c = paged_reference.Cache(rng, B, nkv, hd, kv, page, max(1, -(-int(lens.max()) // page) + 1), lens=lens)
    first = np.cumsum([ahead] + list(new)).astype(np.int32)
    nt = int(first[-1]) + behind
    x = (q_scale * rng.standard_normal((nt, nh * hd))).astype(np.float32)
    if change:
        change(c, x)
    plan = plan or make_plan(nh, nkv, hd, kv)
    cache = Q.PagedKv(plan, *pools_of(c, pool_off, page_gap), dev(c.table))
    q, o = buffers(nt, nh * hd, x, out, stride)
    lse = torch.full((nt, nh), 55.0, device="cuda")
    if workspace is None:
        workspace = torch.full((Q.qkv_prompt_attn_workspace_bytes(plan, cache, nt),), 0xa5, dtype=torch.uint8, device="cuda")
    scale = hd ** -0.5 if scale is None else scale
    args = (plan, cache, q, dev(first), dev(lens), scale, o[:, :nh * hd], workspace)
    Q.qkv_prompt_attn_step(*args, window=window, lse=lse)
    torch.cuda.synchronize()
    assert Q.qkv_check_device_error()[0] == 0
    check(c, x, ref.prompt_places(c, first, lens, nt, window), nh, scale, out, o, lse, nh * hd)
    if twice:  # the same bits again
        o2 = torch.full_like(o, 77.0)
        Q.qkv_prompt_attn_step(*args[:6], o2[:, :nh * hd], workspace, window=window)
        assert torch.equal(o.view(torch.int16 if out == "bf16" else torch.int32), o2.view(torch.int16 if out == "bf16" else torch.int32))


@pytest.mark.parametrize("nh,nkv,hd,kv,page,new,cached,kw", [
    (14, 2, 64, "f32", 16, [17], [0], {}),
    (14, 2, 64, "f16", 16, [17], [0], {}),
    (1, 1, 2, "f32", 1, [1], [0], {}),
    (1, 1, 8, "f16", 1, [3], [2], {}),
    (28, 4, 128, "f16", 16, [1], [0], {}),
    (28, 4, 128, "f16", 16, [130], [0], {}),
    (28, 4, 128, "f16", 16, [40, 0, 3, 77], [5, 9, 300, 0], {}),
    (28, 4, 128, "f16", 16, [40, 0, 3, 77], [5, 9, 300, 0], dict(out="bf16")),
    (40, 8, 128, "f16", 64, [257], [1000], dict(out="bf16")),
    (40, 8, 128, "f16", 64, [4] * 9, [700, 0, 1, 127, 128, 129, 400, 64, 63], {}),
    (40, 8, 128, "f16", 7, [33, 20], [100, 0], dict(out="bf16")),
    (8, 1, 64, "f16", 17, [300], [33], {}),
    (8, 1, 64, "f16", 17, [300], [33], dict(out="bf16")),
    (6, 3, 96, "f16", 32, [70, 5], [0, 200], {}),
    (6, 3, 80, "f16", 32, [70, 5], [0, 200], dict(out="bf16")),
    (6, 3, 80, "f32", 32, [70, 5], [0, 200], dict(out="bf16")),
    (4, 1, 256, "f16", 5, [31], [90], {}),
    (4, 1, 256, "f32", 5, [31], [90], dict(out="bf16")),
    (6, 2, 6, "f16", 4, [9], [30], {}),
    (12, 1, 64, "f16", 16, [50], [0], {}),
    (136, 1, 16, "f32", 16, [3, 2], [40, 0], {}),               # more q heads a kv head than a tile's rows
    (300, 1, 64, "f16", 16, [3, 2], [40, 0], {}),
    (300, 1, 64, "f16", 16, [3, 2], [40, 0], dict(out="bf16")),
    (14, 2, 64, "f16", 16, [60, 20], [100, 0], dict(window=33)),
    (14, 2, 64, "f32", 16, [60, 20], [100, 0], dict(window=1)),
    (28, 4, 128, "f16", 16, [400], [700], dict(window=200, out="bf16")),
    (28, 4, 128, "f16", 16, [400], [700], dict(window=128)),
    (28, 4, 128, "f16", 16, [5, 30], [0, 0], dict(lens=[3, 4])),  # more new tokens than slots: the first see nothing
    (28, 4, 128, "f16", 16, [300], [0], dict(lens=[0])),
    (14, 2, 64, "f16", 16, [9, 4], [30, 2], dict(ahead=3, behind=5)),
    (14, 2, 64, "f32", 16, [9, 4], [30, 2], dict(ahead=3, behind=5, out="bf16")),
    (28, 4, 128, "f16", 16, [40, 9], [5, 300], dict(stride=12, page_gap=32)),
    (28, 4, 128, "f16", 16, [40, 9], [5, 300], dict(stride=5, out="bf16")),
    (28, 4, 128, "f16", 16, [40, 9], [5, 300], dict(pool_off=1)),
    (28, 4, 128, "f16", 16, [40, 9], [5, 300], dict(page_gap=1)),
    (28, 4, 128, "f16", 16, [40, 9], [5, 300], dict(q_scale=12.0)),
    (28, 4, 128, "f16", 16, [40, 9], [5, 300], dict(scale=-0.11, out="bf16")),
    (28, 4, 128, "f16", 16, [40, 9], [5, 300], dict(scale=0.0)),
    (4, 4, 16, "f16", 16, [40, 9], [5, 300], {}),                # heads narrower than a chunk, rows narrower than a box
    (3, 1, 32, "f16", 24, [200, 9], [5, 300], dict(out="bf16")),
    (6, 2, 48, "f16", 8, [70, 9], [5, 300], {}),
    (2, 1, 128, "f16", 64, [1500], [0], dict(out="bf16")),
    (2, 1, 128, "f16", 64, [2], [9000], {}),                     # one tile over many CTAs
    (2, 1, 64, "f32", 64, [2], [9000], {}),
], ids=short)
def test_prompt(qkv, nh, nkv, hd, kv, page, new, cached, kw):
    run_prompt(nh, nkv, hd, kv, page, new, cached, **kw)


@pytest.mark.parametrize("kv,hd", [("f16", 128), ("f16", 64), ("f32", 64), ("f16", 256)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [np.inf, np.nan])
def test_what_later_tokens_hold_does_not_matter(qkv, kv, hd, out, bad):
    """Infinities and NaN in V (or K) of a token reach the rows that see it, and no others."""
    def spoil(c, x):
        c.v[c.row(0, 100)][3] = bad
        c.v[c.row(0, 77)][hd - 1] = -bad
        c.k[c.row(0, 150)][5] = bad if bad != bad else 0
    run_prompt(4, 1, hd, kv, 16, [120], [50], out=out, change=spoil, twice=False)


@pytest.mark.parametrize("kv", ["f16", "f32"])
def test_rows_without_a_finite_score(qkv, kv):
    """Every score -inf gives NaN, as the formula does; the largest and smallest numbers stay finite."""
    def spoil(c, x):
        for s in range(0, 40):
            c.k[c.row(0, s)][:] = 0
            c.k[c.row(0, s)][0] = -np.inf
        x[:, :64] = 0
        x[:, 0] = 1.0
        x[:, 64:] = 0  # the other head: 0 * -inf
    run_prompt(2, 1, 64, kv, 16, [60], [0], change=spoil, twice=False)

    def large(c, x):
        x[:] = np.float32(1e-30) * np.sign(x)
        x[3] *= 1e30
        c.v[:] = np.where(np.isnan(c.v), c.v, 60000 if kv == "f16" else 1e35)
    run_prompt(2, 1, 64, kv, 16, [60], [20], change=large)


def test_flags_what_is_out_of_range(qkv):
    """Bad pairs, lengths and pages are flagged; what they would have addressed is not read, other sequences are right."""
    import torch
    rng = np.random.default_rng(5)
    for kv, hd in (("f16", 128), ("f32", 64)):
        nh, nkv, page = 4, 2, 16
        c = paged_reference.Cache(rng, 3, nkv, hd, kv, page, 6, lens=[60, 60, 60])
        plan = make_plan(nh, nkv, hd, kv)
        pools = pools_of(c)
        nt = 30
        x = rng.standard_normal((nt, nh * hd)).astype(np.float32)
        for first, lens, entry, value in (([0, 10, 5, 5], [60] * 3, None, 5), ([0, 10, 31, 40], [60] * 3, None, None),
                                          ([-1, 10, 20, 30], [60] * 3, None, -1), ([0, 10, 20, 30], [60, 97, 60], None, 97),
                                          ([0, 10, 20, 30], [60, -2, 60], None, -2), ([0, 10, 20, 30], [60] * 3, c.n_pages, c.n_pages),
                                          ([0, 10, 20, 30], [60] * 3, -1, -1)):
            table = c.table.copy()
            if entry is not None:
                table[1, 2] = entry
            cache = Q.PagedKv(plan, *pools, dev(table))
            q, o = buffers(nt, nh * hd, x, "f32", 0)
            ws = torch.empty(Q.qkv_prompt_attn_workspace_bytes(plan, cache, nt), dtype=torch.uint8, device="cuda")
            Q.qkv_prompt_attn_step(plan, cache, q, dev(np.int32(first)), dev(np.int32(lens)), 0.1, o, ws)
            torch.cuda.synchronize()
            flags, bad = Q.qkv_check_device_error()
            assert flags == 4 and (value is None or bad == value)
            good = ref.prompt_places(c, [first[0], first[1], first[1], first[1]], [60] * 3, nt, 0) if first[0] == 0 else [None] * nt
            rows = [i for i, pl in enumerate(good) if pl is not None]
            if not rows:
                continue
            want, _, bo, _ = ref.rows_ref(c.k, c.v, x[rows], [good[i] for i in rows], 0.1, nh, nkv, hd, False)
            close(o.cpu().numpy()[rows], want, bo, "the first sequence")
            if lens[1] != 60:  # counts as empty
                assert (o[first[1]:first[2]] == 0).all()
            if entry is not None:  # slots 32 to 47 are not there: they count as not seen
                places = ref.prompt_places(c, [0, 10, 20, 30], [60] * 3, nt, 0)
                cut = []
                for i in range(10, 20):
                    keep = [j for j in range(len(places[i][0])) if not 32 <= j < 48]
                    cut.append((places[i][0][keep], places[i][1][keep]))
                want, _, bo, _ = ref.rows_ref(c.k, c.v, x[10:20], cut, 0.1, nh, nkv, hd, False)
                close(o.cpu().numpy()[10:20], want, bo, "without the page")


# ---------------------------------------------------------------- prefix

def run_prefix(nh, nkv, hd, kv, page, share, prefix, own, out="f32", seed=0, q_scale=1.5, change=None, stride=0, lens=None,
               pool_off=0, plan=None, workspace=None):
    """own[b]: slots behind the prefix.  Table entries below a sequence's own slots are -1 where it shares another's."""
    import torch
    rng = np.random.default_rng(seed)
    B = len(share)
    full = np.array([p + n for p, n in zip(prefix, own)], np.int32)
    c = paged_reference.Cache(rng, B, nkv, hd, kv, page, max(1, -(-int(full.max()) // page) + 1), lens=full)
    lens = full if lens is None else np.asarray(lens, np.int32)
    for b in range(B):
        if share[b] != b:
            c.table[b, :prefix[b] // page] = -1
    x = (q_scale * rng.standard_normal((B, nh * hd))).astype(np.float32)
    if change:
        change(c, x)
    plan = plan or make_plan(nh, nkv, hd, kv)
    cache = Q.PagedKv(plan, *pools_of(c, pool_off), dev(c.table))
    q, o = buffers(B, nh * hd, x, out, stride)
    lse = torch.full((B, nh), 55.0, device="cuda")
    if workspace is None:
        workspace = torch.full((Q.qkv_prefix_attn_workspace_bytes(plan, cache),), 0xa5, dtype=torch.uint8, device="cuda")
        workspace[:4096] = 0
    scale = hd ** -0.5
    i32 = lambda v: dev(np.asarray(v, np.int32))  # noqa: E731
    for _ in range(2):  # the workspace stays usable
        Q.qkv_prefix_attn_step(plan, cache, q, i32(lens), i32(share), i32(prefix), scale, o[:, :nh * hd], workspace, lse=lse)
        torch.cuda.synchronize()
        assert Q.qkv_check_device_error()[0] == 0
        check(c, x, ref.prefix_places(c, lens, share, prefix), nh, scale, out, o, lse, nh * hd)
        o.fill_(77.0)


@pytest.mark.parametrize("nh,nkv,hd,kv,page,share,prefix,own,kw", [
    (14, 2, 64, "f32", 16, [0] * 4, [509] * 4, [1, 30, 7, 37], {}),
    (14, 2, 64, "f16", 16, [0] * 4, [512] * 4, [1, 30, 7, 37], {}),
    (28, 4, 128, "f16", 16, [0], [100], [3], {}),                      # nobody shares
    (28, 4, 128, "f16", 16, [0, 1, 2], [100, 0, 60], [3, 5, 6], {}),
    (28, 4, 128, "f16", 16, [0, 0], [130, 130], [1, 300], dict(out="bf16")),
    (40, 8, 128, "f16", 64, [0] * 30, [777] * 30, list(range(1, 31)), dict(out="bf16")),
    (40, 8, 128, "f16", 64, [0] * 60, [777] * 60, list(range(1, 61)), {}),      # two tiles
    (40, 8, 128, "f16", 16, [0] * 5 + [5] * 3 + [8] + [9] * 4, [200] * 5 + [33] * 3 + [50] + [16] * 4, [9] * 13, {}),
    (8, 1, 64, "f16", 17, [0] * 7, [3000] * 7, [20] * 7, {}),                   # one tile over many CTAs
    (8, 1, 64, "f32", 17, [0] * 7, [3000] * 7, [20] * 7, dict(out="bf16")),
    (8, 2, 64, "f16", 8, [0] * 6, [64, 64, 64, 40, 0, 7], [5, 1, 0, 30, 12, 90], {}),   # uneven shares of one prefix
    (8, 2, 64, "f16", 8, [0] * 6, [64] * 6, [5] * 6, dict(lens=[69, 64, 63, 30, 1, 0])),  # lengths within the prefix
    (6, 3, 80, "f16", 32, [0, 0, 0, 3], [96, 96, 96, 40], [1, 2, 3, 4], {}),
    (4, 1, 256, "f16", 5, [0, 0, 0], [95] * 3, [1, 20, 3], {}),
    (300, 1, 64, "f16", 16, [0, 0], [200, 200], [5, 60], {}),
    (28, 4, 128, "f16", 16, [0] * 4, [256] * 4, [9] * 4, dict(stride=5, out="bf16")),
    (28, 4, 128, "f16", 16, [0] * 4, [256] * 4, [9] * 4, dict(pool_off=1)),
    (2, 1, 64, "f16", 1, [0] * 600, [40] * 600, [1] * 600, {}),                  # more sequences than the plan takes at once
], ids=short)
def test_prefix(qkv, nh, nkv, hd, kv, page, share, prefix, own, kw):
    run_prefix(nh, nkv, hd, kv, page, share, prefix, own, **kw)


@pytest.mark.parametrize("kv", ["f16", "f32"])
def test_prefix_of_uneven_lengths_with_nan_beyond(qkv, kv):
    """What lies behind a sequence's share of the prefix does not reach it, NaN and infinities neither."""
    def spoil(c, x):
        c.v[c.row(0, 50)][3] = np.nan
        c.v[c.row(0, 45)][4] = np.inf
    run_prefix(8, 1, 64, kv, 8, [0] * 4, [64, 48, 40, 64], [3, 4, 5, 6], change=spoil)


def test_prefix_flags_what_is_out_of_range(qkv):
    import torch
    rng = np.random.default_rng(6)
    nh, nkv, hd, page = 4, 2, 64, 16
    c = paged_reference.Cache(rng, 3, nkv, hd, "f16", page, 6, lens=[90, 90, 90])
    plan = make_plan(nh, nkv, hd, "f16")
    cache = Q.PagedKv(plan, *pools_of(c), dev(c.table))
    x = rng.standard_normal((3, nh * hd)).astype(np.float32)
    i32 = lambda v: dev(np.asarray(v, np.int32))  # noqa: E731
    for share, prefix, lens, bad in (([0, 3, 0], [48] * 3, [60] * 3, 3), ([0, -1, 0], [48] * 3, [60] * 3, -1),
                                     ([0, 0, 0], [48, 97, 48], [60] * 3, 97), ([0, 0, 0], [48, -5, 48], [60] * 3, -5),
                                     ([0, 0, 0], [48] * 3, [60, 97, 60], 97)):
        q, o = buffers(3, nh * hd, x, "f32", 0)
        lse = torch.full((3, nh), 55.0, device="cuda")
        ws = torch.zeros(Q.qkv_prefix_attn_workspace_bytes(plan, cache), dtype=torch.uint8, device="cuda")
        Q.qkv_prefix_attn_step(plan, cache, q, i32(lens), i32(share), i32(prefix), 0.1, o, ws, lse=lse)
        torch.cuda.synchronize()
        assert Q.qkv_check_device_error() == (4, bad)
        places = ref.prefix_places(c, [60, 60 if lens[1] == 60 else 0, 60], [0, 0, 0], [48, 48 if prefix[1] == 48 else 0, 48])
        if share[1] != 0:
            places[1] = tuple(a[48:] for a in ref.prefix_places(c, [60] * 3, [0, 1, 2], [0] * 3)[1])
        want, wl, bo, bl = ref.rows_ref(c.k, c.v, x, places, 0.1, nh, nkv, hd, False)
        close(o.cpu().numpy(), want, bo, "out")
        close(lse.cpu().numpy(), wl, bl, "lse")


def test_prefix_equals_plain_decode(qkv):
    """With tables that name the shared pages in every row, qkv_attn_step gives the same up to both bounds."""
    import torch
    rng = np.random.default_rng(7)
    nh, nkv, hd, page, B = 28, 4, 128, 16, 12
    c = paged_reference.Cache(rng, B, nkv, hd, "f16", page, 40, lens=[320 + 3 * b + 1 for b in range(B)])
    c.table[1:, :20] = c.table[0, :20]
    plan = make_plan(nh, nkv, hd, "f16")
    cache = Q.PagedKv(plan, *pools_of(c), dev(c.table))
    x = rng.standard_normal((B, nh * hd)).astype(np.float32)
    q, a = buffers(B, nh * hd, x, "f32", 0)
    b = torch.empty_like(a)
    ws = torch.zeros(Q.qkv_prefix_attn_workspace_bytes(plan, cache), dtype=torch.uint8, device="cuda")
    i32 = lambda v: dev(np.asarray(v, np.int32))  # noqa: E731
    Q.qkv_attn_step(plan, cache, q, dev(c.lens), 0.09, a, ws)
    Q.qkv_prefix_attn_step(plan, cache, q, dev(c.lens), i32([0] * B), i32([320] * B), 0.09, b, ws)
    _, _, bo, _ = ref.rows_ref(c.k, c.v, x, ref.prefix_places(c, c.lens, [0] * B, [320] * B), 0.09, nh, nkv, hd, False)
    assert (np.abs(a.cpu().numpy() - b.cpu().numpy()) <= 2 * bo).all()


# ---------------------------------------------------------------- many blocks for a CTA

def attend64(q, K, V, hi, scale):
    """q [rows, G, hd] f32 over K, V [n, hd] f16, row i up to hi[i]: out in 64 bits, and the bound of rows_reference.py
    (with sum p |V| in the place of each column's)."""
    import torch
    s = torch.einsum("rgd,nd->rgn", q.double(), K.double()) * scale
    s.masked_fill_(torch.arange(K.shape[0], device="cuda") >= hi[:, None, None], -float("inf"))
    p = torch.softmax(s, -1)
    size = torch.einsum("rgd,nd->rgn", q.double().abs(), K.double().abs()).amax(-1, keepdim=True) * scale
    return torch.einsum("rgn,nd->rgd", p, V.double()), torch.einsum("rgn,nd->rgd", p, V.double().abs()), size


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("page", [64, 7])  # copied by boxes, and row by row
@pytest.mark.parametrize("nh,nkv,hd,new,cached", [(32, 8, 128, 700, 3900), (16, 8, 64, 1500, 2000), (40, 8, 128, 3, 20000)])
def test_long_prompts(qkv, nh, nkv, hd, new, cached, page, out):
    """Pieces of tens of blocks, which sums of several accumulators and rescaled ones go through."""
    import torch
    torch.manual_seed(1)
    n, G = new + cached, nh // nkv
    per = -(-n // page)
    plan = make_plan(nh, nkv, hd, "f16")
    k, v = (torch.randn(per, page, nkv * hd, device="cuda").half() for _ in range(2))
    k.view(-1, nkv, hd)[cached // 2:] *= 1.5  # maxima move on the way
    table = torch.randperm(per, device="cuda").int()[None].contiguous()
    cache = Q.PagedKv(plan, k, v, table)
    q = 2 * torch.randn(new, nh * hd, device="cuda")
    o = torch.empty(new, nh * hd, device="cuda", dtype=torch.bfloat16 if out == "bf16" else torch.float32)
    ws = torch.empty(Q.qkv_prompt_attn_workspace_bytes(plan, cache, new), dtype=torch.uint8, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    scale = hd ** -0.5
    for _ in range(4):
        o.fill_(float("nan"))
        Q.qkv_prompt_attn_step(plan, cache, q, i32(0, new), i32(n), scale, o, ws)
        K, V = (x[table[0].long()].view(-1, nkv, hd)[:n] for x in (k, v))
        hi = torch.arange(cached + 1, n + 1, device="cuda")
        for h in range(nkv):
            want, most, size = attend64(q.view(new, nkv, G, hd)[:, h], K[:, h], V[:, h], hi, scale)
            ds = (hd + 8) * 2 * ref.U * size + 2 * 4 * ref.U * size
            rel = torch.expm1(2 * (ds + (2.0 ** -11 * size if out == "bf16" else 0))) + (n / 8 + 64) * 2 * ref.U
            bound = rel * most
            if out == "bf16":
                bound = bound + 2.0 ** -11 * most + 2.0 ** -8 * (want.abs() + bound)
            got = o.view(new, nkv, G, hd)[:, h].double()
            assert ((got - want).abs() <= bound).all()
            if out == "f32":  # sums of many values are not worse than those of f32 adds one by one: sqrt(n) u of them
                assert (got - want).norm() <= (n ** 0.5 + hd ** 0.5 * size.max()) * ref.U * most.norm()
    assert Q.qkv_check_device_error()[0] == 0


def test_long_shared_prefix(qkv):
    import torch
    torch.manual_seed(2)
    nh, nkv, hd, page, B, P = 28, 4, 128, 64, 60, 12800
    G, per, own = nh // nkv, P // page, 3
    plan = make_plan(nh, nkv, hd, "f16")
    k, v = (torch.randn(per + B, page, nkv * hd, device="cuda").half() for _ in range(2))
    table = torch.full((B, per + 1), -1, dtype=torch.int32, device="cuda")
    table[0, :per] = torch.randperm(per, device="cuda").int()
    table[:, per] = torch.arange(per, per + B, device="cuda").int()
    cache = Q.PagedKv(plan, k, v, table)
    ws = torch.zeros(Q.qkv_prefix_attn_workspace_bytes(plan, cache), dtype=torch.uint8, device="cuda")
    q = 2 * torch.randn(B, nh * hd, device="cuda")
    full = lambda x: torch.full((B,), x, dtype=torch.int32, device="cuda")  # noqa: E731
    for dtype in (torch.float32, torch.bfloat16):
        for _ in range(4):
            torch.zeros(1 << 28, device="cuda")  # caches hold something else: warps of a CTA run further apart
            o = torch.full((B, nh * hd), float("nan"), device="cuda", dtype=dtype)
            Q.qkv_prefix_attn_step(plan, cache, q, full(P + own), full(0), full(P), hd ** -0.5, o, ws)
            for h in range(nkv):
                Kp, Vp = (x[table[0, :per].long()].view(-1, nkv, hd)[:, h] for x in (k, v))
                Ko, Vo = (x[per:].view(B, page, nkv, hd)[:, :own, h] for x in (k, v))
                x = q.view(B, nkv, G, hd)[:, h]
                s = torch.cat([torch.einsum("bgd,nd->bgn", x.double(), Kp.double()),
                               torch.einsum("bgd,bnd->bgn", x.double(), Ko.double())], -1) * hd ** -0.5
                p = torch.softmax(s, -1)
                want = torch.einsum("bgn,nd->bgd", p[..., :P], Vp.double()) + torch.einsum("bgn,bnd->bgd", p[..., P:], Vo.double())
                got = o.view(B, nkv, G, hd)[:, h].double()
                # 2-norms: weights off by 2^-11 at random, and bf16's half step; f32 as in test_long_prompts
                assert (got - want).norm() <= (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -18) * want.norm()
    assert Q.qkv_check_device_error()[0] == 0


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_calls_at_the_same_time(qkv, out):
    """Calls on two streams, each with a workspace of its own, give the bits of calls one after the other."""
    import torch
    torch.manual_seed(3)
    nh, nkv, hd, page, new = 28, 4, 128, 16, 300
    plan = make_plan(nh, nkv, hd, "f16")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    dtype = torch.bfloat16 if out == "bf16" else torch.float32
    sides = []
    for k in range(2):
        n = new + 700 * (k + 1)
        pools = [torch.randn(-(-n // page), page, nkv * hd, device="cuda").half() for _ in range(2)]
        table = torch.randperm(pools[0].shape[0], device="cuda").int()[None].contiguous()
        cache = Q.PagedKv(plan, *pools, table)
        ws = torch.empty(Q.qkv_prompt_attn_workspace_bytes(plan, cache, new), dtype=torch.uint8, device="cuda")
        sides.append((cache, torch.randn(new, nh * hd, device="cuda"), i32(0, new), i32(n), ws, torch.cuda.Stream(), pools, table))

    def call(s, o, stream=None):
        Q.qkv_prompt_attn_step(plan, s[0], s[1], s[2], s[3], hd ** -0.5, o, s[4], stream=stream)
    want = [torch.empty(new, nh * hd, device="cuda", dtype=dtype) for _ in sides]
    for s, o in zip(sides, want):
        call(s, o)
        torch.cuda.synchronize()
    got = [[torch.full_like(o, float("nan")) for _ in range(6)] for o in want]
    torch.cuda.synchronize()
    for k in range(6):
        for s, o in zip(sides, got):
            call(s, o[k], s[5])
    torch.cuda.synchronize()
    for o, w in zip(got, want):
        assert all(torch.equal(x, w) for x in o)
    assert Q.qkv_check_device_error()[0] == 0


# ---------------------------------------------------------------- as they are used

def test_graphs_streams_and_shapes_share_a_workspace(qkv):
    """Captured calls of several shapes, replayed in turn on one workspace, and lengths read at every replay."""
    import torch
    rng = np.random.default_rng(8)
    nh, nkv, hd, page = 28, 4, 128, 16
    plan = make_plan(nh, nkv, hd, "f16")
    c = paged_reference.Cache(rng, 2, nkv, hd, "f16", page, 40, lens=[600, 500])
    cache = Q.PagedKv(plan, *pools_of(c), dev(c.table))
    x = rng.standard_normal((70, nh * hd)).astype(np.float32)
    q = dev(x)
    first, lens = dev(np.int32([0, 40, 70])), dev(np.int32([600, 500]))
    o = torch.empty(70, nh * hd, device="cuda")
    p = torch.empty(2, nh * hd, device="cuda")
    share, prefix = dev(np.int32([0, 0])), dev(np.int32([320, 320]))
    n = max(Q.qkv_prompt_attn_workspace_bytes(plan, cache, 70), Q.qkv_prefix_attn_workspace_bytes(plan, cache))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    ws2 = torch.zeros(n, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        graph, both = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            Q.qkv_prompt_attn_step(plan, cache, q, first, lens, 0.09, o, ws)
        with torch.cuda.graph(both, stream=stream):
            Q.qkv_prefix_attn_step(plan, cache, q[:2], lens, share, prefix, 0.09, p, ws2)
        for lengths in ([600, 500], [41, 450], [600, 500]):
            lens.copy_(torch.tensor(lengths, dtype=torch.int32))
            o.fill_(7.0)
            graph.replay()
            both.replay()
            stream.synchronize()
            want, _, bo, _ = ref.rows_ref(c.k, c.v, x, ref.prompt_places(c, [0, 40, 70], lengths, 70, 0), 0.09, nh, nkv, hd, False)
            close(o.cpu().numpy(), want, bo, "replay")
            want, _, bo, _ = ref.rows_ref(c.k, c.v, x[:2], ref.prefix_places(c, lengths, [0, 0], [320, 320]), 0.09, nh, nkv, hd, False)
            close(p.cpu().numpy(), want, bo, "replay")


def test_serving_run(qkv):
    """A shared beginning and two questions stored with a scaled rotation, attended, then answered token by token: the same
    as with every sequence on its own, in one contiguous cache."""
    import torch
    torch.manual_seed(0)
    nh, nkv, hd, page = 8, 2, 64, 16
    nqt, R = nh * hd, (nh + 2 * nkv) * hd
    plan = make_plan(nh, nkv, hd, "f16")
    rope = Q.qkv_rope_create(hd, 1e4, rot_dim=32, layout=Q.QKV_ROPE_INTERLEAVED, scaling=Q.QKV_ROPE_SCALE_RAMP, factor=4.0,
                             orig_ctx=4096.0, low=1.0, high=32.0, magnitude=1.1)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    P0, n = 40, [9, 23]
    # pages: 0-2 the beginning's (the last one holds 8 slots of it), then each question's own from slot 40 on
    table = torch.tensor([[0, 1, 2, 3, 4, 5], [-1, -1, 6, 7, 8, 9]], dtype=torch.int32, device="cuda")
    pools = [torch.zeros(10, page, nkv * hd, dtype=torch.float16, device="cuda") for _ in range(2)]
    cache = Q.PagedKv(plan, *pools, table)
    alone = [[torch.zeros(1, 96, nkv * hd, dtype=torch.float16, device="cuda") for _ in range(2)] for _ in range(2)]
    each = [Q.PagedKv(plan, *p, torch.zeros(1, 1, dtype=torch.int32, device="cuda")) for p in alone]
    ws = torch.zeros(max(Q.qkv_prompt_attn_workspace_bytes(plan, cache, 80), Q.qkv_prefix_attn_workspace_bytes(plan, cache)),
                     dtype=torch.uint8, device="cuda")
    ws1 = torch.zeros(max(Q.qkv_prompt_attn_workspace_bytes(plan, each[0], 80), Q.qkv_attn_workspace_bytes(plan, each[0])),
                      dtype=torch.uint8, device="cuda")

    def store(where, y, pos, seqs):
        q = torch.empty(y.shape[0], nqt, device="cuda")
        Q.qkv_paged_store_rope_step(plan, where, rope, y, None, None, None, 0.0, i32(*pos), i32(*seqs), None, q)
        return q

    def same(a, b):
        assert (a - b).abs().max().item() < 2e-5  # both f32 sums of values of order 1

    begin = torch.randn(P0, R, device="cuda")
    asks = [torch.randn(k, R, device="cuda") for k in n]
    qb = store(cache, begin, range(P0), [0] * P0)
    out = torch.empty(P0, nqt, device="cuda")
    Q.qkv_prompt_attn_step(plan, cache, qb, i32(0, P0, P0), i32(P0, P0), hd ** -0.5, out, ws)
    want = torch.empty_like(out)
    for b in range(2):
        q1 = store(each[b], torch.cat([begin, asks[b]]), range(P0 + n[b]), [0] * (P0 + n[b]))
        full = torch.empty(P0 + n[b], nqt, device="cuda")
        Q.qkv_prompt_attn_step(plan, each[b], q1, i32(0, P0 + n[b]), i32(P0 + n[b]), hd ** -0.5, full, ws1)
        want = full[:P0]
        same(out, want)
    # the questions' tokens: sequence 1 reads the beginning through its own row, so that names the same pages here; its
    # part of page 2 is copied
    pools[0][6, :8], pools[1][6, :8] = pools[0][2, :8], pools[1][2, :8]
    table[1, :2] = table[0, :2]
    y = torch.cat(asks)
    qa = store(cache, y, [*range(P0, P0 + n[0]), *range(P0, P0 + n[1])], [0] * n[0] + [1] * n[1])
    out = torch.empty(sum(n), nqt, device="cuda")
    Q.qkv_prompt_attn_step(plan, cache, qa, i32(0, n[0], sum(n)), i32(P0 + n[0], P0 + n[1]), hd ** -0.5, out, ws)
    for b in range(2):
        q1 = store(each[b], torch.cat([begin, asks[b]]), range(P0 + n[b]), [0] * (P0 + n[b]))
        full = torch.empty(P0 + n[b], nqt, device="cuda")
        Q.qkv_prompt_attn_step(plan, each[b], q1, i32(0, P0 + n[b]), i32(P0 + n[b]), hd ** -0.5, full, ws1)
        same(out[:n[0]] if b == 0 else out[n[0]:], full[P0:])
    table[1, :2] = -1  # from here on the beginning is read through sequence 0's row only
    lens = [P0 + n[0], P0 + n[1]]
    for _ in range(5):
        y = torch.randn(2, R, device="cuda")
        qd = store(cache, y, lens, [0, 1])
        got = torch.empty(2, nqt, device="cuda")
        Q.qkv_prefix_attn_step(plan, cache, qd, i32(lens[0] + 1, lens[1] + 1), i32(0, 0), i32(32, 32), hd ** -0.5, got, ws)
        for b in range(2):
            q1 = store(each[b], y[b:b + 1], [lens[b]], [0])
            one = torch.empty(1, nqt, device="cuda")
            Q.qkv_attn_step(plan, each[b], q1, i32(lens[b] + 1), hd ** -0.5, one, ws1)
            same(got[b:b + 1], one)
        lens = [lens[0] + 1, lens[1] + 1]
    assert Q.qkv_check_device_error()[0] == 0
