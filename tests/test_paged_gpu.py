"""The paged-cache operators on the GPU against their 64-bit forms (paged_reference.py, which
derives the error bounds), at the sizes, masks and layouts where they can go wrong."""
import numpy as np
import pytest

import paged_reference as ref
import qkv_rope_kv_gb300 as Q

pytestmark = pytest.mark.gpu

KV = {"f16": Q.QKV_F16, "f32": Q.QKV_F32}
EPS = 1e-6


def short(v):
    return str(v).replace(" ", "")[:40]


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def make_plan(nh, nkv, hd, kv, theta=1e6):
    return Q.qkv_plan_create(64, nh, nkv, hd, theta, 64, kv_dtype=KV[kv])


def gpu_cache(plan, c, **track):
    k, v = dev(c.k), dev(c.v)
    return Q.PagedKv(plan, k, v, dev(c.table), **track), k, v


def close(got, want, bound, what):
    """|got - want| <= bound elementwise, infinities and NaN in the same places."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, what
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what + ": NaN elsewhere"
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), what
    off = np.abs(got[fine] - want[fine]) - np.broadcast_to(bound, want.shape)[fine]
    assert not off.size or off.max() <= 0, "%s: %.3g over the bound" % (what, off.max())


# ---------------------------------------------------------------- store

def run_store(nh, nkv, hd, kv, page, y, norm, nt, with_bias=True, y_off=0, pool_off=0, seed=0, positions=None):
    import torch
    rng = np.random.default_rng(seed)
    B, cap = 3, 5 * page
    c = ref.Cache(rng, B, nkv, hd, kv, page, 5, fill=7.0)
    R = (nh + 2 * nkv) * hd
    plan = make_plan(nh, nkv, hd, kv)
    Y = torch.from_numpy(rng.standard_normal((nt, R + y_off)).astype(np.float32)).cuda()[:, y_off:]
    Y = Y.to(torch.bfloat16) if y == "bf16" else Y
    bias = rng.standard_normal(R).astype(np.float32) if with_bias else None
    qw, kw = (rng.standard_normal((2, hd)).astype(np.float32) if norm else (None, None))
    pos = (rng.integers(0, 40000, nt) if positions is None else np.asarray(positions)).astype(np.int32)
    at = rng.choice(B * cap, nt, replace=False)
    seqs, slots = (at // cap).astype(np.int32), (at % cap).astype(np.int32)
    pad = rng.random(nt) < 0.2
    seqs[pad] = -1 - rng.integers(0, 5, pad.sum())
    weight = torch.full((B, nkv, cap), 3.0, device="cuda")
    spos = torch.full((B, nkv, cap), -9, dtype=torch.int32, device="cuda")
    k, v = (torch.zeros(c.k.size + pool_off, dtype=torch.float16 if kv == "f16" else torch.float32, device="cuda")[
        pool_off:].view(c.k.shape) for _ in range(2))
    k.copy_(dev(c.k))
    v.copy_(dev(c.v))
    cache = Q.PagedKv(plan, k, v, dev(c.table), slot_weight=weight, slot_pos=spos)
    q = torch.full((nt, nh * hd), -5.0, device="cuda")
    opt = lambda a: None if a is None else dev(a)  # noqa: E731
    Q.qkv_paged_store_step(plan, cache, Y, opt(bias), opt(qw), opt(kw), EPS, dev(pos), dev(seqs), dev(slots), q)
    torch.cuda.synchronize()
    assert Q.qkv_check_device_error()[0] == 0
    wq, wk, wv, bq, bk = ref.store_ref(Y.float().cpu().numpy(), bias, qw, kw, EPS, pos, nh, nkv, hd, plan.inv_freq())
    got = q.cpu().numpy()
    assert (got[pad] == -5.0).all()
    close(got[~pad], wq[~pad], bq[~pad], "q")
    K, V = c.k.astype(np.float64), c.v.astype(np.float64)
    bK, bV = np.zeros_like(K), np.zeros_like(V)
    ww, wp = np.full((B, nkv, cap), 3.0), np.full((B, nkv, cap), -9)
    for t in np.flatnonzero(~pad):
        r = c.row(seqs[t], slots[t])
        K[r], V[r] = wk[t], wv[t]
        bK[r] = bk[t] + (ref.f16_half_step(wk[t]) * (1 + 2.0 ** -10) if kv == "f16" else 0)
        bV[r] = np.abs(wv[t]) * ref.U + (ref.f16_half_step(wv[t]) * (1 + 2.0 ** -10) if kv == "f16" else 0)
        ww[seqs[t], :, slots[t]], wp[seqs[t], :, slots[t]] = 0, pos[t]
    close(k.cpu().numpy(), K, bK, "K pool")
    close(v.cpu().numpy(), V, bV, "V pool")
    assert np.array_equal(weight.cpu().numpy(), ww) and np.array_equal(spos.cpu().numpy(), wp)


@pytest.mark.parametrize("nh,nkv,hd,kv,page,y,norm,nt,kw", [
    (14, 2, 64, "f32", 16, "f32", False, 1, {}),
    (14, 2, 64, "f32", 16, "bf16", True, 50, {}),
    (28, 4, 128, "f16", 16, "f32", False, 7, {}),
    (40, 8, 128, "f16", 7, "bf16", True, 33, {}),
    (40, 8, 128, "f16", 64, "f32", True, 129, {}),
    (4, 1, 256, "f16", 5, "f32", True, 13, {}),
    (2, 2, 16, "f32", 9, "bf16", True, 20, {}),
    (3, 2, 6, "f16", 4, "f32", True, 17, {}),            # odd head count, a head that is no power of two
    (5, 5, 2, "f32", 3, "bf16", True, 11, {}),
    (6, 3, 96, "f16", 17, "f32", True, 40, {}),
    (8, 2, 80, "f32", 1, "bf16", False, 12, {}),
    (3, 1, 8, "f16", 16, "bf16", True, 30, {}),
    (3, 1, 24, "f32", 16, "f32", True, 30, {}),
    (14, 2, 64, "f16", 1000, "f32", True, 2501, {}),             # enough tokens to share CTAs
    (28, 4, 128, "f16", 1000, "bf16", False, 2500, {}),
    (5, 1, 80, "f32", 1000, "bf16", True, 2503, dict(with_bias=False)),
    (28, 4, 128, "f16", 16, "f32", True, 9, dict(y_off=1)),      # rows at odd addresses
    (28, 4, 128, "f16", 16, "bf16", True, 9, dict(y_off=4)),
    (28, 4, 128, "f16", 16, "f32", True, 9, dict(pool_off=1)),
    (28, 4, 128, "f16", 16, "f32", True, 9, dict(with_bias=False)),
    (28, 4, 128, "f16", 16, "f32", True, 3, dict(positions=[0, 2 ** 24 + 1, -3])),
], ids=short)
def test_store(qkv, nh, nkv, hd, kv, page, y, norm, nt, kw):
    run_store(nh, nkv, hd, kv, page, y, norm, nt, **kw)


def test_store_equals_the_decode_epilogue_bitwise(qkv):
    """Without norms a token's q and cache rows are the bits that qkv_epilogue gives."""
    import torch
    for nh, nkv, hd, kv in ((40, 8, 128, "f16"), (14, 2, 64, "f32"), (6, 3, 96, "f16")):
        rng = np.random.default_rng(3)
        nqt, nkt, n_ctx, nt = nh * hd, nkv * hd, 64, 5
        plan = Q.qkv_plan_create(64, nh, nkv, hd, 1e6, n_ctx, kv_dtype=KV[kv])
        dt = torch.float16 if kv == "f16" else torch.float32
        Y, bias = dev(rng.standard_normal((nt, nqt + 2 * nkt)).astype(np.float32)), dev(
            rng.standard_normal(nqt + 2 * nkt).astype(np.float32))
        pos = dev(rng.permutation(n_ctx)[:nt].astype(np.int32))
        k, v, ke, ve = (torch.zeros(1, n_ctx, nkt, dtype=dt, device="cuda") for _ in range(4))
        cache = Q.PagedKv(plan, k, v, torch.zeros(1, 1, dtype=torch.int32, device="cuda"))
        q = torch.empty(nt, nqt, device="cuda")
        Q.qkv_paged_store_step(plan, cache, Y, bias, None, None, 0.0, pos, torch.zeros(nt, dtype=torch.int32,
                                                                                    device="cuda"), None, q)
        b = (bias[:nqt], bias[nqt:nqt + nkt], bias[nqt + nkt:])
        for t in range(0, nt, max(1, nt // 7)):
            y = Y[t].clone()
            Q.qkv_epilogue(plan, y[:nqt], y[nqt:nqt + nkt], y[nqt + nkt:], *b, pos[t:t + 1], ke, ve)
            assert torch.equal(y[:nqt], q[t])
        assert torch.equal(k, ke) and torch.equal(v, ve)
        # in place: q over Y's own rows
        inplace = Y.clone()
        Q.qkv_paged_store_step(plan, cache, inplace, bias, None, None, 0.0, pos,
                               torch.zeros(nt, dtype=torch.int32, device="cuda"), None, inplace[:, :nqt])
        assert torch.equal(inplace[:, :nqt], q) and torch.equal(inplace[:, nqt:], Y[:, nqt:])


def test_store_flags_what_is_out_of_range(qkv):
    import torch
    rng = np.random.default_rng(5)
    nh, nkv, hd, page = 4, 2, 64, 4
    c = ref.Cache(rng, 2, nkv, hd, "f16", page, 2, fill=1.0)
    plan = make_plan(nh, nkv, hd, "f16")
    Y = dev(rng.standard_normal((1, (nh + 2 * nkv) * hd)).astype(np.float32))
    for seq, slot, entry, flag, value in ((0, 8, None, 1, 8), (1, -1, None, 1, -1), (2, 0, None, 4, 2),
                                          (0, 5, c.n_pages, 4, c.n_pages), (0, 5, -7, 4, -7)):
        table = c.table.copy()
        if entry is not None:
            table[0, 1] = entry
        k, v = dev(c.k), dev(c.v)
        cache = Q.PagedKv(plan, k, v, dev(table))
        q = torch.zeros(1, nh * hd, device="cuda")
        i32 = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")  # noqa: E731
        Q.qkv_paged_store_step(plan, cache, Y, None, None, None, 0.0, i32(3), i32(seq), i32(slot), q)
        torch.cuda.synchronize()
        assert Q.qkv_check_device_error() == (flag, value)
        assert np.array_equal(k.cpu().numpy(), c.k) and np.array_equal(v.cpu().numpy(), c.v)
        assert q.abs().sum().item() > 0
    assert Q.qkv_check_device_error()[0] == 0


# ---------------------------------------------------------------- attention

def run_attn(nh, nkv, hd, kv, page, lens, window=0, out="f32", weights=False, seed=0, q_scale=1.5, change=None,
             stride=0, pool_off=0, page_gap=0, max_pages=None, plan=None, workspace=None):
    import torch
    rng = np.random.default_rng(seed)
    B = len(lens)
    max_pages = max_pages or max(1, -(-max(lens) // page) + 1)
    c = ref.Cache(rng, B, nkv, hd, kv, page, max_pages, lens=lens, fill=np.nan)
    x = (q_scale * rng.standard_normal((B, nh * hd))).astype(np.float32)
    if change:
        change(c, x)
    plan = plan or make_plan(nh, nkv, hd, kv)
    dt = torch.float16 if kv == "f16" else torch.float32
    step = page * nkv * hd + page_gap
    pools = []
    for a in (c.k, c.v):
        flat = torch.full((c.n_pages * step + pool_off,), float("nan"), dtype=dt, device="cuda")
        view = flat[pool_off:].as_strided(a.shape, (step, nkv * hd, 1))
        view.copy_(dev(a))
        pools.append(view)
    w0 = rng.random((B, nkv, c.cap)).astype(np.float32)
    weight = dev(w0) if weights else None
    cache = Q.PagedKv(plan, *pools, dev(c.table), slot_weight=weight)
    q = torch.zeros(B, nh * hd + stride, device="cuda")[:, :nh * hd]
    q.copy_(dev(x))
    o = torch.full((B, nh * hd + stride), 77.0, dtype=torch.bfloat16 if out == "bf16" else torch.float32,
                   device="cuda")
    lse = torch.empty(B, nh, device="cuda")
    ws = workspace if workspace is not None else torch.zeros(Q.qkv_attn_workspace_bytes(plan, cache),
                                                             dtype=torch.uint8, device="cuda")
    scale = hd ** -0.5
    first = None
    for again in range(2):
        if weights:
            weight.copy_(dev(w0))
        Q.qkv_attn_step(plan, cache, q, dev(c.lens), scale, o[:, :nh * hd], ws, window=window, lse=lse,
                        add_weight=weights)
        torch.cuda.synchronize()
        assert Q.qkv_check_device_error()[0] == 0
        got = [t.clone() for t in (o, lse, weight) if t is not None]
        if first is not None:  # the same bits again, with the workspace as the first call left it
            for a, b in zip(first, got):
                assert torch.equal(torch.nan_to_num(a, 1e9), torch.nan_to_num(b, 1e9))
        first = got
    w_out, w_lse, w_w, b_out, b_lse, b_w = ref.attn_ref(c, x, lens, scale, window, nh)
    g = o.float().cpu().numpy()
    assert (g[:, nh * hd:] == 77.0).all()
    close(g[:, :nh * hd], w_out, b_out + (np.abs(w_out) * 2.0 ** -8 if out == "bf16" else 0), "out")
    close(lse.cpu().numpy(), w_lse, b_lse, "lse")
    if weights:
        close(weight.cpu().numpy(), w0 + w_w, b_w + np.abs(w0 + w_w) * 2 * ref.U, "weight")
    return c, got


@pytest.mark.parametrize("nh,nkv,hd,kv,page,lens,kw", [
    (14, 2, 64, "f32", 16, [1], {}),
    (14, 2, 64, "f32", 16, [509], {}),
    (14, 2, 64, "f16", 16, [0, 1, 15, 16, 17, 0, 33], dict(weights=True)),
    (28, 4, 128, "f16", 16, [1641], {}),
    (28, 4, 128, "f16", 32, [700, 1, 64, 2000], dict(weights=True, out="bf16")),
    (40, 8, 128, "f16", 16, [300, 77, 0, 129, 128, 127, 5, 1000], dict(out="bf16")),
    (40, 8, 128, "f16", 7, [350, 21], dict(weights=True)),
    (40, 8, 128, "f32", 13, [260, 90], dict(weights=True)),
    (40, 8, 128, "f16", 1, [100, 3], {}),
    (40, 8, 128, "f16", 1000, [999, 12], {}),
    (8, 8, 128, "f16", 16, [500, 40], dict(weights=True)),          # one q head a kv head
    (32, 2, 128, "f16", 16, [400, 9], dict(weights=True)),          # sixteen
    (24, 2, 64, "f32", 16, [200, 9], dict(weights=True)),           # twelve
    (8, 1, 256, "f16", 16, [300, 31], dict(weights=True)),
    (3, 1, 256, "f32", 8, [120, 31], dict(weights=True)),
    (10, 2, 80, "f16", 16, [150, 31], dict(weights=True)),
    (10, 2, 96, "f32", 16, [150, 31], dict(weights=True)),
    (6, 3, 8, "f16", 4, [50, 3], {}),
    (6, 3, 24, "f32", 4, [50, 3], {}),
    (2, 1, 4, "f32", 4, [50, 3], dict(weights=True)),
    (6, 3, 6, "f16", 4, [50, 3], dict(weights=True)),               # rows of no whole 16 bytes
    (5, 5, 2, "f32", 3, [130, 4], dict(weights=True, out="bf16")),
    (28, 4, 128, "f16", 16, [500, 70, 5], dict(window=64, weights=True)),
    (28, 4, 128, "f16", 16, [500, 70, 5], dict(window=1)),
    (14, 2, 64, "f32", 16, [500, 70, 0], dict(window=77, weights=True)),
    (28, 4, 128, "f16", 16, [90, 200], dict(stride=24, page_gap=8)),
    (28, 4, 128, "f16", 16, [90, 200], dict(stride=1, page_gap=3)),  # pages at odd addresses
    (28, 4, 128, "f16", 16, [90, 200], dict(pool_off=1)),
    (14, 2, 64, "f32", 16, [90, 200], dict(pool_off=4)),
    (28, 4, 128, "f16", 16, [90, 200], dict(q_scale=40.0)),          # one slot takes all the weight
    (28, 4, 128, "f16", 16, [90, 200], dict(q_scale=1e-6, weights=True)),
    (14, 2, 64, "f32", 16, [90, 200], dict(q_scale=40.0)),
    (28, 4, 128, "f16", 16, [0, 0], {}),
    (4, 2, 64, "f16", 16, [17] * 300, dict(weights=True)),           # more sequences than blocks
    (4, 1, 64, "f16", 16, [40 * (i % 7) for i in range(200)], dict(max_pages=20)),
    (40, 8, 128, "f16", 64, [20011], dict(weights=True)),
    (5, 1, 128, "f16", 64, [30011], dict(weights=True)),             # one item over the whole GPU
    (3, 1, 64, "f32", 64, [9000, 50], {}),
    (8, 1, 256, "f16", 64, [9000], {}),
    (2, 2, 64, "f16", 16, [12000] + [33] * 60, dict(weights=True)),  # one long among many short
    (2, 1, 64, "f16", 16, [(7 * i) % 40 if i % 3 else 0 for i in range(1500)], dict(max_pages=3, weights=True)),
    (2, 2, 64, "f32", 16, [0] * 700 + [300] + [0] * 40, {}),
    (28, 4, 128, "f16", 16, [40, 0, 7, 33] * 40, dict(weights=True)),  # items dealt whole, several a CTA
    (28, 4, 128, "f16", 16, [100, 300, 0, 5, 333] * 5, dict(weights=True)),  # clusters of two, and of four
    (14, 2, 64, "f32", 16, [400, 33, 500] * 15, dict(weights=True, window=300)),
    (8, 1, 256, "f16", 16, [400, 33, 500] * 15, {}),
    (10, 2, 80, "f32", 8, [1000, 90, 0, 64] * 5, dict(weights=True, out="bf16")),
    (20, 4, 128, "f32", 16, [400, 33, 250] * 5, {}),
    (12, 1, 64, "f16", 16, [900, 33, 250] * 10, {}),
    (14, 2, 64, "f32", 8, [(37 * i) % 90 for i in range(400)], dict(window=50)),
    (5, 1, 256, "f16", 16, [16, 100, 1] * 150, {}),
], ids=short)
def test_attn(qkv, nh, nkv, hd, kv, page, lens, kw):
    run_attn(nh, nkv, hd, kv, page, lens, **kw)


@pytest.mark.parametrize("nh,nkv,hd,kv,page,lens,kw", [
    (96, 8, 128, "f16", 16, [700, 1, 64, 0, 300, 5], dict(weights=True)),
    (96, 8, 128, "f32", 13, [260, 90, 5, 700], dict(weights=True)),
    (24, 2, 64, "f16", 16, [200, 0, 33, 1] * 9, dict(out="bf16")),
    (24, 2, 64, "f32", 16, [100, 31, 0] * 8, dict(weights=True, window=40)),
    (20, 1, 256, "f16", 16, [100, 31] * 16, dict(weights=True)),     # three blocks of q heads
    (12, 1, 256, "f32", 16, [100, 31] * 16, {}),
    (22, 1, 80, "f16", 16, [100, 31] * 16, dict(weights=True)),
    (17, 1, 96, "f32", 7, [100, 31] * 16, {}),
    (68, 2, 72, "f32", 16, [90, 300, 2] * 3, dict(stride=4, page_gap=4)),
    (136, 1, 64, "f16", 16, [90, 31, 0, 200] * 4, dict(weights=True)),  # seventeen
    (136, 1, 64, "f16", 64, [5000], dict(weights=True)),
    (40, 2, 128, "f16", 64, [6000, 5000] * 6, {}),
    (24, 2, 128, "f16", 64, [20000] + [1] * 30, dict(weights=True)),
    (12, 1, 128, "f16", 64, [20011, 40], dict(weights=True)),
    (33, 1, 128, "f16", 64, [9000], {}),
    (12, 1, 64, "f32", 64, [9000, 50], dict(weights=True)),
    (16, 2, 6, "f16", 4, [50, 3], {}),
], ids=short)
def test_attn_with_blocks_of_q_heads(qkv, nh, nkv, hd, kv, page, lens, kw):
    """More than eight q heads to a kv head."""
    run_attn(nh, nkv, hd, kv, page, lens, **kw)


@pytest.mark.parametrize("kv", ["f16", "f32"])
def test_attn_with_infinite_values(qkv, kv):
    """A slot whose score is -inf has weight 0; an infinite V element reaches only its column; a NaN
    stays in its own column (V) or its own heads (K)."""
    def score(c, x):
        x[0, 0:128] = np.abs(x[0, 0:128])       # q heads 0 and 1 read kv head 0 (hd 64)
        c.k[c.row(0, 5)][3] = -np.inf

    def value(c, x):
        c.v[c.row(0, 7)][2], c.v[c.row(1, 30)][70] = np.inf, -np.inf
        c.v[c.row(0, 9)][4] = np.nan

    def key(c, x):
        c.k[c.row(1, 11)][66] = np.nan

    def all_lost(c, x):
        x[0, 0:128] = np.abs(x[0, 0:128])
        for s in range(40):
            c.k[c.row(0, s)][3] = -np.inf

    def large(c, x):
        x *= 1000.0
        c.k[...] = np.clip(np.nan_to_num(c.k, nan=0.0) * 100, -500, 500)

    for change in (score, value, key, all_lost, large):
        run_attn(4, 2, 64, kv, 16, [40, 90], change=change)


def test_attn_large_magnitudes(qkv):
    """q beyond the range of f16, and cache values at its end."""
    def far(c, x):
        x *= 3e5
        c.k[...] = np.nan_to_num(c.k, nan=0.0) * 1e-6
        c.v[...] = np.clip(np.nan_to_num(c.v, nan=0.0), -4, 4) * 15000

    def tiny(c, x):
        x *= 1e-30
    for kv in ("f16", "f32"):
        run_attn(4, 2, 64, kv, 16, [40, 300], change=far)
        run_attn(4, 2, 64, kv, 16, [40, 300], change=tiny, weights=True)


def test_attn_beyond_32_bit_offsets(qkv):
    """Pages more than 2^31 elements into the pools."""
    import torch
    nh, nkv, hd, page, n = 8, 2, 64, 16, 40
    rng = np.random.default_rng(8)
    plan = make_plan(nh, nkv, hd, "f16")
    step = (1 << 30) + 128
    k, v = (torch.empty(3 * step, dtype=torch.float16, device="cuda").as_strided((3, page, nkv * hd), (step, nkv * hd, 1))
            for _ in range(2))
    c = ref.Cache(rng, 1, nkv, hd, "f16", page, 3, lens=[n], spare=0)
    k.copy_(dev(c.k))
    v.copy_(dev(c.v))
    cache = Q.PagedKv(plan, k, v, dev(c.table))
    x = rng.standard_normal((1, nh * hd)).astype(np.float32)
    out = torch.empty(1, nh * hd, device="cuda")
    ws = torch.zeros(Q.qkv_attn_workspace_bytes(plan, cache), dtype=torch.uint8, device="cuda")
    Q.qkv_attn_step(plan, cache, dev(x), dev(c.lens), 0.125, out, ws)
    want = ref.attn_ref(c, x, c.lens, 0.125, 0, nh)
    close(out.cpu().numpy(), want[0], want[3], "out")
    # and the store: the last page's row gets the token
    Y = dev(rng.standard_normal((1, (nh + 2 * nkv) * hd)).astype(np.float32))
    slot = 47 if c.table[0, 2] == 2 else int(np.flatnonzero(c.table[0] == 2)[0]) * page + 15
    i32 = lambda a: torch.tensor([a], dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.empty(1, nh * hd, device="cuda")
    Q.qkv_paged_store_step(plan, cache, Y, None, None, None, 0.0, i32(0), i32(0), i32(slot), q)
    assert torch.equal(v[2, 15], Y[0, -nkv * hd:].half())
    assert Q.qkv_check_device_error()[0] == 0


def test_attn_flags_bad_lengths_and_pages(qkv):
    """A length out of range counts as 0, a page that is not there holds no slots; the other
    sequences' results stand."""
    import torch
    rng = np.random.default_rng(9)
    for nh, nkv, hd, kv in ((4, 2, 64, "f16"), (4, 2, 64, "f32"), (4, 2, 6, "f16")):
        c = ref.Cache(rng, 3, nkv, hd, kv, 16, 4, lens=[30, 50, 64])
        plan = make_plan(nh, nkv, hd, kv)
        x = rng.standard_normal((3, nh * hd)).astype(np.float32)
        for lens, entry, value in (([65, 50, 64], None, 65), ([-1, 50, 64], None, -1), ([30, 50, 64], 999, 999)):
            table = c.table.copy()
            if entry is not None:
                table[0, 1] = entry
            cache = Q.PagedKv(plan, dev(c.k), dev(c.v), dev(table))
            out = torch.empty(3, nh * hd, device="cuda")
            ws = torch.zeros(Q.qkv_attn_workspace_bytes(plan, cache), dtype=torch.uint8, device="cuda")
            Q.qkv_attn_step(plan, cache, dev(x), dev(np.int32(lens)), 0.1, out, ws)
            torch.cuda.synchronize()
            assert Q.qkv_check_device_error() == (4, value)
            left = [16 if entry is not None else 0, 50, 64]  # the first page of sequence 0 is there
            want = ref.attn_ref(c, x, left, 0.1, 0, nh)
            close(out.cpu().numpy(), want[0], want[3], "out")
    assert Q.qkv_check_device_error()[0] == 0


def test_attn_workspace_serves_other_shapes(qkv):
    """One workspace, zeroed once, for calls of different shapes one after the other."""
    import torch
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    for nh, nkv, hd, kv, lens in ((40, 8, 128, "f16", [3000]), (14, 2, 64, "f32", [700, 20]),
                                  (8, 1, 256, "f16", [900]), (40, 8, 128, "f16", [500, 900, 0, 64])):
        run_attn(nh, nkv, hd, kv, 16, lens, weights=True, workspace=ws)


# ---------------------------------------------------------------- eviction

def run_evict(nkv, hd, kv, page, lens, budget, recent, weights, seed=0, pool_off=0, inplace=False, shuffle=True,
              max_pages=None):
    import torch
    rng = np.random.default_rng(seed)
    B = len(lens)
    c = ref.Cache(rng, B, nkv, hd, kv, page, max_pages or max(1, -(-max(lens) // page)), lens=lens, fill=3.0)
    w = weights(rng, (B, nkv, c.cap)).astype(np.float32)
    pos = np.tile(np.arange(c.cap, dtype=np.int32), (B, nkv, 1))
    if shuffle:
        for b in range(B):
            for h in range(nkv):
                pos[b, h, :lens[b]] = rng.permutation(lens[b])
    plan = make_plan(2 * nkv, nkv, hd, kv)
    k, v = (torch.zeros(c.k.size + pool_off, dtype=torch.float16 if kv == "f16" else torch.float32, device="cuda")[
        pool_off:].view(c.k.shape) for _ in range(2))
    k.copy_(dev(c.k))
    v.copy_(dev(c.v))
    dw, dp, dl = dev(w), dev(pos), dev(c.lens)
    cache = Q.PagedKv(plan, k, v, dev(c.table), slot_weight=dw, slot_pos=dp)
    wo, po = (dw, dp) if inplace else (torch.full_like(dw, -8.0), torch.full_like(dp, -8))
    lo = torch.full_like(dl, -1)
    n = Q.qkv_evict_workspace_bytes(plan, cache)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda") if n else None
    Q.qkv_evict_step(plan, cache, dl, dl, budget, recent, lo, wo, po, ws)
    torch.cuda.synchronize()
    assert Q.qkv_check_device_error()[0] == 0
    rk, rv, rl, rw, rp = ref.evict_ref(c, c.lens, c.lens, w, pos, budget, recent)
    assert np.array_equal(lo.cpu().numpy(), rl)
    bits = np.uint16 if kv == "f16" else np.uint32
    assert np.array_equal(k.cpu().numpy().view(bits), rk.view(bits))
    assert np.array_equal(v.cpu().numpy().view(bits), rv.view(bits))
    gw, gp = wo.cpu().numpy(), po.cpu().numpy()
    for b in range(B):
        m = rl[b]
        assert np.array_equal(gw[b, :, :m].view(np.uint32), rw[b, :, :m].view(np.uint32))
        assert np.array_equal(gp[b, :, :m], rp[b, :, :m])
        rest = (w[b, :, m:], pos[b, :, m:]) if inplace else (np.float32(-8.0), -8)
        assert np.array_equal(gw[b, :, m:].view(np.uint32), np.broadcast_to(rest[0], gw[b, :, m:].shape).view(np.uint32)) \
            if inplace else (gw[b, :, m:] == -8).all()
        assert (gp[b, :, m:] == rest[1]).all()


def heavy(rng, shape):
    return np.exp(2 * rng.standard_normal(shape))


def tied(rng, shape):
    return rng.integers(0, 3, shape) / 4


def flat(rng, shape):
    return np.zeros(shape)


def wild(rng, shape):
    return rng.choice(np.array([np.nan, -np.nan, np.inf, -np.inf, 0.0, -0.0, -1.0, 1.0, 3e-45, -3e-45, 3e38]), shape)


@pytest.mark.parametrize("nkv,hd,kv,page,lens,budget,recent,weights,kw", [
    (2, 64, "f16", 16, [100, 40, 0, 1, 64, 65], 64, 8, heavy, {}),
    (2, 64, "f16", 16, [100, 40, 0, 1, 64, 65], 64, 8, heavy, dict(inplace=True)),
    (8, 128, "f16", 16, [2112, 2048], 2048, 256, heavy, {}),
    (4, 128, "f16", 64, [5001], 1000, 100, heavy, dict(inplace=True)),
    (4, 128, "f16", 64, [5001], 4000, 0, heavy, {}),
    (2, 64, "f32", 7, [333, 70], 50, 50, tied, {}),
    (2, 64, "f32", 7, [333, 70], 50, 0, tied, dict(inplace=True)),
    (3, 6, "f16", 5, [200, 33], 32, 3, tied, {}),
    (1, 2, "f32", 1, [90, 2], 1, 0, flat, {}),
    (1, 2, "f16", 3, [90, 2], 1, 1, heavy, {}),
    (2, 80, "f16", 16, [300, 299], 200, 17, wild, {}),
    (2, 64, "f16", 16, [4097, 1023, 1024, 1025], 33, 0, wild, dict(inplace=True)),
    (2, 64, "f16", 16, [1000], 500, 10, flat, dict(shuffle=False)),
    (2, 64, "f16", 16, [1000], 500, 10, heavy, dict(pool_off=1)),
    (2, 64, "f32", 16, [7], 100, 10, heavy, {}),
    (1, 64, "f16", 256, [40001], 17000, 300, heavy, dict(inplace=True)),
    (1, 8, "f16", 256, [70000], 60000, 300, tied, {}),
    (2, 64, "f16", 16, [30] * 150, 20, 5, tied, {}),
    (2, 64, "f16", 16, [5000, 9], 4500, 5, heavy, dict(max_pages=400, inplace=True)),
    (8, 64, "f16", 64, [20000], 700, 5, wild, {}),
    (160, 2, "f16", 64, [2000, 130], 129, 20, tied, dict(max_pages=520)),        # many heads, large capacity:
    (160, 2, "f32", 64, [130, 2000], 1500, 0, heavy, dict(max_pages=520, inplace=True)),  # keys made again
    (1, 2, "f16", 256, [3001], 2000, 7, tied, dict(max_pages=2100)),
    (1, 2, "f32", 256, [3001], 11, 7, heavy, dict(max_pages=2100, inplace=True)),
    (8, 128, "f16", 16, [600, 550, 551, 33] * 8, 550, 50, tied, dict(inplace=True)),     # more items than SMs
    (8, 64, "f32", 32, [2112, 1999, 2048] * 8, 1000, 100, heavy, {}),
    (8, 16, "f16", 16, [1025, 1024, 1023, 513, 2] * 5, 512, 0, wild, {}),
], ids=short)
def test_evict(qkv, nkv, hd, kv, page, lens, budget, recent, weights, kw):
    run_evict(nkv, hd, kv, page, lens, budget, recent, weights, **kw)


def test_evict_flags_bad_lengths_and_pages(qkv):
    import torch
    rng = np.random.default_rng(11)
    c = ref.Cache(rng, 2, 2, 64, "f16", 16, 4, lens=[64, 64])
    plan = make_plan(4, 2, 64, "f16")
    w = dev(np.tile(np.arange(64, dtype=np.float32), (2, 2, 1)))
    p = dev(np.tile(np.arange(64, dtype=np.int32), (2, 2, 1)))
    for lens, entry, value in (([65, 40], None, 65), ([-2, 40], None, -2), ([64, 30], 77, 77)):
        table = c.table.copy()
        if entry is not None:
            table[0, 3] = entry
        k, v = dev(c.k), dev(c.v)
        cache = Q.PagedKv(plan, k, v, dev(table), slot_weight=w, slot_pos=p)
        lo, wo, po = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros_like(w), torch.zeros_like(p)
        ws = torch.zeros(Q.qkv_evict_workspace_bytes(plan, cache), dtype=torch.uint8, device="cuda")
        dl = dev(np.int32(lens))
        Q.qkv_evict_step(plan, cache, dl, dl, 16, 0, lo, wo, po, ws)
        torch.cuda.synchronize()
        assert Q.qkv_check_device_error() == (4, value)
        assert lo.tolist() == [lens[0] if entry is None else 16, 16]
        after = k.cpu().numpy()
        page = c.table[1, 0]  # sequence 1 was cut to its last 16 slots (its largest weights)
        want = np.concatenate([c.k[c.row(1, s)][None] for s in range(lens[1] - 16, lens[1])])
        order = po[1, 0, :16].cpu().numpy()
        assert sorted(order) == list(range(lens[1] - 16, lens[1]))
        assert np.array_equal(after[page][:, :64], want[order - (lens[1] - 16)][:, :64])
        rest = [np.ascontiguousarray(np.delete(a, page, 0)).view(np.uint16) for a in (after, c.k)]
        assert np.array_equal(rest[0], rest[1])
    assert Q.qkv_check_device_error()[0] == 0


# ---------------------------------------------------------------- together

def reference_step(state, c_rows, x, scale, nh, nkv, hd):
    out = np.zeros(nh * hd)
    for h in range(nh):
        K, V = c_rows[h // (nh // nkv)]
        s = scale * (K @ x[h * hd:(h + 1) * hd])
        p = np.exp(s - s.max())
        out[h * hd:(h + 1) * hd] = (p / p.sum()) @ V
    return out


@pytest.mark.parametrize("kv,hd,captured", [("f16", 128, False), ("f32", 64, False), ("f16", 128, True)])
def test_serving_steps_together(qkv, kv, hd, captured):
    """Prompts stored, then decode steps of a batch (store, attention with running weights) with an
    eviction every few steps, on a stream of its own, eager or as captured graphs that share one
    workspace; every step's output against attention in 64 bits over the keys and values that the
    positions in slot_pos name, and every eviction's choice against the definition."""
    import torch
    nh, nkv, page, B, budget, recent, scale = 8, 2, 16, 3, 40, 6, hd ** -0.5
    rng = np.random.default_rng(12)
    R, nqt, nkt = (nh + 2 * nkv) * hd, nh * hd, nkv * hd
    plan = make_plan(nh, nkv, hd, kv)
    prompt = [30, 1, 44]
    steps = 12
    cap = 64
    dt = torch.float16 if kv == "f16" else torch.float32
    n_pages = B * cap // page
    table = rng.permutation(n_pages).astype(np.int32).reshape(B, -1)
    k, v = (torch.full((n_pages, page, nkt), float("nan"), dtype=dt, device="cuda") for _ in range(2))
    weight = torch.full((B, nkv, cap), float("nan"), device="cuda")
    spos = torch.full((B, nkv, cap), -1, dtype=torch.int32, device="cuda")
    cache = Q.PagedKv(plan, k, v, dev(table), slot_weight=weight, slot_pos=spos)
    bias, qw, kw = (dev(rng.standard_normal(n).astype(np.float32)) for n in (R, hd, hd))
    lens, nxt = torch.tensor(prompt, dtype=torch.int32, device="cuda"), torch.tensor(prompt, dtype=torch.int32,
                                                                                     device="cuda")
    ws = torch.zeros(Q.qkv_attn_workspace_bytes(plan, cache), dtype=torch.uint8, device="cuda")
    wse = torch.zeros(Q.qkv_evict_workspace_bytes(plan, cache), dtype=torch.uint8, device="cuda")
    Y = torch.empty(B, R, device="cuda")
    q, out = torch.empty(B, nqt, device="cuda"), torch.empty(B, nqt, device="cuda")
    lens2 = torch.empty_like(lens)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    # every position's key and value in 64 bits, from its own projection
    keys, vals = [{} for _ in range(B)], [{} for _ in range(B)]

    def remember(b, pos, y):
        rq, rk, rv, *_ = ref.store_ref(y[None], bias.cpu().numpy(), qw.cpu().numpy(), kw.cpu().numpy(), EPS,
                                       np.int32([pos]), nh, nkv, hd, plan.inv_freq())
        keys[b][pos], vals[b][pos] = rk[0].reshape(nkv, hd), rv[0].reshape(nkv, hd)
        return rq[0]

    with torch.cuda.stream(stream):
        toks = sum(prompt)
        Yp = rng.standard_normal((toks, R)).astype(np.float32)
        seq = np.repeat(np.arange(B), prompt).astype(np.int32)
        pp = np.concatenate([np.arange(n) for n in prompt]).astype(np.int32)
        Q.qkv_paged_store_step(plan, cache, dev(Yp), bias, qw, kw, EPS, dev(pp), dev(seq), None,
                               torch.empty(toks, nqt, device="cuda"))
        for b, pos, y in zip(seq, pp, Yp):
            remember(b, int(pos), y)

        def decode():
            Q.qkv_paged_store_step(plan, cache, Y, bias, qw, kw, EPS, nxt, None, lens, q)
            lens.add_(1)
            nxt.add_(1)
            Q.qkv_attn_step(plan, cache, q, lens, scale, out, ws, add_weight=True)

        def evict():
            Q.qkv_evict_step(plan, cache, lens, nxt, budget, recent, lens2, weight, spos, wse)
            lens.copy_(lens2)

        if captured:
            stream.synchronize()
            graphs = []
            for fn in (decode, decode, evict):  # two graphs of the same step share the workspace
                g = torch.cuda.CUDAGraph()
                saved = [t.clone() for t in (k, v, weight, spos, lens, nxt)]
                with torch.cuda.graph(g, stream=stream):
                    fn()
                for t, s in zip((k, v, weight, spos, lens, nxt), saved):
                    t.copy_(s)
                graphs.append(g)
        for step in range(steps):
            y = rng.standard_normal((B, R)).astype(np.float32)
            Y.copy_(dev(y))
            now = nxt.tolist()
            x = np.stack([remember(b, now[b], y[b]) for b in range(B)])
            before = weight.cpu().numpy().astype(np.float64)
            n0 = lens.tolist()
            (graphs[step % 2].replay if captured else decode)()
            stream.synchronize()
            n, sp, w = lens.tolist(), spos.cpu().numpy(), weight.cpu().numpy()
            for b in range(B):
                assert n[b] == n0[b] + 1 and all(len(set(sp[b, h, :n[b]])) == n[b] for h in range(nkv))
                rows = [(np.stack([keys[b][int(t)][h] for t in sp[b, h, :n[b]]]),
                         np.stack([vals[b][int(t)][h] for t in sp[b, h, :n[b]]])) for h in range(nkv)]
                want = reference_step(None, rows, x[b], scale, nh, nkv, hd)
                # cached rows carry f16's half step: scores move by 2^-11 sum |q k| at most, values by 2^-11
                size = scale * max(np.abs(x[b]).max() * np.abs(r[0]).sum(1).max() for r in rows)
                tol = (2 * size * 2.0 ** -11 + 2.0 ** -11 if kv == "f16" else 2.0 ** -15) * max(
                    np.abs(r[1]).max() for r in rows)
                assert np.abs(out[b].cpu().numpy() - want).max() <= tol
                added = w[b, :, :n[b]] - np.where(np.arange(n[b]) < n0[b], before[b, :, :n[b]], 0.0) \
                    if step else w[b, :, :n[b]]
                assert np.allclose(added.sum(1), nh // nkv, atol=2.0 ** -14)
            if step % 4 == 3:
                host = ref.Cache(rng, B, nkv, hd, kv, page, cap // page, lens=[0] * B)
                host.k, host.v, host.table = k.cpu().numpy(), v.cpu().numpy(), table
                rk, rv, rl, rw, rp = ref.evict_ref(host, n, nxt.tolist(), w, sp, budget, recent)
                (graphs[2].replay if captured else evict)()
                stream.synchronize()
                assert lens.tolist() == list(rl)
                bits = np.uint16 if kv == "f16" else np.uint32
                assert np.array_equal(k.cpu().numpy().view(bits), rk.view(bits))
                assert np.array_equal(v.cpu().numpy().view(bits), rv.view(bits))
                for b in range(B):
                    assert np.array_equal(weight.cpu().numpy()[b, :, :rl[b]], rw[b, :, :rl[b]])
                    assert np.array_equal(spos.cpu().numpy()[b, :, :rl[b]], rp[b, :, :rl[b]])
        assert Q.qkv_check_device_error(stream)[0] == 0


def test_two_streams_at_once(qkv):
    """Calls on two streams, each with its own workspace, over one shared cache: the bits of calls one
    after the other."""
    import torch
    rng = np.random.default_rng(14)
    nh, nkv, hd = 28, 4, 128
    c = ref.Cache(rng, 4, nkv, hd, "f16", 16, 130, lens=[2000, 5, 900, 64])
    plan = make_plan(nh, nkv, hd, "f16")
    cache, _, _ = gpu_cache(plan, c)
    lens = dev(c.lens)
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [torch.zeros(Q.qkv_attn_workspace_bytes(plan, cache), dtype=torch.uint8, device="cuda") for _ in range(2)]
    qs = [dev(rng.standard_normal((4, nh * hd)).astype(np.float32)) for _ in range(2)]
    outs = [[torch.empty(4, nh * hd, device="cuda") for _ in range(20)] for _ in range(3)]
    torch.cuda.synchronize()
    for i in range(20):
        for k in range(2):
            Q.qkv_attn_step(plan, cache, qs[k], lens, 0.09, outs[k][i], ws[k], stream=streams[k])
    torch.cuda.synchronize()
    for k in range(2):
        Q.qkv_attn_step(plan, cache, qs[k], lens, 0.09, outs[2][k], ws[k])
        torch.cuda.synchronize()
        assert all(torch.equal(o, outs[2][k]) for o in outs[k])
    assert not torch.equal(outs[2][0], outs[2][1])


FIRST_CALLS = """
import torch, qkv_rope_kv_gb300 as Q
torch.manual_seed(0)
nh, nkv, hd, page = 8, 2, 64, 16
plan = Q.qkv_plan_create(64, nh, nkv, hd, 1e6, 64)
k, v = torch.randn(8, page, nkv * hd, device="cuda").half(), torch.randn(8, page, nkv * hd, device="cuda").half()
table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
w, p = torch.rand(2, nkv, 64, device="cuda"), torch.arange(64, dtype=torch.int32, device="cuda").expand(2, nkv, 64).contiguous()
cache = Q.PagedKv(plan, k, v, table, slot_weight=w, slot_pos=p)
ws = torch.zeros(Q.qkv_attn_workspace_bytes(plan, cache), dtype=torch.uint8, device="cuda")
we = torch.zeros(Q.qkv_evict_workspace_bytes(plan, cache), dtype=torch.uint8, device="cuda")
Y = torch.randn(2, (nh + 2 * nkv) * hd, device="cuda")
q, out = torch.zeros(2, nh * hd, device="cuda"), torch.zeros(2, nh * hd, device="cuda")
lens, n2 = torch.tensor([50, 63], dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
wo, po = w.clone(), p.clone()
state = [k, v, w, p, q, out, n2, wo, po]
saved = [t.clone() for t in state]
def step():
    Q.qkv_paged_store_step(plan, cache, Y, None, None, None, 0.0, lens, None, None, q)
    Q.qkv_attn_step(plan, cache, q, lens, 0.125, out, ws, add_weight=True)
    Q.qkv_evict_step(plan, cache, lens, lens, 32, 4, n2, wo, po, we)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    step()
for t, s in zip(state, saved): t.copy_(s)
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in state]
for t, s in zip(state, saved): t.copy_(s)
step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, state)) and out.abs().sum() > 0 and n2.tolist() == [32, 32]
assert Q.qkv_check_device_error()[0] == 0
print("captured first: ok")
"""


def test_first_calls_inside_a_capture(qkv):
    """A process whose first calls are captured replays what eager calls do."""
    import subprocess
    import sys
    import os
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], capture_output=True, text=True, timeout=120,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "captured first: ok" in r.stdout, r.stderr[-2000:]


def test_attention_reads_what_decode_steps_stored(qkv):
    """qkv_decode_step fills a contiguous region, which is one page to qkv_attn_step."""
    import torch
    H, nh, nkv, hd, n_ctx, n = 256, 4, 2, 64, 48, 37
    rng = np.random.default_rng(13)
    plan = Q.qkv_plan_create(H, nh, nkv, hd, 1e6, n_ctx, w_dtype=Q.QKV_F32, kv_dtype=Q.QKV_F16)
    nqt, nkt = nh * hd, nkv * hd
    W, bias = dev((0.05 * rng.standard_normal((nqt + 2 * nkt, H))).astype(np.float32)), dev(
        rng.standard_normal(nqt + 2 * nkt).astype(np.float32))
    k, v = (torch.zeros(1, n_ctx, nkt, dtype=torch.float16, device="cuda") for _ in range(2))
    out = torch.empty(nqt + 2 * nkt, device="cuda")
    for p in range(n):
        Q.qkv_decode_step(plan, dev(rng.standard_normal(H).astype(np.float32)), W, bias, dev(np.int32([p])), out[:nqt],
                          out[nqt:nqt + nkt], out[nqt + nkt:], k, v)
    cache = Q.PagedKv(plan, k, v, torch.zeros(1, 1, dtype=torch.int32, device="cuda"))
    ws = torch.zeros(Q.qkv_attn_workspace_bytes(plan, cache), dtype=torch.uint8, device="cuda")
    o = torch.empty(1, nqt, device="cuda")
    Q.qkv_attn_step(plan, cache, out[None, :nqt], dev(np.int32([n])), hd ** -0.5, o, ws)
    c = ref.Cache(rng, 1, nkv, hd, "f16", n_ctx, 1, lens=[0])
    c.k, c.v, c.table = k.cpu().numpy(), v.cpu().numpy(), np.int32([[0]])
    want = ref.attn_ref(c, out[None, :nqt].cpu().numpy(), [n], hd ** -0.5, 0, nh)
    close(o.cpu().numpy(), want[0], want[3], "out")


def test_python_refusals(qkv):
    import torch
    plan = make_plan(4, 2, 64, "f16")
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    i32, f16 = torch.int32, torch.float16
    k, table = z(8, 16, 128, dtype=f16), z(3, 4, dtype=i32)
    for args, kw in (((z(8, 16, 128), k, table), {}), ((k, z(8, 16, 64, dtype=f16), table), {}),
                     ((k, k, z(3, 4)), {}), ((k, k, table), dict(slot_weight=z(3, 2, 63))),
                     ((k, k, table), dict(slot_pos=z(3, 2, 64))), ((k.transpose(0, 1), k, table), {}),
                     ((k[:, ::2], k[:, ::2], table), {}), ((k[::2], k[:4], table), {})):
        with pytest.raises(Q.QkvError):
            Q.PagedKv(plan, *args, **kw)
    cache = Q.PagedKv(plan, k, k.clone(), table, slot_weight=z(3, 2, 64), slot_pos=z(3, 2, 64, dtype=i32))
    ws = z(Q.qkv_attn_workspace_bytes(plan, cache), dtype=torch.uint8)
    q, out, lens = z(3, 256), z(3, 256), z(3, dtype=i32)
    Q.qkv_attn_step(plan, cache, q, lens, 0.1, out, ws)
    for a in ((q[:2], lens, 0.1, out, ws), (q, lens[:2], 0.1, out, ws), (q, lens.long(), 0.1, out, ws),
              (q, lens, 0.1, out.half(), ws), (q, lens, 0.1, out, ws[:256]), (q.cpu(), lens, 0.1, out, ws),
              (q, lens, 0.1, z(256, 3).t(), ws), (q, lens, 0.1, out, None)):
        with pytest.raises(Q.QkvError):
            Q.qkv_attn_step(plan, cache, *a)
    Y, pos = z(5, 512), z(5, dtype=i32)
    seqs = pos.clone()
    for a in ((Y[:, :511], None, None, None, 0.0, pos, seqs, None, z(5, 256)),
              (Y.half(), None, None, None, 0.0, pos, seqs, None, z(5, 256)),
              (Y, None, None, None, 0.0, pos[:4], seqs, None, z(5, 256)),
              (Y, None, None, None, 0.0, pos, None, None, z(5, 256)),
              (Y, z(511), None, None, 0.0, pos, seqs, None, z(5, 256)),
              (Y, None, z(64), None, 0.0, pos, seqs, None, z(5, 256)),
              (Y, None, None, None, 0.0, pos, seqs, None, z(4, 256))):
        with pytest.raises(Q.QkvError):
            Q.qkv_paged_store_step(plan, cache, *a)
    wse = z(Q.qkv_evict_workspace_bytes(plan, cache), dtype=torch.uint8)
    w, p = z(3, 2, 64), z(3, 2, 64, dtype=i32)
    for a in ((lens, lens, 4, 1, lens, w, p, wse), (lens, lens, 0, 0, lens.clone(), w, p, wse),
              (lens, lens, 4, 5, lens.clone(), w, p, wse), (lens, lens, 4, 1, lens.clone(), w[:2], p, wse),
              (lens, lens, 4, 1, lens.clone(), w, p, None)):
        with pytest.raises(Q.QkvError):
            Q.qkv_evict_step(plan, cache, *a)
    assert Q.qkv_check_device_error()[0] == 0


def test_readme_example_of_the_paged_cache(qkv):
    """The README's paged example runs as printed: its last attention is that of the cache, and the
    eviction leaves the newest positions and the largest weights."""
    import os
    import re

    import torch
    readme = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
    code = re.findall(r"```python\n(.*?)```", open(readme).read(), re.S)[0]
    before, evict = code.split("# Keep 32 slots")
    env = {}
    exec(compile(before, "README.md", "exec"), env)
    torch.cuda.synchronize()
    assert env["lens"].tolist() == [44, 28]
    c = ref.Cache(np.random.default_rng(0), 2, 8, 128, "f16", 16, 4, lens=[0, 0])
    c.k, c.v, c.table = env["pool_k"].cpu().numpy(), env["pool_v"].cpu().numpy(), env["table"].cpu().numpy()
    want = ref.attn_ref(c, env["step_q"].cpu().numpy(), [44, 28], 128 ** -0.5, 0, 40)
    close(env["attn"].cpu().numpy(), want[0], want[3], "README attention")
    w, p = env["slot_weight"].cpu().numpy(), env["slot_pos"].cpu().numpy()
    assert np.allclose(w[0].sum(1), 4 * 5, atol=1e-3) and (p[0, :, :44] == np.arange(44)).all()
    exec(compile("# Keep 32 slots" + evict, "README.md", "exec"), env)
    torch.cuda.synchronize()
    rk, rv, rl, rw, rp = ref.evict_ref(c, [44, 28], [44, 28], w, p, 32, 8)
    assert env["kept"].tolist() == list(rl) == [32, 28]
    assert np.array_equal(env["pool_k"].cpu().numpy(), rk) and np.array_equal(env["pool_v"].cpu().numpy(), rv)
    assert np.array_equal(env["slot_pos"].cpu().numpy()[0, :, :32], rp[0, :, :32])
    assert np.array_equal(env["slot_weight"].cpu().numpy()[0, :, :32], rw[0, :, :32])
