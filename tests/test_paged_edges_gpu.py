"""Paged-cache calls at their edges on the GPU: values at the ends of their types, the smallest
shapes, calls from several threads, tables and outputs that a caller got wrong."""
import numpy as np
import pytest

import test_paged_gpu as base

pytestmark = pytest.mark.gpu
EPS = base.EPS

# Head sizes and pool alignments that take each of the kernels: tensor cores, and rows of no whole 16 bytes.
LAYOUTS = [(64, 0), (128, 0), (256, 0), (64, 1)]


@pytest.mark.parametrize("hd,pool_off", LAYOUTS)
def test_attn_keeps_all_bits_of_large_f32_keys(qkv, hd, pool_off):
    """Keys of 1e34 and both signs: the part below their leading 11 bits is above 1e30 itself.  q is small, so the
    scores are ordinary; the bound is that of ordinary keys (the remainders of q, 2^-12 * 1e-34, are normal
    numbers)."""
    def large(c, x):
        c.k *= np.float32(1e34)
        x *= np.float32(1e-34)

    base.run_attn(4, 2, hd, "f32", 16, [40, 90], change=large, pool_off=pool_off, weights=True)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("hd,pool_off", LAYOUTS)
def test_attn_infinite_key_against_a_large_query(qkv, hd, pool_off, sign):
    """A score of -inf from an infinite f32 key of either sign has weight 0, however large the query element that
    makes it is (the element's other keys are 0, so all other scores are ordinary)."""
    def change(c, x):
        c.k[..., 3] = 0
        x[0, 3], x[0, hd + 3] = -sign * 1e12, -sign * 3e20  # both q heads of kv head 0
        c.k[c.row(0, 5)][3] = sign * np.inf

    base.run_attn(4, 2, hd, "f32", 16, [40, 90], change=change, pool_off=pool_off)


@pytest.mark.parametrize("kv,hd,pool_off", [(kv, *x) for kv in ("f32", "f16") for x in LAYOUTS])
def test_attn_of_one_slot_is_its_value(qkv, kv, hd, pool_off):
    """One slot has weight 1, kept as a power of two: out is V, off by what the split of an f32 value may
    lose, 2^-23 of it; an f16 value is exact."""
    import torch
    rng = np.random.default_rng(21)
    n_seq, nh, nkv = 5, 6, 2
    plan = base.make_plan(nh, nkv, hd, kv)
    dt = torch.float16 if kv == "f16" else torch.float32
    k, v = (torch.zeros(n_seq * 16 * nkv * hd + pool_off, dtype=dt, device="cuda")[pool_off:].view(n_seq, 16, nkv * hd)
            for _ in range(2))
    host = rng.standard_normal((2, n_seq, 16, nkv * hd)).astype(np.float32)
    k.copy_(base.dev(host[0]))
    v.copy_(base.dev(host[1]))
    cache = base.Q.PagedKv(plan, k, v, torch.arange(n_seq, dtype=torch.int32, device="cuda").view(n_seq, 1))
    ws = torch.zeros(base.Q.qkv_attn_workspace_bytes(plan, cache), dtype=torch.uint8, device="cuda")
    q = base.dev(rng.standard_normal((n_seq, nh * hd)).astype(np.float32))
    out = torch.empty(n_seq, nh * hd, device="cuda")
    base.Q.qkv_attn_step(plan, cache, q, torch.ones(n_seq, dtype=torch.int32, device="cuda"), 0.1, out, ws)
    want = v[:, 0].double().view(n_seq, nkv, 1, hd).expand(n_seq, nkv, nh // nkv, hd).reshape(n_seq, nh * hd)
    bound = want.abs() * (2.0 ** -23 if kv == "f32" else 0.0)
    assert ((out.double() - want).abs() <= bound).all()


@pytest.mark.parametrize("kv", ["f32", "f16"])
@pytest.mark.parametrize("n_seq,n", [(1, 6000), (4, 6000), (300, 1500)])
def test_attn_error_over_long_rows(qkv, kv, n_seq, n):
    """The 2-norm of the error, relative, over rows long enough for sums to lose bits.  With u = 2^-24, standard
    normal K and V of head size 128 and q of twice that (scores of 2.9 in log2 terms), rms values:
      scores: q scaled, q and K split 1.2 u of 2.9; eight blocks of columns, each a sum inside two MMAs that cut
        up to 2 u off a value of 1: 4.5 u; eight additions to nearest 3.3 u; the two halves' sum 1.7 u;
        the difference to the maximum (4 to 16 in size) 4 u: 8 u together, 5.6 u of a weight;
      weights and values: 2^s 1.2 u, the two splits 0.7 u each: 5.9 u with the above.  Independent errors of
        the weights are to the error of the sum as the weights are to the sum;
      sums: a warp adds at most 6000 / 8 / 4 = 190 units to nearest: sqrt(190 / 2) 0.58 u = 5.7 u, and each
        unit's own MMAs cut 1.4 u.
    Together 8.3 u = 5e-7; the bound is twice that.  (Sums left to the MMAs come out at 2.3e-6 and 6.1e-6.)"""
    import torch
    nh, nkv, hd = 10, 2, 128
    gen = torch.Generator(device="cuda").manual_seed(22)
    plan = base.make_plan(nh, nkv, hd, kv)
    dt = torch.float16 if kv == "f16" else torch.float32
    k, v = (torch.randn(n_seq, n, nkv * hd, generator=gen, device="cuda").to(dt) for _ in range(2))
    q = 2.0 * torch.randn(n_seq, nh * hd, generator=gen, device="cuda")
    cache = base.Q.PagedKv(plan, k, v, torch.arange(n_seq, dtype=torch.int32, device="cuda").view(n_seq, 1))
    ws = torch.zeros(base.Q.qkv_attn_workspace_bytes(plan, cache), dtype=torch.uint8, device="cuda")
    out = torch.empty(n_seq, nh * hd, device="cuda")
    lens = torch.full((n_seq,), n, dtype=torch.int32, device="cuda")
    base.Q.qkv_attn_step(plan, cache, q, lens, hd ** -0.5, out, ws)
    off = size = 0.0
    for b in range(n_seq):
        K, V = (t[b].double().view(n, nkv, hd).transpose(0, 1) for t in (k, v))
        p = torch.softmax(q[b].double().view(nkv, nh // nkv, hd) @ K.transpose(1, 2) * hd ** -0.5, -1)
        want = (p @ V).reshape(-1)
        off += (out[b].double() - want).square().sum().item()
        size += want.square().sum().item()
    assert (off / size) ** 0.5 <= 1e-6


@pytest.mark.parametrize("hd,pool_off", LAYOUTS)
def test_attn_of_f32_values_near_the_largest(qkv, hd, pool_off):
    """Values of either sign around 5e35, whose sum over 90 slots is an f32 number, within the bound of ordinary
    ones; and one slot of 3.3e38."""
    def large(c, x):
        c.v *= np.float32(5e35)

    def one(c, x):
        c.v[...] = np.where(np.signbit(c.v), np.float32(-3.3e38), np.float32(3.3e38))

    base.run_attn(4, 2, hd, "f32", 16, [40, 90], change=large, pool_off=pool_off, weights=True)
    base.run_attn(4, 2, hd, "f32", 16, [1, 1, 0], change=one, pool_off=pool_off)


def run_in_threads(works):
    """Run the functions at once, a thread each; what they raise."""
    import threading
    start, raised = threading.Barrier(len(works)), []

    def body(work):
        start.wait()
        try:
            work()
        except Exception as e:
            raised.append(e)
    threads = [threading.Thread(target=body, args=(w,)) for w in works]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return raised


@pytest.mark.parametrize("caps", [(512, 8192), (16384, 49152, 600000)], ids=str)
def test_evictions_of_different_capacities_from_several_threads(qkv, caps):
    """Host threads with caches of different capacities, a stream and a workspace each: no call fails, and each
    keeps what it keeps alone."""
    import torch
    nkv, hd, page, n, budget = 2, 64, 64, 500, 400
    works, states = [], []
    rng = np.random.default_rng(23)
    for cap in caps:
        plan = base.make_plan(2 * nkv, nkv, hd, "f16")
        c = base.ref.Cache(rng, 1, nkv, hd, "f16", page, cap // page, lens=[n], table_fill=0)
        w = torch.zeros(1, nkv, cap, device="cuda")
        w[..., :n] = base.dev(rng.random((1, nkv, n)).astype(np.float32))
        pos = torch.arange(cap, dtype=torch.int32, device="cuda").expand(1, nkv, cap).contiguous()
        k, v = base.dev(c.k), base.dev(c.v)
        cache = base.Q.PagedKv(plan, k, v, base.dev(c.table), slot_weight=w, slot_pos=pos)
        lens, out = base.dev(c.lens), torch.zeros(1, dtype=torch.int32, device="cuda")
        wo, po = torch.zeros_like(w), torch.zeros_like(pos)
        ws = torch.zeros(base.Q.qkv_evict_workspace_bytes(plan, cache), dtype=torch.uint8, device="cuda")
        stream = torch.cuda.Stream()

        def work(a=(plan, cache, lens, lens, budget, 7, out, wo, po, ws), stream=stream):
            for _ in range(1500):
                base.Q.qkv_evict_step(*a, stream=stream)
        works.append(work)
        states.append((c, w.cpu().numpy(), pos.cpu().numpy(), out, wo, po))
    torch.cuda.synchronize()
    assert run_in_threads(works) == []
    torch.cuda.synchronize()
    for c, w, pos, out, wo, po in states:
        _, _, rl, rw, rp = base.ref.evict_ref(c, c.lens, c.lens, w, pos, budget, 7)
        assert out.tolist() == list(rl) == [budget]
        assert np.array_equal(wo.cpu().numpy()[..., :budget], rw[..., :budget])
        assert np.array_equal(po.cpu().numpy()[..., :budget], rp[..., :budget])
    assert base.Q.qkv_check_device_error()[0] == 0


@pytest.mark.parametrize("hd", [128, 6])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("nt", [1, 2, 500, 2500])
def test_store_in_place(qkv, nt, norm, hd):
    """q over Y's own rows, one token or more: the bits of a q of its own, and the rest of Y untouched."""
    import torch
    nh, nkv, page = 6, 2, 16
    gen = torch.Generator(device="cuda").manual_seed(24)
    plan = base.make_plan(nh, nkv, hd, "f16")
    k, v = (torch.zeros(160, page, nkv * hd, dtype=torch.float16, device="cuda") for _ in range(2))
    cache = base.Q.PagedKv(plan, k, v, torch.arange(160, dtype=torch.int32, device="cuda").view(1, 160))
    Y = torch.randn(nt, (nh + 2 * nkv) * hd, generator=gen, device="cuda")
    w = (torch.randn(hd, generator=gen, device="cuda"), torch.randn(hd, generator=gen, device="cuda")) if norm else (None, None)
    at, seqs = torch.arange(nt, dtype=torch.int32, device="cuda"), torch.zeros(nt, dtype=torch.int32, device="cuda")
    got = []
    for inplace in (False, True):
        y = Y.clone()
        q = y[:, :nh * hd] if inplace else torch.empty(nt, nh * hd, device="cuda")
        k.zero_()
        v.zero_()
        base.Q.qkv_paged_store_step(plan, cache, y, None, *w, EPS, at, seqs, None, q)
        got.append((q.clone(), k.clone(), v.clone()))
        assert torch.equal(y[:, nh * hd:], Y[:, nh * hd:])
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert base.Q.qkv_check_device_error()[0] == 0


def test_pools_whose_pages_overlap_are_refused(qkv):
    """An expanded pool (page stride 0, which means "one after the other" to the C call) or overlapping pages."""
    import torch
    plan = base.make_plan(4, 2, 64, "f16")
    table = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    whole = torch.zeros(8, 16, 128, dtype=torch.float16, device="cuda")
    one = whole[:1].expand(8, 16, 128)
    near = whole.as_strided((4, 16, 128), (8 * 128, 128, 1))
    for k, v in ((one, one), (whole, one), (one, whole), (near, near)):
        with pytest.raises(base.Q.QkvError, match="pages of their own"):
            base.Q.PagedKv(plan, k, v, table)
    base.Q.PagedKv(plan, whole[:1].expand(1, 16, 128), whole[1:2], table)  # one page has no stride


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("hd,page,max_pages", [(64, 16, 4), (6, 16, 4), (64, 16, 600)])
def test_evict_leaves_slots_of_bad_pages_as_they_are(qkv, hd, page, max_pages, inplace):
    """A move from or to a page that is not there is not made, and the slot keeps its weight and position with its
    row; in one launch, with rows of no whole 16 bytes, and in clusters."""
    import torch
    rng = np.random.default_rng(25)
    nkv, n, budget = 2, 64, 24
    c = base.ref.Cache(rng, 2, nkv, hd, "f16", page, max_pages, lens=[n, n])
    plan = base.make_plan(2 * nkv, nkv, hd, "f16")
    w = rng.random((2, nkv, c.cap)).astype(np.float32)
    pos = np.tile(rng.permutation(c.cap).astype(np.int32), (2, nkv, 1))
    bad_slots = set(range(page, 2 * page)) | set(range(2 * page, 3 * page))  # 8 below the budget, others above
    table = c.table.copy()
    table[0, 1], table[0, 2] = c.n_pages, -3
    k, v, dw, dp = base.dev(c.k), base.dev(c.v), base.dev(w), base.dev(pos)
    cache = base.Q.PagedKv(plan, k, v, base.dev(table), slot_weight=dw, slot_pos=dp)
    wo, po = (dw, dp) if inplace else (torch.full_like(dw, -8.0), torch.full_like(dp, -8))
    lo = torch.zeros(2, dtype=torch.int32, device="cuda")
    ws = torch.zeros(base.Q.qkv_evict_workspace_bytes(plan, cache), dtype=torch.uint8, device="cuda")
    lens = base.dev(c.lens)
    base.Q.qkv_evict_step(plan, cache, lens, base.dev(np.int32([2 ** 30] * 2)), budget, 0, lo, wo, po, ws)
    torch.cuda.synchronize()
    flags, value = base.Q.qkv_check_device_error()
    assert flags == 4 and value in (c.n_pages, -3) and lo.tolist() == [budget, budget]
    rk, rv, rw, rp, left = c.k.copy(), c.v.copy(), w.copy(), pos.copy(), 0
    for b in range(2):
        for h in range(nkv):
            kept = set(sorted(range(n), key=lambda s: -w[b, h, s])[:budget])
            for to, at in zip([s for s in range(budget) if s not in kept], [s for s in range(budget, n) if s in kept]):
                if b == 0 and (to in bad_slots or at in bad_slots):
                    left += 1
                    continue
                for pool in (rk, rv):
                    pool[c.row(b, to)][h * hd:(h + 1) * hd] = pool[c.row(b, at)][h * hd:(h + 1) * hd]
                rw[b, h, to], rp[b, h, to] = w[b, h, at], pos[b, h, at]
    assert left > 4
    assert np.array_equal(wo.cpu().numpy()[..., :budget], rw[..., :budget])
    assert np.array_equal(po.cpu().numpy()[..., :budget], rp[..., :budget])
    for got, want in ((k, rk), (v, rv)):
        assert np.array_equal(got.cpu().numpy().view(np.uint16), want.view(np.uint16))


STATUS_READS = """
import torch, qkv_rope_kv_gb300 as Q
from torch.profiler import ProfilerActivity, profile
plan = Q.qkv_plan_create(64, 4, 2, 64, 1e6, 64)
k = torch.zeros(4, 16, 128, dtype=torch.float16, device="cuda")
table = torch.full((1, 4), 9, dtype=torch.int32, device="cuda")
cache = Q.PagedKv(plan, k, k.clone(), table)
ws = torch.zeros(Q.qkv_attn_workspace_bytes(plan, cache), dtype=torch.uint8, device="cuda")
q, out, lens = torch.zeros(1, 256, device="cuda"), torch.zeros(1, 256, device="cuda"), torch.ones_like(table[0, :1])
def reads():
    torch.cuda.synchronize()
    with profile(activities=[ProfilerActivity.CUDA, ProfilerActivity.CPU]) as p:
        got = Q.qkv_check_device_error()
    return got, sum(e.count for e in p.key_averages() if "Memcpy DtoH" in e.key)
reads()  # the profiler's first use records nothing
print(reads())
Q.qkv_attn_step(plan, cache, q, lens, 0.1, out, ws)
print(reads())
print(reads())
"""


def test_status_is_read_only_where_it_can_be_set(qkv):
    """A process that launched no paged kernel reads the two words of decode and prefill; the attention's follows once
    it was launched (here on a page that is not there, which sets it)."""
    import os
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-c", STATUS_READS], capture_output=True, text=True, timeout=120,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    lines = [line for line in r.stdout.splitlines() if line.startswith("((")]
    assert lines == ["((0, 0), 2)", "((4, 9), 3)", "((0, 0), 3)"], r.stdout + r.stderr[-2000:]


def test_numbers_that_fit_no_argument_are_refused(qkv):
    """As any other bad argument, by the framework's error."""
    import torch
    plan = base.make_plan(4, 2, 64, "f16")
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    i32 = torch.int32
    k = z(4, 16, 128, dtype=torch.float16)
    w, p, lens = z(1, 2, 64), z(1, 2, 64, dtype=i32), z(1, dtype=i32)
    cache = base.Q.PagedKv(plan, k, k.clone(), z(1, 4, dtype=i32), slot_weight=w, slot_pos=p)
    ws = z(base.Q.qkv_attn_workspace_bytes(plan, cache), dtype=torch.uint8)
    we = z(base.Q.qkv_evict_workspace_bytes(plan, cache), dtype=torch.uint8)
    q, out = z(1, 256), z(1, 256)
    for scale, window in ((0.1, 1 << 31), (0.1, -1), (0.1, 1.5), (0.1, None), (1e39, 0), (None, 0), (float("nan"), 0)):
        with pytest.raises(base.Q.QkvError) as e:
            base.Q.qkv_attn_step(plan, cache, q, lens, scale, out, ws, window=window)
        assert e.value.status == base.Q.QKV_ERR_INVALID_ARG
    for budget, recent in ((1 << 31, 0), (1 << 40, 0), (4, -1), (4, 1 << 40), (2.5, 0)):
        with pytest.raises(base.Q.QkvError) as e:
            base.Q.qkv_evict_step(plan, cache, lens, lens, budget, recent, lens.clone(), w, p, we)
        assert e.value.status == base.Q.QKV_ERR_INVALID_ARG
    for eps in (1e39, None, -1.0):
        with pytest.raises(base.Q.QkvError) as e:
            base.Q.qkv_paged_store_step(plan, cache, z(1, 512), None, z(64), z(64), eps, lens, None, None, q)
        assert e.value.status == base.Q.QKV_ERR_INVALID_ARG
    assert base.Q.qkv_check_device_error()[0] == 0


@pytest.mark.parametrize("nh,nkv,hd,kv,lens,kw", [
    (28, 4, 128, "f16", [3000], {}), (28, 4, 128, "f16", [700, 1, 0, 2000] * 9, dict(window=65)),
    (14, 2, 64, "f32", [509, 33], {}), (5, 1, 128, "f16", [30011], {}), (136, 1, 64, "f16", [90, 31, 0, 200] * 4, {}),
    (8, 1, 256, "f16", [900] * 20, {}), (6, 3, 6, "f16", [50, 3], dict(window=7)),
], ids=str)
def test_attn_workspace_needs_its_head_zero_alone(qkv, nh, nkv, hd, kv, lens, kw):
    """Behind the first 4096 bytes the workspace may hold anything (here NaN)."""
    import torch
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    ws[:4096] = 0
    base.run_attn(nh, nkv, hd, kv, 16, lens, weights=True, workspace=ws, **kw)


@pytest.mark.filterwarnings("ignore:invalid value")  # a signalling NaN on its way to 64 bits
@pytest.mark.parametrize("bits", [0x7f800001, 0xff800001, 0x7f801fff, 0x7fffffff], ids=hex)
@pytest.mark.parametrize("hd,pool_off", LAYOUTS)
def test_attn_f32_nan_of_any_payload(qkv, hd, pool_off, bits):
    """A NaN whose payload is in its lowest bits is one as any other: in V it stays in its column, in K in its heads."""
    nan = np.array(bits, np.uint32).view(np.float32)

    def change(c, x):
        c.v[c.row(0, 9)][4] = nan
        c.k[c.row(1, 11)][hd + 2] = nan

    base.run_attn(4, 2, hd, "f32", 16, [40, 90], change=change, pool_off=pool_off)


@pytest.mark.parametrize("max_pages", [4, 600])
def test_evict_with_more_newest_slots_than_the_budget(qkv, max_pages):
    """Positions that all count as newest: the lowest slots stay, and nothing moves."""
    import torch
    rng = np.random.default_rng(26)
    c = base.ref.Cache(rng, 1, 2, 64, "f16", 16, max_pages, lens=[64])
    plan = base.make_plan(4, 2, 64, "f16")
    w, pos = base.dev(rng.random((1, 2, c.cap)).astype(np.float32)), base.dev(np.tile(np.arange(c.cap, dtype=np.int32), (1, 2, 1)))
    k, v = base.dev(c.k), base.dev(c.v)
    cache = base.Q.PagedKv(plan, k, v, base.dev(c.table), slot_weight=w, slot_pos=pos)
    wo, po, lo = torch.full_like(w, -8.0), torch.full_like(pos, -8), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(base.Q.qkv_evict_workspace_bytes(plan, cache), dtype=torch.uint8, device="cuda")
    for nxt in (-2 ** 31, 0, 5):
        base.Q.qkv_evict_step(plan, cache, base.dev(c.lens), base.dev(np.int32([nxt])), 20, 9, lo, wo, po, ws)
        assert lo.tolist() == [20] and torch.equal(wo[..., :20], w[..., :20]) and torch.equal(po[..., :20], pos[..., :20])
        assert (wo[..., 20:] == -8).all() and (po[..., 20:] == -8).all()
        assert np.array_equal(k.cpu().numpy().view(np.uint16), c.k.view(np.uint16))
        assert np.array_equal(v.cpu().numpy().view(np.uint16), c.v.view(np.uint16))
    assert base.Q.qkv_check_device_error()[0] == 0
