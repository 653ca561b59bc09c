"""Infinities and NaN in long caches, attention of many query rows: they reach the rows that see them and leave the others'
bits alone, raise no flag, and cost about as much as the call itself."""
import pytest

import qkv_rope_kv_gb300 as Q
import rows_reference as ref
from test_paged_gpu import make_plan
from test_rows_gpu import attend64

pytestmark = pytest.mark.gpu


class Call:
    """`new` tokens at the end of `slots` slots of one sequence, on an f16 cache of two kv heads."""
    nkv = 2

    def __init__(self, new, slots, hd, out, page=64, G=4, window=0, seed=0):
        import torch
        torch.manual_seed(seed)
        self.new, self.slots, self.hd, self.G, self.window = new, slots, hd, G, window
        self.nh = G * self.nkv
        self.plan = make_plan(self.nh, self.nkv, hd, "f16")
        per = -(-slots // page)
        self.k, self.v = (torch.randn(per, page, self.nkv * hd, device="cuda").half() for _ in range(2))
        self.table = torch.randperm(per, device="cuda").int()[None].contiguous()
        self.page = page
        self.cache = Q.PagedKv(self.plan, self.k, self.v, self.table)
        self.q = torch.randn(new, self.nh * hd, device="cuda")
        self.dtype = torch.bfloat16 if out == "bf16" else torch.float32
        self.ws = torch.empty(Q.qkv_prompt_attn_workspace_bytes(self.plan, self.cache, new), dtype=torch.uint8, device="cuda")
        self.ints = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, new], [slots])]

    def row(self, slot):
        return int(self.table[0, slot // self.page]), slot % self.page

    def sees(self, slot):
        """Which tokens see it."""
        import torch
        end = torch.arange(self.slots - self.new + 1, self.slots + 1, device="cuda")
        lo = (end - self.window).clamp(min=0) if self.window else torch.zeros_like(end)
        return (slot >= lo) & (slot < end)

    def run(self):
        """out and lse as [new, kv head, q head of it(, hd)], and the time in ms (the second call's)."""
        import torch
        o = torch.full((self.new, self.nh * self.hd), 7.0, dtype=self.dtype, device="cuda")
        lse = torch.full((self.new, self.nh), 7.0, device="cuda")
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        for _ in range(2):
            a.record()
            Q.qkv_prompt_attn_step(self.plan, self.cache, self.q, *self.ints, self.hd ** -0.5, o, self.ws, window=self.window,
                                   lse=lse)
            b.record()
        b.synchronize()
        assert Q.qkv_check_device_error()[0] == 0
        return o.view(self.new, self.nkv, self.G, self.hd), lse.view(self.new, self.nkv, self.G), a.elapsed_time(b)


def same(a, b):
    import torch
    return torch.equal(a.view(torch.int16 if a.dtype == torch.bfloat16 else torch.int32),
                       b.view(torch.int16 if b.dtype == torch.bfloat16 else torch.int32))


def spoil_v(call, bad):
    """bad: (slot, kv head, column, value) each.  What the columns become: a sum of infinities (weights are above zero)."""
    import torch
    total = torch.zeros(call.new, call.nkv, call.hd, device="cuda")
    for slot, h, d, value in bad:
        call.v[call.row(slot)][h * call.hd + d] = value
        total[:, h, d] += torch.where(call.sees(slot), value, 0.0)
    return total[:, :, None].expand(-1, -1, call.G, -1)


INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("new,slots,hd,kw", [
    (8191, 8191, 128, {}),
    (8191, 8191, 64, dict(page=7)),
    (300, 40000, 128, {}),
    (300, 40000, 80, dict(page=12)),
    (2000, 6000, 128, dict(window=1500)),
    (5, 40000, 96, dict(G=1)),
], ids=str)
def test_values(qkv, new, slots, hd, kw, out):
    """V: an early slot that all rows see, later ones that some do, opposite infinities, in one of two kv heads."""
    import torch
    call = Call(new, slots, hd, out, **kw)
    want, lse, t0 = call.run()
    last = slots - new
    bad = [(5, 0, 3, INF), (slots // 2, 0, 3, -INF), (last + new // 2, 0, hd - 1, -INF), (last + new // 3, 0, 17, NAN),
           (slots - 1, 0, 0, INF), (last + new // 2 + 1, 0, 20, INF), (last + new // 2 + 2, 0, 20, INF)]
    total = spoil_v(call, bad)
    got, lse2, t1 = call.run()
    assert same(lse, lse2)  # V has no say in it
    odd = total != 0
    expect = torch.where(odd, total.to(want.dtype), want)
    assert torch.equal(torch.isnan(got), torch.isnan(expect))
    assert same(torch.where(torch.isnan(expect), 0, got), torch.where(torch.isnan(expect), 0, expect))
    assert same(got[:, 1], want[:, 1])
    assert t1 < 5 * t0 + 0.5, "%.3f ms, %.3f without" % (t1, t0)


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_every_value(qkv, out):
    """All of V infinite, of one sign in even columns and of both in odd ones."""
    import torch
    call = Call(600, 5000, 128, out)
    _, _, t0 = call.run()
    sign = torch.where(torch.rand_like(call.v, dtype=torch.float32) < 0.5, INF, -INF)
    sign[..., ::2] = INF
    call.v.copy_(sign)
    got, _, t1 = call.run()
    assert (got[..., ::2] == INF).all() and torch.isnan(got[..., 1::2]).all()
    assert t1 < 20 * t0 + 0.5, "%.3f ms, %.3f without" % (t1, t0)


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_shared_prefix(qkv, out):
    """A V that overflowed in the shared slots reaches every sequence, one in a sequence's own slots that one only."""
    import torch
    torch.manual_seed(4)
    B, P, own, nkv, G, hd, page = 40, 12800, 30, 2, 4, 128, 64
    plan = make_plan(nkv * G, nkv, hd, "f16")
    k, v = (torch.randn(P // page + B, page, nkv * hd, device="cuda").half() for _ in range(2))
    table = torch.full((B, P // page + 1), -1, dtype=torch.int32, device="cuda")
    table[0, :-1] = torch.randperm(P // page, device="cuda").int()
    table[:, -1] = torch.arange(P // page, P // page + B, device="cuda").int()
    cache = Q.PagedKv(plan, k, v, table)
    ws = torch.zeros(Q.qkv_prefix_attn_workspace_bytes(plan, cache), dtype=torch.uint8, device="cuda")
    q = torch.randn(B, nkv * G * hd, device="cuda")
    full = lambda x: torch.full((B,), x, dtype=torch.int32, device="cuda")  # noqa: E731

    def run():
        o = torch.empty(B, nkv * G * hd, dtype=torch.bfloat16 if out == "bf16" else torch.float32, device="cuda")
        Q.qkv_prefix_attn_step(plan, cache, q, full(P + own), full(0), full(P), hd ** -0.5, o, ws)
        assert Q.qkv_check_device_error()[0] == 0
        return o.view(B, nkv, G, hd)
    want = run()
    v[int(table[0, 7]), 5, 2] = INF            # kv head 0, column 2
    v[int(table[9, -1]), 3, hd + 4] = -INF     # kv head 1, column 4, of sequence 9
    got = run()
    expect = want.clone()
    expect[:, 0, :, 2], expect[9, 1, :, 4] = INF, -INF
    assert same(got, expect)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("new,slots,hd,window", [(700, 900, 128, 0), (700, 5000, 64, 0), (2000, 6000, 128, 1500), (900, 1500, 96, 40)])
def test_large_scores_of_others(qkv, out, new, slots, hd, window):
    """K that grows much in slots that a row does not see, but its neighbours do, leaves the row's bits alone."""
    import torch
    call = Call(new, slots, hd, out, page=16, window=window)
    want, lse, _ = call.run()
    half = slots - new // 2
    rows, checked = call.k.clone(), 0
    for changed in (range(half, slots), range(0, half)):  # later slots, and earlier ones, which only a window hides
        call.k.copy_(rows)
        at = torch.tensor([int(call.table[0, s // call.page]) * call.page + s % call.page for s in changed], device="cuda")
        call.k.view(-1, call.nkv * hd)[at] *= 20
        got, lse2, _ = call.run()
        free = ~torch.stack([call.sees(changed[0]), call.sees(changed[-1])]).any(0)
        end = torch.arange(slots - new + 1, slots + 1, device="cuda")
        free &= (end <= changed[0]) | ((end - window > changed[-1]) if window else False)
        checked += int(free.sum())
        assert same(got[free], want[free]) and same(lse[free], lse2[free])
    assert checked


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("new,slots,hd,kw", [
    (8191, 8191, 128, {}),
    (300, 40000, 64, dict(page=12)),
    (2000, 6000, 128, dict(window=1500)),
], ids=str)
def test_nan_scores(qkv, new, slots, hd, kw, out):
    """A NaN in K makes the rows that see it NaN, one in q (or an infinity) its row; the others keep their bits."""
    import torch
    call = Call(new, slots, hd, out, **kw)
    want, lse, t0 = call.run()
    dead = torch.zeros(new, call.nkv, call.G, dtype=torch.bool, device="cuda")
    for slot in (5, slots - new // 2):
        call.k[call.row(slot)][7] = NAN
        dead[:, 0] |= call.sees(slot)[:, None]
    got, lse2, t1 = call.run()
    q = call.q.view(new, call.nkv, call.G, hd)
    q[3, 1, 2, 5], q[new // 2, 1, 0, 0], q[new - 1, 1, 1, hd - 1] = NAN, INF, -INF
    got3, lse3, t2 = call.run()
    for dead, o, l in ((dead, got, lse2), (dead | ~torch.isfinite(q).all(-1), got3, lse3)):
        assert torch.isnan(o[dead]).all() and torch.isnan(l[dead]).all()
        assert same(o[~dead], want[~dead]) and same(l[~dead], lse[~dead])
    assert max(t1, t2) < 5 * t0 + 0.5, "%.3f and %.3f ms, %.3f without" % (t1, t2, t0)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("value,d", [(INF, 0), (-INF, 63)])
def test_infinite_k(qkv, out, value, d):
    """A row whose q has the other sign there sees the slot with no weight, one of the same sign is NaN."""
    import torch
    new, slots, hd, slot = 700, 5000, 64, 1234
    call = Call(new, slots, hd, out, page=16)
    _, _, t0 = call.run()
    call.k[call.row(slot)][d] = value
    got, lse, t1 = call.run()
    q = call.q.view(new, call.nkv, call.G, hd)[:, 0]
    dead = (q[..., d] < 0) == (value < 0)
    assert dead.any() and not dead.all()
    assert torch.isnan(got[:, 0][dead]).all() and torch.isnan(lse[:, 0][dead]).all()
    at = [i for i in range(slots) if i != slot]
    K, V = (x[call.table[0].long()].view(-1, call.nkv, hd)[at][:, 0] for x in (call.k, call.v))
    hi = torch.arange(slots - new + 1, slots + 1, device="cuda") - 1
    want, most, size = attend64(q, K, V, hi, hd ** -0.5)
    ds = (hd + 16) * 2 * ref.U * size + (2.0 ** -11 * size if out == "bf16" else 0)
    bound = (torch.expm1(2 * ds) + (slots / 8 + 64) * 2 * ref.U) * most
    if out == "bf16":
        bound = bound + 2.0 ** -11 * most + 2.0 ** -8 * (want.abs() + bound)
    assert ((got[:, 0].double() - want).abs() <= bound)[~dead].all()
    assert t1 < 5 * t0 + 0.5, "%.3f ms, %.3f without" % (t1, t0)


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_every_k_infinite(qkv, out):
    """Every row is NaN, by +inf or by nothing else than -inf."""
    import torch
    call = Call(600, 5000, 128, out)
    _, _, t0 = call.run()
    call.k[..., 3] = INF
    call.k[..., 128 + 3] = -INF
    got, _, t1 = call.run()
    assert torch.isnan(got).all()
    assert t1 < 40 * t0 + 0.5, "%.3f ms, %.3f without" % (t1, t0)
