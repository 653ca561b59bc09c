"""Attention of many query rows: arguments that the documentation allows or names and ordinary calls do not have."""
import numpy as np
import pytest

import paged_reference
import qkv_rope_kv_gb300 as Q
import rows_reference as ref
from test_paged_gpu import close, dev, make_plan
from test_rows_gpu import attend64, buffers, pools_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv,hd", [("f16", 128), ("f32", 64)])
@pytest.mark.parametrize("first,skipped", [
    ([0, 10, 5, 15], [1, 2]),                  # the last pair is in order and overlaps the first
    ([0, 20, 8, 12, 25, 30], [1, 2, 3]),       # two of them; the last one begins above all
    ([12, 3, 20, 30], [0, 1]),
    ([0, 5, 5, 9, 30], []),
], ids=str)
def test_sequences_that_would_share_rows(qkv, kv, hd, first, skipped):
    """Only one of two sequences that name the same rows gets them, whatever the timing: the earlier one."""
    import torch
    rng = np.random.default_rng(11)
    nh, nkv, page, nt, B = 4, 2, 16, 30, len(first) - 1
    c = paged_reference.Cache(rng, B, nkv, hd, kv, page, 6, lens=[60 + b for b in range(B)])
    plan = make_plan(nh, nkv, hd, kv)
    cache = Q.PagedKv(plan, *pools_of(c), dev(c.table))
    x = rng.standard_normal((nt, nh * hd)).astype(np.float32)
    places = [None] * nt
    for b in range(B):
        if b not in skipped:
            for i, p in enumerate(ref.prompt_places(c, [first[b]] * (b + 1) + [first[b + 1]] * (B - b), c.lens, nt, 0)):
                places[i] = p if p is not None else places[i]
    rows = [i for i, p in enumerate(places) if p is not None]
    want, _, bound, _ = ref.rows_ref(c.k, c.v, x[rows], [places[i] for i in rows], 0.1, nh, nkv, hd, False)
    for _ in range(3):
        q, o = buffers(nt, nh * hd, x, "f32", 0)
        ws = torch.empty(Q.qkv_prompt_attn_workspace_bytes(plan, cache, nt), dtype=torch.uint8, device="cuda")
        Q.qkv_prompt_attn_step(plan, cache, q, dev(np.int32(first)), dev(c.lens), 0.1, o, ws)
        torch.cuda.synchronize()
        assert Q.qkv_check_device_error()[0] == (4 if skipped else 0)
        got = o.cpu().numpy()
        close(got[rows], want, bound, "out")
        assert (got[[i for i in range(nt) if i not in rows]] == 77.0).all()


def test_a_decrease_far_before(qkv):
    """More sequences than the plan takes at once: one far behind a decrease that begins below it is skipped, others are not."""
    import torch
    rng = np.random.default_rng(12)
    nh, nkv, hd, page, B, nt = 2, 1, 64, 4, 1300, 1400
    c = paged_reference.Cache(rng, B, nkv, hd, "f16", page, 2, lens=[5] * B)
    plan = make_plan(nh, nkv, hd, "f16")
    cache = Q.PagedKv(plan, *pools_of(c), dev(c.table))
    first = np.arange(B + 1, dtype=np.int32)
    first[40] = 1000                          # sequences 39 and 40: too long, and down again; none below 1000 after that
    skipped = [40] + [b for b in range(41, 1000)]
    long = 39
    x = rng.standard_normal((nt, nh * hd)).astype(np.float32)
    q, o = buffers(nt, nh * hd, x, "f32", 0)
    ws = torch.empty(Q.qkv_prompt_attn_workspace_bytes(plan, cache, nt), dtype=torch.uint8, device="cuda")
    Q.qkv_prompt_attn_step(plan, cache, q, dev(first), dev(c.lens), 0.125, o, ws)
    torch.cuda.synchronize()
    assert Q.qkv_check_device_error()[0] == 4
    got = o.cpu().numpy()
    for b in [0, 38, 1000, 1001, 1299]:
        assert b not in skipped
        places = ref.prompt_places(c, [b] * (b + 1) + [b + 1] * (B - b), c.lens, nt, 0)
        want, _, bound, _ = ref.rows_ref(c.k, c.v, x[b:b + 1], [places[b]], 0.125, nh, nkv, hd, False)
        close(got[b:b + 1], want, bound, "sequence %d" % b)
    assert (got[long:1000 - 5] == 0).all()    # 961 tokens on 5 slots: all but the last five see nothing
    places = ref.prompt_places(c, [long] * (long + 1) + [1000] * (B - long), c.lens, nt, 0)
    want, _, bound, _ = ref.rows_ref(c.k, c.v, x[995:1000], places[995:1000], 0.125, nh, nkv, hd, False)
    close(got[995:1000], want, bound, "the long one")
    assert (got[1300:] == 77.0).all()


@pytest.mark.parametrize("kv,hd", [("f16", 128), ("f32", 64)])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 40, 96, 95])
def test_windows_as_large_as_the_cache(qkv, kv, hd, window):
    """The capacity is 96 slots; some tokens' ends lie below 0."""
    import torch
    rng = np.random.default_rng(13)
    nh, nkv, page, new, lens = 4, 2, 16, [70, 50], [20, 96]
    c = paged_reference.Cache(rng, 2, nkv, hd, kv, page, 6, lens=lens)
    plan = make_plan(nh, nkv, hd, kv)
    cache = Q.PagedKv(plan, *pools_of(c), dev(c.table))
    first, nt = np.int32([0, 70, 120]), 120
    x = rng.standard_normal((nt, nh * hd)).astype(np.float32)
    q, o = buffers(nt, nh * hd, x, "f32", 0)
    lse = torch.full((nt, nh), 55.0, device="cuda")
    ws = torch.empty(Q.qkv_prompt_attn_workspace_bytes(plan, cache, nt), dtype=torch.uint8, device="cuda")
    Q.qkv_prompt_attn_step(plan, cache, q, dev(first), dev(c.lens), 0.1, o, ws, window=window, lse=lse)
    torch.cuda.synchronize()
    assert Q.qkv_check_device_error()[0] == 0
    want, wl, bound, bl = ref.rows_ref(c.k, c.v, x, ref.prompt_places(c, first, lens, nt, window), 0.1, nh, nkv, hd, False)
    close(o.cpu().numpy(), want, bound, "out")
    close(lse.cpu().numpy(), wl, bl, "lse")


@pytest.mark.parametrize("page", [64, 12])  # copied by boxes, and row by row
@pytest.mark.parametrize("slots,grow", [(262144, 1.0), (65536, 1.0), (65536 + 128, 3.0)])
def test_many_slots_in_one_piece(qkv, slots, grow, page):
    """Out bf16, values above zero: the tensor cores cut less than 2^-23 of a sum off at each 16 slots, always towards zero, so
    2^-12 is lost over the 32768 that are summed in one accumulator, and no more over any number.  That is looked for in
    the mean distance from the exact values' own roundings to bf16; other errors, which may move a value by 2^-8 across a
    rounding's border to either side, leave 2^-8 / sqrt(values) of a mean; 4 times that is allowed."""
    import torch
    torch.manual_seed(0)
    hd, new = 64, 256 * 152                   # every CTA has a whole tile
    plan = make_plan(1, 1, hd, "f16")
    per = -(-slots // page)
    k, v = (torch.randn(per, page, hd, device="cuda").half() for _ in range(2))
    v.copy_(v.abs())
    k[per // 2:] *= grow                      # maxima move on the way
    table = torch.randperm(per, device="cuda").int()[None].contiguous()
    cache = Q.PagedKv(plan, k, v, table)
    q = torch.randn(new, hd, device="cuda")
    o = torch.empty(new, hd, device="cuda", dtype=torch.bfloat16)
    lse = torch.empty(new, 1, device="cuda")
    ws = torch.empty(Q.qkv_prompt_attn_workspace_bytes(plan, cache, new), dtype=torch.uint8, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    Q.qkv_prompt_attn_step(plan, cache, q, i32(0, new), i32(slots), hd ** -0.5, o, ws, lse=lse)
    assert Q.qkv_check_device_error()[0] == 0
    at = torch.arange(7, new, 151, device="cuda")
    K, V = (x[table[0].long()].view(-1, hd)[:slots].double() for x in (k, v))
    want = torch.empty(len(at), hd, device="cuda", dtype=torch.float64)
    most, off = (torch.empty(len(at), 1, device="cuda", dtype=torch.float64) for _ in range(2))
    for i in range(0, len(at), 32):
        t = at[i:i + 32]
        s = q[t].double() @ K.T * hd ** -0.5
        s.masked_fill_(torch.arange(slots, device="cuda") >= (slots - new + 1 + t)[:, None], -float("inf"))
        most[i:i + 32] = torch.logsumexp(s, -1, keepdim=True)
        want[i:i + 32] = torch.softmax(s, -1) @ V
        # each q element is rounded to f16 (2^-11 of it at most), so a score may be off by 2^-11 scale sum |q_d K_d|, besides the
        # f32 sums' (hd + 16) 2^-23 of that; log sum exp is off by no more than the scores are, and its own sum's error
        off[i:i + 32] = (q[t].double().abs() @ K.abs().T).amax(-1, keepdim=True) * hd ** -0.5 * (2.0 ** -11 + (hd + 16) * 2.0 ** -23)
    got = o[at].double()
    shrink = ((got - want.bfloat16().double()) * want).sum().item() / (want * want).sum().item()
    assert abs(shrink) <= 2.0 ** -12 + 4 * 2.0 ** -8 / want.numel() ** 0.5, shrink
    assert (got - want).norm() <= 2.0 ** -9 * want.norm()  # roundings of all kinds, not only towards zero
    assert ((lse[at].double() - most).abs() <= off + (slots / 8 + 64) * 2.0 ** -23).all()


def test_infinities_in_long_pieces(qkv):
    """Pieces that are summed in several goes: an infinity of an earlier or a later go reaches all rows, other columns keep
    their bits."""
    import torch
    torch.manual_seed(1)
    hd, new, slots, page = 64, 256 * 152, 65536, 64
    plan = make_plan(1, 1, hd, "f16")
    k, v = (torch.randn(slots // page, page, hd, device="cuda").half() for _ in range(2))
    cache = Q.PagedKv(plan, k, v, torch.arange(slots // page, device="cuda").int()[None].contiguous())
    q = torch.randn(new, hd, device="cuda")
    ws = torch.empty(Q.qkv_prompt_attn_workspace_bytes(plan, cache, new), dtype=torch.uint8, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    def run():
        o = torch.empty(new, hd, device="cuda", dtype=torch.bfloat16)
        Q.qkv_prompt_attn_step(plan, cache, q, i32(0, new), i32(slots), hd ** -0.5, o, ws)
        assert Q.qkv_check_device_error()[0] == 0
        return o
    want = run()
    first = slots - new                          # the first token's own slot
    for slot, d, value in ((5, 1, float("inf")), (first - 3, 2, -float("inf")), (first - 2, 60, float("nan")), (7, 61, float("inf")),
                           (first - 4, 61, -float("inf"))):
        v.view(-1, hd)[slot, d] = value
    got = run()
    assert (got[:, 1] == float("inf")).all() and (got[:, 2] == -float("inf")).all() and torch.isnan(got[:, 60:62]).all()
    keep = [d for d in range(hd) if d not in (1, 2, 60, 61)]
    assert torch.equal(got[:, keep].view(torch.int16), want[:, keep].view(torch.int16))


def test_long_shared_prefix_in_one_piece(qkv):
    """The same for sequences on a shared prefix: out bf16 against out f32, whose sums are never in one accumulator for long."""
    import torch
    torch.manual_seed(2)
    nkv, hd, page, B, P = 8, 64, 64, 19 * 256, 131072
    plan = make_plan(nkv, nkv, hd, "f16")
    per = P // page
    k, v = (torch.randn(per + 1, page, nkv * hd, device="cuda").half() for _ in range(2))
    v.copy_(v.abs())
    k[per // 2:] *= 2
    table = torch.full((B, per + 1), -1, dtype=torch.int32, device="cuda")
    table[0, :per] = torch.randperm(per, device="cuda").int()
    table[:, per] = per
    cache = Q.PagedKv(plan, k, v, table)
    ws = torch.zeros(Q.qkv_prefix_attn_workspace_bytes(plan, cache), dtype=torch.uint8, device="cuda")
    q = torch.randn(B, nkv * hd, device="cuda")
    full = lambda x: torch.full((B,), x, dtype=torch.int32, device="cuda")  # noqa: E731
    outs = []
    for dtype in (torch.float32, torch.bfloat16):
        o = torch.empty(B, nkv * hd, device="cuda", dtype=dtype)
        Q.qkv_prefix_attn_step(plan, cache, q, full(P + 9), full(0), full(P), hd ** -0.5, o, ws)
        assert Q.qkv_check_device_error()[0] == 0
        outs.append(o.double())
    want, got = outs
    shrink = ((got - want.bfloat16().double()) * want).sum().item() / (want * want).sum().item()
    assert abs(shrink) <= 2.0 ** -12 + 4 * 2.0 ** -8 / want.numel() ** 0.5, shrink
    assert (got - want).norm() <= 2.0 ** -8 * want.norm()


@pytest.mark.parametrize("kind", ["prompt", "prefix"])
@pytest.mark.parametrize("q_scale", [2.0, 8.0, 32.0])
def test_rounded_q_and_weights(qkv, q_scale, kind):
    """Out bf16 on an f16 cache, scores of standard deviation 2 to 32.  q's elements are off by 2^-11 of themselves at most, to
    either side, so a score by 2^-11 / sqrt(3) scale |q o K| (2-norm) as a mean square, twice that with the others of its
    row; a weight by 2^-11 / sqrt(3); the result by 2^-8 / sqrt(3) as bf16.  Out f32 has none of these."""
    import torch
    torch.manual_seed(5)
    nh, nkv, hd, page, n = 8, 1, 128, 64, 4096
    new = 256 if kind == "prompt" else 32
    plan = make_plan(nh, nkv, hd, "f16")
    k, v = (torch.randn(n // page + new, page, hd, device="cuda").half() for _ in range(2))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q = q_scale * torch.randn(new, nh * hd, device="cuda")
    outs = []
    for dtype in (torch.bfloat16, torch.float32):
        o = torch.empty(new, nh * hd, device="cuda", dtype=dtype)
        if kind == "prompt":
            cache = Q.PagedKv(plan, k, v, torch.arange(n // page, device="cuda").int()[None].contiguous())
            ws = torch.empty(Q.qkv_prompt_attn_workspace_bytes(plan, cache, new), dtype=torch.uint8, device="cuda")
            Q.qkv_prompt_attn_step(plan, cache, q, i32([0, new]), i32([n]), hd ** -0.5, o, ws)
            hi = torch.arange(n - new + 1, n + 1, device="cuda")
        else:  # every sequence has the prefix only
            table = torch.arange(n // page, device="cuda").int()[None].repeat(new, 1).contiguous()
            cache = Q.PagedKv(plan, k, v, table)
            ws = torch.zeros(Q.qkv_prefix_attn_workspace_bytes(plan, cache), dtype=torch.uint8, device="cuda")
            Q.qkv_prefix_attn_step(plan, cache, q, i32([n] * new), i32([0] * new), i32([n] * new), hd ** -0.5, o, ws)
            hi = torch.full((new,), n, device="cuda")
        assert Q.qkv_check_device_error()[0] == 0
        outs.append(o.view(new, nh, hd).double())
    K, V = (x[:n // page].view(-1, hd) for x in (k, v))
    want, most, size = attend64(q.view(new, nh, hd), K, V, hi, hd ** -0.5)
    spread = ((q.view(new, nh, hd).double() ** 2) @ (K.double() ** 2).T).mean().sqrt().item() * hd ** -0.5
    rms = (2.0 ** -8 + 2.0 ** -11 + 2 * 2.0 ** -11 * spread) / 3 ** 0.5
    assert (outs[0] - want).norm() <= rms * want.norm()
    assert (outs[1] - want).norm() <= (n ** 0.5 + hd ** 0.5 * size.max()) * ref.U * most.norm()  # as in test_long_prompts
