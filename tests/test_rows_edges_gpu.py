"""Attention of many query rows: arguments that the documentation allows or names and ordinary calls do not have."""
import numpy as np
import pytest

import paged_reference
import qkv_rope_kv_gb300 as Q
import rows_reference as ref
from test_paged_gpu import close, dev, make_plan
from test_rows_gpu import buffers, pools_of

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
