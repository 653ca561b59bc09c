"""Bounded waits of the attention of many query rows on the tensor cores: none runs out while its CTA gets on, however long
a piece of work lasts; one whose end never comes sets the flag and leaves the context usable."""
import time

import pytest

import qkv_rope_kv_gb300 as Q
from test_paged_gpu import make_plan

pytestmark = pytest.mark.gpu


def dtypes(out):
    import torch
    return torch.bfloat16 if out == "bf16" else torch.float32


def problem(new, slots, nh, nkv, hd, out, pages=64, page=64, grow=1.0):
    """Sequences of new[b] tokens at the end of slots[b] slots, of `pages` pages that their rows of the table name again and
    again, and a call of them.  K of the second half of the pages is larger by `grow`."""
    import torch
    torch.manual_seed(1)
    plan = make_plan(nh, nkv, hd, "f16")
    k, v = (torch.randn(pages, page, nkv * hd, device="cuda").half() for _ in range(2))
    k[pages // 2:] *= grow
    per = -(-max(slots) // page)
    table = (torch.arange(per, device="cuda") % pages).int()[None].repeat(len(new), 1).contiguous()
    cache = Q.PagedKv(plan, k, v, table)
    first = [0]
    for n in new:
        first.append(first[-1] + n)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.randn(first[-1], nh * hd, device="cuda")
    ws = torch.empty(Q.qkv_prompt_attn_workspace_bytes(plan, cache, first[-1]), dtype=torch.uint8, device="cuda")
    o = torch.full((first[-1], nh * hd), float("nan"), dtype=dtypes(out), device="cuda")

    def call(fn, o, **kw):
        fn(plan, cache, q, i32(first), i32(slots), hd ** -0.5, o, ws, **kw)
        torch.cuda.synchronize()
        return Q.qkv_check_device_error()[0]
    return call, o


# pieces of 320 blocks, which take some 300 us and more: the warp that copies q waits for the last one's end; and tiles of
# one stream before those of two, whose second stream's warps wait all that time
LONG = {"whole tiles": dict(new=[4864], slots=[40960]), "one stream, then two": dict(new=[128] * 18 + [256], slots=[40960] * 19)}


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("name", list(LONG))
def test_pieces_longer_than_the_limit(qkv, name, out):
    import torch
    call, want = problem(nh=8, nkv=8, hd=64, out=out, **LONG[name])
    assert call(Q.qkv_prompt_attn_step, want) == 0
    for _ in range(3):
        got = torch.full_like(want, float("nan"))
        assert call(Q.qkv_test_prompt_attn, got, wait_limit_us=100) == 0
        assert torch.equal(got, want)


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_a_plan_longer_than_the_limit(qkv, out):
    """200000 sequences, of which the first and the last have tokens: what comes before the attention does not count."""
    import torch
    torch.manual_seed(2)
    nh, nkv, hd, page, B, n = 8, 4, 64, 16, 200000, 300
    plan = make_plan(nh, nkv, hd, "f16")
    per = -(-n // page)
    k, v = (torch.randn(per, page, nkv * hd, device="cuda").half() for _ in range(2))
    table = torch.arange(per, device="cuda").int()[None].repeat(B, 1).contiguous()
    cache = Q.PagedKv(plan, k, v, table)
    first = torch.full((B + 1,), n, dtype=torch.int32, device="cuda")
    first[0], first[B] = 0, 2 * n
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    q = torch.randn(n, nh * hd, device="cuda").repeat(2, 1)
    ws = torch.empty(Q.qkv_prompt_attn_workspace_bytes(plan, cache, 2 * n), dtype=torch.uint8, device="cuda")
    o = torch.full((2 * n, nh * hd), float("nan"), dtype=dtypes(out), device="cuda")
    Q.qkv_test_prompt_attn(plan, cache, q, first, lens, hd ** -0.5, o, ws, wait_limit_us=100)
    torch.cuda.synchronize()
    assert Q.qkv_check_device_error()[0] == 0
    want = torch.empty_like(o[:n])
    one = Q.PagedKv(plan, k, v, table[:1].contiguous())
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    Q.qkv_prompt_attn_step(plan, one, q[:n], i32(0, n), i32(n), hd ** -0.5, want, ws)
    for got in (o[:n], o[n:]):  # (other CTAs may begin in the middle of a tile: the same up to the sums' order)
        assert (got.float() - want.float()).norm() <= (2.0 ** -8 if out == "bf16" else 2.0 ** -18) * want.float().norm()


@pytest.mark.parametrize("page", [64, 12])  # copied by boxes, and row by row
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_withheld_end_is_flagged(qkv, out, page):
    import torch
    call, want = problem([700], [3000], 8, 2, 128, out, page=page)
    assert call(Q.qkv_prompt_attn_step, want) == 0
    got = torch.full_like(want, 5.0)
    t0 = time.perf_counter()
    assert call(Q.qkv_test_prompt_attn, got, wait_limit_us=500, fail=1) == 2
    assert time.perf_counter() - t0 < 10.0
    assert call(Q.qkv_prompt_attn_step, got) == 0  # the context is usable, the workspace too
    assert torch.equal(got, want)


@pytest.mark.parametrize("slots,pages", [(256, 4), (640, 10)])  # where sums are rescaled; where they are added to others too
def test_one_of_two_warps_gives_up(qkv, slots, pages):
    """A row's two warps, which meet at barriers of their own, leave together."""
    import torch
    call, want = problem([700], [slots], 32, 8, 128, "f32", pages=pages, grow=8.0)
    assert call(Q.qkv_prompt_attn_step, want) == 0
    got = torch.full_like(want, 5.0)
    t0 = time.perf_counter()
    assert call(Q.qkv_test_prompt_attn, got, wait_limit_us=500, fail=2) == 2
    assert time.perf_counter() - t0 < 10.0
    assert call(Q.qkv_prompt_attn_step, got) == 0
    assert torch.equal(got, want)


def test_hook_refusals(qkv):
    call, o = problem([3], [40], 2, 1, 64, "f32")
    for kw in (dict(wait_limit_us=0), dict(wait_limit_us=1001), dict(fail=3), dict(fail=-1)):
        with pytest.raises(Q.QkvError):
            call(Q.qkv_test_prompt_attn, o, **kw)
