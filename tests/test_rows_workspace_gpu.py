"""One workspace for the attention of one token, of many and over shared beginnings, in turn."""
import numpy as np
import pytest

import qkv_rope_kv_gb300 as Q
import rows_reference as ref
from test_paged_gpu import make_plan
from test_rows_gpu import attend64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["f16", "f32"])
def test_calls_of_all_kinds_take_turns(qkv, kv):
    """Sequences that are split over many CTAs: prompts of many and of few tokens, a decode step, one over a shared prefix,
    captured on one workspace and replayed in changing orders."""
    import torch
    torch.manual_seed(0)
    nh, nkv, hd, page, P = 28, 4, 128, 16, 3200
    G, lens = nh // nkv, [9000, 4100]
    plan = make_plan(nh, nkv, hd, kv)
    dt = torch.float16 if kv == "f16" else torch.float32
    per = -(-max(lens) // page)
    k, v = (torch.randn(2 * per, page, nkv * hd, device="cuda").to(dt) for _ in range(2))
    table = torch.randperm(2 * per, device="cuda").int().view(2, per)
    table[1, :P // page] = table[0, :P // page]
    table = table.contiguous()
    cache = Q.PagedKv(plan, k, v, table)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    n = max(Q.qkv_prompt_attn_workspace_bytes(plan, cache, 300), Q.qkv_prefix_attn_workspace_bytes(plan, cache),
            Q.qkv_attn_workspace_bytes(plan, cache))
    ws = torch.full((n,), 0xa5, dtype=torch.uint8, device="cuda")
    ws[:4096] = 0
    scale, L = hd ** -0.5, i32(*lens)
    steps = []
    stream = torch.cuda.Stream()
    for name, out, new in (("prompt", "bf16", (200, 100)), ("prompt", "f32", (3, 2)), ("attn", "f32", (1, 1)),
                           ("prefix", "f32", (1, 1)), ("prefix", "bf16", (1, 1))):
        nt = sum(new)
        q = torch.randn(nt, nh * hd, device="cuda")
        o = torch.empty(nt, nh * hd, device="cuda", dtype=torch.bfloat16 if out == "bf16" else torch.float32)
        first, share, prefix = i32(0, new[0], nt), i32(0, 0), i32(P, P)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
            if name == "prompt":
                Q.qkv_prompt_attn_step(plan, cache, q, first, L, scale, o, ws)
            elif name == "attn":
                Q.qkv_attn_step(plan, cache, q, L, scale, o, ws)
            else:
                Q.qkv_prefix_attn_step(plan, cache, q, L, share, prefix, scale, o, ws)
        single = out == "bf16" and kv == "f16"
        want, bound = [], []
        for b in range(2):
            K, V = (x[table[b].long()].view(-1, nkv, hd)[:lens[b]] for x in (k, v))
            rows = q.view(nt, nkv, G, hd)[sum(new[:b]):sum(new[:b + 1])]
            hi = torch.arange(lens[b] - new[b] + 1, lens[b] + 1, device="cuda")
            w, e = torch.empty_like(rows, dtype=torch.float64), torch.empty_like(rows, dtype=torch.float64)
            for h in range(nkv):
                w[:, h], most, size = attend64(rows[:, h], K[:, h], V[:, h], hi, scale)
                ds = (hd + 16) * 2 * ref.U * size + (2.0 ** -11 * size if single else 0)
                e[:, h] = (torch.expm1(2 * ds) + (lens[b] / 8 + 64) * 2 * ref.U + (2.0 ** -11 if single else 0)) * most
            want.append(w)
            bound.append(e + (2.0 ** -8 * (w.abs() + e) if out == "bf16" else 0))
        steps.append((name, graph, o, torch.cat(want).view(nt, -1), torch.cat(bound).view(nt, -1), (q, first, share, prefix)))
    rng = np.random.default_rng(1)
    for _ in range(6):
        order = rng.permutation(len(steps))
        for i in order:
            steps[i][2].fill_(float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            for i in order:
                steps[i][1].replay()
        stream.synchronize()
        for name, _, o, want, bound, _ in steps:
            assert ((o.double() - want).abs() <= bound).all(), name
    assert Q.qkv_check_device_error()[0] == 0


@pytest.mark.parametrize("kv", ["f16", "f32"])
def test_a_prompt_leaves_the_counters(qkv, kv):
    import torch
    plan = make_plan(8, 2, 64, kv)
    k, v = (torch.randn(50, 16, 128, device="cuda").to(torch.float16 if kv == "f16" else torch.float32) for _ in range(2))
    cache = Q.PagedKv(plan, k, v, torch.arange(50, device="cuda").int()[None].contiguous())
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q, o = (torch.randn(300, 512, device="cuda") for _ in range(2))
    ws = torch.arange(Q.qkv_prompt_attn_workspace_bytes(plan, cache, 300), device="cuda").to(torch.uint8)
    before = ws[:4096].clone()
    Q.qkv_prompt_attn_step(plan, cache, q, i32(0, 300), i32(800), 0.125, o, ws)
    torch.cuda.synchronize()
    assert torch.equal(ws[:4096], before)
