"""Decode steps of several host threads at once, each with a layer width, stream and buffers of its own."""
import threading

import pytest

import qkv_rope_kv_gb300 as Q

pytestmark = pytest.mark.gpu


# Widths of one kernel that need different amounts of shared memory: rings of long, middle and short rows, and rows of
# no whole 16 bytes, whose x is staged.
@pytest.mark.parametrize("widths,w_dtype", [((4096, 6144, 8192), "bf16"), ((2048, 2304), "bf16"), ((512, 960), "f32"),
                                            ((13001, 20003), "f32")], ids=str)
def test_widths_from_several_threads(qkv, widths, w_dtype):
    import torch
    nh, nkv, hd, n_ctx = 4, 2, 64, 8
    gen = torch.Generator(device="cuda").manual_seed(31)
    rows = (nh + 2 * nkv) * hd
    works, outs, raised = [], [], []
    start = threading.Barrier(len(widths))
    pos = torch.tensor([3], dtype=torch.int32, device="cuda")
    for H in widths:
        plan = Q.qkv_plan_create(H, nh, nkv, hd, 1e6, n_ctx, w_dtype=Q.QKV_BF16 if w_dtype == "bf16" else Q.QKV_F32)
        w = 0.02 * torch.randn(rows, H, generator=gen, device="cuda")
        w = w.to(torch.bfloat16) if w_dtype == "bf16" else w
        x, bias = (torch.randn(n, generator=gen, device="cuda") for n in (H, rows))
        kv = [torch.zeros(n_ctx, nkv * hd, dtype=torch.float16, device="cuda") for _ in range(2)]
        pair = [torch.zeros(rows, device="cuda") for _ in range(2)]
        cut = [(o[:nh * hd], o[nh * hd:(nh + nkv) * hd], o[(nh + nkv) * hd:]) for o in pair]
        Q.qkv_decode_step(plan, x, w, bias, pos, *cut[0], *kv)  # alone
        stream = torch.cuda.Stream()

        def work(plan=plan, a=(plan.handle, *[t.data_ptr() for t in (x, w, bias, pos, *cut[1], *kv)], stream.cuda_stream),
                 keep=(x, w, bias, cut, kv, stream)):
            call = Q.load().qkv_decode_step  # the bare entry point: the threads meet in it more often
            start.wait()
            raised.append(sum(call(*a) != Q.QKV_OK for _ in range(10000)))
        works.append(work)
        outs.append(pair)
    torch.cuda.synchronize()
    threads = [threading.Thread(target=w) for w in works]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert raised == [0] * len(widths)
    for alone, together in outs:
        assert torch.equal(alone, together) and alone.abs().sum().item() > 0
    assert Q.qkv_check_device_error()[0] == 0
