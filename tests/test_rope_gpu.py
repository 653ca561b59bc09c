"""Rotations of a qkv_rope on the GPU, alone and in the paged store, against their 64-bit form
(rope_reference.py, which derives the bounds)."""
import numpy as np
import pytest

import paged_reference
import qkv_rope_kv_gb300 as Q
import rope_reference as ref
from test_paged_gpu import EPS, KV, close, dev, make_plan, short

pytestmark = pytest.mark.gpu

NAMES = [f["scaling"] for f in ref.FORMS]


def dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def run_rope(nt, heads, hd, rot, neighbours, form, dtype, inverse=False, offset=0, positions=None, in_place=False, seed=0):
    import torch
    rng = np.random.default_rng(seed)
    rope, f = ref.create(Q, hd, rot, neighbours, 1e6, ref.FORMS[NAMES.index(form)])
    magnitude = ref.FORMS[NAMES.index(form)].get("magnitude", 1.0)
    flat = torch.from_numpy(rng.standard_normal((nt, heads * hd + offset)).astype(np.float32)).cuda().to(dt(dtype))
    x, ahead = flat[:, offset:], flat[:, :offset].clone()
    pos = np.asarray(rng.integers(0, 200000, nt) if positions is None else positions, np.int32)
    want, bound = ref.turn(x.float().cpu().numpy().reshape(nt, heads, hd), pos, f, rot, neighbours, magnitude, inverse)
    bound = ref.rounded(bound, want, dtype)
    bound[..., rot:] = 0  # what passes keeps its bits
    out = x if in_place else torch.full((nt, heads * hd + 2 * offset), 9.0, dtype=dt(dtype), device="cuda")[
        :, :heads * hd] if offset else torch.empty(nt, heads * hd, dtype=dt(dtype), device="cuda")
    Q.qkv_rope_step(rope, x, dev(pos), out, inverse=inverse)
    torch.cuda.synchronize()
    close(out.float().cpu().numpy().reshape(nt, heads, hd), want, bound, "turned")
    assert torch.equal(flat[:, :offset], ahead)


@pytest.mark.parametrize("nt,heads,hd,rot,neighbours,form,dtype,kw", [
    (1, 16, 64, 64, False, "none", "f32", {}),
    (1, 1, 2, 2, True, "none", "f32", {}),
    (7, 3, 128, 128, True, "ramp", "bf16", {}),
    (7, 3, 128, 64, False, "bands", "f16", {}),
    (33, 5, 128, 64, True, "linear", "f32", {}),
    (33, 5, 80, 40, False, "base", "bf16", {}),
    (9, 5, 80, 20, False, "table", "f32", {}),           # quads that would straddle the end of the turned part
    (9, 5, 80, 20, True, "table", "f16", {}),
    (5, 2, 7, 4, False, "none", "bf16", {}),             # an odd head
    (5, 2, 9, 2, True, "none", "f32", {}),
    (2501, 11, 128, 128, False, "ramp", "f32", {}),      # enough rows for several heads a thread, the last group short
    (2501, 11, 128, 32, True, "none", "bf16", {}),
    (2501, 13, 96, 96, False, "bands", "f16", dict(inverse=True)),
    (40, 4, 256, 256, True, "ramp", "f32", dict(inverse=True)),
    (40, 4, 64, 32, False, "linear", "f32", dict(offset=1)),
    (40, 4, 64, 64, True, "linear", "bf16", dict(offset=4)),
    (40, 4, 64, 64, False, "linear", "f16", dict(offset=3)),
    (40, 4, 64, 64, False, "none", "f32", dict(in_place=True)),
    (2501, 9, 128, 128, True, "none", "bf16", dict(in_place=True, offset=8)),
    (4, 4, 64, 64, False, "none", "f32", dict(positions=[0, -1, 2 ** 24 + 1, -2 ** 20])),
], ids=short)
def test_rope(qkv, nt, heads, hd, rot, neighbours, form, dtype, kw):
    run_rope(nt, heads, hd, rot, neighbours, form, dtype, **kw)


def test_far_positions_keep_their_angle(qkv):
    """At the ends of int32 the angle is still that of the exact product (decimal arithmetic)."""
    import decimal
    import torch
    decimal.getcontext().prec = 60
    pi = decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494")
    pos = [2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, -1999999999, 16777217]
    rope = Q.qkv_rope_create(128, 1e6)
    f = rope.freqs()
    x = torch.zeros(len(pos), 128, device="cuda")
    x[:, :64] = 1.0
    out = torch.empty_like(x)
    Q.qkv_rope_step(rope, x, torch.tensor(pos, dtype=torch.int32, device="cuda"), out)
    got = out.double().cpu().numpy()
    for i, p in enumerate(pos):
        angle = np.array([float((decimal.Decimal(p) * decimal.Decimal(v)).remainder_near(2 * pi)) for v in f])
        # a turn a position is kept to half a unit of 2^-64: 2^31 positions of it are 2^-34 turns
        assert np.abs(got[i, :64] - np.cos(angle)).max() < 7 * ref.U and np.abs(got[i, 64:] - np.sin(angle)).max() < 7 * ref.U


@pytest.mark.parametrize("neighbours", [False, True])
def test_inverse_is_the_gradient(qkv, neighbours):
    """For a loss sum(w * out), inverse turns w into the differences of the loss by every x."""
    import torch
    rng = np.random.default_rng(4)
    form = ref.FORMS[NAMES.index("ramp")]
    rope, f = ref.create(Q, 16, 8, neighbours, 1e4, form)
    x, w = rng.standard_normal((2, 3, 2, 16))
    pos = np.array([3, 70000, 11], np.int32)
    turn = lambda v: ref.turn(v, pos, f, 8, neighbours, form["magnitude"])[0]  # noqa: E731
    grad = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        step = np.zeros_like(x)
        step[i] = 1.0  # linear: any step
        grad[i] = (w * (turn(x + step) - turn(x))).sum()
    w32 = w.astype(np.float32)
    out = torch.empty(3, 32, device="cuda")
    Q.qkv_rope_step(rope, dev(w32.reshape(3, 32)), dev(pos), out, inverse=True)
    # the bound of a turned value, of |w| up to 4, and w's own rounding
    assert np.abs(out.cpu().numpy().reshape(grad.shape) - grad).max() < 10 * ref.U * form["magnitude"] * 8
    Q.qkv_rope_step(rope, out, dev(pos), out)
    back = form["magnitude"] ** 2 * w32[..., :8]
    assert np.abs(out.cpu().numpy().reshape(w.shape)[..., :8] - back).max() < 20 * ref.U * form["magnitude"] ** 2 * 8


def test_agrees_with_the_plans_rotation_nearby(qkv):
    """Unscaled halves are the plan's rotation up to the rounding of its f32 angle: 2^-24 of it."""
    import torch
    plan = make_plan(4, 2, 64, "f32")
    rope = Q.qkv_rope_create(64, 1e6)
    x = torch.randn(1, 256, device="cuda")
    pos = torch.tensor([100], dtype=torch.int32, device="cuda")
    a, b = x.clone(), torch.empty_like(x)
    Q.qkv_chain_rope(plan, a, 4, pos)
    Q.qkv_rope_step(rope, x, pos, b)
    assert (a - b).abs().max().item() < 2 * (100 + 8) * 2 * ref.U * x.abs().max().item()


def run_store(nh, nkv, hd, rot, neighbours, form, kv, page, y, norm, nt, with_bias=True, y_off=0, in_place=False, seed=0,
              positions=None):
    import torch
    rng = np.random.default_rng(seed)
    B, cap = 3, 5 * page
    c = paged_reference.Cache(rng, B, nkv, hd, kv, page, 5, fill=7.0)
    R = (nh + 2 * nkv) * hd
    plan = make_plan(nh, nkv, hd, kv)
    rope, f = ref.create(Q, hd, rot, neighbours, 1e6, ref.FORMS[NAMES.index(form)])
    magnitude = ref.FORMS[NAMES.index(form)].get("magnitude", 1.0)
    Y = torch.from_numpy(rng.standard_normal((nt, R + y_off)).astype(np.float32)).cuda()[:, y_off:].to(dt(y))
    bias = rng.standard_normal(R).astype(np.float32) if with_bias else None
    qw, kw = (rng.standard_normal((2, hd)).astype(np.float32) if norm else (None, None))
    pos = (rng.integers(0, 200000, nt) if positions is None else np.asarray(positions)).astype(np.int32)
    at = rng.choice(B * cap, nt, replace=False)
    seqs, slots = (at // cap).astype(np.int32), (at % cap).astype(np.int32)
    pad = rng.random(nt) < 0.2
    seqs[pad] = -1 - rng.integers(0, 5, pad.sum())
    k, v = dev(c.k), dev(c.v)
    weight = torch.full((B, nkv, cap), 3.0, device="cuda")
    spos = torch.full((B, nkv, cap), -9, dtype=torch.int32, device="cuda")
    cache = Q.PagedKv(plan, k, v, dev(c.table), slot_weight=weight, slot_pos=spos)
    opt = lambda a: None if a is None else dev(a)  # noqa: E731
    Y0 = Y.float().cpu().numpy()
    q = Y[:, :nh * hd] if in_place else torch.full((nt, nh * hd), -5.0, device="cuda")
    Q.qkv_paged_store_rope_step(plan, cache, rope, Y, opt(bias), opt(qw), opt(kw), EPS, dev(pos), dev(seqs), dev(slots), q)
    torch.cuda.synchronize()
    assert Q.qkv_check_device_error()[0] == 0
    z = (Y0.astype(np.float64) + (0 if bias is None else bias)).reshape(nt, nh + 2 * nkv, hd)
    x, wv = z[:, :nh + nkv], z[:, nh + nkv:].reshape(nt, -1)
    if norm:
        w = np.concatenate([np.tile(qw, (nh, 1)), np.tile(kw, (nkv, 1))]).astype(np.float64)
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + EPS) * w
    want, bound = ref.turn(x, pos, f, rot, neighbours, magnitude)
    # values before the turn: one rounding of the bias's sum, or 18 u with a norm (paged_reference.py)
    ahead = 18 if norm else 1
    bound = bound + ahead * ref.U * (magnitude * bound / (7 * ref.U * magnitude))
    bound[..., rot:] = ahead * ref.U * np.abs(want[..., rot:]) + 1e-37
    got = q.cpu().numpy().reshape(nt, nh, hd)
    if not in_place:
        assert (got[pad] == -5.0).all()
    close(got[~pad], want[~pad, :nh], bound[~pad, :nh], "q")
    K, V = c.k.astype(np.float64), c.v.astype(np.float64)
    bK, bV = np.zeros_like(K), np.zeros_like(V)
    half = lambda t: paged_reference.f16_half_step(t) * (1 + 2.0 ** -10) if kv == "f16" else 0.0  # noqa: E731
    wk, wb = want[:, nh:].reshape(nt, -1), bound[:, nh:].reshape(nt, -1)
    ww, wp = np.full((B, nkv, cap), 3.0), np.full((B, nkv, cap), -9)
    for t in np.flatnonzero(~pad):
        r = c.row(seqs[t], slots[t])
        K[r], V[r], bK[r] = wk[t], wv[t], wb[t] + half(wk[t])
        bV[r] = np.abs(wv[t]) * ref.U + half(wv[t])
        ww[seqs[t], :, slots[t]], wp[seqs[t], :, slots[t]] = 0, pos[t]
    close(k.cpu().numpy(), K, bK, "K pool")
    close(v.cpu().numpy(), V, bV, "V pool")
    assert np.array_equal(weight.cpu().numpy(), ww) and np.array_equal(spos.cpu().numpy(), wp)


@pytest.mark.parametrize("nh,nkv,hd,rot,neighbours,form,kv,page,y,norm,nt,kw", [
    (14, 2, 64, 64, False, "none", "f32", 16, "f32", False, 1, {}),
    (14, 2, 64, 32, True, "linear", "f32", 16, "bf16", True, 50, {}),
    (28, 4, 128, 64, True, "none", "f16", 16, "f32", False, 7, {}),
    (40, 8, 128, 128, False, "ramp", "f16", 7, "bf16", True, 33, {}),
    (40, 8, 128, 32, False, "bands", "f16", 64, "f32", True, 129, {}),
    (4, 1, 256, 256, True, "ramp", "f16", 5, "f32", True, 13, {}),
    (3, 2, 6, 4, False, "none", "f16", 4, "f32", True, 17, {}),
    (3, 2, 6, 2, True, "none", "f32", 4, "bf16", False, 17, {}),
    (6, 3, 80, 20, False, "table", "f16", 17, "f32", True, 40, {}),
    (6, 3, 80, 20, True, "table", "f32", 17, "bf16", True, 40, {}),
    (28, 4, 128, 64, False, "base", "f16", 1000, "bf16", True, 2500, {}),     # enough tokens to share CTAs
    (14, 2, 64, 64, True, "ramp", "f32", 1000, "f32", False, 2501, dict(with_bias=False)),
    (28, 4, 128, 64, True, "none", "f16", 16, "f32", True, 9, dict(y_off=1)),
    (28, 4, 128, 64, False, "none", "f16", 16, "f32", True, 9, dict(in_place=True)),
    (6, 3, 96, 48, True, "none", "f16", 16, "f32", True, 9, dict(in_place=True)),
    (28, 4, 128, 128, False, "none", "f16", 16, "f32", True, 3, dict(positions=[0, 2 ** 24 + 1, -3])),
], ids=short)
def test_store_rope(qkv, nh, nkv, hd, rot, neighbours, form, kv, page, y, norm, nt, kw):
    run_store(nh, nkv, hd, rot, neighbours, form, kv, page, y, norm, nt, **kw)


def test_captured_and_on_another_stream(qkv):
    """One graph with a rotation in place and its inverse leaves the values near where they were; replays add up."""
    import torch
    rope = Q.qkv_rope_create(128, 1e6, layout=Q.QKV_ROPE_INTERLEAVED)
    x = torch.randn(17, 5 * 128, device="cuda")
    y, pos = x.clone(), torch.arange(17, dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    Q.qkv_rope_step(rope, y, pos, y, stream=stream)
    stream.synchronize()
    once = y.clone()
    y.copy_(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Q.qkv_rope_step(rope, y, pos, y)
    for _ in range(2):
        y.copy_(x)
        graph.replay()
        assert torch.equal(y, once)
    pos.fill_(0)  # read on the device at every replay
    y.copy_(x)
    graph.replay()
    assert torch.equal(y, x)
