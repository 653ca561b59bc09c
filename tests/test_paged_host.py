"""Host-side checks of the paged-cache entry points (no GPU): every refusal comes before any
CUDA call, workspace sizes, and the reference forms against brute force."""
import ctypes

import numpy as np
import pytest

import paged_reference as ref
import qkv_rope_kv_gb300 as q

P = 4096  # a plausible, never dereferenced, aligned address


@pytest.fixture(scope="module")
def lib():
    return q.load()


def plan(**kw):
    base = dict(hidden=64, n_head=4, n_head_kv=2, head_dim=64, theta=1e6, n_ctx=64)
    base.update(kw)
    return q.qkv_plan_create(**base)


def cache(**kw):
    base = dict(k=P, v=P << 8, page_table=P, n_pages=8, page_size=16, n_seq=3, max_pages=4, page_stride=0,
                slot_weight=P << 12, slot_pos=P << 13)
    base.update(kw)
    return q.qkv_paged_kv(*[base[f] for f, _ in q.qkv_paged_kv._fields_])


BAD_CACHES = [dict(k=None), dict(v=None), dict(page_table=None), dict(n_pages=0), dict(page_size=0), dict(n_seq=0),
              dict(max_pages=0), dict(max_pages=1 << 28, page_size=8), dict(max_pages=(1 << 30) + 1, page_size=1), dict(page_stride=16 * 128 - 1), dict(k=P + 1),
              dict(page_table=P + 2), dict(slot_pos=P + 1), dict(n_seq=1 << 23), dict(page_stride=-5)]


def _call(fn, pl, c, layout, values):
    """The entry point on an args struct (None among the values: a null pointer)."""
    args = layout.pack(*[0 if v is None else v for v in values])
    return fn(pl.handle if pl else None, ctypes.byref(c) if c else None, args, None)


def store(lib, pl, c, **kw):
    a = dict(Y=P << 4, y_stride=512, y_dtype=q.QKV_F32, nt=3, bias=P, qw=P, kw=P, pos=P, seqs=P, slots=P, q=P << 5,
             q_stride=256, eps=1e-6)
    return _call(lib.qkv_paged_store_step, pl, c, q._STORE_ARGS, {**a, **kw}.values())


def attn(lib, pl, c, **kw):
    a = dict(q=P, q_stride=256, lens=P, out=P << 7, out_stride=256, lse=None, ws=P, ws_bytes=1 << 40, scale=0.125,
             window=0, out_dtype=q.QKV_F32, add=0)
    return _call(lib.qkv_attn_step, pl, c, q._ATTN_ARGS, {**a, **kw}.values())


def evict(lib, pl, c, **kw):
    a = dict(lens=P, next=P, lens_out=P << 6, w=P << 12, pos=P << 13, ws=P, ws_bytes=1 << 40, budget=8, recent=2)
    return _call(lib.qkv_evict_step, pl, c, q._EVICT_ARGS, {**a, **kw}.values())


def test_null_args_are_refused(lib):
    for fn in (lib.qkv_paged_store_step, lib.qkv_attn_step, lib.qkv_evict_step):
        assert fn(plan().handle, ctypes.byref(cache()), None, None) == q.QKV_ERR_INVALID_ARG


def test_args_layouts_match_the_header(tmp_path):
    """The packed layouts have the sizes and field offsets that a C compiler gives the header's structs."""
    import os
    import subprocess
    fields = {"qkv_paged_store_args": ("Y y_stride y_dtype nt bias q_norm_w k_norm_w d_positions d_seqs d_slots q "
                                       "q_stride eps", q._STORE_ARGS),
              "qkv_attn_args": ("q q_stride d_lens out out_stride lse d_workspace workspace_bytes scale window "
                                "out_dtype add_weight", q._ATTN_ARGS),
              "qkv_evict_args": ("d_lens d_next_pos lens_out weight_out pos_out d_workspace workspace_bytes budget "
                                 "recent", q._EVICT_ARGS)}
    lines = ['printf("%s %%zu", sizeof(%s));%s puts("");' % (n, n, "".join(
        'printf(" %%zu", offsetof(%s, %s));' % (n, f) for f in fs.split())) for n, (fs, _) in fields.items()]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include "qkv.h"\nint main(void) {%s return 0; }\n' % "".join(lines))
    exe = str(tmp_path / "layout")
    subprocess.check_call(["gcc", "-I", os.path.dirname(q.HEADER), "-o", exe, str(src)])
    for line in subprocess.check_output([exe], text=True).splitlines():
        name, size, *offsets = line.split()
        names, layout = fields[name]
        assert layout.size == int(size)
        for i in range(len(offsets)):  # each field alone non-zero shows where it is packed
            values = [0] * len(offsets)
            values[i] = 1
            data = layout.pack(*values)
            assert min(k for k, byte in enumerate(data) if byte) - int(offsets[i]) in (0, 2), (name, names.split()[i])


@pytest.mark.parametrize("bad", BAD_CACHES, ids=str)
def test_bad_caches_are_refused(lib, bad):
    pl, c = plan(), cache(**bad)
    for call in (store, attn, evict):
        assert call(lib, pl, c) == q.QKV_ERR_INVALID_ARG
        assert lib.qkv_last_error()
        assert call(lib, None, cache()) == call(lib, pl, None) == q.QKV_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,status", [
    (dict(Y=None), 1), (dict(q=None), 1), (dict(pos=None), 1), (dict(y_stride=511), 1), (dict(q_stride=255), 1),
    (dict(nt=-1), 1), (dict(qw=None), 1), (dict(kw=None), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(seqs=None, nt=4), 1), (dict(y_dtype=q.QKV_F16), 2), (dict(y_dtype=9), 2), (dict(Y=P + 2), 1),
    (dict(bias=P + 1), 1), (dict(q=(P << 4) + 256), 1), (dict(q=P << 4), 1),
    (dict(q=P << 4, y_dtype=q.QKV_BF16, q_stride=512), 1), (dict(nt=0), 0), (dict(nt=0, seqs=None, slots=None), 0),
], ids=str)
def test_store_refusals(lib, kw, status):
    assert store(lib, plan(), cache(), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(lens=None), 1), (dict(out=None), 1), (dict(q_stride=255), 1), (dict(out_stride=1), 1),
    (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1), (dict(window=-1), 1), (dict(ws=None), 1),
    (dict(ws=P + 8), 1), (dict(ws_bytes=1024), 1), (dict(out_dtype=q.QKV_F16), 2), (dict(out=(P << 7) + 2), 1),
    (dict(lse=P + 2), 1), (dict(out=P), 1), (dict(out=P + 4 * (2 * 256 + 255)), 1), (dict(out=P - 4 * 767), 1),
], ids=str)
def test_attn_refusals(lib, kw, status):
    assert attn(lib, plan(), cache(), **kw) == status


def test_attn_refuses_uneven_groups_and_untracked_weights(lib):
    assert attn(lib, plan(n_head=5), cache(), q_stride=999, out_stride=999) == q.QKV_ERR_UNSUPPORTED
    assert attn(lib, plan(), cache(slot_weight=None), add=1) == q.QKV_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(lens=None), dict(next=None), dict(lens_out=None), dict(w=None), dict(pos=None), dict(budget=0),
    dict(recent=-1), dict(recent=9), dict(lens_out=P), dict(lens_out=P + 8), dict(w=(P << 12) + 4),
    dict(pos=(P << 13) - 4), dict(ws=None), dict(ws_bytes=16), dict(ws=P + 2), dict(w=P + 1),
], ids=str)
def test_evict_refusals(lib, kw):
    assert evict(lib, plan(), cache(), **kw) == q.QKV_ERR_INVALID_ARG


def test_evict_needs_a_tracked_cache(lib):
    for bad in (dict(slot_weight=None), dict(slot_pos=None)):
        assert evict(lib, plan(), cache(**bad)) == q.QKV_ERR_INVALID_ARG


def test_workspace_sizes(lib):
    pl, n = plan(), ctypes.c_size_t()
    assert lib.qkv_attn_workspace_bytes(pl.handle, ctypes.byref(cache()), ctypes.byref(n)) == 0
    tracked = n.value
    assert lib.qkv_attn_workspace_bytes(pl.handle, ctypes.byref(cache(slot_weight=None)), ctypes.byref(n)) == 0
    assert tracked - n.value >= 4 * 3 * 4 * 64 and n.value % 256 == 0
    assert attn(lib, pl, cache(slot_weight=None), ws_bytes=n.value - 1) == q.QKV_ERR_INVALID_ARG
    assert lib.qkv_evict_workspace_bytes(pl.handle, ctypes.byref(cache()), ctypes.byref(n)) == 0
    assert n.value == 4 * 3 * 2 * (1 + 64)  # a count and two half lists for each sequence and kv head
    assert lib.qkv_evict_workspace_bytes(pl.handle, ctypes.byref(cache()), None) == q.QKV_ERR_INVALID_ARG
    assert lib.qkv_attn_workspace_bytes(None, ctypes.byref(cache()), ctypes.byref(n)) == q.QKV_ERR_INVALID_ARG


def test_python_refuses_what_its_tensors_show():
    torch = pytest.importorskip("torch")
    pl = plan(kv_dtype=q.QKV_F16)
    k = torch.zeros(8, 16, 128, dtype=torch.float16)
    table = torch.zeros(3, 4, dtype=torch.int32)
    for args in ((k, k, table), (k[0], k, table), (k, k, table[0])):
        with pytest.raises(q.QkvError):
            q.PagedKv(pl, *args)


def test_reference_attention_against_brute_force():
    rng = np.random.default_rng(0)
    c = ref.Cache(rng, 2, 2, 4, "f32", 3, 3, lens=[7, 0])
    x = rng.standard_normal((2, 16)).astype(np.float32)
    out, lse, weight, *_ = ref.attn_ref(c, x, c.lens, 0.5, 5, 4)
    for h in range(4):
        s = [0.5 * sum(float(x[0, h * 4 + d]) * float(c.k[c.row(0, j)][h // 2 * 4 + d]) for d in range(4))
             for j in range(2, 7)]
        e = np.exp(s)
        assert np.isclose(lse[0, h], np.log(e.sum()))
        for d in range(4):
            assert np.isclose(out[0, h * 4 + d], sum(e[i] * float(c.v[c.row(0, 2 + i)][h // 2 * 4 + d])
                                                     for i in range(5)) / e.sum())
    assert np.isclose(weight[0, 0].sum(), 2) and not weight[0, :, :2].any() and not out[1].any()


def test_reference_eviction_on_a_worked_example():
    rng = np.random.default_rng(1)
    c = ref.Cache(rng, 1, 1, 2, "f32", 4, 2, lens=[7])
    w = np.array([[[5, 1, 1, 9, 1, 7, 0, 0]]], np.float32)
    pos = np.array([[[0, 1, 2, 3, 4, 5, 6, -1]]], np.int32)
    k, v, n, w2, p2 = ref.evict_ref(c, c.lens, [7], w, pos, 4, 1)
    # kept: 6 (newest), 3, 5, 0; slots 1 and 2 are free and take 5 and 6
    assert list(n) == [4] and list(p2[0, 0, :4]) == [0, 5, 6, 3] and list(w2[0, 0, :4]) == [5, 7, 0, 9]
    assert np.array_equal(k[c.row(0, 1)], c.k[c.row(0, 5)]) and np.array_equal(v[c.row(0, 2)], c.v[c.row(0, 6)])
    # equal weights: the lowest slots stay (budget 3 of the slots 1, 2, 4 and the newest)
    w[0, 0, [0, 3, 5]] = 0
    _, _, _, _, p2 = ref.evict_ref(c, c.lens, [7], w, pos, 3, 1)
    assert list(p2[0, 0, :3]) == [6, 1, 2]
