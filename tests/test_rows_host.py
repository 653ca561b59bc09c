"""Host-side checks of attention with many q rows (no GPU): refusals before any CUDA call, workspace sizes, struct layouts,
and the reference against brute force."""
import ctypes

import numpy as np
import pytest

import paged_reference
import qkv_rope_kv_gb300 as q
import rows_reference as ref
from test_paged_host import BAD_CACHES, P, _call, cache, plan


@pytest.fixture(scope="module")
def lib():
    return q.load()


def prompt(lib, pl, c, **kw):
    a = dict(q=P, q_stride=256, first=P, lens=P, out=P << 9, out_stride=256, lse=None, ws=P, ws_bytes=1 << 40, scale=0.125,
             window=0, out_dtype=q.QKV_F32, nt=5)
    return _call(lib.qkv_prompt_attn_step, pl, c, q._PROMPT_ARGS, {**a, **kw}.values())


def prefix(lib, pl, c, **kw):
    a = dict(q=P, q_stride=256, lens=P, share=P, prefix=P, out=P << 9, out_stride=256, lse=None, ws=P, ws_bytes=1 << 40,
             scale=0.125, out_dtype=q.QKV_F32)
    return _call(lib.qkv_prefix_attn_step, pl, c, q._PREFIX_ARGS, {**a, **kw}.values())


@pytest.mark.parametrize("bad", BAD_CACHES, ids=str)
def test_bad_caches_are_refused(lib, bad):
    pl, c = plan(), cache(**bad)
    for call in (prompt, prefix):
        assert call(lib, pl, c) == q.QKV_ERR_INVALID_ARG
        assert call(lib, None, cache()) == call(lib, pl, None) == q.QKV_ERR_INVALID_ARG
    for fn in (lib.qkv_prompt_attn_step, lib.qkv_prefix_attn_step):
        assert fn(pl.handle, ctypes.byref(cache()), None, None) == q.QKV_ERR_INVALID_ARG


BOTH = [(dict(q=None), 1), (dict(out=None), 1), (dict(lens=None), 1), (dict(q_stride=255), 1), (dict(out_stride=255), 1),
        (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1), (dict(ws=None), 1), (dict(ws=P + 8), 1),
        (dict(ws_bytes=1024), 1), (dict(out_dtype=q.QKV_F16), 2), (dict(out_dtype=7), 2), (dict(out=(P << 9) + 2), 1),
        (dict(lse=P + 2), 1), (dict(lens=P + 2), 1), (dict(q=P + 2), 1), (dict(out=P), 1), (dict(out=P + 4 * (2 * 256 + 255)), 1)]


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(first=None), 1), (dict(first=P + 1), 1), (dict(window=-1), 1), (dict(nt=-1), 1), (dict(nt=(1 << 28) + 1), 1),
    (dict(nt=0), 0), (dict(nt=0, q=None, out=None, first=None, lens=None, ws=None), 0),
], ids=str)
def test_prompt_refusals(lib, kw, status):
    assert prompt(lib, plan(), cache(), **kw) == status


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(share=None), 1), (dict(prefix=None), 1), (dict(share=P + 2), 1), (dict(prefix=P + 1), 1),
], ids=str)
def test_prefix_refusals(lib, kw, status):
    assert prefix(lib, plan(), cache(), **kw) == status


def test_uneven_groups_are_refused(lib):
    n = ctypes.c_size_t()
    assert prompt(lib, plan(n_head=5), cache(), q_stride=999, out_stride=999) == q.QKV_ERR_UNSUPPORTED
    assert prefix(lib, plan(n_head=5), cache(), q_stride=999, out_stride=999) == q.QKV_ERR_UNSUPPORTED
    c = ctypes.byref(cache())
    assert lib.qkv_prompt_attn_workspace_bytes(plan(n_head=5).handle, c, 3, ctypes.byref(n)) == q.QKV_ERR_UNSUPPORTED
    assert lib.qkv_prefix_attn_workspace_bytes(plan(n_head=5).handle, c, ctypes.byref(n)) == q.QKV_ERR_UNSUPPORTED


def test_workspace_sizes(lib):
    pl, c, n = plan(), cache(), ctypes.c_size_t()
    size = lambda nt: (lib.qkv_prompt_attn_workspace_bytes(pl.handle, ctypes.byref(c), nt, ctypes.byref(n)), n.value)  # noqa: E731
    few, many = size(5), size(100000)
    assert few[0] == many[0] == 0 and few[1] < many[1] and few[1] % 256 == 0
    assert prompt(lib, pl, c, ws_bytes=few[1] - 1) == q.QKV_ERR_INVALID_ARG
    assert size(-1)[0] == q.QKV_ERR_INVALID_ARG
    assert lib.qkv_prompt_attn_workspace_bytes(pl.handle, ctypes.byref(c), 5, None) == q.QKV_ERR_INVALID_ARG
    assert lib.qkv_prompt_attn_workspace_bytes(None, ctypes.byref(c), 5, ctypes.byref(n)) == q.QKV_ERR_INVALID_ARG
    assert lib.qkv_prefix_attn_workspace_bytes(pl.handle, ctypes.byref(c), ctypes.byref(n)) == 0
    assert prefix(lib, pl, c, ws_bytes=n.value - 1) == q.QKV_ERR_INVALID_ARG
    assert lib.qkv_prefix_attn_workspace_bytes(pl.handle, None, ctypes.byref(n)) == q.QKV_ERR_INVALID_ARG
    assert lib.qkv_prefix_attn_workspace_bytes(pl.handle, ctypes.byref(c), None) == q.QKV_ERR_INVALID_ARG


def test_args_layouts_match_the_header(tmp_path):
    import os
    import subprocess
    fields = {"qkv_prompt_attn_args": ("q q_stride d_first d_lens out out_stride lse d_workspace workspace_bytes scale window "
                                       "out_dtype nt", q._PROMPT_ARGS),
              "qkv_prefix_attn_args": ("q q_stride d_lens d_share d_prefix_len out out_stride lse d_workspace "
                                       "workspace_bytes scale out_dtype", q._PREFIX_ARGS)}
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
        for i in range(len(offsets)):
            values = [0] * len(offsets)
            values[i] = 1
            data = layout.pack(*values)
            assert min(k for k, byte in enumerate(data) if byte) - int(offsets[i]) in (0, 2), (name, names.split()[i])


def test_reference_against_brute_force():
    rng = np.random.default_rng(0)
    c = paged_reference.Cache(rng, 3, 1, 4, "f32", 3, 4, lens=[7, 2, 5])
    x = rng.standard_normal((9, 8)).astype(np.float32)
    first = [1, 4, 8, 8]  # three tokens, four of which two see nothing, none; rows 0 and 8 belong to nobody
    places = ref.prompt_places(c, first, c.lens, 9, 4)
    assert places[0] is None and places[8] is None
    assert [len(p[0]) for p in places[1:8]] == [4, 4, 4, 0, 0, 1, 2]
    out, lse, *_ = ref.rows_ref(c.k, c.v, x[1:8], places[1:8], 0.5, 2, 1, 4, False)
    row, seen = 2, [c.row(0, j) for j in (3, 4, 5, 6)]  # the last of the first sequence: slots 3 to 6
    for h in range(2):
        s = [0.5 * sum(float(x[3, h * 4 + d]) * float(c.k[r][d]) for d in range(4)) for r in seen]
        e = np.exp(s)
        assert np.isclose(lse[row, h], np.log(e.sum()))
        for d in range(4):
            assert np.isclose(out[row, h * 4 + d], sum(e[i] * float(c.v[r][d]) for i, r in enumerate(seen)) / e.sum())
    assert not out[3].any() and lse[3, 0] == -np.inf
    share = ref.prefix_places(c, [5, 2, 4], [0, 0, 0], [3, 3, 1])
    assert [list(zip(*p)) for p in share] == [[c.row(0, s) for s in range(5)], [c.row(0, 0), c.row(0, 1)],
                                              [c.row(0, 0), c.row(2, 1), c.row(2, 2), c.row(2, 3)]]
