"""Host-side checks of qkv_rope (no GPU): frequencies, refusals before any CUDA call, struct layouts."""
import ctypes
import math

import numpy as np
import pytest

import qkv_rope_kv_gb300 as q
import rope_reference as ref

P = 4096  # a plausible, never dereferenced, aligned address


@pytest.fixture(scope="module")
def lib():
    return q.load()


@pytest.mark.parametrize("form", ref.FORMS, ids=lambda f: f["scaling"])
@pytest.mark.parametrize("hd,rot,theta", [(128, 128, 1e6), (64, 32, 1e4), (256, 64, 5e5), (80, 20, 1e4), (6, 4, 7.0)])
def test_frequencies(lib, hd, rot, theta, form):
    rope, want = ref.create(q, hd, rot, False, theta, form)
    # pow, log and a handful of products in 64 bits; the ramp's ends are whole numbers on either way
    assert np.allclose(rope.freqs(), want, rtol=1e-13, atol=0)


def test_the_scaled_forms_keep_what_they_should():
    """Fast pairs of the ramp and the bands keep their frequency, slow ones are divided; base leaves the fastest."""
    plain = ref.freqs(128, 1e6)
    for name, form in ((f["scaling"], f) for f in ref.FORMS if f["scaling"] in ("ramp", "bands")):
        f = ref.freqs(128, 1e6, **form)
        assert f[0] == plain[0] and math.isclose(f[-1], plain[-1] / form["factor"]), name
        assert (np.diff(f) < 0).all()
    base = ref.freqs(128, 1e6, scaling="base", factor=8.0)
    assert base[0] == 1 and math.isclose(base[-1], plain[-1] / 8.0)  # theta's power at the last pair is (rot - 2) / rot


GOOD = dict(head_dim=64, theta=1e4)
SCALED = dict(factor=4.0, orig_ctx=4096.0, low=1.0, high=4.0)


@pytest.mark.parametrize("kw", [
    dict(head_dim=1), dict(head_dim=258), dict(head_dim=-64), dict(rot_dim=0), dict(rot_dim=66), dict(rot_dim=3),
    dict(layout=2), dict(scaling=6), dict(scaling=-1), dict(theta=0.0), dict(theta=-1.0), dict(theta=float("nan")),
    dict(theta=float("inf")), dict(magnitude=0.0), dict(magnitude=-1.0), dict(magnitude=float("nan")),
    dict(magnitude=1e39), dict(magnitude=1e-60), dict(scaling=1, factor=0.0), dict(scaling=1, factor=float("inf")),
    dict(scaling=2, factor=-2.0), dict(scaling=2, rot_dim=2, factor=2.0), dict(scaling=3, **{**SCALED, "orig_ctx": 0.0}),
    dict(scaling=3, **{**SCALED, "low": 0.0}), dict(scaling=4, **{**SCALED, "high": 1.0}),
    dict(scaling=4, **{**SCALED, "high": float("nan")}), dict(scaling=3, theta=1.0, **SCALED), dict(scaling=5),
    dict(scaling=5, divisors=[1.0] * 31), dict(scaling=5, divisors=[1.0] * 31 + [0.0]),
    dict(scaling=5, divisors=[float("nan")] + [1.0] * 31), dict(scaling=1, factor=1e-300), dict(theta=1e-300),
], ids=lambda kw: str(kw)[:60])
def test_bad_ropes_are_refused(lib, kw):
    with pytest.raises(q.QkvError) as e:
        q.qkv_rope_create(**{**GOOD, **kw})
    assert e.value.status == q.QKV_ERR_INVALID_ARG


def step(lib, rope, **kw):
    a = dict(x=P << 4, x_stride=256, out=P << 8, out_stride=256, positions=P, dtype=q.QKV_F32, nt=3, heads=4, inverse=0)
    args = q._ROPE_ARGS.pack(*[0 if v is None else v for v in {**a, **kw}.values()])
    return lib.qkv_rope_step(rope.handle if rope else None, args, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(out=None), 1), (dict(positions=None), 1), (dict(x_stride=255), 1), (dict(out_stride=255), 1),
    (dict(nt=-1), 1), (dict(heads=0), 1), (dict(dtype=3), 2), (dict(dtype=-1), 2), (dict(x=P + 2), 1),
    (dict(out=(P << 8) + 2), 1), (dict(positions=P + 1), 1), (dict(x=P << 8, out_stride=512), 1),
    (dict(out=(P << 4) + 4), 1), (dict(out=(P << 4) + 4 * (2 * 256 + 255)), 1), (dict(out=P - 4 * 255), 1),
    (dict(nt=(1 << 31) - 1, x_stride=256, heads=4), 1), (dict(x=P + 1, dtype=q.QKV_F16), 1),
    (dict(nt=0), 0), (dict(nt=0, x=None, out=None, positions=None), 0),
], ids=str)
def test_step_refusals(lib, kw, status):
    rope = q.qkv_rope_create(**GOOD)
    assert step(lib, rope, **kw) == status
    if status:
        assert lib.qkv_last_error()


def test_null_arguments(lib):
    rope = q.qkv_rope_create(**GOOD)
    assert step(lib, None) == q.QKV_ERR_INVALID_ARG
    assert lib.qkv_rope_step(rope.handle, None, None) == q.QKV_ERR_INVALID_ARG
    assert lib.qkv_rope_create(None, ctypes.byref(ctypes.c_void_p())) == q.QKV_ERR_INVALID_ARG
    assert lib.qkv_rope_create(ctypes.byref(q.qkv_rope_desc()), None) == q.QKV_ERR_INVALID_ARG
    out = (ctypes.c_double * 40)()
    assert lib.qkv_rope_freqs(rope.handle, out, 31) == lib.qkv_rope_freqs(None, out, 32) == q.QKV_ERR_INVALID_ARG
    assert lib.qkv_rope_freqs(rope.handle, None, 32) == q.QKV_ERR_INVALID_ARG
    lib.qkv_rope_destroy(None)


def test_store_takes_a_rope_of_its_plans_heads(lib):
    plan = q.qkv_plan_create(64, 4, 2, 64, 1e6, 64)
    cache = q.qkv_paged_kv(P, P << 8, P, 8, 16, 3, 4, 0, None, None)
    args = q._STORE_ARGS.pack(P << 4, 512, 0, 0, P, 0, 0, P, P, P, P << 5, 256, 0.0)
    call = lambda pl, rope: lib.qkv_paged_store_rope_step(  # noqa: E731
        pl, ctypes.byref(cache), rope, args, None)
    rope, other = q.qkv_rope_create(64, 1e4), q.qkv_rope_create(128, 1e4)
    assert call(plan.handle, rope.handle) == q.QKV_OK  # nt == 0
    assert call(plan.handle, other.handle) == call(plan.handle, None) == call(None, rope.handle) == q.QKV_ERR_INVALID_ARG
    assert lib.qkv_paged_store_rope_step(plan.handle, None, rope.handle, args, None) == q.QKV_ERR_INVALID_ARG
    assert lib.qkv_paged_store_rope_step(plan.handle, ctypes.byref(cache), rope.handle, None, None) == 1


def test_layouts_match_the_header(tmp_path):
    import os
    import subprocess
    names = [n for n, _ in q.qkv_rope_desc._fields_]
    args = "x x_stride out out_stride d_positions dtype nt n_heads inverse".split()
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include "qkv.h"\nint main(void) {%s%s return 0; }\n' % (
        'printf("%zu", sizeof(qkv_rope_desc));' + "".join('printf(" %%zu", offsetof(qkv_rope_desc, %s));' % n for n in names),
        'printf("\\n%zu", sizeof(qkv_rope_args));' + "".join('printf(" %%zu", offsetof(qkv_rope_args, %s));' % n for n in args)))
    exe = str(tmp_path / "layout")
    subprocess.check_call(["gcc", "-I", os.path.dirname(q.HEADER), "-o", exe, str(src)])
    desc, step_args = ([int(v) for v in line.split()] for line in subprocess.check_output([exe], text=True).splitlines())
    assert desc == [ctypes.sizeof(q.qkv_rope_desc)] + [getattr(q.qkv_rope_desc, n).offset for n in names]
    assert step_args[0] == q._ROPE_ARGS.size
    for i, at in enumerate(step_args[1:]):
        data = q._ROPE_ARGS.pack(*[int(k == i) for k in range(len(args))])
        assert data[at] == 1 and sum(data) == 1


def test_python_refuses_what_its_tensors_show():
    torch = pytest.importorskip("torch")
    rope = q.qkv_rope_create(**GOOD)
    x, pos = torch.zeros(3, 128), torch.zeros(3, dtype=torch.int32)
    for args in ((x, pos, x), (x[:, :100], pos, x), (x.double(), pos, x)):
        with pytest.raises(q.QkvError):
            q.qkv_rope_step(rope, *args)
