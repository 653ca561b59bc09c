"""Paged-cache calls at their edges, as far as no GPU is needed."""
import ctypes

import pytest

import qkv_rope_kv_gb300 as q

P = 4096  # a plausible, never dereferenced, aligned address


@pytest.fixture(scope="module")
def lib():
    return q.load()


def plan(nh, nkv, hd, kv):
    return q.qkv_plan_create(64, nh, nkv, hd, 1e6, 64, kv_dtype={"f16": q.QKV_F16, "f32": q.QKV_F32}[kv])


def store_args(**kw):
    a = dict(Y=P << 4, y_stride=512, y_dtype=q.QKV_F32, nt=1, bias=0, qw=0, kw=0, pos=P, seqs=P, slots=P, q=P << 4,
             q_stride=256, eps=0.0)
    return q._STORE_ARGS.pack(*{**a, **kw}.values())


@pytest.mark.parametrize("kw", [dict(nt=2), dict(y_dtype=q.QKV_BF16), dict(q=(P << 4) + 4), dict(q=(P << 4) + 4 * 511)],
                         ids=str)
def test_store_over_parts_of_y_is_refused(lib, kw):
    """Rows of two strides, of another type, or shifted against Y's."""
    c = q.qkv_paged_kv(P, P << 8, P, 8, 16, 3, 4, 0, None, None)
    assert lib.qkv_paged_store_step(plan(4, 2, 64, "f16").handle, ctypes.byref(c), store_args(**kw),
                                    None) == q.QKV_ERR_INVALID_ARG


@pytest.mark.parametrize("nh,nkv,hd,kv,n_seq,capacity,want", [
    (40, 8, 128, "f16", 1, 32768, (256, 8)),    # four clusters for each kv head
    (28, 4, 128, "f16", 1, 1648, (64, 8)),      # no more clusters than can have work
    (14, 2, 64, "f32", 1, 512, (16, 8)),      # 32 units: one cluster for each kv head
    (28, 4, 128, "f16", 10, 512, (260, 4)),
    (28, 4, 128, "f16", 25, 512, (270, 2)),
    (40, 8, 128, "f16", 64, 8192, (304, 1)),
    (8, 1, 256, "f16", 1, 9024, (72, 8)),     # 564 units: nine clusters have work
    (8, 1, 256, "f16", 1, 20000, (104, 8)),    # all 13
    (8, 1, 256, "f32", 16, 256, (128, 4)),
    (8, 1, 256, "f16", 100, 4096, (152, 1)),
    (96, 8, 128, "f16", 64, 8192, (304, 1)),
    (20, 1, 256, "f16", 100, 4096, (150, 1)),   # three blocks of q heads abreast
], ids=str)
def test_attention_grid_follows_from_sizes_alone(lib, nh, nkv, hd, kv, n_seq, capacity, want):
    """The order of the sums follows from the grid: nothing that a device or its driver says may
    change it (here there is none to ask)."""
    c = q.qkv_paged_kv(P, P << 8, P, 8, 16, n_seq, capacity // 16, 0, None, None)
    ctas, cluster = ctypes.c_int32(), ctypes.c_int32()
    assert lib.qkv_test_attn_grid(plan(nh, nkv, hd, kv).handle, ctypes.byref(c), ctypes.byref(ctas),
                                  ctypes.byref(cluster)) == q.QKV_OK
    assert (ctas.value, cluster.value) == want


@pytest.mark.parametrize("w,pos", [(P << 13, P << 14), (P << 14, P << 12), (P << 14, P << 14), (P << 14, (P << 14) + 1532),
                                   (P << 12, (P << 12) + 4)], ids=str)
def test_eviction_outputs_over_each_other_are_refused(lib, w, pos):
    """weight_out over slot_pos, pos_out over slot_weight, and one over the other."""
    c = q.qkv_paged_kv(P, P << 8, P, 8, 16, 3, 4, 0, P << 12, P << 13)
    args = q._EVICT_ARGS.pack(P, P, P << 6, w, pos, P, 1 << 40, 8, 2)
    assert lib.qkv_evict_step(plan(4, 2, 64, "f16").handle, ctypes.byref(c), args, None) == q.QKV_ERR_INVALID_ARG


@pytest.mark.parametrize("eps", [float("inf"), float("nan"), -1.0, -float("inf")])
def test_store_eps_is_finite_and_not_negative(lib, eps):
    """A norm with an infinite eps has no value but 0."""
    c = q.qkv_paged_kv(P, P << 8, P, 8, 16, 3, 4, 0, None, None)
    args = store_args(qw=P, kw=P, q=P << 5, eps=eps)
    assert lib.qkv_paged_store_step(plan(4, 2, 64, "f16").handle, ctypes.byref(c), args, None) == q.QKV_ERR_INVALID_ARG
