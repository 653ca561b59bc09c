"""Python wrappers of the rotations and of the attention of many query rows: numbers that fit no argument, and a rope that is
none (no GPU)."""
import types

import pytest
import torch

import qkv_rope_kv_gb300 as q
from test_paged_host import cache, plan


class Tensor:
    """What the wrappers ask of a CUDA tensor."""

    def __init__(self, shape, dtype):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, "cuda:0"

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20


@pytest.mark.parametrize("shape", [(2 ** 31, 64), (3, 2 ** 31 * 64)])
def test_rope_step_of_too_many_rows_or_heads(shape):
    rope = q.qkv_rope_create(64, 1e4)
    rope.current_device, rope.current_stream = lambda: 0, lambda dev: 0
    x = Tensor(shape, torch.float32)
    with pytest.raises(q.QkvError):
        q.qkv_rope_step(rope, x, Tensor(shape[:1], torch.int32), x)


@pytest.mark.parametrize("kw", [dict(head_dim=2 ** 32 + 64), dict(head_dim=64, rot_dim=2 ** 32 + 32), dict(head_dim=64, layout=2 ** 32),
                                dict(head_dim=64, scaling=2 ** 32), dict(head_dim=64, theta=None), dict(head_dim=64.5),
                                dict(head_dim=64, magnitude="1"), dict(head_dim=64, factor=10 ** 400),
                                dict(head_dim=4, scaling=q.QKV_ROPE_SCALE_TABLE, divisors=[1.0, None]),
                                dict(head_dim=4, scaling=q.QKV_ROPE_SCALE_TABLE, divisors=2.0)], ids=str)
def test_rope_create_of_numbers_that_fit_no_argument(kw):
    with pytest.raises(q.QkvError):
        q.qkv_rope_create(**{"theta": 1e4, **kw})


@pytest.mark.parametrize("nt", [2 ** 31, 2 ** 32 + 5, -2 ** 40, 1.5, None])
def test_workspace_of_too_many_tokens(nt):
    c = cache()
    paged = types.SimpleNamespace(address=__import__("ctypes").addressof(c))
    assert q.qkv_prompt_attn_workspace_bytes(plan(), paged, 5) > 0
    with pytest.raises(q.QkvError):
        q.qkv_prompt_attn_workspace_bytes(plan(), paged, nt)


def test_store_with_no_rope():
    """None is not the plan's rotation here."""
    with pytest.raises(q.QkvError):
        q.qkv_paged_store_rope_step(plan(), None, None, None, None, None, None, 0.0, None, None, None, None)
