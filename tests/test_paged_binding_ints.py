"""Integers that a C int does not hold are refused by the paged calls of the binding.

ctypes passes on the low 32 bits of any Python int, so 2^32 would arrive as 0 and 2^32 + 1 as
1: a rotation at other positions, another table, another pool.  No GPU: the refusal comes
before any tensor is looked at, or is asked of the helper that takes a batch's shapes.
"""
import pytest
import torch

import causal_gqa_flash_attention_gb300 as ne
from causal_gqa_flash_attention_gb300 import _build

WIDE = [2 ** 32, 2 ** 32 + 1, 2 ** 31, -2 ** 32 + 1]


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return ne.load()


def host_batch():
    kp = torch.zeros(8, 16, 2, 64, dtype=torch.bfloat16)
    return torch.zeros(2, 4, 64, dtype=torch.bfloat16), kp, torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)


@pytest.mark.parametrize("x", WIDE)
def test_append_refuses_a_position_offset_of_more_than_32_bits(x):
    q, kp, t, ln = host_batch()
    with pytest.raises(ValueError, match="pos_offset"):
        ne.paged_append(q[:, :2], q[:, :2], kp, kp, t, ln, pos_offset=x)


@pytest.mark.parametrize("x", WIDE)
def test_attn_refuses_a_row_count_of_more_than_32_bits(x):
    q, kp, t, ln = host_batch()
    with pytest.raises(ValueError, match="max_new"):
        ne.paged_attn(q, kp, kp, t, ln, max_new=x)


@pytest.mark.parametrize("x", WIDE)
def test_rope_spec_refuses_integers_of_more_than_32_bits(x):
    with pytest.raises(ValueError, match="orig_len"):
        ne.rope_spec(64, scaling="parts", factor=2.0, orig_len=x + 2048)
    with pytest.raises(ValueError, match="rot_dim"):
        ne.rope_spec(64, rot_dim=x + 32)
    with pytest.raises(ValueError, match="D = "):
        ne.rope_spec(x + 64, rot_dim=64)


@pytest.mark.parametrize("x", WIDE)
def test_workspace_sizes_refuse_integers_of_more_than_32_bits(x):
    for i in range(5):
        args = [4, 8, 12, 4, 64]
        args[i] += x
        with pytest.raises(ValueError, match="32 bits"):
            ne.alloc_paged_workspace(*args)
    for i in range(3):
        args = [100, 4, 8]
        args[i] += x
        with pytest.raises(ValueError, match="32 bits"):
            ne.alloc_pages_workspace(*args, device="cpu")


@pytest.mark.parametrize("B,W,N", [(2 ** 32 + 1, 1, 2 ** 32 + 1), (1, 2 ** 32 + 1, 1), (2, 2 ** 31, 2)])
def test_a_batch_of_more_than_32_bits_is_refused(B, W, N):
    """(Shapes alone: tensors without memory.)"""
    table, lens = (torch.empty(s, dtype=torch.int32, device="meta") for s in ((B, W), (B,)))
    with pytest.raises(ValueError, match="32 bits"):
        ne._paged_batch(table, lens, None, N, table.get_device())
