"""Refusals of the binding: shapes of one size but another meaning.  Nothing is launched."""
import pytest
import torch

from int4_linear_b200 import fq

pytestmark = pytest.mark.gpu

i32 = dict(dtype=torch.int32, device="cuda")
f16 = dict(dtype=torch.float16, device="cuda")
u8 = dict(dtype=torch.uint8, device="cuda")


def test_head_vectors_of_another_length():
    """[T, 2 heads, 64] holds as many values as [T, 1 head, 128]."""
    cache, slots = fq.kv_cache(2, 2, 16), torch.zeros(3, **i32)
    good, bad = torch.zeros(3, 2, 128, **f16), torch.zeros(3, 4, 64, **f16)
    fq.fq_kv_write(good, good, torch.tensor([0, 1, 2], **i32), cache)
    for k, v in ((bad, good), (good, bad), (bad[:, ::2], good), (bad.transpose(1, 2), good), (torch.zeros(3, 1, 256, **f16), good)):
        with pytest.raises(ValueError, match="128"):
            fq.fq_kv_write(k, v, slots, cache)
    for q in (torch.zeros(3, 16, 64, **f16), torch.zeros(3, 4, 256, **f16), torch.zeros(3, 128, 8, **f16)):
        with pytest.raises(ValueError, match="128"):
            fq.fq_kv_attn(q, torch.zeros(3, **i32), torch.zeros(3, 1, **i32), cache)
