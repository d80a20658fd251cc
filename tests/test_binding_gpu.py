"""Refusals of the binding: shapes of one size but another meaning, numbers that pass 32 bits, workspaces that are no
plain bytes.  Nothing is launched."""
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


@pytest.mark.parametrize("window", [-1, 2 ** 31, 2 ** 32, 2 ** 32 + 5, -2 ** 32])
def test_windows_that_pass_32_bits(window):
    with pytest.raises(ValueError, match="window"):
        fq.fq_kv_attn(torch.zeros(1, 2, 128, **f16), torch.zeros(1, **i32), torch.zeros(1, 1, **i32),
                      fq.kv_cache(2, 2, 16), window=window)


@pytest.mark.parametrize("page_size,max_tokens", [(2 ** 32 + 16, 4), (-16, 4), (16, -1), (16, 2 ** 32 + 4), (16, 2 ** 30 + 1)])
def test_plan_numbers_that_pass_32_bits(page_size, max_tokens):
    one, table = torch.zeros(1, **i32), torch.zeros(1, 2, **i32)
    with pytest.raises(ValueError, match="page_size|max_tokens"):
        fq.fq_kv_plan(one, one, table, one, one, page_size, max_tokens)


@pytest.mark.parametrize("fmt", [2, -1, 2 ** 32, 2 ** 32 + 1])
def test_formats_that_are_none(fmt):
    """2^32 + 1 would be checked as one format and computed as the other, whose scales are twice as many."""
    x = torch.zeros(8, 128, **f16)
    q, s = fq.fq_mx_quant(x, fq.MXFP4)
    for call in (lambda: fq.fq_mx_quant(x, fmt), lambda: fq.fq_mx_dequant(q, s, fmt), lambda: fq.fq_mx_gemm(q, s, q, s, fmt),
                 lambda: fq.fq_mx_linear(x, fmt, q, s)):
        with pytest.raises(fq.FqError, match="format") as e:
            call()
        assert e.value.status == fq.FQ_ERR_UNSUPPORTED


def test_product_workspaces_that_are_no_plain_bytes():
    """Bytes of a strided or repeated view do not lie where its length says."""
    x = torch.zeros(8, 128, **f16)
    q, s = fq.fq_mx_quant(x, fq.MXFP4)
    n = fq.fq_mx_gemm_workspace_size(8, 8, 128, fq.MXFP4)
    for ws in (torch.zeros(2 * n, **u8)[::2], torch.zeros(1, **u8).expand(n), torch.zeros(n, **i32), torch.zeros(n, dtype=torch.uint8)):
        with pytest.raises(ValueError, match="workspace"):
            fq.fq_mx_gemm(q, s, q, s, fq.MXFP4, workspace=ws)
