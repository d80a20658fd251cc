"""Sizes that pass 32 bits are out of range, not the size that their low bits make."""
import pytest

from int4_linear_b200 import fq


@pytest.fixture(scope="module", autouse=True)
def built():
    from int4_linear_b200 import build
    build.build()


@pytest.mark.parametrize("big", [2 ** 32 + 1, 2 ** 31, -2 ** 32 + 1, 2 ** 64 + 1])
def test_sizes(big):
    assert fq.fq_kv_attn_workspace_size(big, 8, 8) == 0 and fq.fq_kv_attn_workspace_size(1, 8 * big, 8) == 0
    for fmt in (fq.MXFP4, fq.NVFP4):
        for fn in (fq.fq_mx_gemm_workspace_size, fq.fq_mx_linear_workspace_size):
            assert fn(1, 8, 128, fmt) > 0
            assert fn(big, 8, 128, fmt) == 0 and fn(1, 8 * big, 128, fmt) == 0 and fn(1, 8, 128 * big, fmt) == 0
        assert fq.fq_mx_scale_bytes(big, 128, fmt) == 0
    assert fq.fq_mx_scale_bytes(1, 128, big) == 0
