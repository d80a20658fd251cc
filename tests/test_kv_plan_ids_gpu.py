"""Block tables and free lists whose ids are no page: their tokens have no slot, not another page's."""
import numpy as np
import pytest
import torch

from int4_linear_b200 import fq
from oracle import kv_oracle as KO
from tests.test_kv_gpu import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("rows", [64, 5000])     # one CTA, and a cluster of them
def test_ids_that_are_no_page(page, rows):
    wrap = 2 ** 32 // page                       # times the page size this is 0 in 32 bits
    ids = [wrap + 3, wrap // 2, wrap // 2 - 1, wrap // 2 + 2, -1, -wrap + 1, 2 ** 31 - 1, -2 ** 31, 4]
    r = len(ids)
    lens = np.full(r, page - 2, np.int32)
    new = np.full(r, 4, np.int32)                # two tokens in the held page, two in a fresh one
    table = np.full((r, 2), -7, np.int32)
    table[:, 0] = ids
    free = np.array(ids[::-1], np.int64).astype(np.int32)
    want = table.copy()
    out, start, slots, used = KO.plan(lens, new, want, free, 0, page, rows)
    assert slots[:4].tolist() == [-1, -1, 4 * page, 4 * page + 1]
    t = dev(table)
    got = fq.fq_kv_plan(dev(lens), dev(new), t, dev(free), torch.zeros(1, dtype=torch.int32, device="cuda"), page, rows)
    for a, b in zip(got, (out, start, slots, used)):
        assert np.array_equal(a.cpu().numpy(), b)
    assert np.array_equal(t.cpu().numpy(), want)


def test_tokens_of_such_pages_are_not_written():
    page = 16
    table = torch.tensor([[2 ** 28 + 3]], dtype=torch.int32, device="cuda")   # 2^32 + 48 as a slot
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    _, _, slots, _ = fq.fq_kv_plan(one, one, table, one, torch.zeros_like(one), page, 1)
    cache = fq.kv_cache(8, 2, page)
    kv = torch.ones(1, 2, 128, dtype=torch.float16, device="cuda")
    fq.fq_kv_write(kv, kv, slots, cache)
    assert not cache.pool.any()
