"""Block-scaled products on CTA pairs, launched one behind the other without a wait between them.

With early dependent launches the CTAs of one product start on an SM that those of the one before are leaving, and
products of other sizes and formats keep their barriers at other places of shared memory.  A pair that left
before everything sent to it had come would change words, or arrivals, of its successor: a wrong output or a
wait that runs out (FQ_ERR_TIMEOUT).
"""
import itertools

import numpy as np
import pytest
import torch

from int4_linear_b200 import fq

pytestmark = pytest.mark.gpu

# tokens, outputs, K: tiles of 128 and of 256 tokens, half tiles, one stage and many, fewer tiles than pairs and more
SIZES = [(65, 256, 128), (128, 512, 4096), (200, 19072, 256), (300, 1000, 896), (600, 4096, 1024), (129, 8, 384)]


@pytest.mark.parametrize("captured", [False, True])
def test_products_one_behind_the_other(captured):
    g = np.random.Generator(np.random.PCG64(41))
    calls = []
    for (m, n, k), fmt in itertools.product(SIZES, (fq.MXFP4, fq.NVFP4)):
        def quantized(rows):
            x = torch.from_numpy((g.standard_normal((rows, k)) / 8).astype(np.float16)).cuda()
            return fq.fq_mx_quant(x, fmt)
        (xq, sx), (wq, sw) = quantized(m), quantized(n)
        out = torch.empty(m, n, dtype=torch.float16, device="cuda")
        calls.append((lambda a=(xq, sx, wq, sw, fmt), o=out: fq.fq_mx_gemm(*a, Y=o), out))
    alone = []
    for call, out in calls:
        torch.cuda.synchronize()
        call()
        torch.cuda.synchronize()
        alone.append(out.clone())
    orders = [g.permutation(len(calls)) for _ in range(20)]

    def steps():
        for order in orders:
            for i in order:
                calls[i][0]()

    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            steps()
    for _ in range(5):
        for _, out in calls:
            out.fill_(float("nan"))
        graph.replay() if captured else steps()
        torch.cuda.synchronize()
        fq.fq_check_device_error()
        for (_, out), want in zip(calls, alone):
            assert torch.equal(out, want)
