"""The rows8 format on the GPU: bit-exact codes, scales and values against the
definition, non-finite blocks, every width and both types."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from gpu_util import requires_gpu
from linear_util import rows8, rows8_read

pytestmark = [pytest.mark.gpu, requires_gpu]


def _mm():
    import mixture_experts_routing_gemm_amd as mm
    return mm


def rows_of(rows, n, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, n, generator=g) * torch.exp(3 * torch.randn(rows, 1, generator=g))
    x[rows // 2] = 0.0
    if rows > 3:
        x[0] = torch.sign(x[0]) * 127.0   # max|v| = 127 2^e exactly
        x[1] *= 1e-38                      # below the smallest step's range
        x[2, 0] = 3.0e38
        x[3] = torch.round(x[3] * 8) / 16  # many halves: ties
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,n", [(1, 1), (1, 32), (2, 31), (5, 33), (7, 64), (4, 40), (9, 100), (3, 1340), (257, 512),
                                    (1000, 1408)])
def test_pack_and_unpack_are_the_definition(rows, n, dtype):
    mm = _mm()
    x = rows_of(rows, n, dtype, seed=n)
    packed = mm.alloc_rows8(rows, n)
    packed.fill_(0x77)
    mm.moe_pack_rows8(x.cuda(), packed)
    back = torch.full((rows, n), 9.0, dtype=dtype, device="cuda")
    mm.moe_unpack_rows8(packed, back)
    torch.cuda.synchronize()
    ref, step = rows8(x.double().numpy())
    got, codes = rows8_read(packed, rows, n)
    assert np.array_equal(got[:, :n], ref)
    assert not codes[:, n:].any()
    assert np.array_equal(back.double().cpu().numpy(), ref)  # code * 2^e is exact in either type
    assert (np.abs(ref - x.double().numpy()) <= step / 2).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_block_that_is_not_finite_reads_back_as_nan(dtype):
    mm = _mm()
    x = torch.ones(3, 96, dtype=dtype)
    x[0, 5], x[1, 40], x[2, 95] = float("inf"), float("nan"), float("-inf")
    packed, back = mm.alloc_rows8(3, 96), torch.empty(3, 96, dtype=dtype, device="cuda")
    mm.moe_pack_rows8(x.cuda(), packed)
    mm.moe_unpack_rows8(packed, back)
    b = back.float().cpu()
    for r, blk in ((0, 0), (1, 1), (2, 2)):
        for q in range(3):
            part = b[r, 32 * q:32 * q + 32]
            assert torch.isnan(part).all() if q == blk else bool((part == 1.0).all())
