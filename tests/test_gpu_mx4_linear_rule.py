"""The 4-bit layer at the borders between its one launch and its two: rows, size of the
weight, place and stride of the rows."""
from __future__ import annotations

import pytest
import torch

import w8a8_int8_quantized_qk_amd as qk

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qk.library()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m", [1, 2, 15, 16, 17])
@pytest.mark.parametrize("n,k", [(4096, 4096), (4097, 4096), (4095, 4128), (524288, 32), (524289, 32), (32, 524288), (64, 262176)])
def test_both_sides_of_each_border(m, n, k, dtype):
    gen = torch.Generator(device=DEV).manual_seed(m + n)
    w, sw = qk.quant_mx4(torch.randn((n, k), generator=gen, device=DEV).to(torch.bfloat16))
    room = torch.randn((m, k + 24), generator=gen, device=DEV).to(dtype)
    for at in (0, 1, 4, 8):            # places at multiples of 16 bytes and not, rows of a stride that is one
        x = room[:, at:at + k]
        q, s = qk.quant_mx4(x)
        want = qk.gemm_mx4_scaled(q, w, s, sw, out_dtype=torch.float32)
        assert torch.equal(qk.linear_mx4(x, w, sw, out_dtype=torch.float32), want), at
    x = torch.randn((m, k + 1), generator=gen, device=DEV).to(dtype)[:, :k]  # and of one that is not
    q, s = qk.quant_mx4(x)
    assert torch.equal(qk.linear_mx4(x, w, sw, out_dtype=torch.float32), qk.gemm_mx4_scaled(q, w, s, sw, out_dtype=torch.float32))
