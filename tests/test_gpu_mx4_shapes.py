"""The product of microscaled 4-bit operands at sizes that take each of its
kernels: few rows in 16, 32 or 64 columns to a workgroup, and each tile, with k of whole
slices and not, and edges in every dimension.  Sums fit in binary32, so results are exact."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import w8a8_int8_quantized_qk_amd as qk
from tests.test_gpu_mx4 import DEV, TORCH

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qk.library()


LEVELS = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6])


def operand(gen, rows, k):
    """Codes, scales with NaN behind each row, and the values, on the GPU."""
    q = torch.randint(0, 256, (rows, k // 2), generator=gen, dtype=torch.uint8, device=DEV)
    room = torch.full((rows, -(-(k // 32) // 16) * 16 + 16), 255, dtype=torch.uint8, device=DEV)
    s = room[:, :k // 32]
    s.copy_(torch.randint(126, 128, (rows, k // 32), generator=gen, dtype=torch.uint8, device=DEV))
    v = LEVELS.to(DEV)[torch.stack([q & 15, q >> 4], 2).view(rows, k).int()]
    return q, s, v * torch.exp2(s.float() - 127).repeat_interleave(32, 1)


def check(m, n, k, out):
    # products are multiples of 2^-4; sums of magnitudes stay below 2^20, so that binary32 holds every partial
    # sum in any order, the reference's included
    assert k * 36 < 2 ** 20
    gen = torch.Generator(device=DEV).manual_seed(m + 3 * n + 7 * k)
    a, sa, va = operand(gen, m, k)
    b, sb, vb = operand(gen, n, k)
    got = qk.gemm_mx4_scaled(a, b, sa, sb, out_dtype=TORCH[out])
    want = torch.mm(va, vb.t().contiguous()).to(TORCH[out])
    bad = got != want
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m,n,k", [
    (1, 12799, 544), (16, 12801, 2048), (9, 25599, 512), (3, 25601, 96), (16, 26000, 1056),  # 16, 32, 64 columns
    (17, 12799, 1056), (32, 13001, 512), (20, 30000, 96),
    (33, 300, 4096), (64, 4097, 1120), (100, 1001, 512),                                     # 32 x 32
    (64, 14336, 1056), (50, 16001, 128), (60, 30000, 32),                                    # 64 x 64
    (129, 14337, 512), (257, 8191, 1184), (512, 4096, 1024), (1000, 4000, 2080),             # tiles of 128 x 128
    (2048, 4096, 2048), (2047, 4095, 2144), (1025, 8000, 2080),                              # 256 x 128
    (4096, 8192, 256), (4095, 8190, 416), (2300, 16500, 2080), (4000, 4096, 4128)])          # 256 x 256
def test_sizes(m, n, k, out):
    check(m, n, k, out)


@pytest.mark.parametrize("k", [32, 64, 96, 128, 160, 480, 512, 544, 1920, 2016, 2048, 2080, 3968, 4064, 4096, 4128, 8192, 8224])
@pytest.mark.parametrize("m,n", [(5, 70), (40, 70), (300, 9000), (2100, 4200), (4100, 8200)])
def test_every_remainder_of_k(m, n, k):
    check(m, n, k, "f32")


@pytest.mark.parametrize("k", [32, 224, 256, 384, 992, 1024, 1280, 1536, 1792, 1920, 2048, 2176, 2304, 3840, 4096, 4352, 6176, 8192])
@pytest.mark.parametrize("m,n", [(2000, 4000), (700, 4096), (3100, 4096)])
def test_every_number_of_slices_in_the_rings(m, n, k):
    check(m, n, k, "bf16")


def test_a_run_of_products_on_two_streams():
    # nothing is shared between calls
    gen = torch.Generator(device=DEV).manual_seed(1)
    cases = [(operand(gen, m, k), operand(gen, n, k)) for m, n, k in ((4, 4096, 4096), (2048, 4096, 512), (200, 300, 1056))]
    want = [qk.gemm_mx4_scaled(a[0], b[0], a[1], b[1]) for a, b in cases]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append([qk.gemm_mx4_scaled(a[0], b[0], a[1], b[1]) for a, b in cases])
    torch.cuda.synchronize()
    for got in outs:
        assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m,n,k", [(1, 4096, 4096), (16, 1001, 2720), (5, 12801, 544), (16, 26001, 1056), (2, 16, 32), (15, 333, 14336),
                                   (7, 13000, 96), (1, 30000, 160), (17, 500, 512), (3, 4096, 2016)])
def test_few_rows_of_a_linear_are_the_two_calls(m, n, k, dtype):
    # rows that are quantised within the product, and the same rows where they cannot be (a row stride or a place
    # that is no multiple of 16 bytes): the same codes, the same order of sums
    gen = torch.Generator(device=DEV).manual_seed(m * k + n)
    x = torch.randn((m, k), generator=gen, device=DEV).to(TORCH[dtype])
    x[m // 2, k // 2] = 300
    w, sw = qk.quant_mx4(torch.randn((n, k), generator=gen, device=DEV))
    q, s = qk.quant_mx4(x)
    want = qk.gemm_mx4_scaled(q, w, s, sw, 0.5, torch.float32)
    assert torch.equal(qk.linear_mx4(x, w, sw, 0.5, torch.float32), want)
    apart = torch.zeros((m, k + 16), dtype=TORCH[dtype], device=DEV)[:, 8:8 + k]
    odd = torch.zeros((m, k + 17), dtype=TORCH[dtype], device=DEV)[:, 3:3 + k]
    for t in (apart, odd):
        t.copy_(x)
        assert torch.equal(qk.linear_mx4(t, w, sw, 0.5, torch.float32), want)
    for out in ("bf16", "f16"):
        assert torch.equal(qk.linear_mx4(x, w, sw, 0.5, TORCH[out]), want.to(TORCH[out]))


@pytest.mark.parametrize("k", [32, 96, 2048, 2720])
def test_special_values_in_few_rows_of_a_linear(k):
    gen = torch.Generator(device=DEV).manual_seed(k)
    x = torch.randn((6, k), generator=gen, device=DEV)
    x[1, k - 1], x[2, 0], x[3] = float("nan"), float("inf"), 0.0
    x[4] *= 2.0 ** -140
    w, sw = qk.quant_mx4(torch.randn((77, k), generator=gen, device=DEV))
    out = qk.linear_mx4(x, w, sw, out_dtype=torch.float32)
    q, s = qk.quant_mx4(x)
    want = qk.gemm_mx4_scaled(q, w, s, sw, out_dtype=torch.float32)
    assert out[1:3].isnan().all() and not out[3].any() and out[[0, 3, 4, 5]].isfinite().all()
    assert torch.equal(out.nan_to_num(7e20), want.nan_to_num(7e20))
