"""The 4-bit product's tiles (128 x 128, 128 x 256 and 256 x 256 outputs, with k of whole pairs
of slices and not) under scales of any size, NaN ones and the smallest and largest, and the
way back of large calls."""
from __future__ import annotations

import pytest
import torch

import w8a8_int8_quantized_qk_amd as qk
from tests.test_gpu_mx4 import DEV, TORCH
from tests.test_gpu_mx4_shapes import LEVELS

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qk.library()


def codes(gen, rows, k):
    return torch.randint(0, 256, (rows, k // 2), generator=gen, dtype=torch.uint8, device=DEV)


def room_for(scale):
    """The scales in rows whose padding is NaN's byte, which must not matter."""
    rows, n = scale.shape
    room = torch.full((rows, -(-n // 16) * 16 + 16), 255, dtype=torch.uint8, device=DEV)
    room[:, :n] = scale
    return room[:, :n]


def values(q, scale, dtype=torch.float64):
    v = LEVELS.to(DEV).to(dtype)[torch.stack([q & 15, q >> 4], 2).view(q.shape[0], -1).int()]
    s = torch.ldexp(torch.ones((), dtype=dtype, device=DEV), scale.int() - 127)
    return v * torch.where(scale == 255, torch.nan, s).repeat_interleave(32, 1)


# rows, columns, k that the rule sends to each tile; k % 256 == 0 and not, more than one batch of 16 slices
SIZES = [(700, 4096, 1024), (500, 4093, 2336), (1000, 4000, 4096),      # 128 x 128
         (2048, 4096, 2048), (2047, 4095, 2144), (1500, 4090, 4160),    # 128 x 256
         (4096, 8192, 256), (4095, 8190, 416), (4095, 4093, 4128)]      # 256 x 256


def scales(gen, rows, k, lo, hi):
    return torch.randint(lo, hi + 1, (rows, k // 32), generator=gen, dtype=torch.uint8, device=DEV)


@pytest.mark.parametrize("m,n,k", SIZES)
def test_any_scales(m, n, k):
    # binary32 sums of k exact products in any order, each addition off by at most 2^-23 of the sum of magnitudes
    gen = torch.Generator(device=DEV).manual_seed(m + k)
    a, b = codes(gen, m, k), codes(gen, n, k)
    sa, sb = scales(gen, m, k, 100, 140), scales(gen, n, k, 107, 125)
    va, vb = values(a, sa), values(b, sb)
    got = qk.gemm_mx4_scaled(a, b, room_for(sa), room_for(sb), out_dtype=torch.float32).double()
    err, size = (got - va @ vb.t().contiguous()).abs_(), va.abs() @ vb.abs().t().contiguous()
    bad = ~(err <= k * 2.0 ** -23 * size)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, first at {bad.nonzero()[0].tolist()}"
    # no block's products are lost in that: the error is far below what one of them adds
    assert (err / size).median() < 2.0 ** -22


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_nan_scales_reach_their_rows_and_columns_only(m, n, k, out):
    # sums of products in units of 2^-4 below 2^24 of them: exact in any order, the reference's too
    assert k * 36 < 2 ** 20
    gen = torch.Generator(device=DEV).manual_seed(m + n)
    a, b = codes(gen, m, k), codes(gen, n, k)
    sa, sb = scales(gen, m, k, 126, 127), scales(gen, n, k, 126, 127)
    want = (values(a, sa, torch.float32) @ values(b, sb, torch.float32).t().contiguous()).to(TORCH[out])
    blocks = k // 32
    # in each 64 rows of scales one thread transposes a row: first and last of them, each byte of a word, each
    # slice of the first and last batch
    for i, row in enumerate(range(3, m, max(1, m // 40))):
        sa[row, [0, blocks - 1, blocks // 2, i % blocks][i % 4]] = 255
        want[row] = torch.nan
    for i, col in enumerate(range(1, n, max(1, n // 50))):
        sb[col, [blocks - 1, i % blocks, 0, (7 * i + 5) % blocks][i % 4]] = 255
        want[:, col] = torch.nan
    got = qk.gemm_mx4_scaled(a, b, room_for(sa), room_for(sb), out_dtype=TORCH[out])
    bad = ~((got == want) | (got.isnan() & want.isnan()))
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("m,n,k", SIZES)
def test_every_block_has_its_scale(m, n, k):
    # A: one block of each row has the scale 2^8, the others 1; B: one block of each column 2^7.  All codes are 1, so
    # a result is the sum of 32 times its blocks' scales, a whole number below 2^24.
    assert k + 32 * (2 ** 15 + 2 ** 8 + 2 ** 7) < 2 ** 24
    blocks = k // 32
    a, b = (torch.full((r, k // 2), 0x22, dtype=torch.uint8, device=DEV) for r in (m, n))
    at_a, at_b = torch.arange(m, device=DEV) * 7 % blocks, torch.arange(n, device=DEV) * 5 % blocks
    sa, sb = (torch.full((r, blocks), 127, dtype=torch.uint8, device=DEV) for r in (m, n))
    sa[torch.arange(m, device=DEV), at_a] = 127 + 8
    sb[torch.arange(n, device=DEV), at_b] = 127 + 7
    got = qk.gemm_mx4_scaled(a, b, room_for(sa), room_for(sb), out_dtype=torch.float32)
    same = at_a[:, None] == at_b[None]
    want = torch.where(same, 32.0 * (blocks - 1 + 2 ** 15), 32.0 * (blocks - 2 + 2 ** 8 + 2 ** 7))
    bad = got != want
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("m,n,k", [(700, 4096, 1024), (2047, 4095, 2144), (4095, 8190, 416)])
def test_smallest_and_largest_scales(m, n, k):
    # one block of ones in each row of A, under 2^-127 .. 2^127, against ones under 2^-1: sums of 32 equal products, powers
    # of two from 2^-123 on, that are infinity from 2^128 on; what is lost of products below binary32's normal numbers
    # is below the least of those
    a, b = torch.zeros((m, k // 2), dtype=torch.uint8, device=DEV), torch.zeros((n, k // 2), dtype=torch.uint8, device=DEV)
    blocks = k // 32
    row = torch.arange(m, device=DEV)
    at = row % blocks
    for j in range(16):
        a[row, at * 16 + j] = 0x22
    b.fill_(0x22)
    sa = torch.full((m, blocks), 127, dtype=torch.uint8, device=DEV)
    sa[row, at] = (row % 255).to(torch.uint8)
    sb = torch.full((n, blocks), 126, dtype=torch.uint8, device=DEV)
    got = qk.gemm_mx4_scaled(a, b, room_for(sa), room_for(sb), out_dtype=torch.float32)
    want = torch.ldexp(torch.ones((), dtype=torch.float64, device=DEV), row % 255 - 127 + 4).float()
    bad = ~((got == want[:, None]) | ((got - want[:, None]).abs() <= 2.0 ** -126))
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m,k", [(3000, 2720), (65537, 128), (70, 131072)])
def test_way_back_of_large_calls(m, k, dtype):
    t = TORCH[dtype]
    gen = torch.Generator(device=DEV).manual_seed(m)
    q, s = codes(gen, m, k), scales(gen, m, k, 0, 255)
    want = values(q, s).to(t)  # exact, or one rounding from exact values
    assert want.numel() * want.element_size() > 8 << 20

    def check(got):
        bad = ~((got == want) | (got.isnan() & want.isnan()))
        assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, first at {bad.nonzero()[0].tolist()}"

    check(qk.dequant_mx4(q, room_for(s), t))
    wide = torch.full((m, k + 9), 7.0, dtype=t, device=DEV)  # rows apart, at an odd place
    qk.dequant_mx4(q, room_for(s), x=wide[:, 3:3 + k])
    check(wide[:, 3:3 + k])
    assert (wide[:, :3] == 7).all() and (wide[:, 3 + k:] == 7).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_large_calls_of_quantisation_are_their_rows(dtype):
    m, k = 4099, 4128
    gen = torch.Generator(device=DEV).manual_seed(3)
    h = torch.randn((m, 2 * k), generator=gen, device=DEV).to(TORCH[dtype])
    q, s = qk.quant_mx4(h[:, :k])
    qs, ss = qk.silu_mul_quant_mx4(h)
    for r in (0, 1, 2047, 4098):
        one = qk.quant_mx4(h[r:r + 1, :k])
        assert torch.equal(one[0], q[r:r + 1]) and torch.equal(one[1], s[r:r + 1])
        one = qk.silu_mul_quant_mx4(h[r:r + 1])
        assert torch.equal(one[0], qs[r:r + 1]) and torch.equal(one[1], ss[r:r + 1])
