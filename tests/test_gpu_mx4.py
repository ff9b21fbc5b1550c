"""Microscaled 4-bit quantisation, the way back and the product, against the
plain definitions in binary64.  Codes and scales are exact; so are products
whose sums fit in binary32, whatever their order."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import w8a8_int8_quantized_qk_amd as qk
from tests import plain_mx4 as plain

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qk.library()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def check_quant(x, q, scale, what=""):
    code, byte = plain.quantise(x.cpu().double().numpy())
    assert np.array_equal(scale.cpu().numpy(), byte), f"scales {what}"
    got = q.cpu().numpy()
    want = plain.pack(code)
    assert np.array_equal(got, want), f"{(got != want).sum()} of {got.size} bytes differ {what}"


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_every_16_bit_value_under_every_near_maximum(dtype):
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(TORCH[dtype])
    every = every[every.isfinite()]
    for d in range(6):
        x = torch.zeros((every.numel(), 32), dtype=TORCH[dtype])
        x[:, 5] = every
        big = torch.ldexp(every.double().abs(), torch.tensor(d)) * 1.2
        x[:, 17] = -torch.where(big > torch.finfo(TORCH[dtype]).max, torch.zeros(()), big).to(TORCH[dtype])
        x = x.to(DEV)
        check_quant(x, *qk.quant_mx4(x), f"exponent {d} below the maximum")


def test_binary32_around_every_border():
    borders = np.concatenate([plain.LEVELS, (plain.LEVELS[1:] + plain.LEVELS[:-1]) / 2, [7.0, 7.9999995]])
    rows = []
    for e in list(range(-149, -115)) + [-60, -1, 0, 1, 90] + list(range(118, 126)):
        for top in (4.0, 5.5, 7.5):
            b = (borders * 2.0 ** e).astype(np.float32)
            b = np.concatenate([b, np.nextafter(b, np.float32(np.inf)), np.nextafter(b, np.float32(0))])
            b = b[b <= np.float32(top * 2.0 ** e)]
            for i in range(0, len(b), 31):
                r = np.zeros(32, np.float32)
                r[0] = top * 2.0 ** e
                r[1:1 + len(b[i:i + 31])] = b[i:i + 31]
                rows += [r, -r]
    x = dev(np.array(rows))
    check_quant(x, *qk.quant_mx4(x))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m,k", [(1, 32), (1, 4096), (3, 64), (7, 96), (63, 544), (64, 2720), (257, 1024), (1000, 32), (5, 28672)])
def test_quant_sizes(m, k, dtype):
    rng = np.random.default_rng(m * k)
    x = dev((rng.standard_normal((m, k)) * np.exp(rng.uniform(-9, 9, (m, 1)))).astype(np.float32)).to(TORCH[dtype])
    q, scale = qk.quant_mx4(x)
    assert q.shape == (m, k // 2) and scale.shape == (m, k // 32) and q.dtype == scale.dtype == torch.uint8
    assert scale.stride(0) % 16 == 0 or m == 1
    check_quant(x, q, scale)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_quant_of_slices_leaves_what_lies_between(dtype):
    rng = np.random.default_rng(3)
    wide = dev(rng.standard_normal((40, 331)).astype(np.float32)).to(TORCH[dtype])
    x = wide[:, 3:3 + 288]  # any alignment, rows apart
    q = torch.full((40, 144), 0xA5, dtype=torch.uint8, device=DEV)
    room = torch.full((40, 32), 0xA5, dtype=torch.uint8, device=DEV)
    got = qk.quant_mx4(x, q, room[:, :9])
    assert got[0].data_ptr() == q.data_ptr() and got[1].data_ptr() == room.data_ptr()
    check_quant(x, q, room[:, :9])
    assert (room[:, 9:] == 0xA5).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_special_values(dtype):
    x = torch.zeros((8, 64), dtype=TORCH[dtype])
    x[0, 3] = float("nan")
    x[1, 40] = float("inf")
    x[2, 0], x[2, 33] = -float("inf"), 1.0
    x[3] = -0.0
    x[4, :32] = torch.finfo(TORCH[dtype]).max
    x[5, 1] = torch.finfo(TORCH[dtype]).smallest_normal / 4  # subnormal
    x[6, :] = torch.finfo(TORCH[dtype]).tiny
    x = x.to(DEV)
    q, scale = qk.quant_mx4(x)
    check_quant(x, q, scale)
    back = qk.dequant_mx4(q, scale, torch.float32).cpu()
    assert back[0, :32].isnan().all() and back[1, 32:].isnan().all() and back[2, :32].isnan().all()
    assert not back[0, 32:].any() and back[2, 33] == 1 and not back[3].any()


def test_nothing_to_do():
    for m, k in ((0, 64), (5, 0), (0, 0)):
        x = torch.empty((m, k), dtype=torch.bfloat16, device=DEV)
        q, scale = qk.quant_mx4(x)
        assert q.shape == (m, k // 2) and scale.shape == (m, k // 32)
        assert qk.dequant_mx4(q, scale).shape == (m, k)
    w, sw = qk.quant_mx4(torch.randn((33, 64), device=DEV))
    a, sa = qk.quant_mx4(torch.empty((0, 64), device=DEV))
    assert qk.gemm_mx4_scaled(a, w, sa, sw).shape == (0, 33)
    assert qk.gemm_mx4_scaled(w, a, sw, sa).shape == (33, 0)
    empty = torch.empty((33, 0), dtype=torch.uint8, device=DEV)
    assert not qk.gemm_mx4_scaled(empty, empty, empty, empty, out=torch.ones((33, 33), device=DEV)).any()
    assert not qk.linear_mx4(torch.empty((4, 0), device=DEV), empty, empty).any()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m,d", [(1, 32), (9, 224), (300, 1792)])
def test_silu(m, d, dtype):
    rng = np.random.default_rng(d)
    h = dev((rng.standard_normal((m, 2 * d)) * 4).astype(np.float32)).to(TORCH[dtype])
    q, scale = qk.silu_mul_quant_mx4(h)
    want_q, want_s = qk.quant_mx4(qk.silu_mul(h))
    assert torch.equal(q, want_q) and torch.equal(scale, want_s)
    check_quant(qk.silu_mul(h), q, scale)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_every_code_under_every_scale(dtype):
    q = np.zeros((256, 16), np.uint8)
    q[:, :8] = plain.pack(np.arange(16, dtype=np.uint8)[None])
    scale = np.arange(256, dtype=np.uint8)[:, None]
    want = plain.values(q, scale)
    room = torch.zeros((256, 16), dtype=torch.uint8, device=DEV)
    room[:, :1] = dev(scale)
    got = qk.dequant_mx4(dev(q), room[:, :1], TORCH[dtype]).cpu()
    assert torch.equal(got.double().nan_to_num(1.5, 1e300, -1e300),
                       torch.from_numpy(want).to(TORCH[dtype]).double().nan_to_num(1.5, 1e300, -1e300))
    # into rows that lie apart, at any alignment; the types of torch are taken too
    wide = torch.full((256, 75), 7.0, dtype=TORCH[dtype], device=DEV)
    qk.dequant_mx4(dev(q).view(torch.float4_e2m1fn_x2), room[:, :1].view(torch.float8_e8m0fnu), x=wide[:, 5:37])
    assert torch.equal(wide[:, 5:37].cpu().nan_to_num(1.5, 3e4), got.nan_to_num(1.5, 3e4))
    assert (wide[:, :5] == 7).all() and (wide[:, 37:] == 7).all()


class Operand:
    """Random codes and scales of `rows` rows; the scales' padding is NaN's byte,
    which must not matter."""

    def __init__(self, rng, rows, k, lo, hi):
        self.q = rng.integers(0, 256, (rows, k // 2), dtype=np.uint8)
        self.s = rng.integers(lo, hi + 1, (rows, k // 32), dtype=np.uint8)
        room = np.full((rows, (k // 32 + 15) // 16 * 16 + 16), 255, np.uint8)
        room[:, :k // 32] = self.s
        self.dev_q, self.dev_s = dev(self.q), dev(room)[:, :k // 32]

    def values(self):
        return plain.values(self.q, self.s)


SHAPES = [(1, 1, 32), (1, 16, 64), (1, 4096, 4096), (2, 33, 96), (15, 31, 128), (16, 64, 160), (17, 100, 512), (24, 512, 544),
          (33, 65, 1024), (48, 257, 2080), (64, 128, 2720), (65, 130, 96), (100, 1001, 1536), (128, 128, 128), (129, 255, 256),
          (200, 300, 640), (255, 257, 384), (256, 256, 512), (257, 513, 1184), (300, 1000, 32), (513, 384, 2048), (1000, 777, 480),
          (700, 1300, 7168), (2048, 2048, 256), (70, 40, 14336), (3, 50, 28672)]


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product_is_exact_where_sums_fit(m, n, k, out):
    # products are multiples of 2^-2, with scales 2^-1 .. 1 of 2^-4: while the sum of magnitudes stays below
    # 2^20 every partial sum, in any order, is a whole number of 2^-4 below 2^24 of them
    rng = np.random.default_rng(m + 3 * n + 7 * k)
    a, b = Operand(rng, m, k, 126, 127), Operand(rng, n, k, 126, 127)
    va, vb = a.values(), b.values()
    assert k * 36 < 2 ** 20
    want = va @ vb.T
    got = qk.gemm_mx4_scaled(a.dev_q, b.dev_q, a.dev_s, b.dev_s, output_scale=0.5, out_dtype=TORCH[out])
    assert got.dtype == TORCH[out] and got.shape == (m, n)
    want = torch.from_numpy(want * 0.5).to(TORCH[out])
    diff = got.cpu() != want
    assert not diff.any(), f"{int(diff.sum())} of {diff.numel()}, first at {diff.nonzero()[0].tolist()}"


@pytest.mark.parametrize("m,n,k", [(1, 500, 1024), (8, 64, 14336), (40, 100, 2720), (130, 300, 4096), (300, 500, 8192), (600, 520, 96)])
def test_product_of_any_scales(m, n, k):
    # binary32 sums of k exact products in any order, each rounded or cut: off by at most 2^-23 of the sum of
    # magnitudes per addition
    rng = np.random.default_rng(k + m)
    a, b = Operand(rng, m, k, 100, 140), Operand(rng, n, k, 107, 125)
    va, vb = a.values(), b.values()
    got = qk.gemm_mx4_scaled(a.dev_q, b.dev_q, a.dev_s, b.dev_s, out_dtype=torch.float32).cpu().double().numpy()
    err = np.abs(got - va @ vb.T)
    assert (err <= k * 2.0 ** -23 * (np.abs(va) @ np.abs(vb).T)).all()
    # a block's products cannot be lost in that: the error is far below the smallest change a block can make
    assert np.median(err / (np.abs(va) @ np.abs(vb).T)) < 2.0 ** -22


@pytest.mark.parametrize("m,n,k", [(1, 40, 96), (20, 70, 544), (300, 400, 2080), (300, 400, 2048)])
def test_nan_scales_reach_their_row_or_column_only(m, n, k):
    rng = np.random.default_rng(5)
    a, b = Operand(rng, m, k, 126, 127), Operand(rng, n, k, 126, 127)
    want = torch.from_numpy(a.values() @ b.values().T).float()
    row, col = m // 2, n - 1
    a.dev_s[row, k // 32 - 1] = 255
    b.dev_s[col, 0] = 255
    got = qk.gemm_mx4_scaled(a.dev_q, b.dev_q, a.dev_s, b.dev_s, out_dtype=torch.float32).cpu()
    want[row], want[:, col] = float("nan"), float("nan")
    assert torch.equal(got.nan_to_num(1e30), want.nan_to_num(1e30))


def test_extreme_scales():
    # 2^-127 and 2^127: products from 2^-254 (lost: binary32 ends at 2^-149) to beyond the largest number
    q = np.full((1, 16), 0x22, np.uint8)  # all ones
    one = np.zeros((6, 16), np.uint8)
    one[:, 0] = [0, 1, 127, 200, 253, 254]
    b = dev(np.repeat(q, 6, 0)), dev(one)[:, :1]
    for byte in (0, 1, 127, 254):
        s = torch.full((1, 16), byte, dtype=torch.uint8, device=DEV)
        got = qk.gemm_mx4_scaled(dev(q), b[0], s[:, :1], b[1], out_dtype=torch.float32).cpu().double().numpy()[0]
        want = 32.0 * 2.0 ** (one[:, 0].astype(np.float64) + byte - 254)
        ok = (np.abs(got - want) <= 2.0 ** -126) | (np.isinf(got) & (want >= 2.0 ** 128))
        assert ok.all(), (byte, got, want)


@pytest.mark.parametrize("m,n,k,dtype,out", [(1, 1001, 2720, "bf16", "bf16"), (24, 512, 1024, "f16", "f32"), (333, 1001, 2720, "f32", "f16"),
                                             (300, 512, 4096, "bf16", "f32")])
def test_linear_is_its_two_calls(m, n, k, dtype, out):
    rng = np.random.default_rng(n)
    wide = dev(rng.standard_normal((m, k + 9)).astype(np.float32)).to(TORCH[dtype])
    x = wide[:, 2:2 + k]
    w, sw = qk.quant_mx4(dev(rng.standard_normal((n, k)).astype(np.float32)))
    q, s = qk.quant_mx4(x)
    want = qk.gemm_mx4_scaled(q, w, s, sw, 0.25, TORCH[out])
    room = torch.empty((m, n), dtype=TORCH[out], device=DEV)
    got = qk.linear_mx4(x, w, sw, 0.25, out=room)
    assert got.data_ptr() == room.data_ptr() and torch.equal(got, want)
    full = plain.values(q.cpu().numpy(), s.cpu().numpy()) @ plain.values(w.cpu().numpy(), sw.cpu().numpy()).T * 0.25
    # binary32 sums as above, then the output's rounding
    eps = torch.finfo(TORCH[out]).eps / 2
    size = np.abs(plain.values(q.cpu().numpy(), s.cpu().numpy())) @ np.abs(plain.values(w.cpu().numpy(), sw.cpu().numpy()).T) * 0.25
    assert (np.abs(got.cpu().double().numpy() - full) <= eps * np.abs(full) + k * 2.0 ** -23 * size + 2.0 ** -25).all()


def test_codes_beyond_4_gib():
    n, k = (1 << 20) + 5, 8224
    w = torch.zeros((n, k // 2), dtype=torch.uint8, device=DEV)
    room = torch.full((n, 272), 127, dtype=torch.uint8, device=DEV)
    w[-3:] = 0x22  # ones
    a, sa = qk.quant_mx4(torch.ones((2, k), device=DEV))
    got = qk.gemm_mx4_scaled(a, w, sa, room[:, :k // 32], out_dtype=torch.float32)
    assert (got[:, -3:] == k).all() and not got[:, :-3].any()
    back = qk.dequant_mx4(w[-4:], room[-4:, :k // 32], torch.float32)
    assert (back[1:] == 1).all() and not back[0].any()


def test_graph_and_streams():
    rng = np.random.default_rng(9)
    x = dev(rng.standard_normal((70, 1024)).astype(np.float32)).to(torch.bfloat16)
    w, sw = qk.quant_mx4(dev(rng.standard_normal((600, 1024)).astype(np.float32)))
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        qk.linear_mx4(x, w, sw)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            out = qk.linear_mx4(x, w, sw)
    for i in range(3):
        x.copy_(dev(rng.standard_normal((70, 1024)).astype(np.float32)))
        want = qk.linear_mx4(x, w, sw)
        torch.cuda.synchronize()
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i


def test_refusals():
    x = torch.zeros((4, 64), device=DEV)
    q, s = qk.quant_mx4(x)
    with pytest.raises(ValueError, match="multiple of 32"):
        qk.quant_mx4(x[:, :48])
    with pytest.raises(ValueError, match="multiple of 32"):
        qk.silu_mul_quant_mx4(x[:, :32])
    with pytest.raises(TypeError):
        qk.quant_mx4(x.double())
    with pytest.raises(ValueError):
        qk.quant_mx4(x.t())
    with pytest.raises(ValueError):
        qk.quant_mx4(x, q[:3], s[:3])
    with pytest.raises(TypeError):
        qk.quant_mx4(x, q.view(torch.int8), s)
    with pytest.raises(ValueError, match="16"):
        qk.quant_mx4(x, q, torch.zeros((4, 2), dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="16"):
        qk.gemm_mx4_scaled(q, q, s, torch.zeros((4, 2), dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="16"):  # the last row ends early
        qk.gemm_mx4_scaled(q, q, s, torch.zeros(50, dtype=torch.uint8, device=DEV).as_strided((4, 2), (16, 1)))
    with pytest.raises(qk.QKError):             # rows at multiples of 16 from a place that is none
        qk.gemm_mx4_scaled(q, q, s, torch.zeros(100, dtype=torch.uint8, device=DEV)[8:].as_strided((4, 2), (16, 1), 8))
    with pytest.raises(ValueError, match="inner dimensions"):
        qk.gemm_mx4_scaled(q[:, :16].contiguous(), q, s[:, :1], s)
    with pytest.raises(ValueError):
        qk.gemm_mx4_scaled(q, q, s[:3], s)
    with pytest.raises(TypeError):
        qk.gemm_mx4_scaled(q, q, s, s, out_dtype=torch.float64)
    with pytest.raises(ValueError):
        qk.gemm_mx4_scaled(q, q, s, s, out=torch.zeros((4, 5), device=DEV))
    with pytest.raises(ValueError, match="inner dimensions"):
        qk.linear_mx4(torch.zeros((4, 96), device=DEV), q, s)
    with pytest.raises(TypeError):
        qk.dequant_mx4(q, s, torch.float64)
    with pytest.raises(ValueError):
        qk.dequant_mx4(q, s, x=x[:, :32])
    with pytest.raises(ValueError, match="GPU"):
        qk.dequant_mx4(q.cpu(), s)
