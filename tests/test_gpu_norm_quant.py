"""GPU parity of the root-mean-square norm with 8-bit output (qk_rms_norm_quant).

After the binary64 root every step is one IEEE binary32 operation, so codes,
scales and the rounded residual sum must have the plain implementation's bits.
(The binary64 sum's own last bits depend on the order of addition; they move
the rounded root only when it lies within 2^-50 of a rounding boundary, which
none of the seeded rows here does.)
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import w8a8_int8_quantized_qk_amd as qk
from tests import plain_decoder as plain

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qk.library()


def _check(x, w, res, fp8, got, eps=EPS):
    q, s = got[0], got[1]
    codes, scale, r = plain.norm(plain.f32(x), plain.f32(w), eps, None if res is None else plain.f32(res), fp8)
    gq, gs = q.view(torch.uint8).cpu().numpy(), s.cpu().numpy()
    nan = np.isnan(scale)
    assert np.array_equal(np.isnan(gs), nan)
    assert np.array_equal(gs[~nan].view(np.uint32), scale[~nan].view(np.uint32))
    assert np.array_equal(gq, codes), f"{(gq != codes).sum()} codes differ"
    if res is not None:
        want = torch.from_numpy(r).to(x.dtype)
        assert torch.equal(got[2].cpu().nan_to_num(nan=7.0), want.nan_to_num(nan=7.0))


def _inputs(seed, m, k, dtype, residual=True, w32=False):
    g = torch.Generator().manual_seed(seed)
    dt = plain.TORCH[dtype]
    x = torch.randn(m, k, generator=g).to(dt)
    w = (1 + 0.3 * torch.randn(k, generator=g)).to(torch.float32 if w32 else dt)
    res = (torch.randn(m, k, generator=g) * 4).to(dt) if residual else None
    return x.to(DEV), w.to(DEV), None if res is None else res.to(DEV)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m,k", [(1, 1), (3, 7), (5, 64), (9, 512), (4, 1000), (2, 1025), (7, 2047), (3, 4096), (2, 8200),
                                 (2, 16385), (1, 40001)])
def test_codes_scales_and_residual(m, k, dtype, fp8):
    for residual in (True, False):
        x, w, res = _inputs(m * 100003 + k, m, k, dtype, residual, w32=m % 2 == 0)
        _check(x, w, res, fp8, qk.rms_norm_quant(x, w, EPS, residual=res, fp8=fp8))


@pytest.mark.parametrize("k", [96, 4099, 20000])
def test_in_place_residual_and_row_strides(k):
    m = 6
    wide, w, wide_res = _inputs(k, m, k + 13, "bf16")
    x, res, w = wide[:, 3:3 + k], wide_res[:, 5:5 + k], w[:k].contiguous()
    want = plain.norm(plain.f32(x), plain.f32(w), EPS, plain.f32(res), False)
    around = wide_res.clone()
    q, s, out = qk.rms_norm_quant(x, w, EPS, residual=res, residual_out=res)
    assert out is res
    assert np.array_equal(q.cpu().numpy().view(np.uint8), want[0])
    assert np.array_equal(s.cpu().numpy(), want[1])
    assert torch.equal(res.cpu(), torch.from_numpy(want[2]).to(torch.bfloat16))
    assert torch.equal(wide_res[:, :5], around[:, :5]) and torch.equal(wide_res[:, 5 + k:], around[:, 5 + k:])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("k", [65, 4096])
def test_special_rows(k, fp8):
    x, w, res = _inputs(k, 8, k, "f32")
    x[0] = 0
    res[0] = 0                       # an all-zero row: the guard's scale, codes 0
    x[1, k // 2] = float("inf")
    x[2, 3] = float("nan")
    x[3] *= 1e30                     # squares beyond binary32
    res[3] *= 1e30
    x[4] *= 1e-30                    # eps decides
    res[4] *= 1e-30
    x[5, 0] = -float("inf")
    x[6] = 1e-42                     # subnormal
    res[6] = 0
    got = qk.rms_norm_quant(x, w, EPS, residual=res, fp8=fp8)
    _check(x, w, res, fp8, got)
    assert np.isnan(got[1].cpu().numpy()[[1, 2, 5]]).all()
    assert not got[0].view(torch.uint8)[[0, 1, 2, 5]].any()
    # a weight that overflows a row's maximum
    w[1] = float("inf")
    got = qk.rms_norm_quant(x[7:], w, EPS, fp8=fp8)
    _check(x[7:], w, None, fp8, got)
    assert not torch.isfinite(got[1]).any()


def test_eps_zero_and_empty():
    x, w, _ = _inputs(1, 4, 128, "bf16", False)
    _check(x, w, None, False, qk.rms_norm_quant(x, w, 0.0), eps=0.0)
    q, s = qk.rms_norm_quant(x[:0], w)
    assert q.shape == (0, 128) and s.shape == (0,)
    q, s = qk.rms_norm_quant(x[:, :0].contiguous(), w[:0].contiguous())
    assert q.shape == (4, 0) and torch.equal(s.cpu(), torch.full((4,), np.float32(1e-12)) / 127)


def test_feeds_the_linear_layer():
    x, w, res = _inputs(5, 20, 512, "bf16")
    q, s, _ = qk.rms_norm_quant(x, w, EPS, residual=res)
    b = torch.randint(-127, 128, (512, 256), dtype=torch.int8, device=DEV)
    acc = qk.gemm_i8_scaled(q, b, out_dtype=None).cpu()
    assert torch.equal(acc.long(), q.cpu().long() @ b.cpu().long())


def test_on_another_stream():
    x, w, res = _inputs(9, 64, 4096, "bf16")
    want = qk.rms_norm_quant(x, w, EPS, residual=res)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = qk.rms_norm_quant(x, w, EPS, residual=res)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("m", [1, 6])
def test_rows_side_by_side_in_one_buffer(m):
    # x, residual and sum as columns of one buffer (also with a stride of two rows) share no element
    k = 40
    wide, w, _ = _inputs(3, 2 * m, 3 * k, "bf16", False)
    w = w[:k].contiguous()
    x, res = wide[:m, :k], wide[:m, k:2 * k]
    for out in (wide[:m, 2 * k:], wide[::2, 2 * k:], wide[m:, k:2 * k]):
        want = qk.rms_norm_quant(x, w, EPS, residual=res)
        got = qk.rms_norm_quant(x, w, EPS, residual=res, residual_out=out)
        for a, b in zip(want, got):
            assert torch.equal(a, b)
    for inplace in (x.clone(), res.clone()):
        pair = (inplace, res) if torch.equal(inplace, x) else (x, inplace)
        got = qk.rms_norm_quant(pair[0], w, EPS, residual=pair[1], residual_out=inplace)
        for a, b in zip(want, got):
            assert torch.equal(a, b)
    with pytest.raises(qk.QKError, match="INVALID"):
        qk.rms_norm_quant(x, w, EPS, residual=res, residual_out=wide[:m, k + 1:2 * k + 1])


def test_more_rows_than_one_grid():
    m, k = (1 << 24) + 5, 5                       # one workgroup a row
    g = torch.Generator(device=DEV).manual_seed(6)
    x = torch.randn((m, k), generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)
    res = torch.randn((m, k + 1), generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)[:, 1:]
    w = torch.rand((k,), generator=g, device=DEV, dtype=torch.float32)
    got = qk.rms_norm_quant(x, w, EPS, residual=res)
    for at in (0, (1 << 23) - 3, (1 << 24) - 3):
        rows = slice(at, at + 8)
        _check(x[rows], w, res[rows], False, [t[rows] for t in got])


def test_refusals():
    x, w, res = _inputs(2, 4, 64, "bf16")
    with pytest.raises(TypeError):
        qk.rms_norm_quant(x.double(), w)
    with pytest.raises(TypeError):
        qk.rms_norm_quant(x, w.half())
    with pytest.raises(ValueError):
        qk.rms_norm_quant(x, w[:63])
    with pytest.raises(ValueError):
        qk.rms_norm_quant(x.t(), w[:4])
    with pytest.raises(ValueError):
        qk.rms_norm_quant(x, w, residual=res[:3])
    with pytest.raises(TypeError):
        qk.rms_norm_quant(x, w, residual=res.float())
    with pytest.raises(ValueError):
        qk.rms_norm_quant(x, w, residual_out=res)
    with pytest.raises(TypeError):
        qk.rms_norm_quant(x, w, q=torch.empty((4, 64), dtype=torch.uint8, device=DEV))
    with pytest.raises(qk.QKError):
        qk.rms_norm_quant(x, w, eps=-1.0)


@pytest.mark.parametrize("dtype,k,in_place", [(torch.bfloat16, 8195, True), (torch.float32, 4097, False)])
def test_large_calls_give_what_their_rows_give(dtype, k, in_place):
    # more than 160 MB read: past the caches; the same rows a few at a time go through them
    m = 170_000_000 // (2 * k * dtype.itemsize)
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn((m, k + 3), generator=g, device=DEV, dtype=torch.float32).to(dtype)[:, :k]
    res = torch.randn((m, k), generator=g, device=DEV, dtype=torch.float32).to(dtype)
    w = torch.rand((k,), generator=g, device=DEV, dtype=torch.float32).to(dtype)
    rows = [0, 1, m // 2, m - 1]
    want = qk.rms_norm_quant(x[rows], w, EPS, residual=res[rows])
    got = qk.rms_norm_quant(x, w, EPS, residual=res, residual_out=res if in_place else None)
    for a, b in zip(want, got):
        assert torch.equal(a, b[rows])
