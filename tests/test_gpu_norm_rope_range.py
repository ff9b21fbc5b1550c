"""Norm and rotation of heads whose squares leave binary32's range: any finite
head has the formula's norm."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import w8a8_int8_quantized_qk_amd as qk
from tests.test_gpu_norm_rope import Setup, plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qk.library()


def check(t, out, eps, interleaved):
    """Against binary64.  `plain`'s bound is relative; elements far below their head's
    largest come to subnormal numbers, where each of at most eight roundings (two of the
    norm, two of the pair's norms, two products, their sum, the output) is off by up to
    half the type's or binary32's last step instead."""
    for name, x, w, o in (("q", t.q, t.w[0], out[0]), ("k", t.k, t.w[1], out[1])):
        want, bound = plain(x, w, t.pos, t.freqs, eps, interleaved)
        f = torch.finfo(o.dtype)
        last = max(f.tiny * f.eps, 2.0 ** -149)
        tol = bound + f.eps / 2 * (np.abs(want) + bound) + last / 2 + 8 * 2.0 ** -150
        err = np.abs(o.double().cpu().numpy() - want)
        assert np.isfinite(err).all(), f"{name}: {(~np.isfinite(err)).sum()} of {err.size} not finite"
        assert (err <= tol).all(), f"{name}: {(err > tol).sum()} of {err.size}, worst {err[err > tol].max()}"


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rotary", [(16, 16), (64, 64), (80, 20), (128, 64), (192, 192), (256, 128), (256, 254)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [2.0 ** 62, 2.0 ** 64, 1e30, 2.0 ** 120])
def test_large_heads(size, dtype, dim, rotary, interleaved):
    t = Setup(dim + rotary, [3, 4], [0, 900], 5, 2, dim, rotary, dtype)
    t.q[1:3] *= size
    t.k[5, 1] *= size
    t.q[4, 2, dim // 2] = 3e38  # one element among ordinary ones
    check(t, t.run(interleaved=interleaved), 1e-6, interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rotary", [(16, 16), (64, 64), (80, 20), (128, 64), (192, 192), (256, 128), (256, 254)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [2.0 ** -60, 1e-25, 2.0 ** -120, 2.0 ** -130])
def test_small_heads_without_eps(size, dtype, dim, rotary, interleaved):
    t = Setup(dim + rotary, [3, 4], [0, 900], 5, 2, dim, rotary, dtype)
    t.q[1:3] *= size
    t.k[5, 1] *= size
    t.q[4, 2] = 0
    t.q[4, 2, dim // 2] = torch.finfo(t.q.dtype).smallest_normal  # alone in its head
    check(t, t.run(eps=0.0, interleaved=interleaved), 0.0, interleaved)


def test_the_smallest_number():
    # 2^-149 in a head of 256: the root of its mean square is 2^-153
    t = Setup(1, [2], [0], 2, 1, 256, 0, "f32")
    t.q[1, 1] = 0
    t.q[1, 1, 77] = 2.0 ** -149
    assert t.q[1, 1, 77] > 0
    check(t, t.run(eps=0.0), 0.0, False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_other_heads_keep_their_bits(dtype):
    t = Setup(8, [5], [10], 16, 4, 64, 64, dtype)
    want = t.run(eps=0.0)
    t.q[2, 1] *= 1e30
    t.q[3, 7] *= 1e-30
    t.k[0, 2] *= 2.0 ** 100
    out = t.run(eps=0.0)
    for o, w, at in ((out[0], want[0], [(2, 1), (3, 7)]), (out[1], want[1], [(0, 2)])):
        same = torch.ones(o.shape[:2], dtype=torch.bool, device=o.device)
        for i in at:
            same[i] = False
        assert torch.equal(o[same], w[same])
    check(t, out, 0.0, False)


def test_a_head_of_zeros():
    t = Setup(9, [3], [10], 4, 2, 64, 64, "bf16")
    t.q[1, 2] = 0
    assert not t.run()[0][1, 2].any()
    assert t.run(eps=0.0)[0][1, 2].isnan().all()  # 0 / 0
