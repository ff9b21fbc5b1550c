"""Norm and rotation of calls with thousands of rows, where a wave goes on from one
group of heads to the next and from queries to keys, and large outputs are stored past
the caches."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import w8a8_int8_quantized_qk_amd as qk

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qk.library()


def plain(x, w, pos, freqs, eps, interleaved):
    """(y, bound before the output's rounding) in binary64, the bound as for small calls:
    a sum of dim squares, mean, root, quotient and two products in binary32; sine and cosine
    within 2^-22, two products and their sum."""
    y, rel, dim = x.double(), 0.0, x.shape[-1]
    if w is not None:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
        rel = (dim + 8) * 2.0 ** -24
    r = 2 * freqs.numel()
    a = slice(0, r, 2) if interleaved else slice(0, r // 2)
    b = slice(1, r, 2) if interleaved else slice(r // 2, r)
    t = pos.double()[:, None, None] * freqs
    out, bound = y.clone(), rel * y.abs()
    out[..., a] = y[..., a] * t.cos() - y[..., b] * t.sin()
    out[..., b] = y[..., b] * t.cos() + y[..., a] * t.sin()
    bound[..., a] = bound[..., b] = (y[..., a].abs() + y[..., b].abs()) * (rel + 2.0 ** -22 + 2.0 ** -23)
    return out, bound


def check(got, want, bound, what):
    f = torch.finfo(got.dtype)
    err = (got.double() - want).abs_()
    bad = ~(err <= bound + f.eps / 2 * (want.abs() + bound) + f.tiny * f.eps / 2)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}, first at {bad.nonzero()[0].tolist()}"


# Calls of more than 16384 rows times groups of heads give a wave two groups, three (of queries and
# of keys, where three does not divide the queries'), or all of a row's.
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,heads,kv_heads,dim,rotary", [(4001, 32, 8, 128, 128), (6007, 32, 8, 128, 64), (9001, 32, 8, 128, 128),
                                                            (9001, 20, 5, 64, 64), (6001, 9, 3, 256, 256), (9001, 7, 2, 80, 20),
                                                            (17000, 5, 1, 96, 96), (2500, 24, 8, 192, 2)])
def test_many_rows(rows, heads, kv_heads, dim, rotary, dtype, interleaved):
    gen = torch.Generator(device=DEV).manual_seed(rows + dim)
    wide = torch.randn((rows, (heads + 2 * kv_heads) * dim + 3), generator=gen, device=DEV).to(TORCH[dtype])
    q = wide[:, 1:1 + heads * dim].view(rows, heads, dim)
    k = wide[:, 1 + heads * dim:1 + (heads + kv_heads) * dim].view(rows, kv_heads, dim)
    w = [(1 + 0.3 * torch.randn(dim, generator=gen, device=DEV)).to(TORCH[dtype]) for _ in range(2)]
    freqs = 10000.0 ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device=DEV) / rotary)
    # four sequences; rows before the first and behind the last belong to none
    cu = [3, rows // 5, rows // 5, rows - 1000, rows - 7]
    starts = [0, 9, 4095, 60000]
    pos = np.zeros(rows, np.int64)
    for s, a, b in zip(starts, cu, cu[1:]):
        pos[a:b] = np.arange(s, s + b - a)
    pos = torch.from_numpy(pos).to(DEV)
    cu_dev, start = (torch.tensor(v, dtype=torch.int32, device=DEV) for v in (cu, starts))
    mine = slice(cu[0], cu[-1])
    room = torch.full_like(wide, 7.0)  # outputs that lie apart, at an odd place
    outs = (room[:, 1:1 + heads * dim].view(rows, heads, dim),
            room[:, 1 + heads * dim:1 + (heads + kv_heads) * dim].view(rows, kv_heads, dim))
    assert rows * (heads + kv_heads) * dim * q.element_size() > 8 << 20  # stored past the caches
    qk.norm_rope(q, k, start, freqs, cu_dev, w[0], w[1], 1e-6, interleaved, *outs)
    for name, x, weight, o in (("q", q, w[0], outs[0]), ("k", k, w[1], outs[1])):
        check(o[mine], *plain(x[mine], weight, pos[mine], freqs, 1e-6, interleaved), name)
        assert (o[:cu[0]] == 7).all() and (o[cu[-1]:] == 7).all(), "rows of no sequence"
    n = (heads + kv_heads) * dim + 1
    assert (room[:, :1] == 7).all() and (room[:, n:] == 7).all(), "beside the heads"
    # the same call in place, and few rows at a time: the same bits
    few = slice(cu[2], cu[2] + 40)
    part = qk.norm_rope(q[few], k[few], start[2:3], freqs, torch.tensor([0, 40], dtype=torch.int32, device=DEV), w[0], w[1], 1e-6, interleaved)
    assert torch.equal(part[0], outs[0][few]) and torch.equal(part[1], outs[1][few])
    before = wide.clone()
    qk.norm_rope(q, k, start, freqs, cu_dev, w[0], w[1], 1e-6, interleaved, q, k)
    assert torch.equal(q[mine], outs[0][mine]) and torch.equal(k[mine], outs[1][mine])
    before[mine, 1:n] = wide[mine, 1:n]
    assert torch.equal(before, wide)


@pytest.mark.parametrize("heads,kv_heads", [(32, 0), (0, 8), (8, 32)])
def test_many_rows_of_one_kind(heads, kv_heads):
    rows, dim = 9001, 128
    gen = torch.Generator(device=DEV).manual_seed(1)
    q, k = (torch.randn((rows, h, dim), generator=gen, device=DEV).to(torch.bfloat16) for h in (heads, kv_heads))
    start = torch.arange(rows, dtype=torch.int32, device=DEV)
    freqs = 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64, device=DEV) / dim)
    w = torch.ones(dim, dtype=torch.bfloat16, device=DEV)
    out = qk.norm_rope(q, k, start, freqs, None, None, w)
    for name, x, weight, o in (("q", q, None, out[0]), ("k", k, w, out[1])):
        check(o, *plain(x, weight, start, freqs, 1e-6, False), name)
