"""GPU parity of writing and reading the paged 8-bit cache: code bytes and
scales as the plain implementation's, bit for bit, for whole pools (so that
bytes that a call must not touch are covered too)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import w8a8_int8_quantized_qk_amd as qk
from tests import plain_decoder as plain

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qk.library()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def random_cache(rng, blocks, heads, dim, block, fp8):
    """A pool of arbitrary bytes (every FP8 code, NaN among them) and ordinary scales."""
    c = qk.new_kv_cache(blocks, heads, dim, block, fp8, DEV)
    for t in (c.k, c.v):
        t.view(torch.uint8).copy_(dev(rng.integers(0, 256, t.shape, dtype=np.uint8)))
    for t in (c.k_scale, c.v_scale):
        t.copy_(dev(rng.uniform(1e-3, 1e-1, t.shape).astype(np.float32)))
    return c


def same(cache, want, what=""):
    for got, w, name in ((cache.k, want.k, "k"), (cache.v, want.v, "v")):
        got = got.view(torch.uint8).cpu().numpy()
        assert np.array_equal(got, w), f"{what} {name}: {(got != w).sum()} bytes differ"
    for got, w, name in ((cache.k_scale, want.ks, "k_scale"), (cache.v_scale, want.vs, "v_scale")):
        got = got.cpu().numpy()
        ok = (got.view(np.uint32) == w.view(np.uint32)) | (np.isnan(got) & np.isnan(w))
        assert ok.all(), f"{what} {name}: {(~ok).sum()} differ"


def rows(rng, tokens, heads, dim, dtype, grow=None):
    k = rng.standard_normal((tokens, heads, dim)).astype(np.float32)
    v = rng.standard_normal((tokens, heads, dim)).astype(np.float32)
    if grow is not None:
        k *= grow
        v *= grow
    dt = plain.TORCH[dtype]
    return dev(k).to(dt), dev(v).to(dt)


def write(cache, k, v, table, start, counts):
    cu = plain.offsets(counts)
    out = qk.kv_cache_write(cache, k, v, dev(table), dev(np.asarray(start, np.int32)), dev(cu))
    assert out is cache
    return cu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("heads,dim,block", [(1, 16, 16), (2, 64, 32), (3, 80, 64), (2, 128, 16), (2, 112, 128), (1, 256, 64),
                                             (5, 128, 128), (1, 240, 16)])
def test_prompt_then_tokens(heads, dim, block, dtype, fp8):
    rng = np.random.default_rng(heads * 1000 + dim + block)
    counts = [1, 0, block, block + 1, 3 * block - 1, 17]
    more = 5
    table, blocks = plain.tables(rng, [n + 2 * block for n in counts], block)
    cache = random_cache(rng, blocks, heads, dim, block, fp8)
    want = plain.Cache(cache, fp8)
    start = [0, 0, 0, 0, 0, 0]
    k, v = rows(rng, sum(counts), heads, dim, dtype)
    cu = write(cache, k, v, table, start, counts)
    want.write(plain.f32(k), plain.f32(v), table, start, cu)
    same(cache, want, "prompt")
    # further tokens one call at a time, growing, so that scales grow too; some calls skip sequences
    start = list(counts)
    for step in range(more):
        counts = [(step + i) % 3 != 0 for i in range(len(start))] if step < more - 1 else [3, 1, block + 3, 0, 2, 9]
        counts = [int(c) for c in counts]
        k, v = rows(rng, sum(counts), heads, dim, dtype, grow=1 + 0.5 * step)
        cu = write(cache, k, v, table, start, counts)
        want.write(plain.f32(k), plain.f32(v), table, start, cu)
        same(cache, want, f"step {step}")
        start = [a + b for a, b in zip(start, counts)]


@pytest.mark.parametrize("fp8", [False, True])
def test_writing_twice_changes_nothing(fp8):
    rng = np.random.default_rng(3)
    table, blocks = plain.tables(rng, [40, 70], 32)
    cache = random_cache(rng, blocks, 2, 64, 32, fp8)
    k, v = rows(rng, 20, 2, 64, "bf16", grow=3)
    write(cache, k, v, table, [25, 41], [11, 9])
    first = plain.Cache(cache, fp8)
    write(cache, k, v, table, [25, 41], [11, 9])
    same(cache, first)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("block", [16, 64])
def test_non_finite_tokens_and_zero_tokens(block, fp8):
    rng = np.random.default_rng(block)
    table, blocks = plain.tables(rng, [block] * 5, block)
    cache = random_cache(rng, blocks, 1, 32, block, fp8)
    want = plain.Cache(cache, fp8)
    counts = [block - 3] * 5
    k, v = rows(rng, sum(counts), 1, 32, "f32")
    k[3, 0, 5] = float("nan")
    v[counts[0] + 2, 0, 1] = float("inf")
    k[2 * counts[0]:3 * counts[0]] = 0
    k[3 * counts[0]] = 1e-40
    v[4 * counts[0]:] *= 1e30
    cu = write(cache, k, v, table, [0] * 5, counts)
    want.write(plain.f32(k), plain.f32(v), table, [0] * 5, cu)
    same(cache, want)
    # a later finite token does not mend a NaN scale; an infinite one spoils a good block
    k, v = rows(rng, 5, 1, 32, "f32")
    k[4] = -float("inf")
    cu = write(cache, k, v, table, counts, [1] * 5)
    want.write(plain.f32(k), plain.f32(v), table, counts, cu)
    same(cache, want)
    # a block begun anew is finite again
    k, v = rows(rng, 5, 1, 32, "f32")
    cu = write(cache, k, v, table, [0] * 5, [1] * 5)
    want.write(plain.f32(k), plain.f32(v), table, [0] * 5, cu)
    same(cache, want)
    assert torch.isfinite(cache.k_scale).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("block", [16, 64])
def test_every_earlier_code_and_negative_and_zero_scales(block, fp8):
    # a cache filled elsewhere: all 256 codes among the earlier tokens (-128 and NaN too), and scales that
    # are tiny, negative (also beyond the new one in size) or 0 when a block is continued
    rng = np.random.default_rng(block)
    n = 12
    table, blocks = plain.tables(rng, [block] * n, block)
    cache = random_cache(rng, blocks, 1, 64, block, fp8)
    factor = dev(np.resize(np.array([0.999, 0.5, -0.4, -30.0, 0.0, 1e-39], np.float32), (n, 1)))
    top = 448 if fp8 else 127
    for t in (cache.k_scale, cache.v_scale):
        t[dev(table[:, 0].astype(np.int64))] = factor / top
    want = plain.Cache(cache, fp8)
    k, v = rows(rng, n, 1, 64, "f32")
    k[:, 0, 0], v[:, 0, 0] = 4.0, -4.0                  # more than any other token: the new scale is 4 / top
    cu = write(cache, k, v, table, [block - 2] * n, [1] * n)
    want.write(plain.f32(k), plain.f32(v), table, [block - 2] * n, cu)
    if fp8:                                             # which NaN a NaN becomes is not part of the format
        for t in (cache.k, cache.v, want.k, want.v):
            b = t.view(torch.uint8) if isinstance(t, torch.Tensor) else t
            b[(b & 0x7F) == 0x7F] = 0x7F
    same(cache, want)


def test_many_sequences_and_slices_of_a_projection():
    # more sequences than a wave has lanes, rows of one fused projection
    rng = np.random.default_rng(8)
    n, heads, dim, block = 150, 2, 48, 16
    start = rng.integers(0, 40, n).tolist()
    counts = rng.integers(0, 4, n).tolist()
    table, blocks = plain.tables(rng, [a + b for a, b in zip(start, counts)], block)
    cache = random_cache(rng, blocks, heads, dim, block, False)
    want = plain.Cache(cache, False)
    proj = dev(rng.standard_normal((sum(counts), 3 * heads * dim + 7)).astype(np.float32)).to(torch.bfloat16)
    k = proj[:, 1:1 + heads * dim].unflatten(1, (heads, dim))
    v = proj[:, 5 + heads * dim:5 + 2 * heads * dim].unflatten(1, (heads, dim))
    cu = write(cache, k, v, table, start, counts)
    want.write(plain.f32(k), plain.f32(v), table, start, cu)
    same(cache, want)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("heads,dim,block", [(1, 16, 128), (2, 80, 16), (3, 128, 64), (1, 256, 32)])
def test_read_back(heads, dim, block, dtype, fp8):
    rng = np.random.default_rng(heads + dim + block)
    start, counts = [0, 5, block, 0, 3], [1, 2 * block, block + 1, 0, 7]
    lens = [a + b for a, b in zip(start, counts)]
    table, blocks = plain.tables(rng, lens, block)
    cache = random_cache(rng, blocks, heads, dim, block, fp8)
    if fp8:  # NaN codes read as NaN; compare finite ones only through ordinary bytes
        for t in (cache.k, cache.v):
            b = t.view(torch.uint8)
            b[(b & 0x7F) == 0x7F] = 0x3A
    host = plain.Cache(cache, fp8)
    cu = plain.offsets(counts)
    guard = torch.full((sum(counts) + 2, heads, dim), 77.0, dtype=plain.TORCH[dtype], device=DEV)
    vout = guard.clone()
    k, v = qk.kv_cache_read(cache, dev(table), dev(np.asarray(start, np.int32)), dev(cu), sum(counts),
                            k=guard[:sum(counts)], v=vout[:sum(counts)])
    for s, n in enumerate(counts):
        wk, wv = host.values(table[s], lens[s])
        for got, w in ((k, wk), (v, wv)):
            w = torch.from_numpy(w[start[s]:]).to(plain.TORCH[dtype])
            assert torch.equal(got[cu[s]:cu[s + 1]].cpu(), w), s
    assert (guard[-2:] == 77).all() and (vout[-2:] == 77).all()
    a, b = qk.kv_cache_read(cache, dev(table), dev(np.asarray(start, np.int32)), dev(cu), sum(counts),
                            plain.TORCH[dtype])
    assert torch.equal(a, k) and torch.equal(b, v)


def test_indices_out_of_range_touch_nothing():
    # block numbers, table columns and rows that point outside are dropped
    rng = np.random.default_rng(1)
    cache = random_cache(rng, 6, 1, 32, 16, False)
    want = plain.Cache(cache, False)
    k, v = rows(rng, 12, 1, 32, "f32")
    table = np.array([[6, 0], [-1, 1], [2, 3]], np.int32)
    # sequence 0: block 6 of 6; 1: block -1; 2: position 30 on, 4 tokens reach column 2 of 2
    cu = write(cache, k, v, table, [0, 3, 30], [4, 4, 4])
    for s, n in ((2, 2),):
        want.write(plain.f32(k)[8:], plain.f32(v)[8:], table[2:], [30], plain.offsets([n]))
    same(cache, want)
    # offsets beyond the rows that there are
    bad = np.array([0, 4, 8, 13], np.int32)
    qk.kv_cache_write(cache, k, v, dev(table), dev(np.array([0, 3, 0], np.int32)), dev(bad))
    same(cache, want)
    assert cu[-1] == 12


def test_a_pool_beyond_32_bit_offsets():
    # 5 GB of keys and 5 GB of values: byte offsets of the last blocks pass 2^32
    heads, dim, block, blocks = 8, 128, 128, 40000
    cache = qk.new_kv_cache(blocks, heads, dim, block, False, DEV)
    rng = np.random.default_rng(2)
    table = np.array([[blocks - 1, 0, blocks - 2]], np.int32)
    k, v = rows(rng, 300, heads, dim, "bf16")
    cu = write(cache, k, v, table, [0], [300])
    rk, rv = qk.kv_cache_read(cache, dev(table), dev(np.zeros(1, np.int32)), dev(cu), 300, torch.float32)
    for got, x, s in ((rk, k, cache.k_scale), (rv, v, cache.v_scale)):
        step = s[torch.from_numpy(table[0].astype(np.int64)).to(DEV)].repeat_interleave(block, 0)[:300, :, None]
        assert torch.equal(got, (x.float() / step).round() * step)
    q = torch.from_numpy(rng.standard_normal((1, heads, dim)).astype(np.float32)).to(DEV).to(torch.bfloat16)
    out = qk.kv_attention(q, cache, dev(table), dev(np.array([300], np.int32)))
    want, _, bound, _ = plain.attention(plain.f32(q), plain.f32(rk), plain.f32(rv), 300, dim ** -0.5, 0)
    assert plain.within(out, want, bound).all()


def test_refusals():
    rng = np.random.default_rng(0)
    cache = random_cache(rng, 4, 2, 32, 16, False)
    k, v = rows(rng, 3, 2, 32, "bf16")
    table, start, cu = dev(np.zeros((1, 1), np.int32)), dev(np.zeros(1, np.int32)), dev(np.array([0, 3], np.int32))
    qk.kv_cache_write(cache, k, v, table, start, cu)
    with pytest.raises(TypeError):
        qk.kv_cache_write(cache, k, v.float(), table, start, cu)
    with pytest.raises(ValueError):
        qk.kv_cache_write(cache, k[:, :1], v[:, :1], table, start, cu)
    with pytest.raises(ValueError):
        qk.kv_cache_write(cache, k.transpose(1, 2), v.transpose(1, 2), table, start, cu)
    with pytest.raises(TypeError):
        qk.kv_cache_write(cache, k, v, table.long(), start, cu)
    with pytest.raises(ValueError):
        qk.kv_cache_write(cache, k, v, table, start, cu[:1])
    with pytest.raises(ValueError):
        qk.kv_cache_write(cache, k, v, table.repeat(2, 1), start, cu)
    with pytest.raises(ValueError):
        qk.kv_cache_write(cache._replace(v=cache.k), k, v, table, start, cu)
    with pytest.raises(TypeError):
        qk.kv_cache_write(cache._replace(k=cache.k.view(torch.uint8)), k, v, table, start, cu)
    with pytest.raises(ValueError):
        qk.kv_cache_write(cache, k.cpu(), v.cpu(), table, start, cu)
    with pytest.raises(ValueError):
        qk.kv_cache_read(cache, table, start, cu, 3, k=torch.empty((2, 2, 32), device=DEV))
    with pytest.raises(TypeError):
        qk.kv_cache_read(cache, table, start, cu, 3, torch.float64)
