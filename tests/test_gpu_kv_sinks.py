"""Attention with a sliding window and first positions that stay visible,
against the plain implementation in binary64, and against the attention
without them."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import w8a8_int8_quantized_qk_amd as qk
from tests import plain_decoder as plain
from tests.test_gpu_kv_attention import DEV, Setup
from tests.test_gpu_kv_cache import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qk.library()


def attention(q, k, v, length, scale, window, sinks):
    """plain.attention's results and bounds (its docstring has their derivation) for a window with sinks."""
    n, heads, dim = q.shape
    group = heads // k.shape[1]
    out, b_out = np.zeros((n, heads, dim)), np.zeros((n, heads, dim))
    lse, b_lse = np.full((n, heads), -math.inf), np.zeros((n, heads))
    k, v, q = k.astype(np.float64), v.astype(np.float64), q.astype(np.float64)
    for i in range(n):
        pos = length - n + i
        j = np.arange(max(0, min(pos + 1, length)))
        if window:
            j = j[(j > pos - window) | (j < sinks)]
        if not len(j):
            continue
        for h in range(heads):
            kk, vv = k[j, h // group], v[j, h // group]
            s = kk @ q[i, h] * scale
            e = np.exp(s - s.max())
            p = e / e.sum()
            out[i, h] = p @ vv
            lse[i, h] = s.max() + math.log(e.sum())
            size = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(scale) * 1.4427 + 64
            ds = 2 * (dim + 64) * 2.0 ** -24 * size
            b_out[i, h] = p @ np.abs(vv) * (2.0 ** -12 + ds) + len(j) * 2.0 ** -38 * np.abs(vv).max()
            b_lse[i, h] = ds + 2.0 ** -21 * (1 + abs(lse[i, h]))
    return out, lse, b_out, b_lse


def check(t, out, lse, window, sinks, scale=None):
    host, cu, qf = plain.Cache(t.cache, t.fp8), plain.offsets(t.counts), plain.f32(t.q)
    scale = t.q.shape[2] ** -0.5 if scale is None else scale
    for s, n in enumerate(t.lens):
        k, v = host.values(t.table[s], n)
        r = slice(cu[s], cu[s + 1])
        want, wl, bo, bl = attention(qf[r], k, v, n, np.float64(np.float32(scale)), window, sinks)
        ok = plain.within(out[r], want, bo)
        assert ok.all(), f"sequence {s}: {(~ok).sum()} of {ok.size} outputs beyond the bound"
        if lse is not None:
            g = lse[r].cpu().numpy().astype(np.float64)
            empty = np.isinf(wl)
            assert np.array_equal(g[empty], wl[empty])
            assert (np.abs(g[~empty] - wl[~empty]) <= bl[~empty]).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads,kv_heads,dim,block,window,sinks", [
    (1, 1, 16, 16, 1, 1), (4, 2, 64, 32, 64, 4), (8, 1, 80, 64, 30, 64), (6, 2, 128, 16, 100, 65), (7, 1, 112, 128, 17, 130),
    (2, 2, 256, 64, 128, 3), (20, 1, 128, 64, 5, 200), (48, 3, 64, 16, 64, 16), (80, 1, 32, 16, 63, 1), (4, 4, 64, 128, 1, 64)])
def test_single_tokens(heads, kv_heads, dim, block, window, sinks, dtype, fp8):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 200, 0, 301, 700]
    t = Setup(heads * 7 + dim, lens, [1] * len(lens), heads, kv_heads, dim, block, fp8, dtype)
    out, lse = t.run(return_lse=True, window=window, sinks=sinks)
    check(t, out, lse, window, sinks)
    again, lse2 = t.run(return_lse=True, ragged=True, window=window, sinks=sinks)
    check(t, again, lse2, window, sinks)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,kv_heads,dim,block,dtype,window,sinks", [
    (4, 2, 64, 16, "bf16", 20, 4), (6, 2, 128, 64, "f16", 64, 70), (3, 1, 256, 32, "bf16", 1, 1), (5, 5, 48, 128, "bf16", 100, 128),
    (17, 1, 96, 16, "f16", 7, 33), (32, 8, 128, 64, "bf16", 128, 4)])
def test_several_tokens_and_prompts(heads, kv_heads, dim, block, dtype, window, sinks, fp8):
    # rows of a whole prompt, of its later part, single rows, none, and more rows than positions
    lens = [40, 133, 1, 77, 90, 3, 0, 257, 600]
    counts = [40, 20, 1, 0, 5, 9, 2, 70, 300]
    t = Setup(dim + heads, lens, counts, heads, kv_heads, dim, block, fp8, dtype)
    out, lse = t.run(return_lse=True, window=window, sinks=sinks)
    check(t, out, lse, window, sinks)
    assert not out[int(np.sum(counts[:5])):][:6].any()      # 9 rows over 3 positions: 6 see nothing
    tight = t.run(max_q=max(counts), max_kv=max(lens), window=window, sinks=sinks)
    ok = plain.within(tight, out.double().cpu().numpy(), np.abs(out.double().cpu().numpy()) * 2.0 ** -7 + 2.0 ** -9)
    assert ok.all()
    check(t, tight, None, window, sinks)


@pytest.mark.parametrize("window,sinks", [(1, 1), (5, 16), (64, 4), (100, 63), (100, 64), (1000, 100), (64, 300), (16, 10 ** 6), (64, 2 ** 40)])
@pytest.mark.parametrize("fp8", [False, True])
def test_blocks_given_back_are_not_read(window, sinks, fp8):
    lens, counts = [300, 90, 64, 500], [1, 33, 64, 140]
    t = Setup(window, lens, counts, 4, 2, 64, 16, fp8, "bf16")
    full = t.table.copy()
    for s, (n, c) in enumerate(zip(lens, counts)):
        first, kept = max(0, n - c - window + 1) // 16, min(-(-sinks // 16), t.table.shape[1])
        t.table[s, kept:first] = -1
    out, lse = t.run(window=window, sinks=sinks, return_lse=True)
    t.table = full
    check(t, out, lse, window, sinks)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("counts", [[1, 1, 1], [3, 1, 2], [40, 1, 300]])
def test_long_ranges_in_chunks(counts, fp8):
    lens = [5000, 64, 20000]
    t = Setup(11, lens, counts, 8, 2, 64, 64, fp8, "bf16")
    for window, sinks in ((4096, 4), (3000, 1500), (100, 6000)):
        out, lse = t.run(window=window, sinks=sinks, return_lse=True, max_q=max(counts))
        # bounds from a few rows of each sequence: binary64 over all of them takes minutes
        host, cu, qf = plain.Cache(t.cache, t.fp8), plain.offsets(t.counts), plain.f32(t.q)
        for s, n in enumerate(lens):
            k, v = host.values(t.table[s], n)
            c = counts[s]
            for i in sorted({0, c // 2, c - 1}):
                r = slice(cu[s] + i, cu[s] + i + 1)
                want, wl, bo, bl = attention(qf[r], k, v, n - c + i + 1, np.float64(np.float32(0.125)), window, sinks)
                assert plain.within(out[r], want, bo).all(), (window, sinks, s, i)
                assert (np.abs(lse[r].cpu().numpy() - wl) <= bl).all()


def test_sinks_that_hide_nothing_change_nothing():
    lens, counts = [300, 90, 64, 500], [1, 33, 64, 140]
    t = Setup(12, lens, counts, 4, 2, 64, 16, False, "bf16")
    assert torch.equal(t.run(window=50, sinks=0), t.run(window=50))
    plain_out = t.run()
    assert torch.equal(t.run(sinks=5), plain_out)                      # no window
    assert torch.equal(t.run(window=50, sinks=10 ** 6), plain_out)     # every position is a sink
    check(t, t.run(window=2 ** 31 - 1, sinks=3), None, 0, 0)


def test_masked_places_may_hold_anything():
    # NaN scales, NaN codes and bad table entries where nothing is visible, in the gap and behind the sequences
    for fp8 in (False, True):
        t = Setup(13, [400, 333], [1, 60], 4, 2, 64, 16, fp8, "bf16")
        want, lse = t.run(window=40, sinks=20, return_lse=True)
        gap = slice(32 // 16, (333 - 60 - 40) // 16)
        pages = t.table[:, gap].reshape(-1)
        if fp8:
            t.cache.k.view(torch.uint8)[dev(pages).long()] = 0x7F
            t.cache.v.view(torch.uint8)[dev(pages).long()] = 0x7F
        for s in (t.cache.k_scale, t.cache.v_scale):
            s[dev(pages).long()] = float("nan")
        out, lse2 = t.run(window=40, sinks=20, return_lse=True)
        assert torch.equal(out, want) and torch.equal(lse, lse2)


def test_graph_and_own_workspace():
    t = Setup(14, [5000, 64, 700], [1, 1, 1], 32, 2, 64, 64, False, "bf16")
    table, lens = dev(t.table), dev(np.asarray(t.lens, np.int32))
    args = (t.q, t.cache, table, lens)
    kw = dict(window=3000, sinks=500)
    want = qk.kv_attention(*args, **kw)
    size = qk.kv_attention_workspace_size(3, 3, 32, 2, 64, table.shape[1] * 64, **kw)
    ws = qk.new_workspace(size, DEV) if size else None
    assert torch.equal(qk.kv_attention(*args, **kw, workspace=ws), want)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            out = qk.kv_attention(*args, **kw)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_refusals():
    t = Setup(15, [20, 20], [1, 1], 4, 2, 64, 16, False, "bf16")
    table, lens = dev(t.table), dev(np.array([20, 20], np.int32))
    with pytest.raises(qk.QKError):
        qk.kv_attention(t.q, t.cache, table, lens, window=8, sinks=-1)
    with pytest.raises(TypeError):
        qk.kv_attention(t.q, t.cache, table, lens, window=8, sinks=1.5)
