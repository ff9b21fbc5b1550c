"""GPU parity of the attention over the paged 8-bit cache against the plain
implementation in binary64, within the bounds it derives (output rounding,
probabilities in 11 bits, binary32 sums)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import w8a8_int8_quantized_qk_amd as qk
from tests import plain_decoder as plain
from tests.test_gpu_kv_cache import dev, random_cache

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qk.library()


class Setup:
    """A cache of arbitrary bytes in which only the sequences' own positions
    hold ordinary codes; unused table entries are -1."""

    def __init__(self, seed, lens, counts, heads, kv_heads, dim, block, fp8, dtype, spread=1.0):
        rng = self.rng = np.random.default_rng(seed)
        self.lens, self.counts, self.fp8, self.dtype = lens, counts, fp8, dtype
        self.table, blocks = plain.tables(rng, lens, block)
        self.cache = random_cache(rng, blocks, kv_heads, dim, block, fp8)
        top = 110.0 if fp8 else 36.0
        for t in (self.cache.k, self.cache.v):
            flat = t.view(torch.uint8).cpu().numpy()
            for s, n in enumerate(lens):
                for p in range(n):
                    x = np.clip(rng.standard_normal((kv_heads, dim)).astype(np.float32) * top, -448 if fp8 else -127,
                                448 if fp8 else 127)
                    codes = plain.to_codes(x, fp8)
                    if t is self.cache.k:
                        flat[self.table[s][p // block], :, p % block] = codes
                    else:
                        flat[self.table[s][p // block], :, :, p % block] = codes
            t.view(torch.uint8).copy_(dev(flat))
        for t in (self.cache.k_scale, self.cache.v_scale):
            t.copy_(dev((rng.uniform(0.3, 3.0, t.shape) / top).astype(np.float32)))
        q = rng.standard_normal((sum(counts), heads, dim)).astype(np.float32) * spread
        self.q = dev(q).to(plain.TORCH[dtype])

    def run(self, **kw):
        cu = None if all(c == 1 for c in self.counts) and not kw.pop("ragged", False) else dev(plain.offsets(self.counts))
        kw.pop("ragged", None)
        q = kw.pop("q", self.q)
        return qk.kv_attention(q, self.cache, dev(self.table), dev(np.asarray(self.lens, np.int32)), cu, **kw)

    def check(self, out, lse=None, window=0, scale=None):
        host = plain.Cache(self.cache, self.fp8)
        cu = plain.offsets(self.counts)
        scale = self.q.shape[2] ** -0.5 if scale is None else scale
        qf = plain.f32(self.q)
        for s, n in enumerate(self.lens):
            k, v = host.values(self.table[s], n)
            r = slice(cu[s], cu[s + 1])
            want, wl, bo, bl = plain.attention(qf[r], k, v, n, np.float64(np.float32(scale)), window)
            ok = plain.within(out[r], want, bo)
            assert ok.all(), f"sequence {s}: {(~ok).sum()} of {ok.size} outputs beyond the bound"
            if lse is not None:
                g = lse[r].cpu().numpy().astype(np.float64)
                empty = np.isinf(wl)
                assert np.array_equal(g[empty], wl[empty])
                assert (np.abs(g[~empty] - wl[~empty]) <= bl[~empty]).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads,kv_heads,dim,block", [(1, 1, 16, 16), (4, 2, 64, 32), (8, 1, 80, 64), (6, 2, 128, 16), (7, 1, 112, 128),
                                                      (2, 2, 256, 64), (20, 1, 128, 64), (48, 3, 64, 16), (80, 1, 32, 16)])
def test_single_tokens(heads, kv_heads, dim, block, dtype, fp8):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 200, 0, 301]
    t = Setup(heads * 7 + dim, lens, [1] * len(lens), heads, kv_heads, dim, block, fp8, dtype)
    out, lse = t.run(return_lse=True)
    t.check(out, lse)
    again, lse2 = t.run(return_lse=True, ragged=True)
    t.check(again, lse2)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,kv_heads,dim,block,dtype", [(4, 2, 64, 16, "bf16"), (6, 2, 128, 64, "f16"), (3, 1, 256, 32, "bf16"),
                                                            (5, 5, 48, 128, "bf16"), (17, 1, 96, 16, "f16")])
def test_several_tokens_and_prompts(heads, kv_heads, dim, block, dtype, fp8):
    # rows of a whole prompt, of its later part, single rows, none, and more rows than positions
    lens = [40, 133, 1, 77, 90, 3, 0, 257]
    counts = [40, 20, 1, 0, 5, 9, 2, 70]
    t = Setup(dim + heads, lens, counts, heads, kv_heads, dim, block, fp8, dtype)
    out, lse = t.run(return_lse=True)
    t.check(out, lse)
    assert not out[int(np.sum(counts[:5])):][:6].any()      # 9 rows over 3 positions: 6 see nothing
    tight = t.run(max_q=max(counts), max_kv=max(lens))
    assert torch.equal(tight, out)


@pytest.mark.parametrize("window", [1, 5, 64, 100, 1000])
@pytest.mark.parametrize("fp8", [False, True])
def test_window(window, fp8):
    lens, counts = [300, 90, 64, 500], [1, 33, 64, 140]
    t = Setup(window, lens, counts, 4, 2, 64, 16, fp8, "bf16")
    # blocks before every window may have been given back: their entries are not read
    for s, (n, c) in enumerate(zip(lens, counts)):
        first = max(0, n - c - window + 1) // 16
        t.table[s, :first] = -1
    out, lse = t.run(window=window, return_lse=True)
    ok = Setup(window, lens, counts, 4, 2, 64, 16, fp8, "bf16")
    t.table = ok.table
    t.check(out, lse, window=window)


@pytest.mark.parametrize("window", [2 ** 31 - 3, 2 ** 31 - 1, 2 ** 40])
def test_a_window_without_bound(window):
    # as no window, also where rows stand before position 0
    lens, counts = [3, 70, 40, 0, 1], [9, 70, 100, 4, 1]
    t = Setup(17, lens, counts, 4, 2, 64, 16, False, "bf16")
    want, want_lse = t.run(return_lse=True)
    t.check(want, want_lse)
    out, lse = t.run(return_lse=True, window=window)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("fp8", [False, True])
def test_long_cache_is_split(fp8, dtype):
    t = Setup(11, [5000, 1, 2600, 700], [1, 1, 1, 1], 4, 2, 64, 64, fp8, dtype)
    assert qk.kv_attention_workspace_size(4, 4, 4, 2, 64, 5056) > 0
    out, lse = t.run(return_lse=True)
    t.check(out, lse)
    ws = qk.new_workspace(qk.kv_attention_workspace_size(4, 4, 4, 2, 64, 5056), DEV)
    ws[65536:] = 255                              # only the counters have to be zero, and they are zero again
    own = t.run(workspace=ws)
    assert torch.equal(own, out) and not ws[:65536].any()
    for _ in range(3):
        assert torch.equal(t.run(), out)          # the same bits on every run


@pytest.mark.parametrize("heads,kv_heads,counts,max_q", [(8, 8, [1, 16, 1, 1], 1), (8, 2, [3, 1, 1, 1], 1), (6, 2, [2, 2, 7, 21], 2)])
def test_more_rows_than_max_q_stay_out_of_other_results(heads, kv_heads, counts, max_q):
    # some sequences break the bound in a call that is cut into chunks: nothing is written outside the
    # workspace, and the sequences that keep the bound get their results
    lens = [5000, 4100, 700, 4990]
    t = Setup(13, lens, counts, heads, kv_heads, 64, 64, False, "bf16")
    args = (dev(t.table), dev(np.asarray(lens, np.int32)), dev(plain.offsets(counts)))
    need = qk.kv_attention_workspace_size(4, sum(counts), heads, kv_heads, 64, t.table.shape[1] * 64, 0, True, max_q)
    assert need > 0
    room = torch.full((need + 65536,), 165, dtype=torch.uint8, device=DEV)
    ws = room[:need]
    qk.workspace_init(ws)
    out = qk.kv_attention(t.q, t.cache, *args, max_q=max_q, workspace=ws)
    assert (room[need:] == 165).all() and not ws[:65536].any()
    host, cu = plain.Cache(t.cache, False), plain.offsets(counts)
    for s in (s for s, n in enumerate(counts) if n <= max_q):
        r = slice(cu[s], cu[s + 1])
        want, _, bound, _ = plain.attention(plain.f32(t.q[r]), *host.values(t.table[s], lens[s]), lens[s], 0.125, 0)
        assert plain.within(out[r], want, bound).all(), f"sequence {s}"


@pytest.mark.parametrize("heads,kv_heads,dim,fp8", [(4, 2, 128, False), (2, 2, 64, True), (3, 1, 256, True)])
def test_prompt_tiles_are_split(heads, kv_heads, dim, fp8):
    # a few rows behind a long cache: tiles of many columns whose positions are cut into chunks
    lens, counts = [2500, 1900, 700, 50], [90, 1, 150, 50]
    t = Setup(12 + dim, lens, counts, heads, kv_heads, dim, 32, fp8, "bf16")
    assert qk.kv_attention_workspace_size(4, sum(counts), heads, kv_heads, dim, t.table.shape[1] * 32, 0, True, 150) > 0
    out, lse = t.run(return_lse=True, max_q=150)
    t.check(out, lse)
    for _ in range(3):
        assert torch.equal(t.run(max_q=150), out)


@pytest.mark.parametrize("long", [0, 3000])
@pytest.mark.parametrize("heads,kv_heads", [(2, 2), (2, 1)])
def test_prompts_among_short_sequences(heads, kv_heads, long):
    # rows just at, above and below a tile's and the short sequences' columns, and many that have no tile;
    # over a long cache the tiles are cut into chunks
    counts = [1, 64, 0, 65, 1, 1, 127, 128, 3, 129, 32, 33, 1, 0, 191, 1] + [1] * 70 + [66, 2]
    lens = [c + (5 * i) % 40 for i, c in enumerate(counts)]
    lens[3] = max(lens[3], long)
    t = Setup(14, lens, counts, heads, kv_heads, 32, 16, False, "f16")
    out, lse = t.run(return_lse=True)
    t.check(out, lse)
    only = Setup(15, [n + long // 2 for n in (90, 5, 70)], [90, 5, 70], heads, kv_heads, 32, 16, True, "bf16")
    only.check(*only.run(return_lse=True))


def test_sharp_and_flat_rows():
    # scores of several hundred, equal scores, a scale of zero, large and tiny queries
    for spread, scale in ((300.0, None), (0.0, None), (1.0, 0.0), (1e30, 1e-30), (1e-30, 1e30), (1.0, -1.0)):
        t = Setup(21, [700, 64, 33], [1, 3, 33], 4, 2, 128, 16, False, "bf16", spread)
        out, lse = t.run(scale=scale, return_lse=True)
        t.check(out, lse, scale=scale)


@pytest.mark.parametrize("step", [0.9, 1.7, 1.95, 6.0])
@pytest.mark.parametrize("counts", [[1, 1], [60, 33]])
def test_scores_that_keep_rising(step, counts):
    # by `step` binary orders every 64 positions: the maximum that exponents are taken
    # from may lag behind the true one
    lens = [508, 300]
    t = Setup(21, lens, counts, 4, 2, 64, 32, False, "f16")
    flat = t.cache.k.view(torch.uint8).cpu().numpy()
    for s, n in enumerate(lens):
        for p in range(n):
            codes = np.zeros(64, np.int8)
            codes[0] = p // 4
            flat[t.table[s][p // 32], :, p % 32] = codes.view(np.uint8)
    t.cache.k.view(torch.uint8).copy_(dev(flat))
    t.cache.k_scale.fill_(1.0)
    t.q.fill_(step / 16 * 8 / 1.4427)
    out, lse = t.run(return_lse=True)
    t.check(out, lse)


def test_one_large_query_element():
    # elements 2^20 and more below the row's largest still count
    t = Setup(22, [100, 40], [1, 40], 4, 2, 64, 16, False, "bf16")
    t.q[:, :, 0] = 4096.0
    t.q[:, :, 1:] *= 2.0 ** -8
    t.cache.k.view(torch.uint8)[:, :, :, 0] = 0
    out, lse = t.run(return_lse=True)
    t.check(out, lse)


def test_scales_of_very_different_size():
    t = Setup(23, [500, 130], [1, 70], 4, 2, 64, 16, False, "bf16")
    s = np.clip(np.exp(t.rng.standard_normal(t.cache.v_scale.shape) * 8), 1e-13, 1e13)
    t.cache.v_scale.copy_(dev(s.astype(np.float32)))
    t.check(*t.run(return_lse=True))
    # blocks of zeros with the guard's scale among ordinary ones
    t = Setup(24, [500, 130], [1, 70], 4, 2, 64, 16, True, "bf16")
    zero = t.table[0, 3]
    t.cache.v.view(torch.uint8)[zero] = 0
    t.cache.v_scale[zero] = float(np.float32(1e-12) / np.float32(448))
    t.check(*t.run(return_lse=True))


def _check_small(t, out, lse):
    # as Setup.check, with what values below 2^-64 may lose beside the rest: 2^-88 each
    host, cu = plain.Cache(t.cache, t.fp8), plain.offsets(t.counts)
    for s, n in enumerate(t.lens):
        r = slice(cu[s], cu[s + 1])
        want, wl, bo, bl = plain.attention(plain.f32(t.q[r]), *host.values(t.table[s], n), n,
                                           np.float64(np.float32(t.q.shape[2] ** -0.5)), 0)
        ok = plain.within(out[r], want, bo + 2.0 ** -88)
        assert ok.all(), f"sequence {s}: {(~ok).sum()} of {ok.size} outputs beyond the bound"
        assert (np.abs(lse[r].cpu().numpy() - wl) <= bl).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,counts,dim", [([500, 130], [1, 1], 64), ([500, 130], [60, 33], 64), ([1400, 90], [1, 1], 128),
                                             ([1500, 200], [70, 1], 128), ([300, 90], [2, 40], 256)])
def test_scales_that_are_zero_negative_or_subnormal(lens, counts, dim, fp8):
    t = Setup(25, lens, counts, 4, 2, dim, 32, fp8, "bf16")
    k, v = t.cache.k_scale.clone(), t.cache.v_scale.clone()
    # some blocks of each kind among ordinary ones; the first block of either sequence has every second kind
    kinds = [0.0, -1.0, 1e-38, 1e-30, -1e-43, 1.0, 1.0, 1.0]
    factor = np.asarray(kinds, np.float32)[t.rng.integers(0, 8, tuple(k.shape))]
    factor[t.table[0, 0]], factor[t.table[1, 0]] = 0.0, -1.0
    t.cache.v_scale.mul_(dev(factor))
    t.cache.k_scale.mul_(dev(np.asarray([0.0, -1.0, 1e-38, 1.0], np.float32)[t.rng.integers(0, 4, tuple(k.shape))]))
    _check_small(t, *t.run(return_lse=True))
    # all of one kind
    for fk, fv in ((-1.0, 1.0), (1.0, -1.0), (-1.0, 1e-38), (0.0, 1e-22), (1.0, -1e-43), (1.0, 0.0), (0.0, 0.0), (1.0, 1e13)):
        t.cache.k_scale.copy_(k * fk)
        t.cache.v_scale.copy_(v * fv)
        out, lse = t.run(return_lse=True)
        _check_small(t, out, lse)
        if fv == 0.0:
            assert not out.any()


@pytest.mark.parametrize("counts", [[1, 1, 1], [3, 70, 1]])
def test_a_fresh_cache_reads_as_zeros(counts):
    lens = [20, 300, 1]
    cache = qk.new_kv_cache(32, 2, 64, 16, device=DEV)
    table, _ = plain.tables(np.random.default_rng(1), lens, 16)
    q = torch.randn((sum(counts), 4, 64), device=DEV).to(torch.bfloat16)
    out, lse = qk.kv_attention(q, cache, dev(table), dev(np.asarray(lens, np.int32)), dev(plain.offsets(counts)), return_lse=True)
    assert not out.any()
    seen = np.concatenate([np.arange(n - c, n) + 1 for n, c in zip(lens, counts)])
    assert np.allclose(lse.cpu().numpy(), np.log(seen)[:, None], rtol=0, atol=2.0 ** -20)


def test_the_largest_scales():
    t = Setup(26, [90, 70], [1, 40], 2, 1, 64, 16, False, "bf16")
    t.cache.v.view(torch.uint8).fill_(1)
    t.cache.v_scale.fill_(2.0 ** 126.7)
    t.cache.v_scale[::2] = 2.0 ** 125
    t.check(*t.run(return_lse=True))


@pytest.mark.parametrize("fp8", [False, True])
def test_non_finite_values_reach_only_rows_that_see_them(fp8):
    lens, counts = [80, 64], [40, 1]
    t = Setup(31, lens, counts, 2, 1, 64, 16, fp8, "bf16")
    clean, lse = t.run(return_lse=True)
    t.check(clean, lse)
    last = t.table[0, 4]                      # positions 64 to 79
    t.cache.k_scale[last] = float("nan")
    t.cache.v_scale[last] = float("nan")
    for c in (t.cache.k, t.cache.v):
        c.view(torch.uint8)[last] = 0
    out = t.run()
    blind = 64 - (80 - 40)                    # rows at positions below 64
    assert torch.equal(out[:blind], clean[:blind]) and torch.equal(out[40:], clean[40:])
    assert torch.isnan(out[blind:40]).all()
    t.cache.v_scale[last] = float("inf")
    t.cache.k_scale[last] = 1.0
    out = t.run()
    assert torch.equal(out[:blind], clean[:blind]) and torch.isnan(out[blind:40]).all()
    # a query that is not finite spoils its own row and head alone
    t = Setup(31, lens, counts, 2, 1, 64, 16, fp8, "bf16")
    t.q[3, 1, 7] = float("nan")
    t.q[9, 0, 0] = float("inf")
    out = t.run()
    assert torch.isnan(out[3, 1]).all() and torch.isnan(out[9, 0]).all()
    out[3, 1] = clean[3, 1]
    out[9, 0] = clean[9, 0]
    assert torch.equal(out, clean)


@pytest.mark.parametrize("lens,counts", [([80, 40], [1, 1]), ([80, 40], [5, 40]), ([80, 200], [70, 90]), ([5000, 90], [1, 1]),
                                         ([2500, 90], [90, 1])])
def test_scores_that_are_all_minus_infinity(lens, counts):
    # 0 / 0 by the formula, unlike a row that sees nothing; the log of their sum is -infinity either way
    t = Setup(33, lens, counts, 4, 2, 64, 16, False, "f16")
    t.cache.k.view(torch.uint8)[:, :, :, 0] = 1
    t.q[0, 1, 0] = -float("inf")
    cu = plain.offsets(counts)
    t.q[cu[1], 2, 0] = -float("inf")
    out, lse = t.run(return_lse=True, max_q=max(counts))
    for row, head in ((0, 1), (int(cu[1]), 2)):
        assert torch.isnan(out[row, head]).all() and lse[row, head] == -float("inf")
        t.q[row, head, 0] = out[row, head] = 0
    other, other_lse = t.run(return_lse=True, max_q=max(counts))
    for row, head in ((0, 1), (int(cu[1]), 2)):
        other[row, head] = 0
        lse[row, head] = other_lse[row, head]
    assert torch.equal(out, other) and torch.equal(lse, other_lse)


def test_table_entries_out_of_range_give_nan():
    t = Setup(32, [80, 200], [1, 1], 2, 1, 64, 16, False, "bf16")
    clean = t.run()
    t.table[0, 2] = t.cache.k.shape[0]
    out = t.run()
    assert torch.isnan(out[0]).all() and torch.equal(out[1], clean[1])
    t.table[0, 2] = -5
    out = t.run()
    assert torch.isnan(out[0]).all() and torch.equal(out[1], clean[1])


def test_strided_queries_output_buffer_and_stream():
    t = Setup(41, [150, 77, 9], [30, 1, 9], 6, 2, 64, 32, False, "bf16")
    want = t.run()
    wide = torch.zeros((t.q.shape[0], 6 * 64 + 129), dtype=t.q.dtype, device=DEV)
    wide[:, 1:1 + 6 * 64] = t.q.flatten(1)
    out = torch.empty_like(t.q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = t.run(q=wide[:, 1:1 + 6 * 64].unflatten(1, (6, 64)), out=out)
    torch.cuda.current_stream().wait_stream(side)
    assert got is out and torch.equal(out, want)


def test_many_sequences():
    rng = np.random.default_rng(51)
    counts = rng.integers(0, 4, 140).tolist()
    lens = [int(c + rng.integers(0, 40)) for c in counts]
    t = Setup(52, lens, counts, 4, 1, 32, 16, True, "f16")
    t.check(*t.run(return_lse=True))


def test_graph_replay():
    t = Setup(61, [1300, 64, 700], [1, 1, 1], 4, 2, 64, 64, False, "bf16")
    want = t.run().clone()
    table, lens = dev(t.table), dev(np.asarray(t.lens, np.int32))
    out = torch.empty_like(t.q)
    ws = qk.new_workspace(qk.kv_attention_workspace_size(3, 3, 4, 2, 64, table.shape[1] * 64), DEV)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qk.kv_attention(t.q, t.cache, table, lens, out=out, workspace=ws)
    for _ in range(4):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert torch.equal(t.run(), want)


def test_graph_captured_before_any_eager_call_and_kept_past_larger_ones():
    t = Setup(62, [1300, 64, 700], [1, 1, 1], 4, 2, 64, 64, False, "bf16")
    big = Setup(63, [5000] * 4, [1] * 4, 16, 8, 64, 64, False, "bf16")
    want, want_big = t.run().clone(), big.run().clone()
    args = (t.q, t.cache, dev(t.table), dev(np.asarray(t.lens, np.int32)))
    big_args = (big.q, big.cache, dev(big.table), dev(np.asarray(big.lens, np.int32)))
    for warm in (False, True):
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            if warm:
                qk.kv_attention(*args)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                out = qk.kv_attention(*args)
                out_big = qk.kv_attention(*big_args)
            for _ in range(3):
                got = qk.kv_attention(*big_args)      # eager, on the same stream, with more workspace
                g.replay()
                torch.cuda.synchronize()
                assert torch.equal(got, want_big)
                assert torch.equal(out, want) and torch.equal(out_big, want_big)
                out.zero_()
                out_big.zero_()
        torch.cuda.current_stream().wait_stream(stream)


def test_graphs_share_no_workspace_with_other_calls(monkeypatch):
    # captured on a stream that has a workspace already, twice: a replay on any stream may run beside the
    # other graph and beside eager calls, so each call in a graph has a workspace of its own
    made, of_package = [], qk._workspace_on

    def spy(nbytes, index):
        made.append(of_package(nbytes, index))
        return made[-1]

    monkeypatch.setattr(qk, "_workspace_on", spy)
    qk._bind_to(qk.library())
    try:
        t = Setup(64, [5000, 64, 700], [1, 1, 1], 4, 2, 64, 64, False, "bf16")
        big = Setup(65, [5000] * 8, [1] * 8, 32, 16, 64, 64, False, "bf16")
        args, big_args = ((s.q, s.cache, dev(s.table), dev(np.asarray(s.lens, np.int32))) for s in (t, big))
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            qk.kv_attention(*big_args)           # the stream's workspace is large enough for all that follows
            before = len(made)
            want = qk.kv_attention(*args)
            assert len(made) == before
            torch.cuda.synchronize()
            graphs, outs = [], []
            for _ in range(2):
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=stream):
                    outs.append(qk.kv_attention(*args))
                graphs.append(g)
            own = [w.data_ptr() for w in made[before:]]
            assert len(set(own)) == 2 and not {w.data_ptr() for w in made[:before]} & set(own)
            again = qk.kv_attention(*args)       # eager calls go on with the stream's
            assert len(made) == before + 2
        torch.cuda.synchronize()
        assert torch.equal(again, want)
        kept = [(w, w.clone()) for w in made[:before]]
        for _ in range(3):
            for g, out in zip(graphs, outs):
                out.zero_()
                g.replay()
                torch.cuda.synchronize()
                assert torch.equal(out, want)
        assert all(torch.equal(w, c) for w, c in kept)
    finally:
        monkeypatch.undo()
        qk._bind_to(qk.library())


def test_refusals():
    t = Setup(71, [20, 20], [1, 1], 4, 2, 64, 16, False, "bf16")
    table, lens, cu = dev(t.table), dev(np.array([20, 20], np.int32)), dev(np.array([0, 1, 2], np.int32))
    with pytest.raises(TypeError):
        qk.kv_attention(t.q.float(), t.cache, table, lens)
    with pytest.raises(ValueError):
        qk.kv_attention(t.q[:, :3], t.cache, table, lens)
    with pytest.raises(ValueError):
        qk.kv_attention(t.q[:, :, :48], t.cache, table, lens)
    with pytest.raises(ValueError):
        qk.kv_attention(t.q[:1], t.cache, table, lens)
    with pytest.raises(ValueError):
        qk.kv_attention(t.q, t.cache, table[:1], lens)
    with pytest.raises(TypeError):
        qk.kv_attention(t.q, t.cache, table, lens.long())
    with pytest.raises(ValueError):
        qk.kv_attention(t.q, t.cache, table, lens, cu[:2])
    with pytest.raises(qk.QKError):
        qk.kv_attention(t.q, t.cache, table, lens, scale=float("inf"))
    with pytest.raises(qk.QKError):
        qk.kv_attention(t.q, t.cache, table, lens, window=-1)
    with pytest.raises(qk.QKError):
        qk.kv_attention(t.q, t.cache, table, lens, max_q=0)
    big = dev(np.zeros((2, 4000), np.int32))
    with pytest.raises(qk.QKError, match="WORKSPACE"):
        qk.kv_attention(t.q, t.cache, big, lens, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        qk.new_kv_cache(4, 2, 64, block=48, device=DEV)
    with pytest.raises(ValueError):
        qk.new_kv_cache(4, 2, 72, device=DEV)
