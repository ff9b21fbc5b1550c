"""The example decoder layer with 4-bit projections, normed and rotated heads,
and a window with sinks: each of those operators against its plain form on
what it was really given, and replayed tokens against eager ones."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import w8a8_int8_quantized_qk_amd as qk
from examples import decoder_layer as ex
from tests import plain_decoder as plain
from tests import plain_mx4
from tests.test_gpu_kv_sinks import attention
from tests.test_gpu_norm_rope import check
from tests.test_gpu_norm_rope import plain as plain_rope

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qk.library()


def _shape(fp8, **kw):
    return ex.Shape(hidden=256, heads=6, kv_heads=2, dim=64, inner=384, block=16, fp8=fp8, mx4=True, rope=10000.0, window=12, sinks=3, **kw)


@pytest.mark.parametrize("fp8", [False, True])
def test_operators_of_a_step_against_their_plain_forms(fp8, monkeypatch):
    shape = _shape(fp8)
    dec = ex.Decoder(shape, 1, 4, 64)
    table = dec.table.cpu().numpy()
    host = plain.Cache(dec.layers[0].cache, fp8)
    seen = []

    def rope(q, k, start, freqs, cu, q_weight, k_weight, eps):
        got = was["norm_rope"](q, k, start, freqs, cu, q_weight, k_weight, eps)
        at = cu.tolist() if cu is not None else list(range(len(start) + 1))
        pos = np.concatenate([np.arange(s, s + at[i + 1] - at[i]) for i, s in enumerate(start.tolist())])
        for x, w, o in ((q, q_weight, got[0]), (k, k_weight, got[1])):
            check(o, *plain_rope(x, w, pos, freqs.cpu().numpy(), eps, False), "rope")
        seen.append("rope")
        return got

    def write(cache, k, v, tab, start, cu):
        got = was["kv_cache_write"](cache, k, v, tab, start, cu)
        host.write(plain.f32(k), plain.f32(v), table, start.tolist(), cu.tolist())
        return got

    def attend(q, cache, tab, lens, cu, **kw):
        got = was["kv_attention"](q, cache, tab, lens, cu, **kw)
        at = cu.tolist() if cu is not None else list(range(len(lens) + 1))
        for s, n in enumerate(lens.tolist()):
            rows = slice(at[s], at[s + 1])
            want, _, bound, _ = attention(plain.f32(q[rows]), *host.values(table[s], n), n, np.float64(np.float32(shape.dim ** -0.5)),
                                          shape.window, shape.sinks)
            assert plain.within(got[rows], want, bound).all()
        seen.append("attend")
        return got

    def quant(x):
        q, s = was["quant_mx4"](x)
        code, byte = plain_mx4.quantise(x.cpu().double().numpy())
        assert np.array_equal(q.cpu().numpy(), plain_mx4.pack(code)) and np.array_equal(s.cpu().numpy(), byte)
        seen.append("quant")
        return q, s

    def gemm(a, b, scale_a, scale_b):
        out = was["gemm_mx4_scaled"](a, b, scale_a, scale_b)
        va, vb = (plain_mx4.values(t.cpu().numpy(), s.cpu().numpy()) for t, s in ((a, scale_a), (b, scale_b)))
        want, size = va @ vb.T, np.abs(va) @ np.abs(vb).T
        # binary32 sums of k exact products in any order, then bf16
        assert (np.abs(out.cpu().double().numpy() - want) <= 2.0 ** -8 * np.abs(want) + va.shape[1] * 2.0 ** -23 * size).all()
        seen.append("gemm")
        return out

    fakes = {"norm_rope": rope, "kv_cache_write": write, "kv_attention": attend, "quant_mx4": quant, "gemm_mx4_scaled": gemm}
    was = {n: getattr(qk, n) for n in fakes}
    for n, f in fakes.items():
        monkeypatch.setattr(qk, n, f)
    g = torch.Generator(device=DEV).manual_seed(1)
    for counts in ([3, 21, 1, 40], [1, 1, 1, 1], [5, 1, 12, 1]):
        x = torch.randn((sum(counts), shape.hidden), generator=g, device=DEV).to(torch.bfloat16)
        out = dec.prompt(x, counts)
        assert out.shape == x.shape and out.isfinite().all()
    assert seen == ["rope", "attend", "quant", "gemm", "gemm"] * 3


@pytest.mark.parametrize("fp8", [False, True])
def test_replayed_tokens_are_the_eager_ones(fp8):
    shape, counts = _shape(fp8), [5, 33, 16]
    one, two = (ex.Decoder(shape, 3, 3, 60, seed=4) for _ in range(2))
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randn((sum(counts), shape.hidden), generator=g, device=DEV).to(torch.bfloat16)
    assert torch.equal(one.prompt(x, counts), two.prompt(x, counts))
    step = ex.TokenGraph(one)
    for i in range(20):
        new = torch.randn((3, shape.hidden), generator=g, device=DEV).to(torch.bfloat16)
        out = step(new)
        want = two.prompt(new, [1, 1, 1])
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"token {i}"


def test_positions_count():
    outs = []
    for rope in (0.0, 10000.0):
        shape = ex.Shape(hidden=256, heads=6, kv_heads=2, dim=64, inner=384, block=16, rope=rope)
        x = torch.randn((6, shape.hidden), generator=torch.Generator(device=DEV).manual_seed(4), device=DEV).to(torch.bfloat16)
        outs.append(ex.Decoder(shape, 1, 1, 64, seed=5).prompt(x, [6]))
    assert outs[0].isfinite().all() and outs[1].isfinite().all() and not torch.equal(outs[0], outs[1])
