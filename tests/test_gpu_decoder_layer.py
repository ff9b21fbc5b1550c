"""The example decoder layer: each operator in it against its plain form on what
it was really given, prompts and graph-replayed tokens, and both ways of
filling the cache."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import w8a8_int8_quantized_qk_amd as qk
from examples import decoder_layer as ex
from tests import plain_decoder as plain

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qk.library()


def _shape(fp8):
    return ex.Shape(hidden=256, heads=6, kv_heads=2, dim=64, inner=384, block=16, fp8=fp8)


@pytest.mark.parametrize("fp8", [False, True])
def test_operators_of_a_step_against_their_plain_forms(fp8, monkeypatch):
    shape, counts = _shape(fp8), [3, 21, 1, 40]
    dec = ex.Decoder(shape, 1, 4, 64)
    table = dec.table.cpu().numpy()
    host = plain.Cache(dec.layers[0].cache, fp8)
    seen = []

    def norm(x, w, eps, residual=None, fp8=False):
        got = qk_norm(x, w, eps, residual, fp8)
        codes, scale, r = plain.norm(plain.f32(x), plain.f32(w), eps, None if residual is None else plain.f32(residual), fp8)
        assert np.array_equal(got[0].view(torch.uint8).cpu().numpy(), codes)
        assert np.array_equal(got[1].cpu().numpy(), scale)
        if residual is not None:
            assert torch.equal(got[2].cpu(), torch.from_numpy(r).to(x.dtype))
        seen.append("norm")
        return got

    def write(cache, k, v, tab, start, cu):
        got = qk_write(cache, k, v, tab, start, cu)
        host.write(plain.f32(k), plain.f32(v), table, start.tolist(), cu.tolist())
        assert np.array_equal(cache.k.view(torch.uint8).cpu().numpy(), host.k)
        assert np.array_equal(cache.v.view(torch.uint8).cpu().numpy(), host.v)
        assert np.array_equal(cache.k_scale.cpu().numpy(), host.ks)
        assert np.array_equal(cache.v_scale.cpu().numpy(), host.vs)
        seen.append("write")
        return got

    def attend(q, cache, tab, lens, cu, **kw):
        got = qk_attend(q, cache, tab, lens, cu, **kw)
        at = cu.tolist() if cu is not None else list(range(len(lens) + 1))
        for s, n in enumerate(lens.tolist()):
            rows = slice(at[s], at[s + 1])
            want, _, bound, _ = plain.attention(plain.f32(q[rows]), *host.values(table[s], n), n,
                                                np.float64(np.float32(shape.dim ** -0.5)), 0)
            assert plain.within(got[rows], want, bound).all()
        seen.append("attend")
        return got

    qk_norm, qk_write, qk_attend = qk.rms_norm_quant, qk.kv_cache_write, qk.kv_attention
    monkeypatch.setattr(qk, "rms_norm_quant", norm)
    monkeypatch.setattr(qk, "kv_cache_write", write)
    monkeypatch.setattr(qk, "kv_attention", attend)
    g = torch.Generator(device=DEV).manual_seed(1)
    for counts in (counts, [1, 1, 1, 1], [5, 1, 12, 1]):
        x = torch.randn((sum(counts), shape.hidden), generator=g, device=DEV).to(torch.bfloat16)
        out = dec.prompt(x, counts)
        assert out.shape == x.shape and out.isfinite().all()
    assert seen == ["norm", "write", "attend", "norm"] * 3


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
    for a, b in zip(one.layers, two.layers):
        for p, q in zip(a.cache, b.cache):
            assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))


@pytest.mark.parametrize("fp8", [False, True])
def test_a_token_graph_has_its_own_workspaces(fp8, monkeypatch):
    shape = ex.Shape(hidden=256, heads=6, kv_heads=2, dim=64, inner=384, block=16, fp8=fp8)
    dec = ex.Decoder(shape, 2, 3, 3000)
    g = torch.Generator(device=DEV).manual_seed(5)
    dec.prompt(torch.randn((1200, shape.hidden), generator=g, device=DEV).to(torch.bfloat16), [700, 300, 200])
    seen = []

    def attend(*a, workspace=None, **kw):
        seen.append(workspace)
        return qk_attend(*a, workspace=workspace, **kw)

    qk_attend = qk.kv_attention
    monkeypatch.setattr(qk, "kv_attention", attend)
    one, two = ex.TokenGraph(dec), ex.TokenGraph(dec)
    half = len(seen) // 2
    assert all(w is one.step.attention_workspace for w in seen[:half]) and one.step.attention_workspace is not None
    assert all(w is two.step.attention_workspace for w in seen[half:])
    assert one.step.attention_workspace.data_ptr() != two.step.attention_workspace.data_ptr()
    if not fp8:
        assert one.step.linear_workspace.data_ptr() != two.step.linear_workspace.data_ptr()
    x = torch.randn((3, shape.hidden), generator=g, device=DEV).to(torch.bfloat16)
    a = one(x).clone()
    torch.cuda.synchronize()
    b = two(x).clone()                           # both begin at the same position and write the same token
    assert torch.equal(a, b) and a.isfinite().all()


@pytest.mark.parametrize("fp8", [False, True])
def test_a_prompt_in_pieces_of_whole_blocks_fills_the_same_cache(fp8):
    shape = _shape(fp8)
    one, two = (ex.Decoder(shape, 1, 2, 96, seed=9) for _ in range(2))
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn((2, 90, shape.hidden), generator=g, device=DEV).to(torch.bfloat16)
    one.prompt(x.reshape(180, -1), [90, 90])
    for at, n in ((0, 32), (32, 48), (80, 10)):
        two.prompt(x[:, at:at + n].reshape(2 * n, -1), [n, n])
    for p, q in zip(one.layers[0].cache, two.layers[0].cache):
        assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))
