"""Host-side refusals of the norm, cache and attention entry points.  None of
these calls launches a kernel."""
import ctypes

import pytest

import w8a8_int8_quantized_qk_amd as qk
from tests.test_abi import FAKE, FAKE_ODD, NULL, _header_constants

C = _header_constants()
INVALID, UNSUP, WS = C["QK_ERR_INVALID_VALUE"], C["QK_ERR_UNSUPPORTED"], C["QK_ERR_WORKSPACE"]


def at(offset):
    return ctypes.c_void_p(FAKE.value + offset)


def call(fn, defaults, **kw):
    args = dict(defaults)
    assert set(kw) <= set(args)
    args.update(kw)
    return fn(*args.values())


NORM = dict(m=4, k=64, x=FAKE, ldx=64, residual=FAKE, ldr=64, weight=FAKE, dtype=1, weight_dtype=1, eps=1e-6, code=0,
            residual_out=FAKE, ldo=64, q=FAKE, scale=FAKE, stream=NULL)
ROWS = dict(seqs=2, tokens=5, kv_heads=2, dim=64, k=FAKE, ldk=128, v=FAKE, ldv=128, dtype=1, k_cache=FAKE, v_cache=FAKE,
            k_scale=FAKE, v_scale=FAKE, blocks=4, block=16, code=0, table=FAKE, ldt=3, width=3, start=FAKE, cu=FAKE,
            stream=NULL)
ATTEND = dict(seqs=2, tokens=5, heads=4, kv_heads=2, dim=64, q=FAKE, ldq=256, dtype=1, k_cache=FAKE, v_cache=FAKE, k_scale=FAKE,
              v_scale=FAKE, blocks=4, block=16, code=0, table=FAKE, ldt=3, width=3, lens=FAKE, cu=FAKE, max_q=5, max_kv=48,
              scale=0.125, window=0, out=FAKE, lse=NULL, workspace=NULL, workspace_bytes=0, stream=NULL)


def test_constants():
    assert (C["QK_CODE_I8"], C["QK_CODE_FP8"]) == (qk.CODE_I8, qk.CODE_FP8)


@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), INVALID), (dict(k=-1), INVALID), (dict(dtype=3), INVALID), (dict(weight_dtype=2), INVALID),
    (dict(dtype=0, weight_dtype=1), INVALID), (dict(code=2), INVALID), (dict(eps=-1e-9), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(x=NULL), INVALID), (dict(weight=NULL), INVALID), (dict(q=NULL), INVALID),
    (dict(scale=NULL), INVALID), (dict(residual_out=NULL), INVALID), (dict(ldx=63), INVALID), (dict(ldr=63), INVALID),
    (dict(ldo=63), INVALID), (dict(x=FAKE_ODD), UNSUP), (dict(residual=FAKE_ODD), UNSUP), (dict(weight=FAKE_ODD), UNSUP),
    (dict(scale=FAKE_ODD), UNSUP), (dict(k=(1 << 30) + 1, ldx=1 << 31, ldr=1 << 31, ldo=1 << 31), UNSUP),
    (dict(m=0, x=NULL, q=NULL, scale=NULL), 0),
    # rows of the sum that overlap rows of x or the residual: shifted by a row, within a row, by the last element,
    # another stride from the same start, one row
    (dict(residual_out=at(128)), INVALID), (dict(residual_out=at(2)), INVALID), (dict(x=at(2), residual=at(1 << 20)), INVALID),
    (dict(x=at(1 << 20), residual_out=at(128), ldr=65, ldo=65), INVALID), (dict(x=at(1 << 20), residual_out=at(-126), ldr=100, ldo=100), INVALID),
    (dict(x=at(1 << 20), ldo=65), INVALID), (dict(x=at(1 << 20), residual_out=at(128), ldo=128), INVALID),
    (dict(m=1, residual_out=at(126)), INVALID),
])
def test_norm(kw, status):
    assert call(qk.library().qk_rms_norm_quant, NORM, **kw) == status


@pytest.mark.parametrize("name", ["qk_kv_cache_write", "qk_kv_cache_read"])
def test_grids_beyond_a_launch_are_refused_before_it(name):
    assert call(getattr(qk.library(), name), ROWS, tokens=1 << 27, kv_heads=64, ldk=4096, ldv=4096) == UNSUP
    many = dict(seqs=1 << 20, tokens=1 << 20, heads=64, kv_heads=64, ldq=4096, cu=NULL, max_q=1)
    assert call(qk.library().qk_kv_attention, ATTEND, **many) == UNSUP
    assert call(qk.library().qk_kv_attention, ATTEND, tokens=1 << 27, heads=64, kv_heads=64, ldq=4096, max_q=1 << 27) == UNSUP


CACHE = [
    (dict(seqs=-1), INVALID), (dict(tokens=-1), INVALID), (dict(kv_heads=0), INVALID), (dict(dim=24), INVALID),
    (dict(dim=0), INVALID), (dict(dim=272), INVALID), (dict(block=8), INVALID), (dict(block=48), INVALID),
    (dict(block=256), INVALID), (dict(code=7), INVALID), (dict(blocks=-1), INVALID), (dict(blocks=0), INVALID),
    (dict(width=-1), INVALID), (dict(ldt=2), INVALID), (dict(table=NULL), INVALID), (dict(k_cache=NULL), INVALID),
    (dict(v_cache=NULL), INVALID), (dict(k_scale=NULL), INVALID), (dict(v_scale=NULL), INVALID),
    (dict(k_cache=ctypes.c_void_p(0x100008)), UNSUP), (dict(v_cache=FAKE_ODD), UNSUP), (dict(table=FAKE_ODD), UNSUP),
    (dict(cu=FAKE_ODD), UNSUP), (dict(seqs=0), 0), (dict(tokens=0), 0),
]


@pytest.mark.parametrize("name", ["qk_kv_cache_write", "qk_kv_cache_read"])
@pytest.mark.parametrize("kw,status", CACHE + [
    (dict(dtype=3), INVALID), (dict(k=NULL), INVALID), (dict(v=NULL), INVALID), (dict(ldk=127), INVALID), (dict(ldv=127), INVALID),
    (dict(start=NULL), INVALID), (dict(cu=NULL), INVALID), (dict(k=FAKE_ODD), UNSUP), (dict(start=FAKE_ODD), UNSUP),
])
def test_rows(name, kw, status):
    assert call(getattr(qk.library(), name), ROWS, **kw) == status


@pytest.mark.parametrize("kw,status", CACHE + [
    (dict(dtype=0), INVALID), (dict(heads=3), INVALID), (dict(heads=0), INVALID), (dict(q=NULL), INVALID), (dict(out=NULL), INVALID),
    (dict(ldq=255), INVALID), (dict(lens=NULL), INVALID), (dict(cu=NULL), INVALID), (dict(max_q=0), INVALID),
    (dict(max_kv=-1), INVALID), (dict(window=-1), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(q=FAKE_ODD), UNSUP), (dict(out=FAKE_ODD), UNSUP), (dict(lens=FAKE_ODD), UNSUP),
    (dict(lse=FAKE_ODD), UNSUP),
    (dict(ldt=1000, width=1000, max_kv=16000), WS),
    # positions that 32-bit arithmetic has no room for, whatever the workspace; the bound as the table holds it counts
    (dict(ldt=1 << 24, width=1 << 24, block=128, max_kv=(1 << 31) - 1), UNSUP),
    (dict(ldt=1 << 24, width=1 << 24, block=128, max_kv=(1 << 30) - 127), UNSUP),
    (dict(ldt=1 << 24, width=1 << 24, block=128, max_kv=(1 << 30) - 128), WS),
    (dict(ldt=1000, width=1000, max_kv=(1 << 31) - 1), WS),
    (dict(ldt=1000, width=1000, max_kv=16000, workspace=FAKE, workspace_bytes=64), WS),
    (dict(ldt=1000, width=1000, max_kv=16000, workspace=ctypes.c_void_p(0x100010), workspace_bytes=1 << 30), WS),
])
def test_attention(kw, status):
    assert call(qk.library().qk_kv_attention, ATTEND, **kw) == status


def test_binding_refuses_on_the_host():
    import torch
    x, w = torch.zeros(2, 16), torch.zeros(16)
    with pytest.raises(ValueError, match="x must be a GPU tensor"):
        qk.rms_norm_quant(x, w)
    with pytest.raises(TypeError, match="x must be a torch.Tensor"):
        qk.rms_norm_quant([1.0], w)
    cache = qk.new_kv_cache(2, 1, 16, 16, device="cpu")
    with pytest.raises(ValueError, match="k must be a GPU tensor"):
        qk.kv_cache_write(cache, x, x, x, x, x)
    with pytest.raises(ValueError, match="GPU"):
        qk.kv_cache_read(cache, x, x, x, 2)
    with pytest.raises(TypeError):
        qk.kv_cache_read(cache, x, x, x, 2, torch.float64)
    with pytest.raises(ValueError, match="q must be a GPU tensor"):
        qk.kv_attention(x, cache, x, x)
    with pytest.raises(TypeError):
        qk.kv_attention(None, cache, x, x)


@pytest.mark.parametrize("seqs,tokens,heads,kv_heads,dim,max_q", [
    (16, 28, 32, 8, 128, 28),        # 65 to 127 columns in all: at most one sequence has a prompt's
    (40, 109, 32, 32, 128, 70), (1, 17, 32, 8, 128, 17), (3, 40, 8, 4, 256, 40),
    (32, 32, 32, 8, 128, 32),        # single tokens, max_q left at all rows
    (500, 520, 32, 8, 128, 520), (64, 4096, 32, 8, 128, 4096), (9, 1300, 16, 16, 256, 700),
    (2048, 2048, 128, 8, 128, 1),    # 16384 tiles of single tokens
    (1000, 4000, 64, 8, 256, 4),
])
@pytest.mark.parametrize("max_kv", [4096, 131072, 1 << 20])
def test_attention_workspace_stays_small(seqs, tokens, heads, kv_heads, dim, max_q, max_kv):
    size = qk.kv_attention_workspace_size(seqs, tokens, heads, kv_heads, dim, max_kv, 0, True, max_q)
    assert size <= (1 << 30) + (400 << 20)           # single tokens, prompts
    if tokens * heads // kv_heads <= 64:
        # no sequence can have a prompt's columns: as with the tight bound
        assert size == qk.kv_attention_workspace_size(seqs, tokens, heads, kv_heads, dim, max_kv, 0, True, 64 * kv_heads // heads)


def test_attention_workspace_size():
    size = qk.kv_attention_workspace_size
    assert size(1, 1, 4, 2, 64, 64) == 0                     # one piece: nothing to join
    assert size(1, 1, 4, 2, 64, 100000) > 0
    assert size(0, 1, 4, 2, 64, 100000) == 0
    assert size(1, 1, 4, 3, 64, 100000) == 0                 # refused shapes need none
    assert size(1, 1, 4, 2, 64, 100000, window=100) == 0     # a window bounds the range
    assert size(1, 1, 4, 2, 64, (1 << 30) - 128) > 0
    assert size(1, 1, 4, 2, 64, (1 << 30) - 127) == 0
    assert size(1, 200, 4, 2, 64, 100000, ragged=True, max_q=200) > 0
