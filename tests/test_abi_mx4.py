"""Host-side refusals of the 4-bit, rotation and sinks entry points.  None of
these calls launches a kernel."""
import ctypes

import pytest

import w8a8_int8_quantized_qk_amd as qk
from tests.test_abi import FAKE, FAKE_ODD, NULL
from tests.test_abi_decoder import ATTEND, CACHE, INVALID, UNSUP, WS, at, call

OFF16 = ctypes.c_void_p(FAKE.value + 8)
QUANT = dict(m=4, k=64, x=FAKE, ldx=64, dtype=1, q=FAKE, scale=FAKE, lds=16, stream=NULL)
BACK = dict(m=4, k=64, q=FAKE, scale=FAKE, lds=16, x=FAKE, ldx=64, dtype=1, stream=NULL)
GEMM = dict(m=4, n=5, k=64, a=FAKE, scale_a=FAKE, ldsa=16, b=FAKE, scale_b=FAKE, ldsb=16, output_scale=1.0, out=FAKE, out_dtype=1,
            stream=NULL)
LINEAR = dict(m=40, n=5, k=64, x=FAKE, ldx=64, x_dtype=1, b=FAKE, scale_b=FAKE, ldsb=16, output_scale=1.0, out=FAKE, out_dtype=1, q=FAKE,
              scale=FAKE, lds=16, stream=NULL)
ROPE = dict(seqs=2, tokens=5, heads=4, kv_heads=2, dim=64, q=FAKE, ldq=512, k=at(512), ldk=512, q_weight=NULL, k_weight=NULL, dtype=1,
            weight_dtype=1, eps=1e-6, freqs=FAKE, rotary=64, interleaved=0, start=FAKE, cu=FAKE, q_out=at(1 << 20), ldqo=256,
            k_out=at(1 << 21), ldko=128, stream=NULL)

ROWS = [(dict(m=-1), INVALID), (dict(k=-32), INVALID), (dict(k=48), UNSUP), (dict(dtype=3), INVALID), (dict(x=NULL), INVALID),
        (dict(q=NULL), INVALID), (dict(scale=NULL), INVALID), (dict(ldx=63), INVALID), (dict(lds=1), INVALID), (dict(lds=24), UNSUP),
        (dict(x=FAKE_ODD), UNSUP), (dict(q=OFF16), UNSUP), (dict(scale=OFF16), UNSUP), (dict(dtype=0, x=at(2)), UNSUP),
        (dict(m=(1 << 31) - 1, k=64), UNSUP), (dict(m=0, x=NULL, q=NULL), 0), (dict(k=0, x=NULL, q=NULL), 0)]


@pytest.mark.parametrize("kw,status", ROWS)
def test_quant(kw, status):
    assert call(qk.library().qk_quant_mx4, QUANT, **kw) == status
    wide = dict(kw)
    if "ldx" not in kw:
        wide["ldx"] = 128
    assert call(qk.library().qk_silu_mul_quant_mx4, QUANT, **wide) == status
    assert call(qk.library().qk_dequant_mx4, BACK, **kw) == status


def test_silu_rows_hold_both_halves():
    assert call(qk.library().qk_silu_mul_quant_mx4, QUANT, ldx=127) == INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), INVALID), (dict(n=-1), INVALID), (dict(k=-32), INVALID), (dict(k=33), UNSUP), (dict(out_dtype=3), INVALID),
    (dict(a=NULL), INVALID), (dict(b=NULL), INVALID), (dict(scale_a=NULL), INVALID), (dict(scale_b=NULL), INVALID), (dict(out=NULL), INVALID),
    (dict(ldsa=1), INVALID), (dict(ldsb=1), INVALID), (dict(ldsa=8), UNSUP), (dict(ldsb=20), UNSUP), (dict(a=OFF16), UNSUP),
    (dict(b=OFF16), UNSUP), (dict(scale_a=OFF16), UNSUP), (dict(scale_b=OFF16), UNSUP), (dict(out=FAKE_ODD), UNSUP),
    (dict(out=at(2), out_dtype=0), UNSUP), (dict(m=(1 << 24) + 1), UNSUP), (dict(n=(1 << 24) + 1), UNSUP),
    (dict(k=(1 << 24) + 32, ldsa=1 << 20, ldsb=1 << 20), UNSUP), (dict(ldsa=(1 << 23) + 16), UNSUP), (dict(ldsb=1 << 40), UNSUP),
    (dict(m=0, a=NULL), 0), (dict(n=0, b=NULL), 0)])
def test_product(kw, status):
    assert call(qk.library().qk_gemm_mx4_scaled, GEMM, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), INVALID), (dict(k=40), UNSUP), (dict(x=NULL), INVALID), (dict(b=NULL), INVALID), (dict(out=NULL), INVALID),
    (dict(q=NULL), INVALID), (dict(scale=NULL), INVALID), (dict(lds=8), UNSUP), (dict(ldsb=8), UNSUP), (dict(ldx=60), INVALID),
    (dict(x_dtype=5), INVALID), (dict(out_dtype=5), INVALID), (dict(lds=(1 << 23) + 16), UNSUP), (dict(m=4, ldsb=1 << 40), UNSUP), (dict(out=FAKE_ODD), UNSUP), (dict(n=(1 << 24) + 1), UNSUP),
    (dict(m=0, x=NULL), 0), (dict(m=4, x=at(8), q=NULL), INVALID), (dict(m=4, ldx=68, q=NULL), INVALID), (dict(m=4, x=NULL), INVALID),
    (dict(m=4, b=NULL), INVALID), (dict(m=4, ldx=60), INVALID), (dict(m=4, x=FAKE_ODD), UNSUP), (dict(m=4, out=FAKE_ODD), UNSUP)])
def test_linear(kw, status):
    assert call(qk.library().qk_linear_mx4, LINEAR, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(seqs=-1), INVALID), (dict(tokens=-1), INVALID), (dict(heads=-1), INVALID), (dict(kv_heads=-1), INVALID), (dict(dim=24), INVALID),
    (dict(dim=272, ldq=5000, ldk=5000), INVALID), (dict(rotary=66), INVALID), (dict(rotary=63), INVALID), (dict(rotary=-2), INVALID),
    (dict(dtype=3), INVALID), (dict(weight_dtype=2), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(q=NULL), INVALID), (dict(k=NULL), INVALID), (dict(q_out=NULL), INVALID), (dict(k_out=NULL), INVALID), (dict(freqs=NULL), INVALID),
    (dict(start=NULL), INVALID), (dict(cu=NULL), INVALID), (dict(ldq=255), INVALID), (dict(ldk=127), INVALID), (dict(ldqo=255), INVALID),
    (dict(ldko=127), INVALID), (dict(q=FAKE_ODD), UNSUP), (dict(k_out=FAKE_ODD), UNSUP), (dict(q_weight=FAKE_ODD), UNSUP),
    (dict(freqs=at(4)), UNSUP), (dict(start=FAKE_ODD), UNSUP), (dict(tokens=0), 0), (dict(seqs=0), 0), (dict(heads=0, kv_heads=0), 0),
    (dict(tokens=1 << 24, q_out=at(1 << 40), k_out=at(1 << 41)), UNSUP),
    (dict(heads=(1 << 18) + 1, ldq=1 << 25, ldqo=1 << 25, q_out=at(1 << 40), k_out=at(1 << 41)), UNSUP),
    # outputs over inputs: shifted in place, over the other input, over each other
    (dict(q_out=at(2), ldqo=512), INVALID), (dict(q_out=at(1024), ldqo=512), INVALID), (dict(q_out=FAKE, ldqo=256), INVALID),
    (dict(k_out=FAKE), INVALID), (dict(k_out=at(384), ldko=512), INVALID), (dict(q_out=at(512), ldqo=512), INVALID),
    (dict(k_out=at(1 << 20)), INVALID), (dict(k_out=at((1 << 20) + 510)), INVALID), (dict(q=at((1 << 21) + 100)), INVALID),
])
def test_rope(kw, status):
    assert call(qk.library().qk_norm_rope, ROPE, **kw) == status


SINKS = {}
for _name, _value in ATTEND.items():
    SINKS[_name] = _value
    if _name == "window":
        SINKS["sinks"] = 0


@pytest.mark.parametrize("kw,status", CACHE + [
    (dict(sinks=-1), INVALID), (dict(window=-1, sinks=4), INVALID), (dict(dtype=0), INVALID), (dict(q=NULL), INVALID),
    (dict(ldt=4000, width=4000, max_kv=64000, window=20000, sinks=4), WS), (dict(ldt=4000, width=4000, max_kv=64000, window=10, sinks=64000), WS),
    (dict(ldt=4000, width=4000, max_kv=64000, window=10, sinks=20000), WS),
])
def test_attention(kw, status):
    assert call(qk.library().qk_kv_attention_sinks, SINKS, **kw) == status


def test_workspace_size():
    size = qk.kv_attention_workspace_size
    for window, sinks in ((0, 0), (0, 5), (100, 0), (20000, 0)):
        assert size(1, 1, 4, 2, 64, 100000, window=window, sinks=sinks) == size(1, 1, 4, 2, 64, 100000, window=window)
    assert size(1, 1, 4, 2, 64, 100000, window=100, sinks=4) == 0
    assert size(1, 1, 4, 2, 64, 100000, window=100, sinks=50000) > 0
    assert size(1, 1, 4, 2, 64, 100000, window=100, sinks=100000) == size(1, 1, 4, 2, 64, 100000)
    assert size(1, 1, 4, 2, 64, 100000, window=100, sinks=2 ** 40) == size(1, 1, 4, 2, 64, 100000)
    assert size(1, 1, 4, 2, 64, 100000, window=100, sinks=-1) == 0


def test_binding_refuses_on_the_host():
    import torch
    x = torch.zeros(2, 64)
    for fn in (qk.quant_mx4, qk.silu_mul_quant_mx4):
        with pytest.raises(ValueError, match="must be a GPU tensor"):
            fn(x)
        with pytest.raises(TypeError):
            fn([1.0])
    s = qk.new_mx4_scales(2, 64, device="cpu")
    assert s.shape == (2, 2) and s.stride(0) == 16
    with pytest.raises(ValueError):
        qk.new_mx4_scales(2, 48)
    with pytest.raises(ValueError, match="GPU"):
        qk.gemm_mx4_scaled(x, x, s, s)
    with pytest.raises(ValueError, match="GPU"):
        qk.linear_mx4(x, x, s)
    with pytest.raises(ValueError, match="GPU"):
        qk.norm_rope(x, x, x, x)
