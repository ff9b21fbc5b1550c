"""Norm and rotation of queries and keys against the formulas in binary64."""
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
    """(y, bound on its error before the output's rounding) in binary64.

    The bound: the sum of dim squares, its mean, the root, the quotient and two
    products in binary32, (dim + 8) 2^-24 of y in all; cosine and sine
    within 2^-22 (their argument, a Taylor sum of rounded terms, and positions whose angle
    is off by less), of either element of the pair; two products and their sum, 2^-23."""
    y = x.double().cpu().numpy()
    dim = y.shape[-1]
    rel = 0.0
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + np.float64(np.float32(eps))) * w.double().cpu().numpy()
        rel = (dim + 8) * 2.0 ** -24
    r = 2 * len(freqs)
    a = np.arange(0, r, 2) if interleaved else np.arange(r // 2)
    b = a + 1 if interleaved else a + r // 2
    t = pos[:, None, None].astype(np.longdouble) * freqs.astype(np.longdouble)
    cos, sin = np.cos(t).astype(np.float64), np.sin(t).astype(np.float64)
    out, bound = y.copy(), rel * np.abs(y)
    out[..., a] = y[..., a] * cos - y[..., b] * sin
    out[..., b] = y[..., b] * cos + y[..., a] * sin
    both = (np.abs(y[..., a]) + np.abs(y[..., b])) * (rel + 2.0 ** -22 + 2.0 ** -23)
    bound[..., a] = bound[..., b] = both
    return out, bound


def check(got, want, bound, what):
    t = got.dtype
    g = got.double().cpu().numpy()
    tol = bound + torch.finfo(t).eps / 2 * (np.abs(want) + bound) + torch.finfo(t).tiny * torch.finfo(t).eps / 2
    bad = np.abs(g - want) > tol
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.abs(g - want)[bad].max()}"


class Setup:
    def __init__(self, seed, counts, starts, heads, kv_heads, dim, rotary, dtype, norm=True, w32=False):
        rng = np.random.default_rng(seed)
        n = sum(counts)
        self.counts, self.starts = counts, starts
        rows = torch.from_numpy(rng.standard_normal((n, (heads + 2 * kv_heads) * dim + 5)).astype(np.float32)).to(DEV).to(TORCH[dtype])
        # slices of one projection, at an odd place
        self.q = rows[:, 3:3 + heads * dim].view(n, heads, dim)
        self.k = rows[:, 3 + heads * dim:3 + (heads + kv_heads) * dim].view(n, kv_heads, dim)
        self.freqs = 10000.0 ** (-np.arange(0, rotary, 2) / max(rotary, 1))
        wt = torch.float32 if w32 else TORCH[dtype]
        self.w = [torch.from_numpy(1 + 0.3 * rng.standard_normal(dim)).to(DEV).to(wt) if norm else None for _ in range(2)]
        self.pos = np.concatenate([np.arange(s, s + c) for s, c in zip(starts, counts)]) if n else np.zeros(0, np.int64)
        self.cu = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).to(DEV)
        self.start = torch.tensor(starts, dtype=torch.int32, device=DEV)

    def run(self, **kw):
        kw.setdefault("cu", self.cu)
        return qk.norm_rope(self.q, self.k, self.start, torch.from_numpy(self.freqs).to(DEV), q_weight=self.w[0], k_weight=self.w[1], **kw)

    def check(self, out, eps=1e-6, interleaved=False):
        for name, x, w, o in (("q", self.q, self.w[0], out[0]), ("k", self.k, self.w[1], out[1])):
            check(o, *plain(x, w, self.pos, self.freqs, eps, interleaved), name)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("heads,kv_heads,dim,rotary", [(1, 1, 16, 16), (4, 2, 64, 64), (3, 1, 80, 80), (3, 3, 80, 20), (5, 1, 96, 48),
                                                       (7, 1, 112, 112), (32, 8, 128, 128), (6, 2, 128, 64), (4, 2, 128, 2), (16, 4, 256, 256),
                                                       (2, 1, 256, 254), (2, 2, 48, 6), (9, 1, 32, 0), (64, 1, 64, 24), (1, 2, 192, 64)])
def test_heads(heads, kv_heads, dim, rotary, dtype, interleaved):
    t = Setup(heads + dim, [3, 0, 1, 17, 2], [0, 9, 4095, 100, 70000], heads, kv_heads, dim, rotary, dtype)
    t.check(t.run(interleaved=interleaved), interleaved=interleaved)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("which", ["none", "q", "k", "fp32"])
def test_weights(which, dtype):
    t = Setup(1, [5, 4], [3, 1000], 4, 2, 128, 64, dtype, w32=which == "fp32")
    if which in ("none", "k"):
        t.w[0] = None
    if which in ("none", "q"):
        t.w[1] = None
    t.check(t.run(eps=0.25), eps=0.25)


def test_far_positions():
    # at 2^30 the angle's turns are taken off a product good to 2^-52 of some 2^28 turns: 2^-21 of an angle
    starts = [2 ** 20 - 1, 2 ** 24, 2 ** 27 + 12345, 999_999_999]
    t = Setup(2, [1] * 4, starts, 4, 1, 128, 128, "f32", norm=False)
    out = t.run()
    for x, o in ((t.q, out[0]), (t.k, out[1])):
        want, bound = plain(x, None, t.pos, t.freqs, 1e-6, False)
        far = np.abs(t.pos)[:, None, None] * 2.0 ** -50 * np.abs(x.double().cpu().numpy()).max()
        check(o, want, bound + far, "far")


def test_single_tokens_without_offsets():
    t = Setup(3, [1] * 70, list(range(0, 7000, 100)), 4, 2, 64, 64, "bf16")
    out = t.run()
    t.check(out)
    again = t.run(cu=None)
    assert all(torch.equal(a, b) for a, b in zip(out, again))


def test_many_sequences():
    rng = np.random.default_rng(4)
    counts = rng.integers(0, 4, 300).tolist()
    t = Setup(5, counts, rng.integers(0, 5000, 300).tolist(), 2, 1, 64, 32, "f16")
    t.check(t.run())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rotary", [(128, 128), (80, 20), (256, 64)])
def test_in_place(dim, rotary, interleaved):
    t = Setup(6, [9, 4], [0, 50], 6, 2, dim, rotary, "bf16")
    want = t.run(interleaved=interleaved)
    before = t.q._base.clone() if t.q._base is not None else None
    got = t.run(interleaved=interleaved, q_out=t.q, k_out=t.k)
    assert got[0] is t.q and got[1] is t.k
    assert torch.equal(t.q, want[0]) and torch.equal(t.k, want[1])
    # what lies beside the heads in the same rows is as it was
    after = t.q._base
    n = (6 + 2) * dim
    assert before is None or (torch.equal(before[:, :3], after[:, :3]) and torch.equal(before[:, 3 + n:], after[:, 3 + n:]))


def test_rows_of_no_sequence_stay():
    t = Setup(7, [4, 3, 6], [0, 5, 9], 4, 2, 64, 64, "bf16")
    want = t.run()
    cu = t.cu.clone()
    cu[0], cu[3] = 2, 11  # two rows before the first sequence, two behind the last
    outs = [torch.full_like(o, 7.0) for o in want]
    t.run(cu=cu, q_out=outs[0], k_out=outs[1])
    for o, w in zip(outs, want):
        assert (o[:2] == 7).all() and (o[11:] == 7).all()
        assert torch.equal(o[4:11], w[4:11])


@pytest.mark.parametrize("value", [float("inf"), float("nan"), 3e38])
def test_rows_do_not_touch_each_other(value):
    t = Setup(8, [5], [10], 4, 2, 64, 64, "bf16")
    want = t.run()
    t.q[2, 1, 3] = value
    out = t.run()
    same = torch.ones((5, 4), dtype=torch.bool)
    same[2, 1] = False
    assert torch.equal(out[0][same.to(DEV)], want[0][same.to(DEV)]) and torch.equal(out[1], want[1])


def test_zero_rows_are_zero():
    t = Setup(9, [3], [10], 4, 2, 64, 64, "f16")
    t.q.zero_()
    out = t.run()
    assert not out[0].any() and out[1].any()
    t = Setup(9, [], [], 4, 2, 64, 64, "f16")
    assert t.run()[0].shape == (0, 4, 64)


def test_graph():
    t = Setup(10, [1] * 8, list(range(8)), 8, 2, 128, 128, "bf16")
    freqs = torch.from_numpy(t.freqs).to(DEV)

    def call():
        return qk.norm_rope(t.q, t.k, t.start, freqs, None, t.w[0], t.w[1])

    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            out = call()
    for i in range(3):
        t.start.add_(100)
        want = call()
        torch.cuda.synchronize()
        out[0].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]), i


def test_refusals():
    t = Setup(11, [2, 3], [0, 5], 4, 2, 64, 64, "bf16")
    freqs = torch.from_numpy(t.freqs).to(DEV)

    def call(q=t.q, k=t.k, start=t.start, f=freqs, cu=t.cu, **kw):
        return qk.norm_rope(q, k, start, f, cu, **kw)

    call()
    for kw, error in ((dict(q=t.q.double()), TypeError), (dict(k=t.k.float()), TypeError), (dict(k=t.k[:4]), ValueError),
                      (dict(k=t.k[:, :, :32]), ValueError), (dict(start=t.start.long()), TypeError), (dict(f=freqs.float()), TypeError),
                      (dict(cu=t.cu[:2]), ValueError), (dict(cu=None), ValueError), (dict(q_weight=t.w[0][:32]), ValueError),
                      (dict(q_weight=t.w[0].half()), TypeError), (dict(q_weight=t.w[0], k_weight=t.w[1].float()), TypeError),
                      (dict(q_out=t.q[:, :2]), ValueError), (dict(k_out=t.k.float()), TypeError), (dict(eps=-1.0), qk.QKError),
                      (dict(eps=float("nan")), qk.QKError), (dict(f=torch.cat([freqs, freqs])), qk.QKError),
                      (dict(q=t.q[:, :, :40], k=t.k[:, :, :40]), ValueError)):
        with pytest.raises(error):
            call(**kw)
    # outputs over another input, or over each other
    room = torch.zeros((5, 6, 64), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(qk.QKError):
        call(q_out=room[:, :4], k_out=room[:, 3:5])
    with pytest.raises(qk.QKError):
        call(k_out=t.q[:, 1:3])
    with pytest.raises(qk.QKError):
        call(q=room[:, :4], q_out=room[:, 1:5])
    call(q_out=room[:, :4], k_out=room[:, 4:])
