"""Plain implementations of the norm and of the paged 8-bit cache (test helper).

Written from the formulas in include/qk.h, one sequence and one block at a
time, on numpy arrays.  Codes and scales are formed with single IEEE binary32
operations (numpy's), so they are exact expectations; the attention and the
bounds of its error are in binary64.
"""
from __future__ import annotations

import math

import numpy as np
import torch

QMAX = {False: np.float32(127), True: np.float32(448)}
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def f32(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().float().numpy()


def to_codes(v: np.ndarray, fp8: bool) -> np.ndarray:
    """Values in units of their scale as code bytes (uint8)."""
    if fp8:
        return torch.from_numpy(np.clip(v, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    return np.clip(np.rint(v), -127, 127).astype(np.int8).view(np.uint8)


def from_codes(c: np.ndarray, fp8: bool) -> np.ndarray:
    if fp8:
        return torch.from_numpy(np.ascontiguousarray(c)).view(torch.float8_e4m3fn).float().numpy()
    return c.view(np.int8).astype(np.float32)


def norm(x, weight, eps, residual, fp8):
    """(code bytes, scales, r in binary32) of rows of binary32 values."""
    r = x + residual if residual is not None else x
    k = x.shape[1]
    with np.errstate(all="ignore"):
        mean = (r.astype(np.float64) ** 2).sum(1) / k
        inv = (1.0 / np.sqrt(mean + eps)).astype(np.float32)
        y = (r * inv[:, None]) * weight[None]
        top = np.abs(y).max(1) if k else np.zeros(len(x), np.float32)
        scale = np.where(np.isnan(top), top, np.maximum(top, np.float32(1e-12))) / QMAX[fp8]
        finite = np.isfinite(top)
        v = np.where(finite[:, None], y / scale[:, None], np.float32(0))
    codes = to_codes(v, fp8)
    codes[~finite] = 0
    return codes, np.where(finite, scale, top).astype(np.float32), r


class Cache:
    """Code bytes and scales of a cache, on the host."""

    def __init__(self, cache, fp8):
        self.fp8 = fp8
        self.k = cache.k.view(torch.uint8).cpu().numpy().copy()
        self.v = cache.v.view(torch.uint8).cpu().numpy().copy()
        self.ks = cache.k_scale.cpu().numpy().copy()
        self.vs = cache.v_scale.cpu().numpy().copy()
        self.block, self.dim, self.heads = self.k.shape[2], self.k.shape[3], self.k.shape[1]

    def write(self, k, v, table, start, cu):
        for s in range(len(start)):
            n = cu[s + 1] - cu[s]
            at = start[s]
            while at < start[s] + n:
                page, lo = table[s][at // self.block], at % self.block
                hi = min(self.block, lo + start[s] + n - at)
                row = cu[s] + at - start[s]
                earlier = lo if at == start[s] else 0
                for h in range(self.heads):
                    self._put(self.k[page, h], self.ks, (page, h), k[row:row + hi - lo, h], lo, hi, earlier)
                    self._put(self.v[page, h].T, self.vs, (page, h), v[row:row + hi - lo, h], lo, hi, earlier)
                at += hi - lo

    def _put(self, tile, scales, where, x, lo, hi, earlier):
        """tile: [position][dim] view of code bytes, written in place."""
        with np.errstate(all="ignore"):
            top = np.abs(x).max()
            need = np.float32(top if np.isnan(top) else max(top, np.float32(1e-12))) / QMAX[self.fp8]
            if not np.isfinite(top):
                need = top
            before = scales[where]
            s = np.float32(np.maximum(need, before)) if earlier else np.float32(need)
            if not np.isfinite(s):
                tile[lo:hi] = 0
                if earlier:
                    tile[:lo] = 0
            else:
                if earlier and s != before:
                    tile[:lo] = to_codes((from_codes(tile[:lo], self.fp8) * before) / s, self.fp8)
                tile[lo:hi] = to_codes(x / s, self.fp8)
        scales[where] = s

    def values(self, table, length):
        """Keys and values [length, heads, dim] of one sequence, binary32."""
        k = np.empty((length, self.heads, self.dim), np.float32)
        v = np.empty_like(k)
        for p in range(length):
            page, i = table[p // self.block], p % self.block
            with np.errstate(all="ignore"):
                k[p] = from_codes(self.k[page, :, i], self.fp8) * self.ks[page][:, None]
                v[p] = from_codes(self.v[page, :, :, i], self.fp8) * self.vs[page][:, None]
        return k, v


def within(got: torch.Tensor, want: np.ndarray, bound: np.ndarray) -> np.ndarray:
    """Whether each element of got (16-bit) is the rounding of a value no further
    than bound from want: rounding is monotone, so it lies between the rounded ends."""
    g = got.detach().cpu().double().numpy()

    def rounded(x):
        return torch.from_numpy(x).to(got.dtype).double().numpy()

    return (g >= rounded(want - bound)) & (g <= rounded(want + bound))


def attention(q, k, v, length, scale, window):
    """One sequence: q [n, heads, dim] binary32, k and v [length, kv heads, dim].

    Returns (out, lse, bound on |out error| before the output's own rounding,
    bound on |lse error|) in binary64.  The bounds: probabilities rounded to 11
    bits, 2^-12 of sum p |v|; binary32 sums of dim products, the scale's factors and
    the exponent's argument, (dim + 64) 2^-24 of the largest sum of absolute
    products plus the exponents' size (64 covers log2 of any scale), which
    moves p and l by that much relatively; p below 2^-38 of the largest lost.
    """
    n, heads, dim = q.shape
    group = heads // k.shape[1]
    out = np.zeros((n, heads, dim))
    lse = np.full((n, heads), -math.inf)
    b_out, b_lse = np.zeros_like(out), np.zeros_like(lse)
    k, v, q = k.astype(np.float64), v.astype(np.float64), q.astype(np.float64)
    for i in range(n):
        pos = length - n + i
        lo = max(0, pos - window + 1) if window else 0
        hi = min(pos + 1, length)
        if hi <= lo:
            continue
        for h in range(heads):
            kk, vv = k[lo:hi, h // group], v[lo:hi, h // group]
            s = kk @ q[i, h] * scale
            m = s.max()
            e = np.exp(s - m)
            p = e / e.sum()
            out[i, h] = p @ vv
            lse[i, h] = m + math.log(e.sum())
            size = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(scale) * 1.4427 + 64
            ds = 2 * (dim + 64) * 2.0 ** -24 * size
            a = p @ np.abs(vv)
            b_out[i, h] = a * (2.0 ** -12 + ds) + (hi - lo) * 2.0 ** -38 * np.abs(vv).max()
            b_lse[i, h] = ds + 2.0 ** -21 * (1 + abs(lse[i, h]))
    return out, lse, b_out, b_lse


def tables(rng, lens, block, spare=3):
    """A random block table for sequences of the given lengths: (table int32
    array with unused entries -1, number of blocks in the pool)."""
    each = [(n + block - 1) // block for n in lens]
    total = sum(each) + spare
    order = rng.permutation(total)
    t = np.full((len(lens), max(1, max(each, default=1))), -1, np.int32)
    at = 0
    for i, n in enumerate(each):
        t[i, :n] = order[at:at + n]
        at += n
    return t, total


def offsets(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
