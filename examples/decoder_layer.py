"""A decoder layer in 8 bits, over a paged 8-bit cache: prompts, then tokens.

    norm + quantization -> QKV GEMM -> cache write -> attention -> quantization
    -> output GEMM -> residual + norm + quantization -> gate/up GEMM
    -> silu(gate) * up + quantization -> down GEMM

Every step is a call of the framework; between two of them activations are
either 8-bit codes with per-token scales or bf16.  Positional encoding is left
out.  `python -m examples.decoder_layer` runs prompts of mixed lengths through
a few layers, then single tokens replayed from a HIP graph, and prints times.
"""
from __future__ import annotations

import argparse
import time
from dataclasses import dataclass

import torch

import w8a8_int8_quantized_qk_amd as qk


@dataclass
class Shape:
    hidden: int = 4096
    heads: int = 32
    kv_heads: int = 8
    dim: int = 128
    inner: int = 14336
    block: int = 64
    fp8: bool = False       # both the linears' codes and the cache
    eps: float = 1e-6


class Linear:
    """An 8-bit weight [k, n] with per-channel scales, random."""

    def __init__(self, k, n, fp8, gen, device):
        if fp8:
            w = torch.randn((k, n), generator=gen, device=device) * 100
            self.w = w.clamp_(-448, 448).to(torch.float8_e4m3fn)
        else:
            self.w = torch.randint(-127, 128, (k, n), generator=gen, device=device, dtype=torch.int8)
        size = 100 if fp8 else 73           # the codes' root mean square
        self.s = torch.full((n,), k ** -0.5 / size, device=device)

    def __call__(self, q, s, workspace=None):
        if q.dtype == torch.float8_e4m3fn:
            return qk.gemm_fp8_scaled(q, self.w, s, self.s)
        return qk.gemm_i8_scaled(q, self.w, s, self.s, workspace=workspace)


@dataclass
class Step:
    """What one call does for its sequences: all int32 on the GPU but the bounds."""
    table: torch.Tensor     # [seqs, width] blocks of each sequence
    start: torch.Tensor     # [seqs] positions in the cache before the step
    lens: torch.Tensor      # [seqs] and after it
    cu: torch.Tensor        # [seqs + 1] rows of each sequence
    max_q: int
    max_kv: int
    linear_workspace: torch.Tensor | None = None    # of a graph's own; None: the stream's
    attention_workspace: torch.Tensor | None = None


class Layer:
    def __init__(self, shape: Shape, blocks: int, gen: torch.Generator, device="cuda"):
        c = self.shape = shape
        self.norm1 = torch.ones(c.hidden, dtype=torch.bfloat16, device=device)
        self.norm2 = torch.ones(c.hidden, dtype=torch.bfloat16, device=device)
        wide = (c.heads + 2 * c.kv_heads) * c.dim
        self.qkv = Linear(c.hidden, wide, c.fp8, gen, device)
        self.o = Linear(c.heads * c.dim, c.hidden, c.fp8, gen, device)
        self.gate_up = Linear(c.hidden, 2 * c.inner, c.fp8, gen, device)
        self.down = Linear(c.inner, c.hidden, c.fp8, gen, device)
        self.cache = qk.new_kv_cache(blocks, c.kv_heads, c.dim, c.block, c.fp8, device)

    def __call__(self, x, residual, step: Step):
        """x [tokens, hidden] bf16 and the running sum (None before the first
        layer) to the next pair."""
        c, n = self.shape, x.shape[0]
        if residual is None:
            residual = x
            q, s = qk.rms_norm_quant(x, self.norm1, c.eps, fp8=c.fp8)
        else:
            q, s, residual = qk.rms_norm_quant(x, self.norm1, c.eps, residual, c.fp8)
        ws = step.linear_workspace
        rows = self.qkv(q, s, ws).view(n, c.heads + 2 * c.kv_heads, c.dim)
        query, key, value = rows.split([c.heads, c.kv_heads, c.kv_heads], 1)
        qk.kv_cache_write(self.cache, key, value, step.table, step.start, step.cu)
        a = qk.kv_attention(query, self.cache, step.table, step.lens, step.cu if step.max_q > 1 else None,
                            max_q=step.max_q, max_kv=step.max_kv, workspace=step.attention_workspace)
        quant, silu = ((qk.quant_per_token_fp8, qk.silu_mul_quant_per_token_fp8) if c.fp8
                       else (qk.quant_per_token, qk.silu_mul_quant_per_token))
        x = self.o(*quant(a.view(n, c.heads * c.dim)), ws)
        q, s, residual = qk.rms_norm_quant(x, self.norm2, c.eps, residual, c.fp8)
        return self.down(*silu(self.gate_up(q, s, ws)), ws), residual


class Decoder:
    """A few layers and the blocks of their sequences."""

    def __init__(self, shape: Shape, layers: int, seqs: int, longest: int, seed: int = 0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        width = -(-longest // shape.block)
        self.shape, self.longest, self.device = shape, longest, torch.device(device)
        self.table = torch.randperm(seqs * width, generator=gen, device=device).to(torch.int32).view(seqs, width)
        self.layers = [Layer(shape, seqs * width, gen, device) for _ in range(layers)]
        self.lens = torch.zeros(seqs, dtype=torch.int32, device=device)

    def run(self, x, step: Step):
        residual = None
        for layer in self.layers:
            x, residual = layer(x, residual, step)
        return x + residual

    def prompt(self, x, counts):
        """counts[s] new rows of every sequence, one after the other in x."""
        new = torch.tensor(counts, dtype=torch.int32, device=self.device)
        cu = torch.zeros(len(counts) + 1, dtype=torch.int32, device=self.device)
        cu[1:] = new.cumsum(0)
        start, self.lens = self.lens, self.lens + new
        return self.run(x, Step(self.table, start, self.lens, cu, max(counts), self.longest))


class TokenGraph:
    """One row of every sequence per replay: from x, added to the caches, its
    result in out.  Holds what the graph reads and the workspaces that it uses,
    so that a replay shares nothing with calls on other streams."""

    def __init__(self, dec: Decoder):
        seqs = dec.table.shape[0]
        self.x = torch.zeros((seqs, dec.shape.hidden), dtype=torch.bfloat16, device=dec.device)
        self.cu = torch.zeros(seqs + 1, dtype=torch.int32, device=dec.device)
        self.start, self.lens = dec.lens.clone(), dec.lens.clone()
        c, layer = dec.shape, dec.layers[0]
        linear = max(qk.gemm_workspace_size(seqs, m.w.shape[1], m.w.shape[0])
                     for m in (layer.qkv, layer.o, layer.gate_up, layer.down))
        attention = qk.kv_attention_workspace_size(seqs, seqs, c.heads, c.kv_heads, c.dim, dec.longest)
        self.step = Step(dec.table, self.start, self.lens, self.cu, 1, dec.longest,
                         *(qk.new_workspace(n, dec.device) for n in (linear, attention)))
        self.stream = torch.cuda.Stream()
        self.stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(self.stream):
            self._step(dec)             # what happens on first use is out of the capture; no sequence has a row yet
            self.start.copy_(dec.lens)
            self.lens.copy_(dec.lens + 1)
            self.cu.copy_(torch.arange(seqs + 1))
        torch.cuda.current_stream().wait_stream(self.stream)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph, stream=self.stream):
            self.out = self._step(dec)

    def _step(self, dec):
        out = dec.run(self.x, self.step)
        self.start.add_(1)
        self.lens.add_(1)
        return out

    def __call__(self, x):
        self.x.copy_(x)
        self.graph.replay()
        return self.out


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--prompts", type=int, nargs="+", default=[37, 2048, 700, 301])
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--fp8", action="store_true")
    a = ap.parse_args()
    shape = Shape(fp8=a.fp8)
    dec = Decoder(shape, a.layers, len(a.prompts), max(a.prompts) + a.tokens)
    x = torch.randn((sum(a.prompts), shape.hidden), device="cuda").to(torch.bfloat16)
    empty = dec.lens
    dec.prompt(x, a.prompts)
    dec.lens = empty                    # the second run writes the same again
    torch.cuda.synchronize()
    t = time.perf_counter()
    out = dec.prompt(x, a.prompts)
    torch.cuda.synchronize()
    print(f"{sum(a.prompts)} tokens of {len(a.prompts)} prompts: {(time.perf_counter() - t) * 1e6 / a.layers:.0f} us a layer")
    last = torch.tensor(a.prompts, device="cuda").cumsum(0) - 1
    step, y = TokenGraph(dec), out[last]
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.tokens):
        y = step(y)
    torch.cuda.synchronize()
    print(f"{a.tokens} single tokens of each: {(time.perf_counter() - t) * 1e6 / a.layers / a.tokens:.1f} us a layer and step; "
          f"all finite: {bool(y.isfinite().all())}")


if __name__ == "__main__":
    main()
