"""One attention block served from coded weights: a prompt in two pieces, then
token by token.

    python examples/attention_block.py [--hidden 4096 --heads 32 --kv-heads 8 --head-dim 128 --prompt 600 --new 32]

The q, k, v and o matrices are quantized to 4 bits, Huffman-coded and kept
coded on the GPU.  A piece of the prompt goes through the fused decode + GEMM,
its keys and values into the 8-bit cache and its attention through
``attn_prompt`` (the second piece reads the first one's keys and values back
from the cache); a new token goes through the fused decode + GEMV, the cache
and ``attn_cache``.  Outputs are compared with the same block in float32 on the
decoded weights without a cache: what differs is the cache's 8 bits.
"""
from __future__ import annotations

import argparse
import math
import os
import sys
import time

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import entropy_coded_weight_canonical_amd as ent  # noqa: E402

LANES, REFILL, MAX_LEN = 64, 2, 12


class CodedMatrix:
    """A [rows][cols] matrix in the layout of the fused products: 4-bit codes,
    64 lanes, one row per chunk."""

    def __init__(self, w: np.ndarray):
        import torch

        self.rows, self.cols = w.shape
        q, scale, zp, _ = ent.quantize(w, 4, "mixed")
        lengths = ent.code_lengths(q, 4, MAX_LEN)
        words, offs = ent.encode(q, lengths, 4, self.cols, LANES, refill_steps=REFILL, ahead=True)
        lut = ent.lut_build(lengths, 4, MAX_LEN, scale, zp)
        self.t = ent.DeviceTensor.upload(lut, words, offs, q.size, self.cols, LANES, 4, MAX_LEN, refill_steps=REFILL,
                                         ahead=True)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def dense(self):
        """The decoded weights, bf16 [rows][cols]."""
        import torch

        out = torch.empty(self.rows, self.cols, dtype=torch.bfloat16, device="cuda")
        ent.decode_dequant([self.t.desc], [out.data_ptr()], self.status.data_ptr())
        return out


def product(matrices, x):
    """x [tokens][cols] (bf16) times each matrix, float32 [tokens][rows]; one
    fused launch over the coded weights for all of them."""
    import torch

    n = x.shape[0]
    ys = [torch.empty(n, m.rows, dtype=torch.float32, device="cuda") for m in matrices]
    items = [ent.GemvItem(m.rows, m.cols, x.data_ptr(), y.data_ptr()) for m, y in zip(matrices, ys)]
    status = torch.zeros(len(matrices), dtype=torch.int32, device="cuda")
    fused = ent.decode_gemv if n <= 8 else ent.decode_gemm
    fused([m.t.desc for m in matrices], items, n, status.data_ptr())
    return ys


def rotate(x, first: int, base: float = 10000.0):
    """Rotary position embedding of x [tokens][heads][dim] at positions first on."""
    import torch

    half = x.shape[2] // 2
    freq = base ** (-torch.arange(half, device=x.device, dtype=torch.float32) / half)
    angle = (first + torch.arange(x.shape[0], device=x.device, dtype=torch.float32))[:, None, None] * freq
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()], -1)


class Block:
    """The attention block with its cache, for one sequence."""

    def __init__(self, hidden, heads, kv_heads, dim, tokens, page=64, seed=0):
        import torch

        rng = np.random.default_rng(seed)
        coded = lambda rows, cols: CodedMatrix((rng.standard_t(4, size=(rows, cols)) * 0.02).astype(np.float32))  # noqa: E731
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.q, self.k, self.v = coded(heads * dim, hidden), coded(kv_heads * dim, hidden), coded(kv_heads * dim, hidden)
        self.o = coded(hidden, heads * dim)
        pages = -(-tokens // page)
        self.cache = ent.KVCache.empty(pages, kv_heads, dim, page)
        self.table = torch.randperm(pages, device="cuda").to(torch.int32)[None].contiguous()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.held = 0

    def _ints(self, *v):
        import torch

        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def __call__(self, x):
        """x [tokens][hidden] (bf16), the tokens after those held -> float32
        [tokens][hidden]."""
        import torch

        n, first = x.shape[0], self.held
        q, k, v = product((self.q, self.k, self.v), x)
        q = rotate(q.view(n, self.heads, self.dim), first).to(torch.bfloat16)
        k = rotate(k.view(n, self.kv_heads, self.dim), first).to(torch.bfloat16)
        v = v.view(n, self.kv_heads, self.dim).to(torch.bfloat16)
        if n > 1:
            # the tokens in front from the cache, then this piece's own
            kk, vv = (torch.empty(first + n, self.kv_heads, self.dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
            ent.kv_load(self.cache, self.table, self._ints(0), self._ints(0, first), first, self.status,
                        out=(kk[:first], vv[:first]))
            kk[first:], vv[first:] = k, v
            y = ent.attn_prompt(q, kk, vv, self._ints(0, n), self._ints(0, first + n), self.status)
        ent.kv_store(self.cache, k, v, self.table, self._ints(first), self._ints(0, n), self.status)
        if n == 1:
            y = ent.attn_cache(q, self.cache, self.table, self._ints(first + 1), self.status)
        self.held = first + n
        return product((self.o,), y.view(n, self.heads * self.dim))[0]

    def plain(self, x):
        """All tokens at once in float32 on the decoded weights, no cache."""
        import torch

        n, g = x.shape[0], self.heads // self.kv_heads
        x = x.float()
        q, k, v = (x @ m.dense().float().t() for m in (self.q, self.k, self.v))
        q = rotate(q.view(n, self.heads, self.dim), 0)
        k = rotate(k.view(n, self.kv_heads, self.dim), 0).repeat_interleave(g, 1)
        v = v.view(n, self.kv_heads, self.dim).repeat_interleave(g, 1)
        s = torch.bmm(q.transpose(0, 1).contiguous(), k.permute(1, 2, 0).contiguous()) / math.sqrt(self.dim)
        s = s.masked_fill(torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1), -math.inf)
        y = torch.bmm(s.softmax(-1), v.transpose(0, 1).contiguous()).transpose(0, 1).reshape(n, -1)
        return y @ self.o.dense().float().t()


def run(hidden=4096, heads=32, kv_heads=8, head_dim=128, prompt=600, new=32, seed=0):
    """-> (relative error against the plain block, ms of the prompt, ms a token)."""
    import torch

    block = Block(hidden, heads, kv_heads, head_dim, prompt + new, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(prompt + new, hidden, device="cuda", generator=g).to(torch.bfloat16)

    def serve():
        block.held = 0
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        out = [block(piece) for piece in x[:prompt].split(max(2, min(512, -(-prompt // 2))))]   # the fused GEMM takes up to 512
        torch.cuda.synchronize()
        t1 = time.perf_counter()
        out += [block(x[i: i + 1]) for i in range(prompt, prompt + new)]
        torch.cuda.synchronize()
        return torch.cat(out), 1e3 * (t1 - t0), 1e3 * (time.perf_counter() - t1) / max(new, 1)

    serve()
    got, prompt_ms, token_ms = serve()
    if block.status.any():
        raise RuntimeError(f"faults flagged: {block.status.tolist()}")
    want = block.plain(x)
    return float((got - want).norm() / want.norm()), prompt_ms, token_ms


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("hidden", 4096), ("heads", 32), ("kv-heads", 8), ("head-dim", 128), ("prompt", 600), ("new", 32)):
        p.add_argument(f"--{name}", type=int, default=value)
    a = p.parse_args()
    err, prompt_ms, token_ms = run(a.hidden, a.heads, a.kv_heads, a.head_dim, a.prompt, a.new)
    print(f"{a.prompt} prompt tokens {prompt_ms:.2f} ms, {a.new} new tokens {token_ms:.3f} ms each; "
          f"relative error against the plain float32 block {err:.2e}")


if __name__ == "__main__":
    main()
