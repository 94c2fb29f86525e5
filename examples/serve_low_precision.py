"""One attention block of a decoder served in low precision: weights and
activations in 4 bits (NVFP4 or MXFP4), keys and values in a paged 8-bit cache.

    python examples/serve_low_precision.py [--format nvfp4] [--batch 8] [--prompt 512] [--steps 32]

A ragged batch of prompts goes through the block once (``prefill``), then single
tokens step by step, the step captured in a CUDA graph. The block, per token x:

    h = x / rms(x);  q, k, v = W_qkv h;  cache += k, v;  y = x + W_o attention(q, cache)

(no rotary embedding: the example is about the operators.) Both products run
as quantize_fp4 -> gemm_fp4, the cache as kv8_append -> attention_kv8. At the
end the same tokens go through the block in plain fp32, without any rounding,
and the difference is printed: it is what the two formats cost.
"""
import argparse
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_bf16_gemm_02_gb300 as hk  # noqa: E402


class Block:
    def __init__(self, hidden, heads, kv_heads, head_dim, batch, max_tokens, format="nvfp4", page_size=64, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.kv_heads, self.head_dim, self.format = heads, kv_heads, head_dim, format
        qkv = (heads + 2 * kv_heads) * head_dim
        self.w_qkv = torch.randn(qkv, hidden, generator=g, device="cuda") / math.sqrt(hidden)
        self.w_o = torch.randn(hidden, heads * head_dim, generator=g, device="cuda") / math.sqrt(heads * head_dim)
        self.q_qkv, self.q_o = self._quantize(self.w_qkv), self._quantize(self.w_o)
        pages = -(-max_tokens // page_size)
        self.cache = hk.Kv8Cache.empty(batch * pages, kv_heads, head_dim, page_size)
        self.table = torch.randperm(batch * pages, generator=g, device="cuda").view(batch, pages).to(torch.int32)
        self.lengths = torch.zeros(batch, dtype=torch.int32, device="cuda")

    def _quantize(self, x):
        scale = x.float().abs().amax().reshape(1) / 2688 if self.format == "nvfp4" else None
        return hk.quantize_fp4(x, format=self.format, global_scale=scale)

    def forward(self, x, counts=None):
        """x [B, T, hidden] bf16, of each sequence the first ``counts`` tokens (None: all); returns y like x."""
        B, T, hidden = x.shape
        h = (x.float() * torch.rsqrt(x.float().pow(2).mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)
        qkv = hk.gemm_fp4(self._quantize(h.view(B * T, hidden)), self.q_qkv)
        qkv = qkv.view(B, T, self.heads + 2 * self.kv_heads, self.head_dim)
        q, k, v = qkv.split((self.heads, self.kv_heads, self.kv_heads), 2)       # views: rows keep their strides
        hk.kv8_append(self.cache, k, v, self.table, self.lengths, counts=counts)
        self.lengths.add_(T if counts is None else counts)
        o = hk.attention_kv8(q, self.cache, self.table, self.lengths, counts=counts)
        return x + hk.gemm_fp4(self._quantize(o.view(B * T, -1)), self.q_o).view(B, T, hidden)

    def reference(self, x, b):
        """The block on all tokens of sequence b, [n, hidden], in fp32."""
        h = x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + 1e-6)
        q, k, v = (h @ self.w_qkv.t()).view(len(x), -1, self.head_dim).split((self.heads, self.kv_heads, self.kv_heads), 1)
        k, v = (t.repeat_interleave(self.heads // self.kv_heads, 1) for t in (k, v))
        s = torch.einsum("qhd,khd->hqk", q, k) / math.sqrt(self.head_dim)
        s = s.masked_fill(torch.ones_like(s[0], dtype=torch.bool).triu(1), float("-inf"))
        return x + torch.einsum("hqk,khd->qhd", s.softmax(-1), v).reshape(len(x), -1) @ self.w_o.t()


def run(hidden=4096, heads=32, kv_heads=8, head_dim=128, batch=8, prompt=512, steps=32, format="nvfp4", verbose=True):
    """Prefill and decode; returns the relative error against the plain block (over the tokens' updates)."""
    say = print if verbose else lambda *a: None
    g = torch.Generator(device="cuda").manual_seed(1)
    block = Block(hidden, heads, kv_heads, head_dim, batch, prompt + steps, format)
    counts = torch.randint(max(1, prompt // 2), prompt + 1, (batch,), generator=g, device="cuda").to(torch.int32)
    tokens = torch.randn(batch, prompt + steps, hidden, generator=g, device="cuda").to(torch.bfloat16)
    first = block.forward(tokens[:, :prompt], counts)

    x = torch.zeros(batch, 1, hidden, dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    kept = block.lengths.clone()
    with torch.cuda.graph(graph):               # (captured, not run: the cache and the lengths stay as they are)
        y = block.forward(x)
    assert torch.equal(kept, block.lengths)
    outputs = []
    began = time.perf_counter()
    for i in range(steps):
        x.copy_(tokens[:, prompt + i:prompt + i + 1])
        graph.replay()
        outputs.append(y.clone())
    torch.cuda.synchronize()
    took = (time.perf_counter() - began) / steps
    say(f"{batch} sequences, prompts of {counts.min().item()} to {counts.max().item()} tokens: {took * 1e6:.0f} us a step")
    if hk.hk_gemm_last_device_status(torch.cuda.current_device()) != hk.HK_OK:
        raise RuntimeError(hk.hk_gemm_last_error_string())

    off = norm = 0.0
    for b, n in enumerate(counts.tolist()):
        mine = torch.cat([first[b, :n]] + [o[b] for o in outputs]).float()
        seen = torch.cat([tokens[b, :n], tokens[b, prompt:]]).float()
        want = block.reference(seen, b)
        off += (mine - want).square().sum().item()
        norm += (want - seen).square().sum().item()
    error = math.sqrt(off / norm)
    say(f"{format}: the block's update is {100 * error:.1f} % off the same block in fp32")
    return error


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--format", choices=("nvfp4", "mxfp4"), default="nvfp4")
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=512)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args()
    run(batch=a.batch, prompt=a.prompt, steps=a.steps, format=a.format)
