"""Several answers to one prompt, decoded as a batch that shares the prompt's pages.

    python examples/serve_shared_prompt.py [--answers 16] [--prompt 2000] [--steps 24] [--beams]

One attention block of a decoder with a norm of each head's queries and keys and rotary positions, over
the 8-bit cache. The prompt goes through it once, in one row of the pool; then the row is forked
into all others (``kv8_arrange``: its whole pages are shared, the last one copied), and every decoding
step, captured in a CUDA graph, does

    kv8_arrange (room for one token)  ->  q, k, v = W_qkv h  ->  qk_norm_rope  ->  kv8_append
    ->  attention_kv8_shared (the prompt read once for all answers)  ->  y = x + W_o o

With ``--beams`` the rows are reordered in the same kv8_arrange call, as a step of beam search does: row i
goes on with the tokens of a row drawn at random. At the end some rows end, the pool is compacted (``kv8_compact``)
and another step runs. The same tokens go through the block in plain fp32 without any rounding,
and the difference is printed: it is what the cache's 8 bits and bf16 cost.
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
    def __init__(self, hidden, heads, kv_heads, head_dim, rows, max_tokens, page_size=64, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        qkv = (heads + 2 * kv_heads) * head_dim
        self.w_qkv = torch.randn(qkv, hidden, generator=g, device="cuda").mul_(hidden ** -0.5).to(torch.bfloat16)
        self.w_o = torch.randn(hidden, heads * head_dim, generator=g, device="cuda").mul_((heads * head_dim) ** -0.5).to(torch.bfloat16)
        self.q_weight, self.k_weight = (1 + 0.2 * torch.randn(2, head_dim, generator=g, device="cuda")).to(torch.bfloat16)
        half = head_dim // 2
        self.inv_freq = (10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)).float()
        width = -(-max_tokens // page_size)
        pages = 2 * rows * (-(-max_tokens // page_size))
        self.cache = hk.Kv8Cache.empty(pages, kv_heads, head_dim, page_size)
        self.pool = hk.Kv8Pool.empty(pages, rows, width, page_size)
        self.tokens = torch.zeros(rows, dtype=torch.int32, device="cuda")       # appended to each row

    def arrange(self, keep, room, parents=None):
        return hk.kv8_arrange(self.pool, keep, room, parents, caches=self.cache)

    def forward(self, x, rows, starts, attend):
        """x [B, T, hidden] for the table rows ``rows`` (a slice), whose tokens begin at ``starts``."""
        B, T, hidden = x.shape
        h = (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)
        qkv = hk.gemm(h.view(B * T, hidden), self.w_qkv).view(B, T, self.heads + 2 * self.kv_heads, self.head_dim)
        q, k, v = qkv.split((self.heads, self.kv_heads, self.kv_heads), 2)
        positions = starts[:, None] + torch.arange(T, device="cuda", dtype=torch.int32)
        q, k = hk.qk_norm_rope(q, k, positions, self.inv_freq, self.q_weight, self.k_weight)
        table = self.pool.table[rows]
        hk.kv8_append(self.cache, k, v, table, starts)
        o = attend(q, table, starts + T)
        return x + hk.gemm(o.reshape(B * T, -1), self.w_o).view(B, T, hidden)

    def reference(self, x):
        """The block on all tokens of one row, [n, hidden], in fp32."""
        n = len(x)
        h = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
        q, k, v = (h @ self.w_qkv.float().t()).view(n, -1, self.head_dim).split((self.heads, self.kv_heads, self.kv_heads), 1)
        angle = torch.arange(n, device="cuda").double()[:, None] * self.inv_freq.double()
        cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

        def turned(t, w):
            t = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6) * w.float()
            a, b = t.chunk(2, -1)
            return torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
        q, k = turned(q, self.q_weight), turned(k, self.k_weight)
        k, v = (t.repeat_interleave(self.heads // self.kv_heads, 1) for t in (k, v))
        s = torch.einsum("qhd,khd->hqk", q, k) / math.sqrt(self.head_dim)
        s = s.masked_fill(torch.ones_like(s[0], dtype=torch.bool).triu(1), float("-inf"))
        return x + torch.einsum("hqk,khd->qhd", s.softmax(-1), v).reshape(n, -1) @ self.w_o.float().t()


def run(hidden=2048, heads=32, kv_heads=8, head_dim=128, answers=16, prompt=2000, steps=24, beams=False, page_size=64, verbose=True):
    """Prompt, fork, captured steps, compaction; returns the relative error against the plain block (over the tokens' updates)."""
    say = print if verbose else lambda *a: None
    g = torch.Generator(device="cuda").manual_seed(1)
    block = Block(hidden, heads, kv_heads, head_dim, answers, prompt + steps + 1, page_size)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    draw = lambda *shape: torch.randn(*shape, hidden, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731

    # the prompt, in row 0
    keep = torch.zeros(answers, dtype=torch.int32, device="cuda")
    room = keep.clone()
    room[0] = prompt
    missing = block.arrange(keep, room)
    text = draw(1, prompt)
    first = block.forward(text, slice(0, 1), i32(0), lambda q, t, n: hk.attention_kv8(q, block.cache, t, n))
    # every row becomes a fork of it
    tokens = torch.full((answers,), prompt, dtype=torch.int32, device="cuda")
    missing = missing + block.arrange(tokens, tokens, torch.zeros(answers, dtype=torch.int32, device="cuda"))

    groups, shared = i32(0, answers), i32(prompt)
    x, parents = draw(answers, 1), torch.arange(answers, device="cuda", dtype=torch.int32)

    def step():
        lacked = block.arrange(tokens, tokens + 1, parents if beams else None)
        y = block.forward(x, slice(0, answers), tokens,
                          lambda q, t, n: hk.attention_kv8_shared(q, block.cache, t, n, groups, shared))
        return y, lacked

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        y, lacked = step()
        missing.add_(lacked)
        tokens.add_(1)
    identity = parents.clone()
    given, orders, got = [], [], []
    for _ in range(steps):
        given.append(draw(answers, 1))
        orders.append(torch.randint(0, answers, (answers,), generator=g, device="cuda").int() if beams else identity)
    torch.cuda.synchronize()
    began = time.perf_counter()
    for new, order in zip(given, orders):
        x.copy_(new)
        parents.copy_(order)
        graph.replay()
        got.append(y.clone())
    torch.cuda.synchronize()
    say(f"{answers} answers to {prompt} tokens: {(time.perf_counter() - began) / steps * 1e6:.0f} us a step, "
        f"{int((block.pool.refs > 0).sum())} pages in use where unshared ones would be {answers * -(-(prompt + steps) // page_size)}")

    texts = [[text[0]] for _ in range(answers)]          # what each row has been given, and what came out
    outs = [[first[0]] for _ in range(answers)]
    for new, order, out in zip(given, orders, got):
        texts, outs = ([list(rows[p]) for p in order.tolist()] for rows in (texts, outs))
        for i in range(answers):
            texts[i].append(new[i])
            outs[i].append(out[i])

    # all rows but every other one end, the pool is moved together, and one more step
    gone = torch.arange(answers, device="cuda") % 2 == 1
    tokens.masked_fill_(gone, 0)
    parents.copy_(identity)
    missing = missing + block.arrange(tokens, tokens)
    hk.kv8_compact(block.pool, block.cache)
    if int((block.pool.refs > 0).sum()) != int(block.pool.refs.nonzero().max()) + 1:
        raise RuntimeError("the pages in use are not the first ones")
    x.copy_(draw(answers, 1))
    y, lacked = step()
    missing = missing + lacked
    for i in range(answers):
        if i % 2 == 0:
            texts[i].append(x[i].clone())
            outs[i].append(y[i].clone())
    if missing.item() or hk.hk_gemm_last_device_status(torch.cuda.current_device()) != hk.HK_OK:
        raise RuntimeError(f"pages lacked, or {hk.hk_gemm_last_error_string()}")

    off = norm = 0.0
    for row, out in zip(texts, outs):
        row, out = torch.cat(row).float(), torch.cat(out).float()
        want = block.reference(row)
        off += (out - want).square().sum().item()
        norm += (want - row).square().sum().item()
    error = math.sqrt(off / norm)
    say(f"the block's update is {100 * error:.2f} % off the same block in fp32")
    return error


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--answers", type=int, default=16)
    ap.add_argument("--prompt", type=int, default=2000)
    ap.add_argument("--steps", type=int, default=24)
    ap.add_argument("--beams", action="store_true")
    a = ap.parse_args()
    run(answers=a.answers, prompt=a.prompt, steps=a.steps, beams=a.beams)
