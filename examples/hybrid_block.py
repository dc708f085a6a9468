"""A small hybrid model on the library's operators: GDN-2 layers, which carry a
state per sequence, alternate with softmax-attention layers, which carry a paged
key/value cache.  Both read the same packed batch (cu_seqlens), so a chunk of a
prefill and a decode step are the same call with other lengths.

    python examples/hybrid_block.py                 # prefill in chunks, then decode
    python examples/hybrid_block.py --layers 8 --prompt 16384 --seqs 4 --graph

The projections, norms and gates around the operators are plain torch, with
random weights.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from gated_deltanet_prefill_gb300 import attn, gdn2  # noqa: E402

# Up to this many new tokens per sequence the token-by-token call is the faster one.
RECURRENT_TOKENS = 16


def matrix(g, rows, cols):
    return (torch.randn(rows, cols, device="cuda", generator=g) * rows ** -0.5).to(torch.bfloat16)


class Batch:
    """One call's packed batch: ``new[n]`` tokens of each sequence, and the
    cached lengths with them."""

    def __init__(self, new, kv_lens):
        self.new = max(new)
        self.cu = torch.tensor([0] + new, device="cuda").cumsum(0, dtype=torch.int32)
        self.kv_lens = kv_lens


class Pages:
    """Page tables of a batch of sequences.  The layers' caches have the same
    pages; a sequence's pages are handed out as it grows."""

    def __init__(self, seqs, max_tokens, page_size):
        self.size = page_size
        width = -(-max_tokens // page_size)
        self.table = torch.full((seqs, width), -1, dtype=torch.int32, device="cuda")
        self.held = [0] * seqs
        self.free = list(range(seqs * width))

    def grow(self, lens):
        for n, tokens in enumerate(lens):
            more = -(-tokens // self.size) - self.held[n]
            if more > 0:
                ids = [self.free.pop() for _ in range(more)]
                self.table[n, self.held[n]:self.held[n] + more] = torch.tensor(ids, dtype=torch.int32)
                self.held[n] += more


class Gdn2Layer:
    def __init__(self, g, dim, heads, head_dim, seqs):
        self.heads, self.d = heads, head_dim
        self.w_in = matrix(g, dim, 6 * heads * head_dim)  # q, k, v, write gate, erase gate, decay
        self.w_out = matrix(g, heads * head_dim, dim)
        self.state = torch.zeros(seqs, heads, head_dim, head_dim, device="cuda")

    def __call__(self, x, batch):
        y = (x @ self.w_in).view(-1, 6 * self.heads, self.d)
        q, k, v, w, beta, g = y.split(self.heads, dim=1)
        w, beta, g = torch.sigmoid(w), torch.sigmoid(beta), -F.softplus(g.float() - 2)
        args = (q, k, v, g, beta, w)
        kw = dict(initial_state=self.state, cu_seqlens=batch.cu, use_qk_l2norm=True)
        if batch.new <= RECURRENT_TOKENS:
            o, _ = gdn2.recurrent_gdn2_fwd(*args, final_state=self.state, **kw)  # state in place
        else:
            o, self.state = gdn2.chunk_gdn2_fwd(*args, **kw)
        return o.flatten(1) @ self.w_out


class AttentionLayer:
    def __init__(self, g, dim, heads, kv_heads, head_dim, pages):
        self.hq, self.hkv, self.d, self.pages = heads, kv_heads, head_dim, pages
        self.w_in = matrix(g, dim, (heads + 2 * kv_heads) * head_dim)
        self.w_out = matrix(g, heads * head_dim, dim)
        self.q_weight, self.k_weight = (1 + matrix(g, head_dim, 2) / 4).t().contiguous()
        self.inv_freq, self.rope_factor = attn.rope_frequencies(head_dim // 2)  # half of each head turns
        shape = (pages.table.numel(), pages.size, kv_heads, head_dim)
        self.k_cache = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        self.v_cache = torch.empty(shape, dtype=torch.bfloat16, device="cuda")

    def __call__(self, x, batch):
        y = (x @ self.w_in).view(-1, self.hq + 2 * self.hkv, self.d)
        q, k, v = y.split([self.hq, self.hkv, self.hkv], dim=1)  # views: no copy
        cache = (self.k_cache, self.v_cache, self.pages.table, batch.kv_lens, batch.cu)
        q = attn.append_kv(k, v, *cache, q=q, inv_freq=self.inv_freq, rope_factor=self.rope_factor,
                           q_weight=self.q_weight, k_weight=self.k_weight)
        return attn.paged_attn_fwd(q, *cache).flatten(1) @ self.w_out


class HybridModel:
    """``layers`` layers, every second one (the odd ones) with attention."""

    def __init__(self, seqs, max_tokens, dim=512, layers=2, heads=4, kv_heads=1, head_dim=128, page_size=32, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.seqs, self.lens = seqs, [0] * seqs
        self.kv_lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        self.pages = Pages(seqs, max_tokens, page_size)
        self.layers = [AttentionLayer(g, dim, heads, kv_heads, head_dim, self.pages) if i % 2 else
                       Gdn2Layer(g, dim, heads, head_dim, seqs) for i in range(layers)]

    def reserve(self, new):
        """Pages and a batch for ``new[n]`` more tokens of each sequence."""
        self.lens = [a + b for a, b in zip(self.lens, new)]
        self.pages.grow(self.lens)
        return Batch(new, self.kv_lens)

    def run(self, x, batch):
        """x [tokens, dim]: the new tokens' embeddings; the device's lengths have them counted in."""
        for layer in self.layers:
            x = x + layer(F.rms_norm(x, x.shape[-1:]), batch)
        return x

    def __call__(self, x, new):
        batch = self.reserve(new)
        self.kv_lens += torch.tensor(new, dtype=torch.int32, device="cuda")
        return self.run(x, batch)


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, default in (("layers", 4), ("dim", 2048), ("heads", 16), ("kv-heads", 4), ("seqs", 8), ("prompt", 4096),
                          ("chunk", 2048), ("tokens", 64)):
        p.add_argument("--" + name, type=int, default=default)
    p.add_argument("--graph", action="store_true", help="decode steps replayed from a CUDA graph")
    a = p.parse_args()
    model = HybridModel(a.seqs, a.prompt + a.tokens + 8, a.dim, a.layers, a.heads, a.kv_heads)
    x = torch.randn(a.seqs, a.prompt, a.dim, device="cuda").to(torch.bfloat16)

    def timed(f):
        t0, t1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        t0.record()
        y = f()
        t1.record()
        t1.synchronize()
        return y, t0.elapsed_time(t1)

    def prefill():
        for i in range(0, a.prompt, a.chunk):
            part = x[:, i:i + a.chunk]
            y = model(part.reshape(-1, a.dim), [part.shape[1]] * a.seqs)
        return y.view(a.seqs, -1, a.dim)[:, -1]

    step = [1] * a.seqs
    y, ms = timed(prefill)
    print("prefill: %d x %d tokens in chunks of %d: %.2f ms, %.0f tokens/s (first calls included)" % (
        a.seqs, a.prompt, a.chunk, ms, a.seqs * a.prompt / ms * 1e3))
    token = y.clone()
    for _ in range(3):
        token.copy_(F.rms_norm(model(token, step), (a.dim,)))
    model.reserve([a.tokens] * a.seqs)  # pages of all tokens to come
    batch = Batch(step, model.kv_lens)

    def decode():  # the output stands in for the next token's embedding
        model.kv_lens.add_(1)
        token.copy_(F.rms_norm(model.run(token, batch), (a.dim,)))

    if a.graph:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            decode()
        call = graph.replay
    else:
        call = decode
    _, ms = timed(lambda: [call() for _ in range(a.tokens)])
    assert torch.isfinite(token.float()).all()
    print("decode:  %d steps of %d sequences%s: %.3f ms per step, %.0f tokens/s" % (
        a.tokens, a.seqs, " (graph)" if a.graph else "", ms / a.tokens, a.seqs * a.tokens / ms * 1e3))


if __name__ == "__main__":
    main()
