"""One decoder layer of a served model, from compressed weights to its output.

    h = x + residual;  y = norm(h)              uw_rmsnorm
    qkv = y Wqkv^T                              uw_matmul, weights compressed
    rotate q, k; append k, v to the 4-bit cache uw_kv4_append
    a = attention over the cache                uw_kv4_attention
    o = a Wo^T                                  uw_matmul, weights compressed
    h' = h + o;  y' = norm(h')                  uw_rmsnorm
    m = MLP(y')                                 uw_mlp_forward, weights compressed

The next layer adds m to h' in its first norm.  The demonstration takes in a few
prompts of different lengths at once, then generates a few tokens for all of
them, and prints what the layer holds in memory and how long the steps take:

    python examples/decoder_layer.py [--hidden 4096 --mlp 14336 --q-heads 32 --kv-heads 8]
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import lossless_bf16_weight_gb300 as uw  # noqa: E402
import workloads as wl  # noqa: E402


class Matrix:
    """A weight matrix, compressed on the host, its blob on the device."""

    def __init__(self, w: np.ndarray):
        self.w = w
        blob = uw.compress(w)
        self.desc, self.blob = uw.blob_info(blob), torch.from_numpy(blob).cuda()

    def nbytes(self) -> int:
        return int(self.desc.blob_bytes)


def rope_table(positions: int, dim: int, base: float = 10000.0):
    angle = torch.arange(positions, device="cuda").double()[:, None] * base ** (
        -torch.arange(0, dim, 2, device="cuda").double() / dim)
    return angle.cos().float(), angle.sin().float()


class DecoderLayer:
    """Weights, the cache of one layer, and the workspaces of its calls.  Batches
    of up to `max_tokens` new tokens; `pages` pages shared by all sequences."""

    def __init__(self, hidden, mlp, q_heads, kv_heads, head_dim, pages, page_size, max_tokens, max_positions, seed=0):
        self.hidden, self.q_heads, self.kv_heads, self.head_dim = hidden, q_heads, kv_heads, head_dim
        self.page_size, self.eps = page_size, 1e-5
        heads = q_heads + 2 * kv_heads
        shapes = {"qkv": (heads * head_dim, hidden), "o": (hidden, q_heads * head_dim), "gate": (mlp, hidden),
                  "up": (mlp, hidden), "down": (hidden, mlp)}
        self.m = {name: Matrix(wl.normal_weights(r, c, c ** -0.5, seed + i))
                  for i, (name, (r, c)) in enumerate(shapes.items())}
        rng = np.random.default_rng(seed)
        self.norms = [torch.from_numpy(wl.bf16_bits(1 + 0.1 * rng.standard_normal(hidden)).view(np.int16)).cuda()
                      .view(torch.bfloat16) for _ in range(2)]
        self.pages = torch.zeros(pages, uw.kv4_page_bytes(kv_heads, head_dim, page_size), dtype=torch.uint8,
                                 device="cuda")
        self.cos, self.sin = rope_table(max_positions, head_dim)
        self.mlp = uw.mlp_matrices([(self.m[n].desc, self.m[n].blob, None, None) for n in ("gate", "up", "down")])
        empty = uw.kv4_cache(self.pages, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), kv_heads, head_dim,
                             page_size)
        # A call finds its counters in its workspace as its last one left them, so every matrix
        # shape, the chain and the cache have workspaces of their own.
        # (A smaller batch may need more than a larger one, which is cut up less.)
        batches = range(1, max_tokens + 1)
        need = {n: max(uw.workspace_size(self.m[n].desc, b) for b in batches) for n in ("qkv", "o")}
        need["mlp"] = max(uw.mlp_workspace_size(self.mlp, b) for b in batches)
        need["kv"] = uw.kv4_workspace_size(empty, q_heads)
        self.ws = {n: torch.empty(size, dtype=torch.uint8, device="cuda") for n, size in need.items()}
        for ws in self.ws.values():
            uw.workspace_init(ws)

    def forward(self, x, residual, cache, start, length, max_new, max_len):
        """x, residual [tokens, hidden] BF16 (residual None in the first layer).  Returns (MLP's output, h')."""
        t, hq, hk, d = x.shape[0], self.q_heads, self.kv_heads, self.head_dim
        y = torch.empty_like(x)
        if residual is None:
            h = x
            uw.rmsnorm(x, self.norms[0], y, self.eps)
        else:
            h = torch.empty_like(x)
            uw.rmsnorm(x, self.norms[0], y, self.eps, residual=residual, residual_out=h)
        qkv = torch.empty(t, hq + 2 * hk, d, dtype=x.dtype, device=x.device)
        uw.matmul(self.m["qkv"].desc, self.m["qkv"].blob, y, qkv, self.ws["qkv"])
        q = torch.empty(t, hq, d, dtype=x.dtype, device=x.device)
        uw.kv4_append(cache, start, length, qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:], q, self.cos, self.sin,
                      self.ws["kv"])
        a = torch.empty_like(q)
        uw.kv4_attention(cache, start, length, q, a, self.ws["kv"], max_new, max_len)
        o = torch.empty_like(x)
        uw.matmul(self.m["o"].desc, self.m["o"].blob, a.view(t, hq * d), o, self.ws["o"])
        h2 = torch.empty_like(x)
        uw.rmsnorm(o, self.norms[1], y, self.eps, residual=h, residual_out=h2)
        out = torch.empty_like(x)
        uw.mlp_forward(self.mlp, y, out, self.ws["mlp"])
        return out, h2

    def check(self):
        """Synchronises; errors that a kernel recorded raise."""
        for ws in self.ws.values():
            status = uw.check_status(ws)
            if status != uw.UW_OK:
                raise uw.UwError(status, "decoder layer")


class Sequences:
    """Lengths and page table of a batch of sequences over a layer's pages."""

    def __init__(self, layer: DecoderLayer, count: int, max_len: int):
        self.layer, self.len = layer, [0] * count
        self.width = -(-max_len // layer.page_size)
        self.table = torch.full((count, self.width), -1, dtype=torch.int32, device="cuda")
        self.free = list(range(layer.pages.shape[0]))
        self.cache = uw.kv4_cache(layer.pages, self.table, layer.kv_heads, layer.head_dim, layer.page_size)

    def extend(self, new):
        """Room for new[s] more tokens of every sequence; the arguments of the layer's call."""
        size = self.layer.page_size
        for s, n in enumerate(new):
            have, want = -(-self.len[s] // size), -(-(self.len[s] + n) // size)
            if want > have:
                self.table[s, have:want] = torch.tensor([self.free.pop() for _ in range(want - have)],
                                                        dtype=torch.int32, device="cuda")
            self.len[s] += n
        start = torch.tensor([0] + list(new), dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()
        length = torch.tensor(self.len, dtype=torch.int32).cuda()
        return self.cache, start, length, max(new), max(self.len)


def timed(f, repeat=20):
    f()
    torch.cuda.synchronize()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(repeat):
        f()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / repeat * 1e3


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--hidden", type=int, default=1024)
    p.add_argument("--mlp", type=int, default=2048)
    p.add_argument("--q-heads", type=int, default=8)
    p.add_argument("--kv-heads", type=int, default=2)
    p.add_argument("--head-dim", type=int, default=128)
    p.add_argument("--prompts", default="700,64,1,333")
    p.add_argument("--tokens", type=int, default=16)
    a = p.parse_args()
    prompts = [int(n) for n in a.prompts.split(",")]
    longest = max(prompts) + a.tokens
    page = 64
    layer = DecoderLayer(a.hidden, a.mlp, a.q_heads, a.kv_heads, a.head_dim,
                         sum(-(-(n + a.tokens) // page) for n in prompts), page, sum(prompts), longest)
    plain = sum(2 * m.w.size for m in layer.m.values())
    held = sum(m.nbytes() for m in layer.m.values())
    print("weights %.1f MB, compressed %.1f MB; cache %.1f MB for %d positions (BF16: %.1f MB)" % (
        plain / 1e6, held / 1e6, layer.pages.numel() / 1e6, layer.pages.shape[0] * page,
        layer.pages.shape[0] * page * a.kv_heads * a.head_dim * 4 / 1e6))
    seqs = Sequences(layer, len(prompts), longest)
    x = torch.randn(sum(prompts), a.hidden, device="cuda").bfloat16()
    args = seqs.extend(prompts)
    print("prompts of %s tokens: %.1f us" % (a.prompts, timed(lambda: layer.forward(x, None, *args), 5)))
    for i in range(a.tokens):
        x = torch.randn(len(prompts), a.hidden, device="cuda").bfloat16()
        args = seqs.extend([1] * len(prompts))
        out, h = layer.forward(x, x, *args)
    print("one token each, %d keys at most: %.1f us" % (longest, timed(lambda: layer.forward(x, x, *args))))
    layer.check()
    assert torch.isfinite(out.float()).all() and torch.isfinite(h.float()).all()


if __name__ == "__main__":
    main()
