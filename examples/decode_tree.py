"""Tree-drafted decoding through one attention block with ternary projections,
from a cache that is kept within a budget.

    python examples/decode_tree.py [steps]

Each step drafts a tree of tokens for every sequence and runs, for all of them
at once: INT8 quantization and the ternary QKV projection, norm + rotation +
append to the cache, tree attention, INT8 quantization and the ternary output
projection; then, once the accepted path of each tree is known, the attention
weights of the accepted tokens are added to the cache's running sums, and the
rejected drafts and the least attended tokens beyond the budget leave the
cache.  Hidden states and weights are random: what is shown is the path.
"""
from __future__ import annotations

import os
import random
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import xnor_popcount_gemm_amd as bnn  # noqa: E402


class TernaryLinear:
    """y = gamma * (t x), t = RoundClip(W / gamma) in {-1, 0, +1}, x in INT8."""

    def __init__(self, W: torch.Tensor):
        self.K = W.shape[1]
        self.gamma = bnn.weight_scale_tensor(W)
        self.sign, self.nonzero, _ = bnn.pack_weights_ternary(W, gamma=self.gamma)

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        q = bnn.quantize_act_i8(x)
        return bnn.bwn_i8_linear(self.sign, self.K, bnn.EPI_SCALE_F32 | bnn.EPI_ALPHA_TENSOR | bnn.W_TERNARY, Zp=self.nonzero,
                                 alpha=self.gamma, **q)["Y"]


class Block:
    """The attention half of a decoder block, with its cache."""

    def __init__(self, sequences: int, *, hidden=1024, heads=8, kv_heads=2, dim=128, budget=96, recent=32, nodes=16, page=16,
                 max_pos=4096, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *shape: torch.randn(shape, generator=g, device="cuda")
        self.heads, self.kv_heads, self.dim, self.budget, self.recent, self.nodes = heads, kv_heads, dim, budget, recent, nodes
        self.qkv = TernaryLinear(normal((heads + 2 * kv_heads) * dim, hidden))
        self.out = TernaryLinear(normal(hidden, heads * dim))
        self.q_weight, self.k_weight = 1 + 0.1 * normal(dim), 1 + 0.1 * normal(dim)
        self.turns = bnn.rope_turns(max_pos, dim, kind="ramp", factor=4.0, old_ctx=max_pos / 4, device="cuda")
        per = -(-(budget + nodes) // page)                       # pages that a sequence can need
        k, v = (torch.zeros((sequences * per, page, kv_heads, dim), dtype=dtype, device="cuda") for _ in range(2))
        table = torch.randperm(sequences * per, generator=g, device="cuda").reshape(sequences, per).to(torch.int32)
        slots = (sequences, kv_heads, per * page)
        self.cache = bnn.KVCache(k, v, table, pos=torch.full(slots, -1, dtype=torch.int32, device="cuda"),
                                 score=torch.zeros(slots, device="cuda"))
        self.ctx = torch.zeros(sequences, dtype=torch.int32, device="cuda")
        self.workspace = bnn.tree_attention_workspace(self.cache, sequences * nodes, heads, nodes, budget)
        self.evict_workspace = bnn.cache_evict_workspace(self.cache)

    def attend(self, x, indptr, positions, mask):
        """x fp32 [rows, hidden] of the drafted tokens -> the block's output and
        what the later calls need of it."""
        h, kv, d = self.heads, self.kv_heads, self.dim
        q, k, v = (t.unflatten(1, (-1, d)) for t in self.qkv(x).split([h * d, kv * d, kv * d], dim=1))
        q = bnn.qk_norm_rope(q, k, v, self.cache, indptr, self.ctx, positions, self.turns, q_weight=self.q_weight, k_weight=self.k_weight)
        y, lse = bnn.tree_attention(q, self.cache, indptr, self.ctx, max_nodes=self.nodes, max_ctx=self.budget, mask=mask,
                                    out_dtype=torch.float32, workspace=self.workspace)
        return self.out(y.flatten(1)), (q, lse, indptr, mask)

    def accept(self, seen, accepted):
        """Keep the accepted drafts (packed bits per sequence) and the budget."""
        q, lse, indptr, mask = seen
        sizes = dict(max_nodes=self.nodes, max_ctx=self.budget, accept=accepted)
        bnn.cache_score_add(q, lse, self.cache, indptr, self.ctx, mask=mask, **sizes)
        bnn.cache_evict(self.cache, indptr, self.ctx, budget=self.budget, recent=self.recent, workspace=self.evict_workspace, **sizes)


def draft(rng: random.Random, nodes: int):
    """Parents of a random tree and an accepted path from its root."""
    parents = [-1] + [rng.randrange(i) for i in range(1, nodes)]
    path, node = [], rng.randrange(nodes)
    while node >= 0:
        path.append(node)
        node = parents[node]
    return parents, path[::-1]


def packed(path, nodes: int):
    """A set of nodes as signed 32-bit words, bit i % 32 of word i / 32 for node i."""
    words = [0] * ((nodes + 31) // 32)
    for i in path:
        words[i // 32] |= 1 << (i % 32)
    return [w - (1 << 32) if w >> 31 else w for w in words]


def run(steps: int = 40, sequences: int = 4, seed: int = 0, **kw):
    """Decodes; returns the block, the last outputs and each sequence's length."""
    block = Block(sequences, seed=seed, **kw)
    rng, g = random.Random(seed), torch.Generator(device="cuda").manual_seed(seed + 1)
    indptr = torch.arange(sequences + 1, dtype=torch.int32, device="cuda") * block.nodes
    length = [0] * sequences
    for _ in range(steps):
        trees = [draft(rng, block.nodes) for _ in range(sequences)]
        depth = [[0] * block.nodes for _ in trees]
        for d, (parents, _) in zip(depth, trees):
            for i, p in enumerate(parents):
                d[i] = d[p] + 1 if p >= 0 else 0
        mask = torch.cat([bnn.tree_mask(parents) for parents, _ in trees]).cuda()
        positions = torch.tensor([n + x for n, d in zip(length, depth) for x in d], dtype=torch.int32).cuda()
        bits = torch.tensor([packed(path, block.nodes) for _, path in trees], dtype=torch.int32).cuda()
        x = torch.randn((sequences * block.nodes, block.qkv.K), generator=g, device="cuda")
        y, seen = block.attend(x, indptr, positions, mask)
        block.accept(seen, bits)
        length = [n + len(path) for n, (_, path) in zip(length, trees)]
    return block, y, length


if __name__ == "__main__":
    block, y, length = run(int(sys.argv[1]) if len(sys.argv) > 1 else 40)
    torch.cuda.synchronize()
    print("tokens decoded:", length)
    print("tokens in the cache:", block.ctx.tolist(), "of a budget of", block.budget)
    print("output:", tuple(y.shape), "rms %.3f" % float(y.square().mean().sqrt()))
