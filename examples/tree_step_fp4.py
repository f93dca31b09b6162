"""Speculative decoding with a KV cache held in 4 bits, end to end on one GPU.

A one-layer attention model with random weights stands in for the target. Each step drafts a
trie for every request, builds its mask, runs the target's tree forward (projection, head norm
and rotation at the tree positions, attention over the 4-bit cache and the tree), verifies the
draft greedily and commits the accepted nodes' K/V to the cache in 4 bits.

    python examples/tree_step_fp4.py [--steps 8] [--batch 4] [--nodes 24]
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from speculative_decoding_tree_mask_gb300 import binding as G  # noqa: E402


class Model:
    """Embedding, one attention layer with head norms and rotated positions, output head."""

    def __init__(self, vocab, Hq, Hkv, D, device, seed=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.Hq, self.Hkv, self.D, self.width = Hq, Hkv, D, Hq * D

        def weight(rows, cols):
            w = torch.randn((rows, cols), generator=g, device=device) * cols ** -0.5
            return w.to(torch.bfloat16)

        self.emb = weight(vocab, self.width) * self.width ** 0.5
        self.qkv = weight((Hq + 2 * Hkv) * D, self.width)
        self.proj = weight(self.width, self.width)
        self.head = weight(vocab, self.width)
        self.q_weight = torch.ones(D, dtype=torch.bfloat16, device=device)
        self.k_weight = torch.ones(D, dtype=torch.bfloat16, device=device)
        self.inv_freq = 10000.0 ** (-torch.arange(D // 2, device=device).float() / (D // 2))

    def project(self, h, tokens, pos, depth):
        """Rows q, k (normalised and rotated) and v of tokens [B, N] at pos[b] + depth[b][n].
        q, k and v are columns of one projection; q and k are rotated in place."""
        B, N = tokens.shape
        rows = self.emb[tokens] @ self.qkv.T
        q, k, v = rows.split([self.Hq * self.D, self.Hkv * self.D, self.Hkv * self.D], -1)
        q, k, v = (t.unflatten(2, (-1, self.D)) for t in (q, k, v))
        G.spec_qk_norm_rope(h, q, k, self.inv_freq, pos, depth, q, k, self.q_weight,
                            self.k_weight)
        return q, k, v

    def logits(self, tokens, out):
        """Vocabulary rows [B, N, V] of tokens whose attention gave out [B, N, Hq, D]."""
        x = self.emb[tokens] + 0.3 * (out.flatten(2) @ self.proj.T)
        return (x @ self.head.T).contiguous()


def draft(model, root, nodes, branch, rng):
    """A trie per request: children are the likeliest tokens of the model without attention."""
    B = len(root)
    parent = np.full((B, nodes), -1, np.int32)
    for b in range(B):
        at, i = 0, 1
        while i < nodes:
            for _ in range(int(rng.integers(1, branch + 1))):
                if i < nodes:
                    parent[b, i] = at
                    i += 1
            at += 1
    token = torch.zeros((B, nodes), dtype=torch.int64, device=root.device)
    token[:, 0] = root
    each = torch.arange(B, device=root.device)
    rank = np.zeros((B, nodes), np.int64)
    for i in range(1, nodes):
        rank[:, i] = (parent[:, :i] == parent[:, i:i + 1]).sum(1)
        up = token[each, torch.from_numpy(parent[:, i].astype(np.int64)).to(root.device)]
        top = (model.emb[up] @ model.head.T).topk(branch, -1).indices
        token[:, i] = top[each, torch.from_numpy(rank[:, i]).to(root.device)]
    return torch.from_numpy(parent).to(root.device), token


def decode(steps=8, batch=4, nodes=24, vocab=2048, Hq=8, Hkv=2, D=64, block_size=16, seed=0,
           device="cuda:0"):
    """-> dict(model, cache, table, length [B] cached positions, tokens: per request the tokens
    of those positions and the one to come, accepted: nodes accepted in each step)."""
    rng = np.random.default_rng(seed)
    model = Model(vocab, Hq, Hkv, D, device, seed)
    pages = (steps * nodes + block_size - 1) // block_size + 1
    table = torch.from_numpy(rng.permutation(batch * pages).reshape(batch, pages).astype(
        np.int32)).to(device)
    cache = G.Fp4Cache.empty(batch * pages, block_size, Hkv, D, device, G.SPEC_KV_HND)
    root = torch.from_numpy(rng.integers(0, vocab, batch)).to(device)
    length = torch.zeros(batch, dtype=torch.int32, device=device)
    tokens = [[int(t)] for t in root.tolist()]
    accepted = []
    with G.Handle(batch, nodes, vocab, torch.device(device).index or 0) as h:
        size = G.spec_tree_attention_workspace(h, batch, nodes, Hq, Hkv, D)
        workspace = torch.empty(size, dtype=torch.uint8, device=device)
        attended, kept = (torch.empty(batch, dtype=torch.int32, device=device) for _ in range(2))
        for _ in range(steps):
            parent, token = draft(model, root, nodes, 3, rng)
            tree = G.build_tree_mask(h, parent)
            q, k, v = model.project(h, token, length, tree["depth"])
            out, _ = G.tree_attention_fp4(h, q, k, v, cache, table, length, tree["anc_mask"],
                                          D ** -0.5, workspace, status=attended)
            res = G.verify_greedy(h, model.logits(token, out), token.int(), parent)
            G.spec_kv_commit_fp4(h, k, v, cache, table, length, res["kv_commit"],
                                 res["accept_len"], kept)
            met = torch.stack((tree["status"], attended, res["status"], kept))
            if met.any():
                raise RuntimeError(f"mask, attention, verification, commit: {met.tolist()}")
            length = length + res["accept_len"] + 1
            root = res["bonus"].long()
            n = res["accept_len"].tolist()
            for b, row in enumerate(res["out_tokens"].tolist()):
                tokens[b] += row[:n[b] + 1]
            accepted.append(n)
    return dict(model=model, cache=cache, table=table, length=length, tokens=tokens,
                accepted=accepted)


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--nodes", type=int, default=24)
    a = ap.parse_args()
    r = decode(a.steps, a.batch, a.nodes)
    print("accepted nodes per step:", r["accepted"])
    print("cached positions:", r["length"].tolist())
