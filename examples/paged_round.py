"""Decoding rounds of a one-layer model on a paged cache, with the library's calls in the order
a serving loop makes them:

  tree_build                   the draft tree: tokens, depths, ancestor mask
  paged_append_rope            the tree's keys and values into the cache, rotated by depth
  tree_attention_paged         every node's attention over the cache and its ancestors
  verify_tree_fused_lmhead     target logits of every node and the accept walk
  commit_accepted_path_paged   the accepted path's cache rows to consecutive positions

Random weights and random draft candidates; what it shows is the data flow.  Run on a GPU:
  python examples/paged_round.py
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from speculative_decoding_tree_spec_gb300 import binding  # noqa: E402
from speculative_decoding_tree_spec_gb300 import workloads as wl  # noqa: E402

BF = torch.bfloat16


class PagedRounds:
    """B sequences; `length[b]` cached positions each, the last accepted token in `root`."""

    def __init__(self, B=4, vocab=1000, q_heads=8, kv_heads=2, head_dim=64, page_size=16,
                 max_pages=16, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        dim = q_heads * head_dim

        def weight(*shape):
            return (torch.randn(shape, generator=g, device=device) * shape[-1] ** -0.5).to(BF)

        self.B, self.vocab, self.heads, self.page_size = B, vocab, (q_heads, kv_heads, head_dim), page_size
        self.device = device
        self.embed = torch.randn((vocab, dim), generator=g, device=device).to(BF)
        self.w_qkv = weight(dim + 2 * kv_heads * head_dim, dim)
        self.w_head = weight(vocab, dim)
        # keys and values as the two planes of one cache; the pages of a sequence in any order
        self.cache = torch.zeros((2, B * max_pages, page_size, kv_heads, head_dim), dtype=BF,
                                 device=device)
        order = torch.randperm(B * max_pages, generator=g, device=device)
        self.table = order.view(B, max_pages).to(torch.int32).contiguous()
        r = torch.arange(max_pages * page_size, device=device, dtype=torch.float64)[:, None]
        f = 10000.0 ** (-torch.arange(head_dim // 2, device=device, dtype=torch.float64) * 2 / head_dim)
        self.cos_sin = torch.cat([(r * f).cos(), (r * f).sin()], dim=1).float()
        self.length = torch.zeros(B, dtype=torch.int32, device=device)
        self.root = torch.zeros(B, dtype=torch.int32, device=device)
        self.round = 0

    def _qkv(self, tokens):
        """Queries, keys and values [B, N, heads, head_dim]: views of one projection."""
        hq, hkv, d = self.heads
        x = self.embed[tokens.long()] @ self.w_qkv.t()
        return x.view(*tokens.shape, hq + 2 * hkv, d).split([hq, hkv, hkv], dim=2)

    def attend(self, tokens, position_ids=None, mask=None, counts=None):
        """Appends tokens [B, N] behind each sequence and returns their attention's output."""
        q, k, v = self._qkv(tokens)
        q = binding.paged_append_rope(q, k, v, self.cache[0], self.cache[1], self.table, self.length,
                                      self.cos_sin, position_ids=position_ids, counts=counts)
        return binding.tree_attention_paged(q, self.cache[0], self.cache[1], self.table, self.length,
                                            mask=mask, counts=counts)["out"]

    def prefill(self, prompt, counts):
        """prompt [B, N] int32, of which counts[b] tokens are real; the last one of each becomes
        the first round's root and is cached with its tree."""
        self.attend(prompt, counts=counts - 1)
        self.length += counts - 1
        self.root = prompt.gather(1, (counts.long() - 1)[:, None])[:, 0].contiguous()

    def step(self, m=15, temperature=0.8, seed=1):
        """One round; returns (accepted lengths, tokens [B, depth + 1])."""
        self.round += 1
        d = wl.make_draft_candidates(self.B, layers=4, expand_k=4, children=5, vocab=self.vocab,
                                     seed=1000 * seed + self.round)
        dev = [torch.from_numpy(np.ascontiguousarray(x)).to(self.device)
               for x in (d.parent, d.token, d.prob)]
        tree = binding.tree_build(*dev, self.root, m)
        out = self.attend(tree["tokens"], tree["position_ids"], tree["mask"])
        features = out.reshape(self.B * (m + 1), -1)
        # the draft distribution the children came from: flat here
        pitch = (self.vocab + 7) // 8 * 8
        q_logits = torch.zeros((self.B, m + 1, pitch), dtype=BF, device=self.device)[..., :self.vocab]
        res = binding.verify_tree_fused_lmhead(features, self.w_head, q_logits, tree["tokens"],
                                               tree["parent_idx"], 4, temperature, seed=seed,
                                               offset=self.round)
        binding.commit_accepted_path_paged(self.cache, self.table, self.length, res["path"],
                                           res["accept_len"])
        self.length += res["accept_len"] + 1  # the root and the accepted nodes
        self.root = res["tokens"].gather(1, res["accept_len"].long()[:, None])[:, 0].contiguous()
        return res["accept_len"], res["tokens"]


def main():
    r = PagedRounds()
    prompt = torch.randint(0, r.vocab, (r.B, 40), dtype=torch.int32, device=r.device)
    r.prefill(prompt, torch.tensor([40, 1, 17, 33], dtype=torch.int32, device=r.device))
    for i in range(5):
        accepted, tokens = r.step()
        print(f"round {i}: accepted {accepted.tolist()}, cached {r.length.tolist()}")


if __name__ == "__main__":
    main()
