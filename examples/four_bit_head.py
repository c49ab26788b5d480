"""Draft and target heads kept in 4 bits, and the log probabilities of what a round emits, with the library's
calls in the order a serving loop makes them:

  fp4_quantize                 both heads, once
  draft_topk_fused_fp4         children and confidences of each expanded node, layer by layer
  tree_expand_topk, tree_build the draft tree from them
  fp4_quantize, fp4_linear     the target's logits of every node
  verify_tree                  the accept walk
  token_logprobs               the emitted tokens' log probabilities, from their nodes' rows

Random weights, and features that are a random function of the token instead of a model's; what it shows is
the data flow.  Run on a GPU:
  python examples/four_bit_head.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from speculative_decoding_tree_spec_gb300 import binding  # noqa: E402

BF, I32 = torch.bfloat16, torch.int32


class FourBitRounds:
    """B sequences, each with its last token in `root`."""

    def __init__(self, B=4, vocab=1000, dim=256, fmt="nv", layers=3, expand=3, children=4, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.B, self.vocab, self.fmt, self.device = B, vocab, fmt, device
        self.layers, self.expand, self.children = layers, expand, children
        # tensor scales that move the block scales of unit features and of these weights into e4m3's range
        self.scale = 2.0 ** -4 if fmt == "nv" else 1.0
        weight_scale = 2.0 ** -10 if fmt == "nv" else 1.0
        self.embed = torch.randn((vocab, dim), generator=g, device=device).to(BF)
        target = torch.randn((vocab, dim), generator=g, device=device) * 0.1
        draft = target + torch.randn((vocab, dim), generator=g, device=device) * 0.02
        self.target, self.draft = (binding.fp4_quantize(w.to(BF), fmt, weight_scale) for w in (target, draft))
        self.root = torch.zeros(B, dtype=I32, device=device)
        self.round = 0

    def features(self, tokens):
        return self.embed[tokens.long().reshape(-1)]

    def drafts(self):
        """Candidates of every sequence in creation order: parent [B, n], token [B, n], confidence [B, n]."""
        B, k = self.B, self.children
        d = binding.draft_topk_fused_fp4(self.features(self.root), self.draft, k, 1.0, self.scale)
        parent, token, prob = [torch.full((B, k), -1, dtype=I32, device=self.device)], [d["tokens"]], [d["probs"]]
        begin = 0
        for _ in range(self.layers - 1):
            p, t, c = (torch.cat(x, 1).contiguous() for x in (parent, token, prob))
            chosen = binding.tree_expand_topk(p, c, begin, p.shape[1], min(self.expand, p.shape[1] - begin))
            begin = p.shape[1]
            d = binding.draft_topk_fused_fp4(self.features(t.gather(1, chosen.long())), self.draft, k, 1.0, self.scale)
            parent.append(chosen.repeat_interleave(k, 1))
            token.append(d["tokens"].view(B, -1))
            prob.append(d["probs"].view(B, -1))
        return [torch.cat(x, 1).contiguous() for x in (parent, token, prob)]

    def logits(self, features, head):
        return binding.fp4_linear(binding.fp4_quantize(features, self.fmt, self.scale), head)

    def step(self, m=12, temperature=0.8, seed=1):
        """One round: accepted lengths, tokens [B, depth + 1] and their log probabilities (-inf behind the last)."""
        self.round += 1
        tree = binding.tree_build(*self.drafts(), self.root, m)
        x = self.features(tree["tokens"])
        shape = (self.B, m + 1, self.vocab)
        p, q = self.logits(x, self.target), self.logits(x, self.draft)
        res = binding.verify_tree(p.view(shape), q.view(shape), tree["tokens"], tree["parent_idx"], self.layers,
                                  temperature, seed=seed, offset=self.round)
        first = torch.arange(self.B, dtype=I32, device=self.device)[:, None] * (m + 1)
        rows = torch.where(res["path"] >= 0, first + res["path"], -1)
        lp = binding.token_logprobs(p, res["tokens"].view(-1), 3, temperature, rows=rows.view(-1))
        self.root = res["tokens"].gather(1, res["accept_len"].long()[:, None])[:, 0].contiguous()
        return res["accept_len"], res["tokens"], lp["logprobs"].view(res["tokens"].shape)


def main():
    r = FourBitRounds()
    for i in range(5):
        accepted, tokens, logprobs = r.step()
        print(f"round {i}: accepted {accepted.tolist()}, log probabilities of the first tokens "
              f"{[round(x, 3) for x in logprobs[:, 0].tolist()]}")


if __name__ == "__main__":
    main()
