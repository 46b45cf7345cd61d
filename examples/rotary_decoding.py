"""Greedy speculative decoding with token trees for a model whose queries and keys
have head norms and rotary positions, with the log probabilities of what it
emits.

The model and the draft are tree_decoding's, with a norm for each head of the
queries and keys and positions for long contexts.  Each round

  1. the draft proposes a tree below the last emitted token (7 nodes, depth 2);
  2. kv_append norms and turns the nodes' queries and keys by their depths
     (tree_mask's, behind the context) and puts keys and values into the cache;
  3. kv_attention, verify_tree and kv_commit as there: an accepted node's depth is
     its place on the path, so its key stays as it was turned;
  4. token_logprobs reports the emitted tokens' log probabilities, the entropy at
     each of them and the likeliest alternatives.

Run:  python examples/rotary_decoding.py [rounds]
"""
import os
import sys

import torch
from torch.nn.functional import pad

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import speculative_decoding_verification_63_gb300 as sv  # noqa: E402
from tree_decoding import (DEPTH, DIM, HEADS, KV_HEADS, PAGE, PARENT, Target,  # noqa: E402
                           draft_tree)

EPS = 1e-6


class RotaryTarget(Target):
    def __init__(self, seed=0):
        super().__init__(seed)
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        self.q_norm, self.k_norm = (torch.exp(0.2 * torch.randn(DIM, generator=g, device="cuda"))
                                    .to(torch.bfloat16) for _ in "qk")
        self.rope = sv.rope(DIM, 5e5, scaling=dict(type="yarn", factor=4, context=8192))

    def append(self, cache, table, length, tokens, num=None, offset=None):
        """The layer's input and the tokens' queries, ready for the attention; their
        keys and values go into the cache."""
        x, q, k, v = self.qkv(tokens)
        q = sv.kv_append(cache, table, length, q, k, v, num_new=num, offset=offset, rope=self.rope,
                         q_weight=self.q_norm, k_weight=self.k_norm, eps=EPS)["q"]
        return x, q


def decode(prompts, rounds, model=None, top=3, check=None):
    """For each prompt the emitted tokens as (token, log probability, entropy, likeliest
    tokens).  check, if given, is called with every round's tensors."""
    model = model or RotaryTarget()
    B, N = len(prompts), len(PARENT)
    dev = torch.device("cuda")
    slots = (max(map(len, prompts)) + rounds * (DEPTH + 1) + N + PAGE - 1) // PAGE
    cache = sv.kv_cache(B * slots, PAGE, KV_HEADS, DIM)
    table = torch.randperm(B * slots, device=dev).to(torch.int32).view(B, slots)
    parent = torch.tensor([PARENT] * B, dtype=torch.int32, device=dev)
    q_row = parent.clamp(min=0)
    tree = sv.tree_mask(parent)
    greedy = torch.zeros(B, device=dev)

    longest = max(map(len, prompts)) - 1
    context = torch.zeros(B, longest, dtype=torch.long, device=dev)
    for b, p in enumerate(prompts):
        context[b, :len(p) - 1] = torch.tensor(p[:-1], device=dev)
    length = torch.tensor([len(p) - 1 for p in prompts], dtype=torch.int32, device=dev)
    if longest:
        model.append(cache, table, torch.zeros_like(length), context, num=length)
    root = torch.tensor([p[-1] for p in prompts], device=dev)

    emitted = [[] for _ in prompts]
    for _ in range(rounds):
        tokens, draft = draft_tree(model, root)
        x, q = model.append(cache, table, length, tokens, offset=tree["depth"])
        attention = sv.kv_attention(q, cache, table, length, mask=tree["mask"])["out"]
        logits = model.logits(x, attention)
        zero = torch.zeros(B, N, device=dev)
        got = sv.verify_tree(logits, draft, tokens.to(torch.int32), parent, q_row, greedy, zero,
                             zero[:, 0].contiguous(), max_depth=DEPTH)
        sv.kv_commit(cache, table, length, got["accept_len"], got["accepted_nodes"])
        # the rows that emitted: the root's, then the accepted nodes'
        said = sv.token_logprobs(logits, got["out_tokens"], num_rows=got["out_len"],
                                 rows=pad(got["accepted_nodes"], (1, 0)), top=top)
        if check:
            check(cache=cache, table=table, length=length, tokens=tokens, q=q, logits=logits,
                  got=got, said=said)
        length = length + 1 + got["accept_len"]
        for b, n in enumerate(got["out_len"].tolist()):
            emitted[b] += zip(got["out_tokens"][b, :n].tolist(), said["logprobs"][b, :n].tolist(),
                              said["entropy"][b, :n].tolist(), said["top_tokens"][b, :n].tolist())
        root = torch.tensor([e[-1][0] for e in emitted], device=dev)
    return emitted


def main(rounds=8):
    prompts = [[5, 17, 301, 44, 9], [700], list(range(100, 140))]
    for prompt, tokens in zip(prompts, decode(prompts, rounds)):
        print(f"{len(prompt)} prompt tokens, {len(tokens)} emitted in {rounds} rounds:")
        for token, lp, entropy, best in tokens:
            print(f"  {token:5d}  log p {lp:7.3f}  entropy {entropy:6.3f}  likeliest {best}")


if __name__ == "__main__":
    main(*map(int, sys.argv[1:2]))
