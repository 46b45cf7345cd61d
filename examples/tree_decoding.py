"""Greedy speculative decoding with token trees on the 8-bit key/value cache.

A toy target model of one attention layer (embedding, queries, keys and values,
attention over the cache, output layer) and a toy draft that leaves the
attention out.  Each round

  1. the draft proposes a tree below the last emitted token: two candidates for
     each of the next two positions (7 nodes, depth 2);
  2. kv_write puts the keys and values of all nodes behind the context;
  3. kv_attention runs the target's attention over context and tree, each node
     seeing its ancestors (tree_mask);
  4. verify_tree walks the tree and emits the accepted tokens and one more;
  5. kv_commit moves the accepted path's keys and values up behind the context.

Run:  python examples/tree_decoding.py [rounds]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_63_gb300 as sv  # noqa: E402

VOCAB, WIDTH, HEADS, KV_HEADS, DIM, PAGE = 1024, 256, 8, 2, 64, 16
PARENT = [-1, 0, 1, 1, 0, 4, 4]  # depth-first: two children below the root, two below each
DEPTH = 2


class Target:
    def __init__(self, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(rows, cols):
            w = torch.randn(rows, cols, generator=g, device="cuda") / rows ** 0.5
            return w.to(torch.bfloat16)

        self.embedding = torch.randn(VOCAB, WIDTH, generator=g, device="cuda").to(torch.bfloat16)
        self.wq, self.wo = weight(WIDTH, HEADS * DIM), weight(HEADS * DIM, WIDTH)
        self.wk, self.wv = weight(WIDTH, KV_HEADS * DIM), weight(WIDTH, KV_HEADS * DIM)
        self.out = weight(WIDTH, VOCAB) * 3

    def qkv(self, tokens):
        x = self.embedding[tokens]
        return (x, (x @ self.wq).unflatten(-1, (HEADS, DIM)),
                (x @ self.wk).unflatten(-1, (KV_HEADS, DIM)),
                (x @ self.wv).unflatten(-1, (KV_HEADS, DIM)))

    def logits(self, x, attention):
        return (x + attention.flatten(-2) @ self.wo) @ self.out


def draft_tree(model, root):
    """Node tokens [B][7] and the draft's logits at every node."""
    first = (model.embedding[root] @ model.out).topk(2).indices  # [B][2]
    below = (model.embedding[first] @ model.out).topk(2).indices  # [B][2][2]
    tokens = torch.cat([root[:, None], first[:, :1], below[:, 0], first[:, 1:], below[:, 1]], 1)
    return tokens.long(), model.embedding[tokens] @ model.out


def decode(prompts, rounds, model=None, check=None):
    """Emitted tokens of each prompt (lists of token ids).  check, if given, is
    called with every round's queries, cache and attention output."""
    model = model or Target()
    B, N = len(prompts), len(PARENT)
    dev = torch.device("cuda")
    slots = (max(map(len, prompts)) + rounds * (DEPTH + 1) + N + PAGE - 1) // PAGE
    cache = sv.kv_cache(B * slots, PAGE, KV_HEADS, DIM)
    table = torch.randperm(B * slots, device=dev).to(torch.int32).view(B, slots)
    parent = torch.tensor([PARENT] * B, dtype=torch.int32, device=dev)
    q_row = parent.clamp(min=0)
    mask = sv.tree_mask(parent)["mask"]
    greedy = torch.zeros(B, device=dev)

    # the prompts, all but their last tokens, which are the first roots
    longest = max(map(len, prompts)) - 1
    context = torch.zeros(B, longest, dtype=torch.long, device=dev)
    for b, p in enumerate(prompts):
        context[b, :len(p) - 1] = torch.tensor(p[:-1], device=dev)
    length = torch.tensor([len(p) - 1 for p in prompts], dtype=torch.int32, device=dev)
    if longest:
        _, _, k, v = model.qkv(context)
        sv.kv_write(cache, table, torch.zeros_like(length), k, v, num_new=length)
    root = torch.tensor([p[-1] for p in prompts], device=dev)

    emitted = [[] for _ in prompts]
    for _ in range(rounds):
        tokens, draft = draft_tree(model, root)
        x, q, k, v = model.qkv(tokens)
        sv.kv_write(cache, table, length, k, v)
        attention = sv.kv_attention(q, cache, table, length, mask=mask)["out"]
        if check:
            check(q, cache, table, length, mask, attention)
        zero = torch.zeros(B, N, device=dev)
        got = sv.verify_tree(model.logits(x, attention), draft, tokens.to(torch.int32), parent,
                             q_row, greedy, zero, zero[:, 0].contiguous(), max_depth=DEPTH)
        sv.kv_commit(cache, table, length, got["accept_len"], got["accepted_nodes"])
        length = length + 1 + got["accept_len"]
        for b, (row, n) in enumerate(zip(got["out_tokens"].tolist(), got["out_len"].tolist())):
            emitted[b] += row[:n]
        root = torch.tensor([e[-1] for e in emitted], device=dev)
    return emitted


def main(rounds=8):
    prompts = [[5, 17, 301, 44, 9], [700], list(range(100, 140))]
    for prompt, tokens in zip(prompts, decode(prompts, rounds)):
        print(f"{len(prompt):3d} prompt tokens, {len(tokens)} emitted in {rounds} rounds: {tokens}")


if __name__ == "__main__":
    main(*map(int, sys.argv[1:2]))
