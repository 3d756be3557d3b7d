"""A server's steps over a paged cache that grows and gives back, run with libred.

    python examples/serve_step.py [--requests 9]

A toy model (one attention layer with random weights) answers a queue of
requests, a few at a time. Every step takes one more token of each sequence that
is being answered and up to a chunk of the prompt of each that has just begun:

    red_plan_slots        pages and slots for the step's tokens; those of ended sequences come back
    red_qk_norm_rope      norms and rotates the heads
    red_cache_write       writes keys and values into a paged cache
    red_page_bounds       least and largest keys of the pages that were written
    red_select_pages      the pages worth reading, for each kv head
    red_sparse_attention  attends over those
    red_sample            the next tokens, from temperature, top-k, top-p and min-p

The products around them are torch's. A request waits until the cache has pages
for all of it.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import reduction_libred_amd as rl  # noqa: E402

HEADS, KV_HEADS, DIM, HIDDEN, VOCAB = 16, 4, 128, 512, 4100
PLACES, CHUNK = 16, 32


class Toy:
    """Weights, and a paged cache of `pages` pages for `batch` sequences of up to max_len tokens."""

    def __init__(self, batch, max_len, pages, budget, device, seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape, gain=1.0):
            return (gain * torch.randn(*shape, device=device, generator=g) / shape[0] ** 0.5).to(torch.bfloat16)

        self.embed = torch.randn(VOCAB, HIDDEN, device=device, generator=g).to(torch.bfloat16)
        self.qkv = weight(HIDDEN, (HEADS + 2 * KV_HEADS) * DIM)
        self.out = weight(HEADS * DIM, HIDDEN)
        self.head = weight(HIDDEN, VOCAB, gain=2.0)
        i = torch.arange(DIM // 2, device=device, dtype=torch.float64)
        self.freq = (10000.0 ** (-2.0 * i / DIM)).float()
        self.batch, self.budget, self.most = batch, budget, -(-CHUNK // PLACES) + 1
        cols = -(-max_len // PLACES)
        int32 = dict(device=device, dtype=torch.int32)
        self.table, self.held = torch.full((batch, cols), -1, **int32), torch.zeros(batch, **int32)
        self.free_pages, self.free_count = torch.randperm(pages, device=device, generator=g).to(torch.int32), torch.full((1,), pages, **int32)
        self.k_pages, self.v_pages = (torch.zeros(pages, KV_HEADS, PLACES, DIM, device=device, dtype=torch.bfloat16) for _ in range(2))
        self.lo, self.hi = (torch.zeros(pages, KV_HEADS, DIM, device=device, dtype=torch.bfloat16) for _ in range(2))
        self.lens = torch.zeros(batch, **int32)   # tokens in the cache

    def step(self, tokens, counts, done, r, **settings):
        """One step: counts[b] <= CHUNK more tokens of every sequence, one
        sequence's after the other's in `tokens` (batch * CHUNK of them, the rest
        anything). -> (the next token of every sequence, granted)"""
        self.lens *= 1 - done
        lens = self.lens.clone()
        slots, pos, starts, granted = rl.red_plan_slots(lens, counts, self.table, self.held, self.free_pages, self.free_count, PLACES,
                                                        tokens.shape[0], done=done)
        x = self.embed[tokens]
        qkv = (x @ self.qkv).view(-1, HEADS + 2 * KV_HEADS, DIM)
        q, k, v = torch.split(qkv, [HEADS, KV_HEADS, KV_HEADS], dim=1)
        q, k = rl.red_qk_norm_rope(q, k, pos, self.freq)
        rl.red_cache_write(k, v, slots, self.k_pages, self.v_pages)
        self.lens += granted
        rl.red_page_bounds(self.k_pages, self.table, self.lens, self.lo, self.hi, first=lens, most=self.most)
        # Queries of a sequence side by side, those behind its tokens are not looked at.
        rows = (starts[:-1, None].long() + torch.arange(CHUNK, device=tokens.device)).clamp(max=tokens.shape[0] - 1)
        q = q[rows]
        table, left = rl.red_select_pages(q, self.lo, self.hi, self.table, lens, PLACES, self.budget, node_count=granted)
        out, _ = rl.red_sparse_attention(q, self.k_pages, self.v_pages, table, left, DIM ** -0.5, node_count=granted)
        last = (granted.long() - 1).clamp(min=0)
        each = torch.arange(self.batch, device=tokens.device)
        x = x[rows[each, last]] + out[each, last].view(self.batch, HEADS * DIM) @ self.out
        return rl.red_sample(x @ self.head, r, **settings)[0], granted


def serve(model, requests, answer, seed=1):
    """requests: prompts (lists of tokens). -> the answers, `answer` tokens each (one at least), and the steps taken."""
    device, batch = model.table.device, model.batch
    g = torch.Generator(device=device).manual_seed(seed)
    settings = dict(temperature=torch.linspace(0.0, 1.2, batch, device=device), top_k=torch.full((batch,), 50, device=device, dtype=torch.int32),
                    top_p=torch.full((batch,), 0.95, device=device), min_p=torch.full((batch,), 0.01, device=device))
    assert all(len(p) > 0 for p in requests) and answer > 0
    queue, answers, steps = list(range(len(requests))), [[] for _ in requests], 0
    need = [-(-(len(p) + answer) // PLACES) for p in requests]
    assert max(need) <= model.free_pages.shape[0], "no request may need more pages than there are"
    assert max(need) <= model.table.shape[1], "no request may need more pages than a row of the table has"
    who, todo, ended = [None] * batch, [[] for _ in range(batch)], [0] * batch
    while queue or any(w is not None for w in who):
        for b in range(batch):
            if who[b] is None and queue and need[queue[0]] + sum(need[w] for w in who if w is not None) <= model.free_pages.shape[0]:
                who[b] = queue.pop(0)
                todo[b] = list(requests[who[b]])
        now = [t[:CHUNK] for t in todo]
        flat = [t for part in now for t in part]
        tokens = torch.tensor(flat + [0] * (batch * CHUNK - len(flat)), device=device)
        counts, done = (torch.tensor(x, device=device, dtype=torch.int32) for x in ([len(part) for part in now], ended))
        got, granted = model.step(tokens, counts, done, torch.rand(batch, device=device, generator=g), **settings)
        ended = [0] * batch
        for b, (token, n) in enumerate(zip(got.tolist(), granted.tolist())):
            todo[b] = todo[b][n:]
            if n == 0 or todo[b]:
                continue                # has none, or more of its prompt
            answers[who[b]].append(token)
            todo[b] = [token]
            if len(answers[who[b]]) == answer:
                who[b], todo[b], ended[b] = None, [], 1
        steps += 1
    return answers, steps


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--requests", type=int, default=9)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--answer", type=int, default=12)
    args = ap.parse_args()
    g = torch.Generator().manual_seed(2)
    requests = [torch.randint(0, VOCAB, (int(torch.randint(1, 300, (1,), generator=g)),), generator=g).tolist() for _ in range(args.requests)]
    longest = max(len(p) for p in requests) + args.answer
    model = Toy(args.batch, longest, max(args.batch * 16, -(-longest // PLACES)), 8, torch.device("cuda:0"))
    answers, steps = serve(model, requests, args.answer)
    for i, (prompt, answer) in enumerate(zip(requests, answers)):
        print(f"request {i}, {len(prompt)} tokens: {answer}")
    print(f"{steps} steps")


if __name__ == "__main__":
    main()
