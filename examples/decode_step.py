"""One layer's decoding steps with drafted tokens, run with libred.

    python examples/decode_step.py [--steps 8]

A toy target (one attention layer with random weights and a vocabulary of a few
thousand tokens) decodes a batch of sequences. Every step drafts a few tokens,
then runs the calls of such a step one after the other:

    red_qk_norm_rope    norms and rotates the heads of the fused projection
    red_cache_write     writes keys and values into an int8 paged cache
    red_tree_attention  attends from the last token and the drafts over it
    red_verify_drafts   accepts a prefix of the drafts and samples one token more

The products around them are torch's. The draft is the target's own
probabilities of the last step, flattened, so that some drafts are accepted.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import reduction_libred_amd as rl  # noqa: E402

HEADS, KV_HEADS, DIM, HIDDEN, VOCAB = 16, 4, 128, 512, 4096
PLACES, DRAFTS = 16, 4


class Toy:
    """Weights, and the paged cache of `batch` sequences of up to max_len tokens."""

    def __init__(self, batch, max_len, device, seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape, gain=1.0):
            return (gain * torch.randn(*shape, device=device, generator=g) / shape[0] ** 0.5).to(torch.bfloat16)

        self.embed = torch.randn(VOCAB, HIDDEN, device=device, generator=g).to(torch.bfloat16)
        self.qkv = weight(HIDDEN, (HEADS + 2 * KV_HEADS) * DIM)
        self.out = weight(HEADS * DIM, HIDDEN)
        self.head = weight(HIDDEN, VOCAB, gain=2.0)
        self.q_weight = torch.ones(DIM, device=device, dtype=torch.bfloat16)
        self.k_weight = torch.ones(DIM, device=device, dtype=torch.bfloat16)
        i = torch.arange(DIM // 2, device=device, dtype=torch.float64)
        self.freq = (10000.0 ** (-2.0 * i / DIM)).float()
        self.max_len = max_len
        per = -(-max_len // PLACES)
        self.table = torch.randperm(batch * per, device=device, generator=g).to(torch.int32).view(batch, per)
        pages = (batch * per, KV_HEADS, PLACES, DIM)
        self.k_pages, self.v_pages = (torch.zeros(pages, device=device, dtype=torch.int8) for _ in range(2))
        self.k_scales, self.v_scales = (torch.zeros(pages[:3], device=device) for _ in range(2))
        self.lens = torch.zeros(batch, device=device, dtype=torch.int32)   # tokens in the cache

    def forward(self, tokens):
        """Probabilities after each of `tokens` (batch, nodes), a chain that
        continues the sequences; their keys and values go into the cache."""
        batch, nodes = tokens.shape
        x = self.embed[tokens]
        qkv = (x @ self.qkv).view(batch * nodes, HEADS + 2 * KV_HEADS, DIM)
        q, k, v = torch.split(qkv, [HEADS, KV_HEADS, KV_HEADS], dim=1)
        pos = (self.lens.long()[:, None] + torch.arange(nodes, device=tokens.device)).view(-1)
        q, k = rl.red_qk_norm_rope(q, k, pos, self.freq, self.q_weight, self.k_weight)
        row = torch.arange(batch, device=tokens.device).repeat_interleave(nodes)
        slots = self.table[row, pos // PLACES].long() * PLACES + pos % PLACES
        rl.red_cache_write(k, v, slots, self.k_pages, self.v_pages, self.k_scales, self.v_scales)
        out, _ = rl.red_tree_attention(q.view(batch, nodes, HEADS, DIM), self.k_pages, self.v_pages, self.table, self.lens,
                                       DIM ** -0.5, max_len=self.max_len, k_scales=self.k_scales, v_scales=self.v_scales)
        x = x + out.view(batch, nodes, HEADS * DIM) @ self.out
        return torch.softmax((x @ self.head).float(), -1)


def decode(model, prompt, steps, seed=1):
    """-> the sequences' tokens (lists), and how many drafts were accepted."""
    device, batch = prompt.device, prompt.shape[0]
    g = torch.Generator(device=device).manual_seed(seed)
    model.forward(prompt[:, :-1])
    model.lens += prompt.shape[1] - 1
    last, draft = prompt[:, -1:], None
    tokens, accepted = [[] for _ in range(batch)], 0
    for _ in range(steps):
        if draft is None:
            draft = torch.full((batch, DRAFTS, VOCAB), 1.0 / VOCAB, device=device)
        drafted = torch.multinomial(draft.view(-1, VOCAB), 1, generator=g).view(batch, DRAFTS)
        p = model.forward(torch.cat((last, drafted), 1))
        u, r = torch.rand(batch, DRAFTS, device=device, generator=g), torch.rand(batch, device=device, generator=g)
        n, got = rl.red_verify_drafts(p, draft, drafted, u, r)
        # The accepted tokens (and the one before them) stay in the cache; the
        # sampled one is fed in the next step.
        model.lens += n + 1
        last = got.gather(1, n.long()[:, None])
        draft = p[:, -1:].expand(-1, DRAFTS, -1).contiguous()
        accepted += int(n.sum())
        for b, row in enumerate(got.tolist()):
            tokens[b] += [t for t in row if t >= 0]
    return tokens, accepted


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--batch", type=int, default=3)
    args = ap.parse_args()
    device = torch.device("cuda:0")
    model = Toy(args.batch, 64 + (DRAFTS + 1) * args.steps, device)
    prompt = torch.randint(0, VOCAB, (args.batch, 32), generator=torch.Generator().manual_seed(2)).to(device)
    tokens, accepted = decode(model, prompt, args.steps)
    for b, row in enumerate(tokens):
        print(f"sequence {b}: {row}")
    print(f"{accepted} of {args.batch * args.steps * DRAFTS} drafts accepted")


if __name__ == "__main__":
    main()
