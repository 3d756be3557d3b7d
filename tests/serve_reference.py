"""The serving step's operators on the CPU, straight from their definitions: one
sequence after the other, on lists, in float64 or wider."""
import math

import numpy as np
import torch

F64 = torch.float64


def plan_slots(lens, counts, done, table, held, stack, height, places, tokens, pages=None):
    """Everything as lists; -> dict of what a call leaves and returns."""
    batch, cols, pages = len(lens), len(table[0]) if table else 0, len(stack)
    table, stack = [list(r) for r in table], list(stack)
    held = [min(max(h, 0), cols) for h in held]
    top = min(max(height, 0), pages)
    for b in range(batch):
        if done is not None and done[b]:
            for j in range(held[b]):
                if top < pages:
                    stack[top] = table[b][j]
                    top += 1
            held[b] = 0
    starts, granted, wants, asked, full = [0], [], [], 0, False
    for b in range(batch):
        n, length = max(counts[b], 0), max(lens[b], 0)
        starts.append(starts[-1] + n)
        need = -(-(length + n) // places)
        fits = n > 0 and need <= cols and starts[-1] <= tokens
        want = max(0, need - held[b]) if fits else 0
        if want:
            full = full or asked + want > top
            if not full:
                asked += want
        good = fits and (want == 0 or not full)
        granted.append(n if good else 0)
        wants.append(want if good else 0)
    at = top - asked
    for b in range(batch):
        for j in range(wants[b]):
            table[b][held[b] + j] = stack[at]
            stack[at] = -1
            at += 1
        held[b] += wants[b]
    slots, pos = [-1] * tokens, [0] * tokens
    for b in range(batch):
        for i in range(max(counts[b], 0)):
            t = starts[b] + i
            if t < tokens:
                p = max(lens[b], 0) + i
                pos[t] = p
                if granted[b]:
                    slots[t] = table[b][p // places] * places + p % places
    return dict(slots=slots, pos=pos, starts=[min(s, tokens) for s in starts], granted=granted, table=table, held=held, stack=stack,
                height=[top - asked])


def page_bounds(k, scales, table, lens, lo, hi, first, most):
    """k (pages, heads, places, dim), scales or None; -> lo, hi with the pages of the sequences written."""
    lo, hi = lo.clone(), hi.clone()
    pages, places = k.shape[0], k.shape[2]
    for b, length in enumerate(lens):
        begin = max(first[b], 0) if first is not None else 0
        if begin >= length:
            continue
        for j in range(begin // places, min(-(-length // places), table.shape[1], begin // places + most)):
            page = int(table[b, j])
            if not 0 <= page < pages:
                continue
            x = k[page, :, :min(places, length - j * places)].float()
            if scales is not None:
                x = x * scales[page, :, :x.shape[1], None]       # one product in float32
            none = x.isnan()
            lo[page] = torch.where(none, math.inf, x).amin(1).to(lo.dtype)
            hi[page] = torch.where(none, -math.inf, x).amax(1).to(hi.dtype)
    return lo, hi


def select_pages(q, lo, hi, table, length, count, places, budget, first, last, max_len):
    """One sequence: q (nodes, q heads, dim), table (columns) -> per kv head the
    logical pages chosen (ascending), and the length that is left."""
    pages, heads, _ = lo.shape
    total = min(max(length, 0) + count, max_len, len(table) * places)
    have = -(-total // places) if count > 0 else 0
    if count == 0:
        return [[] for _ in range(heads)], 0
    keep = min(have, budget)
    group = q.shape[1] // heads
    chosen = []
    for h in range(heads):
        rows = q[:count, h * group:(h + 1) * group].to(F64).reshape(-1, q.shape[2])
        up, down = torch.where(rows < 0, 0.0, rows).sum(0), torch.where(rows > 0, 0.0, rows).sum(0)
        keys = []
        for p in range(have):
            page = int(table[p])
            score = math.nan
            if 0 <= page < pages:
                score = float((up * hi[page, h].to(F64) + down * lo[page, h].to(F64)).sum())
            forced = p < first or p >= max(max(length, 0) // places - last, 0)
            # forced before numbers, numbers before NaN
            keys.append((0, 0.0, p) if forced else (2, 0.0, p) if score != score else (1, -score, p))
        chosen.append(sorted(p for _, _, p in sorted(keys)[:keep]))
    return chosen, max(length, 0) - places * (have - keep)


LONG = np.longdouble


def sample(x, t=None, k=None, p=None, m=None):
    """One row of logits (float64 numpy) -> (kept weights in 80 bits, how close a
    border came to its target, relative to the largest weight)."""
    x = np.where(np.isnan(x), -np.inf, x)
    vocab, top = len(x), x.max()
    if top == -np.inf:
        return np.zeros(vocab, dtype=LONG), np.inf
    if top == np.inf:
        x, top = np.where(x == np.inf, 0.0, -np.inf), 0.0
    order = np.argsort(-x, kind="stable")
    t = 1.0 if t is None else float(t)
    k = vocab if k is None or k < 1 or k > vocab else int(k)
    if not t > 0:
        k, t = 1, 1.0
    with np.errstate(invalid="ignore", over="ignore", under="ignore"):
        u = (x[order] - top).astype(LONG) / LONG(t)
    w = np.where(x[order] == -np.inf, LONG(0), np.exp(np.where(np.isnan(u), LONG(0), u)))
    w[k:] = 0
    near = np.inf
    if p is not None and float(p) < 1 and k > 1:
        run = np.cumsum(w)
        target = LONG(max(float(p), 0.0)) * run[-1]
        before = np.concatenate(([LONG(0)], run[:-1]))
        near = float(np.abs(before[1:] - target).min()) if vocab > 1 else np.inf
        w = np.where((before < target) | (np.arange(vocab) == 0), w, LONG(0))
    if m is not None and float(m) > 0:
        w = np.where(w >= LONG(min(float(m), 1.0)), w, LONG(0))
    kept = np.zeros(vocab, dtype=LONG)
    kept[order] = w
    return kept, near


def token_of(kept, r):
    """-> (token, how close its border came to the running sum)"""
    run = np.cumsum(kept)
    if run[-1] == 0:
        return -1, np.inf
    positive = np.nonzero(kept > 0)[0]
    if not float(r) < 1:
        return int(positive[-1]), np.inf
    target = LONG(max(float(r), 0.0)) * run[-1]
    after = positive[run[positive] > target]
    return int(after[0] if len(after) else positive[-1]), float(np.abs(run[positive] - target).min())
