"""Operators of a serving step around the paged cache: cases, inputs and plain forms.

Four groups:

  plan    where the next tokens of every sequence go: finished rows give their pages back, pages are taken
          from the free ones, and every token gets its slot and position
  bounds  the least and largest elements of the keys of every page and kv head, for the pages that changed
  sparse  pages chosen by the bounds for each sequence and kv head, and attention over those pages alone
  sample  temperature, top-k, top-p and min-p, and the token drawn by a given random number
          ("probs": the filtered probabilities as well)

`own` false computes them with elementary torch operations, `own` true calls the library.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
          "i8": torch.int8, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "i8": 1, "e4m3": 1}
SCALED = ("i8", "e4m3")


def listed():
    return [
        # A decoding step: the drafted tokens of every sequence, a few rows taken over by new requests.
        dict(name="plan decode", op="plan", batch=32, cols=1024, page=16, low=9, high=9, longest=16384, done=4, free=1.0),
        # Prompts of many lengths come in at once.
        dict(name="plan prompts", op="plan", batch=256, cols=160, page=64, low=1, high=1021, longest=8192, done=256, free=1.0),
        # More is asked for than there are free pages: the later sequences have to wait.
        dict(name="plan short", op="plan", batch=101, cols=700, page=24, low=0, high=517, longest=16001, done=9, free=0.6),
        # A decoding step's new keys: the last page or two of every sequence.
        dict(name="bounds decode", op="bounds", batch=32, kv_heads=8, dim=128, page=16, longest=16384, shortest=1500, new=9,
             dtype="bf16", cache="bf16"),
        # Prompts are in the cache: all their pages.
        dict(name="bounds prompts", op="bounds", batch=8, kv_heads=8, dim=128, page=64, longest=16384, shortest=7001, new=0,
             dtype="bf16", cache="i8"),
        # One long sequence, a single token.
        dict(name="sparse single", op="sparse", batch=1, nodes=1, q_heads=32, kv_heads=8, dim=128, longest=32767, shortest=32767,
             page=16, budget=128, first=1, last=2, tree=False, ragged=False, dtype="f16", cache="f16"),
        # A serving batch of sequences of many lengths, an 8-bit cache.
        dict(name="sparse batch", op="sparse", batch=32, nodes=1, q_heads=32, kv_heads=8, dim=128, longest=16384, shortest=1500,
             page=32, budget=64, first=1, last=2, tree=False, ragged=False, dtype="bf16", cache="i8"),
        # Long sequences with small trees of drafted tokens.
        dict(name="sparse trees", op="sparse", batch=8, nodes=8, q_heads=32, kv_heads=8, dim=128, longest=131072, shortest=30011,
             page=64, budget=67, first=2, last=3, tree=True, ragged=True, dtype="bf16", cache="bf16"),
        # One sequence's next token, a small vocabulary, all filters.
        dict(name="sample single", op="sample", batch=1, steps=1, vocab=32000, dtype="f32", top_k=50, top_p=True, min_p=False,
             masked=False, probs=None),
        # A serving batch, a large vocabulary of odd size, sequences with settings of their own.
        dict(name="sample batch", op="sample", batch=192, steps=1, vocab=131071, dtype="f32", top_k=None, top_p=True, min_p=False,
             masked=True, probs=None),
        # The smaller logits of a model that leaves them in 16 bits: many are equal.
        dict(name="sample ties", op="sample", batch=64, steps=1, vocab=131071, dtype="bf16", top_k=1000, top_p=False, min_p=True,
             masked=True, probs=None),
        # The target's probabilities after every drafted token, for their verification.
        dict(name="sample drafts", op="sample", batch=32, steps=7, vocab=131071, dtype="bf16", top_k=None, top_p=True, min_p=True,
             masked=False, probs="f32"),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over the logarithm."""
    return min(high, int(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))


def draw(rng):
    op = rng.choice(["plan", "bounds", "sparse", "sparse", "sample", "sample"])
    if op == "plan":
        batch, page, longest = _spread(rng, 1, 256), rng.choice([1, 8, 16, 24, 32, 64, 128]), _spread(rng, 1, 16384)
        low = rng.randint(0, 9)
        high = max(low, _spread(rng, 1, 1021))
        return dict(op=op, batch=batch, cols=-(-(longest + high) // page) + rng.randint(0, 9), page=page, low=low, high=high,
                    longest=longest, done=rng.randint(0, batch), free=rng.choice([1.0, 1.0, rng.random()]))
    if op == "bounds":
        kv_heads, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 80, 96, 128, 128, 192, 256])
        batch, longest = _spread(rng, 1, 64), _spread(rng, 1, 32768)
        while batch * longest * kv_heads * dim > 8 * 12000 * 8 * 128:
            batch, longest = max(1, batch // 2), longest // 2 + 1
        return dict(op=op, batch=batch, kv_heads=kv_heads, dim=dim, page=rng.choice([1, 8, 16, 24, 32, 64, 128]), longest=longest,
                    shortest=rng.randint(1, longest), new=rng.choice([0, 1, rng.randint(1, 300)]), dtype=rng.choice(["bf16", "f16"]),
                    cache=rng.choice(["i8", "e4m3", "own", "own"]))
    if op == "sparse":
        kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8])
        batch, nodes = _spread(rng, 1, 32), rng.choice([1, 1, 1, _spread(rng, 1, 64)])
        longest = _spread(rng, 1, 131072)
        dim, page = rng.choice([64, 80, 96, 128, 128, 192, 256]), rng.choice([8, 16, 24, 32, 64, 128])
        while batch * longest * kv_heads * dim > 8 * 80000 * 8 * 128:
            batch, longest = max(1, batch // 2), longest // 2 + 1
        first, last = rng.randint(0, 3), rng.randint(0, 4)
        budget = first + last + 1 + -(-nodes // page) + _spread(rng, 1, max(1, 4096 // page))
        return dict(op=op, batch=batch, nodes=nodes, q_heads=kv_heads * group, kv_heads=kv_heads, dim=dim, longest=longest,
                    shortest=rng.randint(0, longest), page=page, budget=budget, first=first, last=last, tree=rng.random() < 0.7,
                    ragged=rng.random() < 0.5, dtype=rng.choice(["bf16", "f16"]), cache=rng.choice(["i8", "e4m3", "own"]))
    batch, steps, vocab = _spread(rng, 1, 192), rng.choice([1, 1, 1, rng.randint(2, 8)]), _spread(rng, 1000, 131072)
    while batch * steps * vocab > 224 * 131071:
        batch = batch // 2 + 1
    return dict(op=op, batch=batch, steps=steps, vocab=vocab, dtype=rng.choice(["f32", "f32", "bf16", "f16"]),
                top_k=rng.choice([None, None, _spread(rng, 1, vocab)]), top_p=rng.random() < 0.6, min_p=rng.random() < 0.4,
                masked=rng.random() < 0.4, probs=rng.choice([None, None, "f32", "bf16", "f16"]))


def _cache_type(case):
    return case["dtype"] if case["cache"] == "own" else case["cache"]


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _rand(g, *shape):
    return torch.rand(*shape, device="cuda", generator=g)


def _lengths(h, c):
    """The sequences' tokens, from the shortest to the longest, in no order."""
    b = c["batch"]
    x = torch.linspace(c["shortest"], c["longest"], b).round().to(torch.int32) if b > 1 else torch.tensor([c["longest"]], dtype=torch.int32)
    return x[torch.randperm(b, generator=h)]


def _paged(g, c, kind, pages):
    """Pages of a cache and their scales; the tokens of a page resemble each other, and some dimensions are large."""
    shape = (pages, c["kv_heads"], c["page"], c["dim"])
    x = _randn(g, *shape)
    x += _randn(g, pages, c["kv_heads"], 1, c["dim"])
    x *= torch.exp(0.5 * _randn(g, c["kv_heads"], 1, c["dim"]))
    if kind == "i8":
        x = (x * 18.0).clamp_(-127, 127).round_().to(torch.int8)
    elif kind == "e4m3":
        x = (x * 60.0).clamp_(-448, 448).to(DTYPES[kind])
    else:
        return x.to(DTYPES[kind]), None
    return x, (0.5 + _rand(g, *shape[:3])) * (1.0 / (18.0 if kind == "i8" else 60.0))


def _trees(h, batch, nodes):
    """Ancestor bits of random trees: bit j of word i is set where node i sees node j (itself and the nodes above it)."""
    above = torch.zeros(batch, nodes, nodes, dtype=torch.bool)
    pick = torch.rand(batch, nodes, generator=h)
    for i in range(nodes):
        if i:
            above[:, i] = above[torch.arange(batch), (pick[:, i] * i).long()]
        above[:, i, i] = True
    word = torch.zeros(batch, nodes, dtype=torch.int64)
    for j in range(nodes):
        word |= above[:, :, j].to(torch.int64) << j
    return word


def _prepare_plan(c, s, h):
    b, page, cols = c["batch"], c["page"], c["cols"]
    lens = torch.randint(0, c["longest"] + 1, (b,), generator=h, dtype=torch.int32)
    s["held"] = ((lens + page - 1) // page).clamp(max=cols).to(torch.int32)
    done = torch.zeros(b, dtype=torch.int32)
    done[torch.randperm(b, generator=h)[:c["done"]]] = 1
    s["lens"] = torch.where(done > 0, 0, lens)          # a finished row's new sequence has no tokens yet
    s["done"] = done
    s["counts"] = torch.randint(c["low"], c["high"] + 1, (b,), generator=h, dtype=torch.int32)
    need = ((s["lens"] + s["counts"] + page - 1) // page - torch.where(done > 0, 0, s["held"])).clamp(min=0)
    spare = int(c["free"] * float(need.sum())) if c["free"] < 1 else int(need.sum()) + 100
    held = int(s["held"].sum())
    s["spare"] = max(0, spare - int(s["held"][done > 0].sum())) if c["free"] < 1 else spare
    pages = b * (cols + 1) + 100                                  # the cache's; other programs' sequences hold what is left
    order = torch.randperm(pages, generator=h, dtype=torch.int64).to(torch.int32)
    table = torch.full((b, cols), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(s["held"].tolist()):
        table[i, :n] = order[at:at + n]
        at += n
    s["table"] = table
    free = torch.full((pages,), -1, dtype=torch.int32)
    free[:s["spare"]] = order[held:held + s["spare"]]
    s["free"] = free
    s["height"] = torch.tensor([s.pop("spare")], dtype=torch.int32)
    s["tokens"] = int(0.53 * b * (c["low"] + c["high"])) + c["high"] + 7     # a captured step has room for some more
    for k in ("lens", "counts", "held", "done", "table", "free", "height"):
        s[k] = s[k].cuda()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    h = torch.Generator()
    h.manual_seed(seed)
    s = dict(case=dict(c))
    if c["op"] == "plan":
        _prepare_plan(c, s, h)
    elif c["op"] in ("bounds", "sparse"):
        kind, b, dt = _cache_type(c), c["batch"], DTYPES[c["dtype"]]
        lens, more = _lengths(h, c), c.get("nodes", 0)
        s["lens"] = lens.cuda()
        s["max_len"] = c["longest"] + more
        per = -(-s["max_len"] // c["page"])
        s["table"] = torch.randperm(b * per, device="cuda", generator=g).to(torch.int32).view(b, per)
        s["kp"], s["ks"] = _paged(g, c, kind, b * per)
        shape = (b * per, c["kv_heads"], c["dim"])
        if c["op"] == "bounds":
            s["lo"], s["hi"] = torch.zeros(shape, device="cuda", dtype=dt), torch.zeros(shape, device="cuda", dtype=dt)
            # the keys that are new since the last call: all of them, or the last few
            first = (lens - c["new"]).clamp(min=0) if c["new"] else torch.zeros_like(lens)
            s["first"] = first.cuda()
            s["most"] = int(((lens + c["page"] - 1) // c["page"] - first // c["page"]).max())
        else:
            t = c["nodes"]
            s["vp"], s["vs"] = _paged(g, c, kind, b * per)
            s["lo"], s["hi"] = (torch.empty(shape, device="cuda", dtype=dt) for _ in range(2))
            for i in range(0, b * per, 4096):
                x = s["kp"][i:i + 4096].float()
                if s["ks"] is not None:
                    x *= s["ks"][i:i + 4096][..., None]
                s["lo"][i:i + 4096], s["hi"][i:i + 4096] = x.amin(2).to(dt), x.amax(2).to(dt)
            s["q"] = (1.5 * _randn(g, b, t, c["q_heads"], c["dim"])).to(dt)
            s["mask"] = _trees(h, b, t).cuda() if c["tree"] else None
            s["count"] = torch.randint((t + 1) // 2, t + 1, (b,), generator=h, dtype=torch.int32).cuda() if c["ragged"] else None
            s["scale"] = c["dim"] ** -0.5
    else:
        b, k, v, dt = c["batch"], c["steps"], c["vocab"], DTYPES[c["dtype"]]
        x = _randn(g, b, k, v) * (1.0 + 3.0 * _rand(g, b, k, 1))    # some are sure of the next token, others are not
        if c["masked"]:
            # tokens that a grammar forbids, for some of the sequences
            x[(_rand(g, b, k, v) < 0.4) & (_rand(g, b, 1, 1) < 0.5)] = -math.inf
        s["x"] = x.to(dt)
        s["r"] = _rand(g, b, k)
        t = 0.5 + torch.rand(b, generator=h)
        t[torch.rand(b, generator=h) < 0.1] = 0.0                   # some sequences take the likeliest token
        s["t"] = t.cuda()
        s["k"] = None
        if c["top_k"]:
            s["k"] = torch.randint((c["top_k"] + 1) // 2, c["top_k"] + 1, (b,), generator=h, dtype=torch.int32).cuda()
        s["p"] = (0.8 + 0.19 * torch.rand(b, generator=h)).cuda() if c["top_p"] else None
        s["m"] = (0.1 * torch.rand(b, generator=h)).cuda() if c["min_p"] else None
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _plain_plan(c, s):
    page, cols = c["page"], c["cols"]
    table, held, free, height = s["table"], s["held"], s["free"], s["height"]
    dev = table.device
    col = torch.arange(cols, device=dev)
    # Finished rows: their pages go onto the stack, row after row.
    back = (col < held[:, None]) & (s["done"] > 0)[:, None]
    at = back.flatten().cumsum(0).view(back.shape) - 1 + height
    free[at[back]] = table[back]
    now = height + back.sum().to(torch.int32)
    have = torch.where(s["done"] > 0, 0, held)
    # What every sequence needs, and which of them get it.
    n, held_tokens = s["counts"].clamp(min=0).long(), s["lens"].clamp(min=0).long()
    upto = n.cumsum(0)
    need = (held_tokens + n + page - 1) // page
    fits = (n > 0) & (upto <= s["tokens"]) & (need <= cols)
    want = torch.where(fits, (need - have).clamp(min=0), 0)
    run = want.cumsum(0)
    good = fits & ((run <= now) | (want == 0))
    want = torch.where(good, want, 0)
    taken = want.sum()
    base = now - taken
    mine = (col >= have[:, None]) & (col < (have + want)[:, None])
    order = mine.flatten().cumsum(0).view(mine.shape) - 1 + base
    table[mine] = free[order[mine]]
    place = torch.arange(free.shape[0], device=dev)
    free[(place >= base) & (place < now)] = -1
    held.copy_(have + want)
    height.copy_(base)
    # The tokens.
    starts = torch.cat((torch.zeros_like(upto[:1]), upto)).clamp(max=s["tokens"])
    t = torch.arange(s["tokens"], device=dev)
    owner = (t[:, None] >= upto).sum(1)
    real = owner < n.shape[0]
    owner = owner.clamp(max=n.shape[0] - 1)
    pos = held_tokens[owner] + t - (upto - n)[owner]
    slot = table[owner, (pos // page).clamp(0, cols - 1)].long() * page + pos % page
    return {"slots": torch.where(real & good[owner], slot, -1), "pos": torch.where(real, pos, 0), "starts": starts.to(torch.int32),
            "granted": torch.where(good, n, 0).to(torch.int32), "table": table, "held": held, "free": free, "height": height}


def _rows(kind, pages, scales, page, at):
    """Rows of the cache (page, at: tensors that broadcast) as float32, heads after them."""
    if kind == "e4m3":
        x = pages.view(torch.int8)[page, :, at].view(DTYPES[kind]).float()
    else:
        x = pages[page, :, at].float()
    return x * scales[page, :, at][..., None] if kind in SCALED else x


def _plain_bounds(c, s):
    size, kind, dt = c["page"], _cache_type(c), DTYPES[c["dtype"]]
    low, high = s["first"] // size, (s["lens"] + size - 1) // size
    # Sequences with fewer pages do their last one again.
    j = torch.minimum(low[:, None] + torch.arange(s["most"], device="cuda"), high[:, None] - 1).long()
    page = s["table"].long().gather(1, j)
    at = torch.arange(size, device="cuda")
    x = _rows(kind, s["kp"], s["ks"], page[..., None], at)          # (batch, pages, places, heads, dim)
    there = (j[..., None] * size + at < s["lens"][:, None, None])[..., None, None]
    s["lo"][page] = torch.where(there, x, math.inf).amin(2).to(dt)
    s["hi"][page] = torch.where(there, x, -math.inf).amax(2).to(dt)
    return {"lo": s["lo"], "hi": s["hi"]}


def _select(c, s):
    """-> (logical pages chosen (batch, heads, budget), -1 behind them; how many; how many there are)"""
    b, t, hk, size, budget = c["batch"], c["nodes"], c["kv_heads"], c["page"], c["budget"]
    count = s["count"] if s["count"] is not None else torch.full_like(s["lens"], t)
    q = s["q"].double()                                             # scores need 64 bits where pages are close
    q = torch.where((torch.arange(t, device="cuda") < count[:, None])[..., None, None], q, 0.0)
    q = q.view(b, t, hk, -1, c["dim"])
    up, down = q.clamp(min=0).sum((1, 3)), q.clamp(max=0).sum((1, 3))     # (batch, heads, dim)
    table = s["table"].long()
    score = torch.empty(b, hk, table.shape[1], device="cuda", dtype=torch.float64)
    for i in range(0, table.shape[1], 1024):
        lo, hi = s["lo"][table[:, i:i + 1024]].double(), s["hi"][table[:, i:i + 1024]].double()
        score[:, :, i:i + 1024] = (hi * up[:, None] + lo * down[:, None]).sum(-1).transpose(1, 2)
    page = torch.arange(table.shape[1], device="cuda")
    pages = ((s["lens"] + count + size - 1) // size)[:, None, None]
    tail = (s["lens"] // size - c["last"])[:, None, None]
    score = torch.where((page < c["first"]) | (page >= tail), math.inf, score)
    score = torch.where(page < pages, score, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True)[1][..., :budget]
    n = pages.clamp(max=budget)
    at = torch.arange(order.shape[-1], device="cuda")
    chosen = torch.sort(torch.where(at < n, order, 1 << 40), dim=-1)[0]
    chosen = torch.where(at < n, chosen, -1)
    if chosen.shape[-1] < budget:
        chosen = torch.cat((chosen, torch.full((b, hk, budget - chosen.shape[-1]), -1, device="cuda")), -1)
    return chosen, n[:, 0, 0], pages[:, 0, 0], count


def _visible(c, s, lens, count, pos):
    """Which tokens of the chosen pages each node sees: (batch, nodes, positions)."""
    t = c["nodes"]
    j = pos[None, None, :] - lens[:, None, None]
    node = torch.arange(t, device="cuda")[None, :, None]
    seen = j <= node if s["mask"] is None else ((s["mask"][:, :, None] >> j.clamp(0, t - 1)) & 1).bool()
    return ((j < 0) | (seen & (j < count[:, None, None]))) & (node < count[:, None, None])


def _plain_sparse(c, s):
    b, t, hk, size = c["batch"], c["nodes"], c["kv_heads"], c["page"]
    kind = _cache_type(c)
    chosen, n, pages, count = _select(c, s)
    selected = torch.where(chosen >= 0, s["table"].long()[:, None].expand(-1, hk, -1).gather(2, chosen.clamp(min=0)), -1)
    lens = s["lens"] - (pages - n) * size
    rows = selected.clamp(min=0)
    head = torch.arange(hk, device="cuda")[None, :, None]
    k, v = (s[p].view(torch.int8)[rows, head].view(DTYPES[kind]).float() if kind == "e4m3" else s[p][rows, head].float() for p in ("kp", "vp"))
    if kind in SCALED:
        k, v = k * s["ks"][rows, head][..., None], v * s["vs"][rows, head][..., None]
    k, v = (x.reshape(b, hk, -1, c["dim"]) for x in (k, v))
    q = s["q"].float().view(b, t, hk, -1, c["dim"]).permute(0, 2, 1, 3, 4)
    group = q.shape[3]
    q = q.reshape(b, hk, t * group, -1)
    pos = torch.arange(k.shape[2], device="cuda")
    seen = _visible(c, s, lens, count, pos)[:, None, :, None, :].expand(b, 1, t, group, -1).reshape(b, 1, t * group, -1)
    x = torch.where(seen, torch.matmul(q, k.transpose(2, 3).contiguous()) * s["scale"], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    o = o.view(b, hk, t, group, -1).permute(0, 2, 1, 3, 4).reshape(b, t, c["q_heads"], -1)
    lse = (torch.log(total) + top)[..., 0].view(b, hk, t, group).permute(0, 2, 1, 3).reshape(b, t, c["q_heads"])
    return {"selected": selected.to(torch.int32), "lens": lens.to(torch.int32), "out": o.to(s["q"].dtype), "lse": lse}


def _plain_sample(c, s):
    b, k, v = c["batch"], c["steps"], c["vocab"]
    x = s["x"].float()
    xs, order = torch.sort(x, dim=-1, descending=True, stable=True)
    t = s["t"].double()[:, None, None]
    greedy = ~(t > 0)
    w = torch.exp((xs.double() - xs[..., :1].double()) / torch.where(greedy, 1.0, t))     # borders need 64 bits
    at = torch.arange(v, device="cuda")
    most = s["k"].long()[:, None, None] if s["k"] is not None else torch.full_like(greedy, v, dtype=torch.int64)
    most = torch.where(greedy, 1, torch.where(most > 0, most, v))
    w = torch.where(at < most, w, 0.0)
    if s["p"] is not None:
        run = w.cumsum(-1)
        before = torch.cat((torch.zeros_like(run[..., :1]), run[..., :-1]), -1)
        w = torch.where((before < s["p"].double()[:, None, None] * run[..., -1:]) | (at == 0), w, 0.0)
    if s["m"] is not None:
        w = torch.where(w >= s["m"].double()[:, None, None], w, 0.0)
    w = torch.zeros_like(w).scatter_(-1, order, w)
    run = w.cumsum(-1)
    total = run[..., -1:]
    found = {"tokens": (run <= s["r"].double()[..., None] * total).sum(-1)}
    if c["probs"]:
        found["probs"] = (w / total).to(DTYPES[c["probs"]])
    return found


def run(state):
    s, c = state, state["case"]
    if own:
        return _own(c, s)
    return {"plan": _plain_plan, "bounds": _plain_bounds, "sparse": _plain_sparse, "sample": _plain_sample}[c["op"]](c, s)


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------
def _own(c, s):
    import reduction_libred_amd as rl

    if c["op"] == "plan":
        slots, pos, starts, granted = rl.red_plan_slots(s["lens"], s["counts"], s["table"], s["held"], s["free"], s["height"],
                                                        c["page"], s["tokens"], done=s["done"])
        return {"slots": slots, "pos": pos, "starts": starts, "granted": granted, "table": s["table"], "held": s["held"],
                "free": s["free"], "height": s["height"]}
    if c["op"] == "bounds":
        rl.red_page_bounds(s["kp"], s["table"], s["lens"], s["lo"], s["hi"], first=s["first"], most=s["most"], k_scales=s["ks"])
        return {"lo": s["lo"], "hi": s["hi"]}
    if c["op"] == "sparse":
        selected, lens = rl.red_select_pages(s["q"], s["lo"], s["hi"], s["table"], s["lens"], c["page"], c["budget"], first=c["first"],
                                             last=c["last"], max_len=s["max_len"], node_count=s["count"])
        out, lse = rl.red_sparse_attention(s["q"], s["kp"], s["vp"], selected, lens, s["scale"], tree_mask=s["mask"],
                                           node_count=s["count"], k_scales=s["ks"], v_scales=s["vs"])
        return {"selected": selected, "lens": lens, "out": out, "lse": lse}
    x, r = (s["x"][:, 0], s["r"][:, 0]) if c["steps"] == 1 else (s["x"], s["r"])
    tokens, probs = rl.red_sample(x, r, temperature=s["t"], top_k=s["k"], top_p=s["p"], min_p=s["m"],
                                  probs=DTYPES[c["probs"]] if c["probs"] else None)
    found = {"tokens": tokens.view(c["batch"], c["steps"])}
    if c["probs"]:
        found["probs"] = probs.view(c["batch"], c["steps"], c["vocab"])
    return found


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "plan":
        tokens = c["batch"] * (c["low"] + c["high"]) / 2         # what is left of the slots is written as well
        return {"bytes": 36 * c["batch"] + 17 * tokens + 12 * tokens / c["page"], "flops": 4 * tokens}
    if c["op"] == "sample":
        n = c["batch"] * c["steps"] * c["vocab"]
        return {"bytes": n * (BYTES[c["dtype"]] + (BYTES[c["probs"]] if c["probs"] else 0)), "flops": n * 30}
    kind = _cache_type(c)
    tokens = c["batch"] * (c["shortest"] + c["longest"]) / 2 if c["batch"] > 1 else c["longest"]
    stored = c["dim"] * BYTES[kind] + (4 if kind in SCALED else 0)
    bound = 2 * c["dim"] * BYTES[c["dtype"]]                     # both bounds of a page and kv head
    if c["op"] == "bounds":
        pages = tokens / c["page"]
        if c["new"]:                                             # only the pages of the last few tokens
            pages = min(pages, c["batch"] * (1 + (c["new"] - 1) / c["page"]))
            tokens = min(tokens, pages * c["page"])
        return {"bytes": c["kv_heads"] * (tokens * stored + pages * bound), "flops": 2 * tokens * c["kv_heads"] * c["dim"]}
    seen = min(tokens, c["batch"] * c["budget"] * c["page"]) + c["batch"] * c["nodes"]
    pages, rows = tokens / c["page"], c["batch"] * c["nodes"] * c["q_heads"]
    return {"bytes": c["kv_heads"] * (pages * bound + 2 * seen * stored) + 2 * rows * c["dim"] * BYTES[c["dtype"]],
            "flops": 4 * pages * c["kv_heads"] * c["dim"] + 4 * seen * c["nodes"] * c["q_heads"] * c["dim"]}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_plan(c, s):
    """One sequence after the other, on lists."""
    lens, counts, done, held = (s[k].tolist() for k in ("lens", "counts", "done", "held"))
    table, size = s["table"].tolist(), c["page"]
    stack = s["free"].tolist()
    top = int(s["height"])
    for b in range(c["batch"]):
        if done[b]:
            for j in range(held[b]):
                stack[top] = table[b][j]
                top += 1
            held[b] = 0
    starts, granted, asked, wanted, full = [0], [], [], [], False
    for b in range(c["batch"]):
        starts.append(starts[-1] + max(counts[b], 0))
        pages = -(-(lens[b] + counts[b]) // size)
        want = max(0, pages - held[b])
        okay = counts[b] > 0 and pages <= c["cols"] and starts[-1] <= s["tokens"]
        if okay and want:
            full = full or sum(asked) + want > top
            if full:
                okay = False
            else:
                asked.append(want)
        granted.append(counts[b] if okay else 0)
        wanted.append(want if okay else 0)
    at = top - sum(asked)
    for b in range(c["batch"]):
        for j in range(wanted[b]):
            table[b][held[b] + j] = stack[at]
            stack[at] = -1
            at += 1
        held[b] += wanted[b]
    slots, pos = [-1] * s["tokens"], [0] * s["tokens"]
    for b in range(c["batch"]):
        for i in range(counts[b]):
            if starts[b] + i < s["tokens"]:
                p = lens[b] + i
                pos[starts[b] + i] = p
                if granted[b]:
                    slots[starts[b] + i] = table[b][p // size] * size + p % size
    whole = dict(slots=(slots, torch.int64), pos=(pos, torch.int64), starts=([min(x, s["tokens"]) for x in starts], torch.int32),
                 granted=(granted, torch.int32), table=(table, torch.int32), held=(held, torch.int32), free=(stack, torch.int32),
                 height=([top - sum(asked)], torch.int32))
    return {k: torch.tensor(x, dtype=t) for k, (x, t) in whole.items()}


def _exact_keys(c, s, name, b, pages):
    """The keys or values of these logical pages of a sequence: (pages, heads, places, dim) in 64 bits."""
    page = s["table"][b, pages].long()
    x = s[name + "p"][page].double()
    return x * s[name + "s"][page].double()[..., None] if s[name + "s"] is not None else x


def _exact_bounds(c, s):
    lo, hi = s["lo"].double(), s["hi"].double()
    for b, (n, first) in enumerate(zip(s["lens"].tolist(), s["first"].tolist())):
        a, e = first // c["page"], -(-n // c["page"])
        pages = torch.arange(a, e, device="cuda")
        x = _exact_keys(c, s, "k", b, pages)
        whole = s["table"][b, a:e].long()
        lo[whole], hi[whole] = x.amin(2), x.amax(2)
        rest = n - (e - 1) * c["page"]
        lo[whole[-1]], hi[whole[-1]] = x[-1, :, :rest].amin(1), x[-1, :, :rest].amax(1)
    return {"lo": lo, "hi": hi}


def _exact_sparse(c, s):
    size, hk, group = c["page"], c["kv_heads"], c["q_heads"] // c["kv_heads"]
    selected = torch.full((c["batch"], hk, c["budget"]), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(c["batch"], dtype=torch.int32)
    out = torch.zeros(s["q"].shape, device="cuda", dtype=torch.float64)
    lse = torch.full(s["q"].shape[:3], -math.inf, device="cuda", dtype=torch.float64)
    for b, ctx in enumerate(s["lens"].tolist()):
        nodes = int(s["count"][b]) if s["count"] is not None else c["nodes"]
        pages = -(-(ctx + nodes) // size)
        keep = min(pages, c["budget"])
        lens[b] = ctx - (pages - keep) * size
        here = s["table"][b, :pages].long()
        lo, hi = s["lo"][here].double(), s["hi"][here].double()
        hidden = torch.zeros(nodes, lens[b] + nodes, dtype=torch.bool)
        for i in range(nodes):
            word = int(s["mask"][b, i]) if s["mask"] is not None else (1 << (i + 1)) - 1
            for j in range(nodes):
                hidden[i, lens[b] + j] = not (word >> j) & 1
        hidden = hidden.cuda()
        for h in range(hk):
            q = s["q"][b, :nodes, h * group:(h + 1) * group].double()
            score = torch.zeros(pages, device="cuda", dtype=torch.float64)
            for row in q.reshape(-1, c["dim"]):
                score += torch.maximum(row * lo[:, h], row * hi[:, h]).sum(-1)
            score = score.cpu().numpy()
            forced = [p for p in range(pages) if p < c["first"] or p >= ctx // size - c["last"]]
            others = [p for p in range(pages) if not (p < c["first"] or p >= ctx // size - c["last"])]
            others.sort(key=lambda p: (-score[p], p))
            chosen = torch.tensor(sorted(forced + others[:keep - len(forced)]), device="cuda")
            selected[b, h, :keep] = s["table"][b, chosen]
            k, v = (_exact_keys(c, s, x, b, chosen)[:, h].reshape(-1, c["dim"])[:lens[b] + nodes] for x in "kv")
            x = (q.transpose(0, 1) @ k.t().contiguous()) * s["scale"]
            x = x.masked_fill(hidden, -math.inf)                   # (group, nodes, tokens)
            out[b, :nodes, h * group:(h + 1) * group] = (torch.softmax(x, -1) @ v).transpose(0, 1)
            lse[b, :nodes, h * group:(h + 1) * group] = torch.logsumexp(x, -1).t()
    return {"selected": selected, "lens": lens, "out": out, "lse": lse}


def _exact_sample(c, s):
    """Row by row on the host, with sums of 80 bits."""
    b, k, v = c["batch"], c["steps"], c["vocab"]
    logits, chance = s["x"].double().cpu().numpy(), s["r"].double().cpu().numpy()
    t, top_k, top_p, min_p = (None if s[n] is None else s[n].double().cpu().numpy() for n in "tkpm")
    tokens = np.zeros((b, k), dtype=np.int64)
    probs = np.zeros((b, k, v)) if c["probs"] else None
    for i in range(b):
        for j in range(k):
            x = logits[i, j]
            if not t[i] > 0:
                tokens[i, j] = int(np.argmax(x))
                if c["probs"]:
                    probs[i, j, tokens[i, j]] = 1.0
                continue
            order = np.argsort(-x, kind="stable")
            if top_k is not None and 0 < top_k[i] < v:
                order = order[:int(top_k[i])]
            w = np.exp((x[order] - x[order[0]]).astype(np.longdouble) / np.longdouble(t[i]))
            keep = len(w)
            if top_p is not None:
                run = np.cumsum(w)
                keep = max(1, 1 + int(np.searchsorted(run[:-1], np.longdouble(top_p[i]) * run[-1], side="left")))
            if min_p is not None:
                keep = min(keep, int((w >= min_p[i]).sum()))
            kept = np.zeros(v, dtype=np.longdouble)
            kept[order[:keep]] = w[:keep]
            run = np.cumsum(kept)
            tokens[i, j] = int(np.searchsorted(run, chance[i, j] * run[-1], side="right"))
            if c["probs"]:
                probs[i, j] = kept / run[-1]
    found = {"tokens": torch.from_numpy(tokens)}
    if c["probs"]:
        found["probs"] = torch.from_numpy(probs)
    return found


def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "bounds": _exact_bounds, "sparse": _exact_sparse, "sample": _exact_sample}[case["op"]](case, s)
