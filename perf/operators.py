"""The operators of one decoding step of drafted tokens: cases, inputs and plain forms.

Four groups, in the order in which such a step runs them:

  norm    RMS norm of every query and key head with the rotary position rotation in the same pass
          ("back": its backward pass, with the gradients of both norm weights)
  cache   keys and values quantised as they are written into a paged cache, and read back
          ("read": only the reading back of tokens that are in the cache already)
  attend  attention of drafted tokens (a tree, a chain, or a single token) over that cache
  verify  which drafted tokens the target's probabilities accept, and the token sampled after them

`own` false computes them with elementary torch operations, `own` true calls the library.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
          "i8": torch.int8, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "i8": 1, "e4m3": 1}
TOP = {"i8": 127.0, "e4m3": 448.0}   # the largest value that a cache type stands for


def listed():
    return [
        # One decoding step of a few sequences with drafted tokens: latency counts.
        dict(name="norm decode", op="norm", back=False, tokens=12, q_heads=32, k_heads=8, dim=128, rot=128,
             interleaved=False, packed=True, dtype="bf16", far=1 << 17),
        # A batch of prompts, q and k still inside the product of the fused projection.
        dict(name="norm prompt", op="norm", back=False, tokens=16384, q_heads=32, k_heads=8, dim=128, rot=128,
             interleaved=False, packed=True, dtype="bf16", far=1 << 15),
        # A training step's micro-batch: gradients of q, k and both weights.
        dict(name="norm training", op="norm", back=True, tokens=16384, q_heads=32, k_heads=8, dim=128, rot=128,
             interleaved=False, packed=True, dtype="bf16", far=1 << 13),
        # An odd number of tokens, a head that is rotated in part, neighbours as pairs, 32-bit training.
        dict(name="norm odd training", op="norm", back=True, tokens=1009, q_heads=10, k_heads=5, dim=96, rot=36,
             interleaved=True, packed=False, dtype="f32", far=1 << 20),
        # The drafted tokens of a few sequences go into the cache.
        dict(name="cache decode", op="cache", read=False, tokens=20, heads=8, dim=128, page=16, pages=4096,
             dtype="bf16", cache="i8"),
        # Prompts are written, and their keys and values taken back in 16 bits.
        dict(name="cache prompt", op="cache", read=False, tokens=32768, heads=8, dim=128, page=64, pages=1024,
             dtype="bf16", cache="e4m3"),
        # A prompt's next part needs the earlier parts in 16 bits.
        dict(name="cache read", op="cache", read=True, tokens=100003, heads=4, dim=80, page=24, pages=6000,
             dtype="f16", cache="i8"),
        # A single sequence, a single token.
        dict(name="attend single", op="attend", batch=1, nodes=1, q_heads=32, kv_heads=8, dim=128, longest=8191,
             shortest=8191, page=16, tree=False, ragged=False, dtype="f16", cache="f16"),
        # A serving batch with sequences of many lengths, small trees, an 8-bit cache.
        dict(name="attend batch", op="attend", batch=32, nodes=8, q_heads=32, kv_heads=8, dim=128, longest=16384,
             shortest=1500, page=64, tree=True, ragged=True, dtype="bf16", cache="i8"),
        # Few sequences with large trees: as many products as bytes.
        dict(name="attend large trees", op="attend", batch=4, nodes=64, q_heads=64, kv_heads=8, dim=128,
             longest=8192, shortest=7001, page=32, tree=True, ragged=True, dtype="bf16", cache="bf16"),
        # One sequence's drafts, a small vocabulary.
        dict(name="verify single", op="verify", batch=1, drafts=4, vocab=32000, dtype="f32", given=True),
        # A serving batch, a large vocabulary of odd size.
        dict(name="verify batch", op="verify", batch=192, drafts=6, vocab=131071, dtype="f32", given=True),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over the logarithm."""
    return min(high, int(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "cache", "attend", "attend", "verify"])
    if op == "norm":
        k_heads = rng.choice([1, 2, 4, 5, 8])
        dim = rng.choice([32, 64, 72, 80, 96, 100, 128, 192, 256])
        c = dict(op=op, back=rng.random() < 0.5, tokens=_spread(rng, 1, 16384), q_heads=k_heads * rng.choice([1, 2, 3, 4]),
                 k_heads=k_heads, dim=dim, rot=rng.choice([dim, dim, dim // 4 * 2, 2 * rng.randint(1, dim // 2)]),
                 interleaved=rng.random() < 0.4, packed=rng.random() < 0.5, dtype=rng.choice(["bf16", "f16", "f32"]),
                 far=_spread(rng, 1024, 1 << 20))
        while c["tokens"] * (c["q_heads"] + k_heads) * dim * BYTES[c["dtype"]] > 16384 * 40 * 128 * 2:
            c["tokens"] = c["tokens"] // 2 + 1
        return c
    if op == "cache":
        heads, dim, page = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 80, 96, 112, 128, 192, 256]), rng.choice([1, 8, 16, 24, 32, 64, 128])
        tokens = min(_spread(rng, 1, 120000), 32768 * 8 * 128 // (heads * dim))
        return dict(op=op, read=rng.random() < 0.4, tokens=tokens, heads=heads, dim=dim, page=page,
                    pages=-(-tokens // page) + rng.randint(1, 50), dtype=rng.choice(["bf16", "f16"]),
                    cache=rng.choice(["i8", "i8", "e4m3", "e4m3", "own"]))
    if op == "attend":
        kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8])
        batch, nodes = _spread(rng, 1, 32), _spread(rng, 1, 64)
        longest = _spread(rng, 1, 16384)
        dim = rng.choice([64, 80, 96, 128, 128, 192, 256])
        while batch * longest * kv_heads * dim > 16 * 16384 * 8 * 128 or batch * longest * kv_heads * group * nodes * dim > 2 * 64 * 64 * 8192 * 128:
            batch, longest = max(1, batch // 2), longest // 2 + 1
        dtype = rng.choice(["bf16", "f16"])
        return dict(op=op, batch=batch, nodes=nodes, q_heads=kv_heads * group, kv_heads=kv_heads, dim=dim, longest=longest,
                    shortest=rng.randint(0, longest), page=rng.choice([1, 8, 16, 24, 32, 64, 128]), tree=rng.random() < 0.7,
                    ragged=rng.random() < 0.5, dtype=dtype, cache=rng.choice(["i8", "e4m3", "own"]))
    batch, drafts, vocab = _spread(rng, 1, 192), rng.randint(1, 10), _spread(rng, 1000, 131072)
    while batch * (2 * drafts + 1) * vocab > 192 * 13 * 131071:
        batch = batch // 2 + 1
    return dict(op=op, batch=batch, drafts=drafts, vocab=vocab, dtype=rng.choice(["f32", "f32", "bf16", "f16"]),
                given=rng.random() < 0.8)


def _cache_type(case):
    return case["dtype"] if case["cache"] == "own" else case["cache"]


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _rand(g, *shape):
    return torch.rand(*shape, device="cuda", generator=g)


def _heads(g, tokens, heads, dim, packed, dtype):
    """Projections of `tokens` tokens with these numbers of heads, one tensor each: parts of one product or tensors of their own."""
    gain = torch.exp(0.5 * _randn(g, sum(heads), 1))   # heads differ in size
    if packed:
        x = (_randn(g, tokens, sum(heads), dim) * gain).to(dtype)
        return list(torch.split(x, heads, dim=1))
    return [(_randn(g, tokens, h, dim) * s).to(dtype) for h, s in zip(heads, torch.split(gain, heads))]


def _paged(g, c, kind, pages, heads):
    """A paged cache that holds values of the path's kind everywhere: pages and scales."""
    shape = (pages, heads, c["page"], c["dim"])
    if kind in TOP:
        x = _randn(g, *shape)
        if kind == "i8":
            x = (x * 36.0).clamp_(-127, 127).round_().to(torch.int8)   # the largest of a row of 128 is near 127
        else:
            x = (x * 120.0).clamp_(-448, 448).to(DTYPES[kind])
        return x, (0.5 + _rand(g, *shape[:3])) * (1.0 / (36.0 if kind == "i8" else 120.0))
    return _randn(g, *shape).to(DTYPES[kind]), None


def _trees(g, batch, nodes):
    """Ancestor bits of random trees: bit j of word i is set where node i sees node j (itself and the nodes above it)."""
    above = torch.zeros(batch, nodes, nodes, dtype=torch.bool)
    pick = torch.rand(batch, nodes, generator=g)
    for i in range(nodes):
        if i:
            parent = (pick[:, i] * i).long()
            above[:, i] = above[torch.arange(batch), parent]
        above[:, i, i] = True
    word = torch.zeros(batch, nodes, dtype=torch.int64)
    for j in range(nodes):
        word |= above[:, :, j].to(torch.int64) << j
    return word


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    h = torch.Generator()
    h.manual_seed(seed)
    s = dict(case=dict(c))
    if c["op"] == "norm":
        dt = DTYPES[c["dtype"]]
        s["q"], s["k"] = _heads(g, c["tokens"], [c["q_heads"], c["k_heads"]], c["dim"], c["packed"], dt)
        s["qw"], s["kw"] = ((1.0 + 0.2 * _randn(g, c["dim"])).to(dt) for _ in range(2))
        s["pos"] = torch.randint(0, c["far"], (c["tokens"],), device="cuda", generator=g)
        i = torch.arange(c["rot"] // 2, device="cuda", dtype=torch.float64)
        s["freq"] = torch.pow(10000.0, -2.0 * i / c["rot"]).to(torch.float32)
        if c["back"]:
            s["dq"], s["dk"] = (_randn(g, c["tokens"], n, c["dim"]).to(dt) for n in (c["q_heads"], c["k_heads"]))
    elif c["op"] == "cache":
        kind = _cache_type(c)
        slots = torch.randperm(c["pages"] * c["page"], device="cuda", generator=g)[:c["tokens"]]
        run = torch.sort(slots.view(-1)[:c["tokens"] // 2])[0]   # half of them in order, as a prompt's are
        slots[:c["tokens"] // 2] = run
        s["slots"] = slots
        s["kp"], s["ks"] = _paged(g, c, kind, c["pages"], c["heads"])
        s["vp"], s["vs"] = _paged(g, c, kind, c["pages"], c["heads"])
        if not c["read"]:
            s["k"], s["v"] = _heads(g, c["tokens"], [c["heads"], c["heads"]], c["dim"], True, DTYPES[c["dtype"]])
    elif c["op"] == "attend":
        kind, b, t = _cache_type(c), c["batch"], c["nodes"]
        lens = torch.linspace(c["shortest"], c["longest"], b).round().to(torch.int32) if b > 1 else torch.tensor([c["longest"]], dtype=torch.int32)
        lens = lens[torch.randperm(b, generator=h)]
        s["max_len"] = c["longest"] + t
        per = -(-s["max_len"] // c["page"])
        pages = b * per
        s["table"] = torch.randperm(pages, device="cuda", generator=g).to(torch.int32).view(b, per)
        s["lens"] = lens.cuda()
        s["kp"], s["ks"] = _paged(g, c, kind, pages, c["kv_heads"])
        s["vp"], s["vs"] = _paged(g, c, kind, pages, c["kv_heads"])
        s["q"] = (1.5 * _randn(g, b, t, c["q_heads"], c["dim"])).to(DTYPES[c["dtype"]])
        s["mask"] = _trees(h, b, t).cuda() if c["tree"] else None
        s["count"] = torch.randint((t + 1) // 2, t + 1, (b,), generator=h, dtype=torch.int32).cuda() if c["ragged"] else None
        s["scale"] = c["dim"] ** -0.5
    else:
        b, k, v, dt = c["batch"], c["drafts"], c["vocab"], DTYPES[c["dtype"]]
        x = 2.5 * _randn(g, b, k + 1, v)
        s["p"] = torch.softmax(x, -1).to(dt)
        y = x[:, :k]
        y += 0.7 * _randn(g, b, k, v)
        s["q"] = torch.softmax(y, -1).to(dt) if c["given"] else None
        # tokens drawn from the draft's distribution: the largest of logits with Gumbel noise
        s["drafted"] = (y - torch.log(-torch.log(_rand(g, b, k, v).clamp_(1e-7, 1 - 1e-7)))).argmax(-1)
        s["u"], s["r"] = _rand(g, b, k), _rand(g, b)
        s["count"] = torch.randint((k + 1) // 2, k + 1, (b,), generator=h, dtype=torch.int32).cuda()
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _angles(c, s):
    a = s["pos"].double()[:, None] * s["freq"].double()   # far positions need 64 bits
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _rotate(c, x, cos, sin):
    rot = c["rot"]
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((y, x[..., rot:]), -1)


EPS = 1e-6


def _norm(c, x, w, cos, sin):
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return _rotate(c, x * r * w.float(), cos, sin)


def _norm_back(c, x, w, dy, cos, sin):
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    g = _rotate(c, dy.float(), cos, -sin)
    h = g * w.float()
    dx = r * (h - x * (r * r * (h * x).mean(-1, keepdim=True)))
    return dx, (g * x * r).sum((0, 1))


def _quantise(x, kind):
    x = x.float()
    top = x.abs().amax(-1, keepdim=True)
    y = x * torch.where(top > 0, TOP[kind] / top, 0.0)
    return (y.round().to(torch.int8) if kind == "i8" else y.to(DTYPES[kind])), (top / TOP[kind])[..., 0]


def _write(c, kind, x, pages, scales, page, at):
    if kind in TOP:
        x, top = _quantise(x, kind)
        scales[page, :, at] = top
    if kind == "e4m3":
        pages.view(torch.int8)[page, :, at] = x.view(torch.int8)
    else:
        pages[page, :, at] = x


def _read(kind, pages, scales, page, at):
    if kind == "e4m3":
        x = pages.view(torch.int8)[page, :, at].view(DTYPES[kind]).float()
    else:
        x = pages[page, :, at].float()
    return x * scales[page, :, at][..., None] if kind in TOP else x


def _plain_cache(c, s):
    kind, dt = _cache_type(c), DTYPES[c["dtype"]]
    page, at = torch.div(s["slots"], c["page"], rounding_mode="floor"), s["slots"] % c["page"]
    if not c["read"]:
        _write(c, kind, s["k"], s["kp"], s["ks"], page, at)
        _write(c, kind, s["v"], s["vp"], s["vs"], page, at)
    return {"k": _read(kind, s["kp"], s["ks"], page, at).to(dt), "v": _read(kind, s["vp"], s["vs"], page, at).to(dt),
            "ks": s["ks"], "vs": s["vs"]}


def _visible(c, s, pos):
    """Which cached tokens each node sees: (batch, nodes, positions)."""
    t = c["nodes"]
    lens = s["lens"][:, None, None].long()
    j = pos[None, None, :] - lens                     # the node that lies at this position
    node = torch.arange(t, device=pos.device)[None, :, None]
    if s["mask"] is None:
        seen = j <= node
    else:
        seen = ((s["mask"][:, :, None] >> j.clamp(0, t - 1)) & 1).bool()
    count = (s["count"].long() if s["count"] is not None else torch.full_like(s["lens"], t).long())[:, None, None]
    return ((j < 0) | (seen & (j < count))) & (node < count)


def _plain_attend(c, s):
    b, t, hk = c["batch"], c["nodes"], c["kv_heads"]
    group, kind = c["q_heads"] // hk, _cache_type(c)
    pos = torch.arange(s["max_len"], device="cuda")
    page, at = s["table"].long()[:, pos // c["page"]], (pos % c["page"]).expand(b, -1)
    k = _read(kind, s["kp"], s["ks"], page, at).permute(0, 2, 3, 1).contiguous()     # (batch, heads, dim, positions)
    v = _read(kind, s["vp"], s["vs"], page, at).permute(0, 2, 1, 3).contiguous()
    q = s["q"].float().view(b, t, hk, group, -1).permute(0, 2, 1, 3, 4).reshape(b, hk, t * group, -1)
    seen = _visible(c, s, pos)[:, None, :, None, :].expand(b, 1, t, group, -1).reshape(b, 1, t * group, -1)
    x = torch.where(seen, torch.matmul(q, k) * s["scale"], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    o = o.view(b, hk, t, group, -1).permute(0, 2, 1, 3, 4).reshape(b, t, c["q_heads"], -1)
    lse = (torch.log(total) + top)[..., 0].view(b, hk, t, group).permute(0, 2, 1, 3).reshape(b, t, c["q_heads"])
    return {"out": o.to(DTYPES[c["dtype"]]), "lse": lse}


def _plain_verify(c, s):
    b, k = c["batch"], c["drafts"]
    d, row = s["drafted"], torch.arange(b, device="cuda")
    at_p = s["p"][:, :k].gather(-1, d[..., None])[..., 0].double()   # borders need 64 bits
    at_q = s["q"].gather(-1, d[..., None])[..., 0].double() if s["q"] is not None else torch.ones_like(at_p)
    i = torch.arange(k, device="cuda")
    good = (s["u"].double() * at_q < at_p) & (i < s["count"][:, None])
    n = good.long().cumprod(-1).sum(-1)
    w = s["p"][row, n].double()
    used = n.clamp(max=k - 1)
    if s["q"] is not None:
        less = s["q"][row, used].double()
    else:
        less = torch.zeros_like(w).scatter_(-1, d[row, used][:, None], 1.0)
    left = torch.where((n < s["count"])[:, None], (w - less).clamp(min=0.0), w)
    left = torch.where(left.sum(-1, keepdim=True) > 0, left, w)
    run = left.cumsum(-1)
    last = run[:, -1:]
    token = (run <= s["r"].double()[:, None] * last).sum(-1)
    j = torch.arange(k + 1, device="cuda")
    padded = torch.cat((d, d[:, :1]), -1)
    tokens = torch.where(j < n[:, None], padded, torch.where(j == n[:, None], token[:, None], -1))
    return {"accepted": n.to(torch.int32), "tokens": tokens}


def run(state):
    s, c = state, state["case"]
    if own:
        return _own(c, s)
    if c["op"] == "norm":
        cos, sin = _angles(c, s)
        if c["back"]:
            dq, dqw = _norm_back(c, s["q"], s["qw"], s["dq"], cos, sin)
            dk, dkw = _norm_back(c, s["k"], s["kw"], s["dk"], cos, sin)
            return {"dq": dq.to(s["q"].dtype), "dk": dk.to(s["q"].dtype), "dqw": dqw, "dkw": dkw}
        return {"q": _norm(c, s["q"], s["qw"], cos, sin).to(s["q"].dtype), "k": _norm(c, s["k"], s["kw"], cos, sin).to(s["q"].dtype)}
    if c["op"] == "cache":
        return _plain_cache(c, s)
    if c["op"] == "attend":
        return _plain_attend(c, s)
    return _plain_verify(c, s)


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------
def _own(c, s):
    import reduction_libred_amd as rl

    if c["op"] == "norm":
        if c["back"]:
            dq, dk, dqw, dkw = rl.red_qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["pos"], s["freq"], q_weight=s["qw"],
                                                            k_weight=s["kw"], eps=EPS, interleaved=c["interleaved"])
            return {"dq": dq, "dk": dk, "dqw": dqw, "dkw": dkw}
        q, k = rl.red_qk_norm_rope(s["q"], s["k"], s["pos"], s["freq"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS,
                                   interleaved=c["interleaved"])
        return {"q": q, "k": k}
    if c["op"] == "cache":
        if not c["read"]:
            rl.red_cache_write(s["k"], s["v"], s["slots"], s["kp"], s["vp"], k_scales=s["ks"], v_scales=s["vs"])
        k, v = rl.red_cache_read(s["kp"], s["vp"], s["slots"], DTYPES[c["dtype"]], k_scales=s["ks"], v_scales=s["vs"])
        return {"k": k, "v": v, "ks": s["ks"], "vs": s["vs"]}
    if c["op"] == "attend":
        out, lse = rl.red_tree_attention(s["q"], s["kp"], s["vp"], s["table"], s["lens"], s["scale"], max_len=s["max_len"],
                                         tree_mask=s["mask"], node_count=s["count"], k_scales=s["ks"], v_scales=s["vs"])
        return {"out": out, "lse": lse}
    accepted, tokens = rl.red_verify_drafts(s["p"], s["q"], s["drafted"], s["u"], s["r"], draft_count=s["count"])
    return {"accepted": accepted, "tokens": tokens}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "norm":
        n = c["tokens"] * (c["q_heads"] + c["k_heads"]) * c["dim"]
        return {"bytes": n * BYTES[c["dtype"]] * (3 if c["back"] else 2) + 8 * c["tokens"], "flops": n * (16 if c["back"] else 8)}
    if c["op"] == "cache":
        rows, kind = 2 * c["tokens"] * c["heads"], _cache_type(c)
        stored = c["dim"] * BYTES[kind] + (4 if kind in TOP else 0)
        wide = c["dim"] * BYTES[c["dtype"]]
        return {"bytes": rows * (stored + wide + (0 if c["read"] else stored + wide)) + 8 * c["tokens"],
                "flops": rows * c["dim"] * (1 if c["read"] else 5)}
    if c["op"] == "attend":
        kind = _cache_type(c)
        tokens = c["batch"] * (c["nodes"] + (c["shortest"] + c["longest"]) / 2 if c["batch"] > 1 else c["longest"] + c["nodes"])
        stored = c["dim"] * BYTES[kind] + (4 if kind in TOP else 0)
        rows = c["batch"] * c["nodes"] * c["q_heads"]
        return {"bytes": 2 * tokens * c["kv_heads"] * stored + 2 * rows * c["dim"] * BYTES[c["dtype"]],
                "flops": 4 * tokens * c["nodes"] * c["q_heads"] * c["dim"]}
    return {"bytes": c["batch"] * ((2 if c["given"] else 1) * c["vocab"] * BYTES[c["dtype"]] + 28 * c["drafts"]),
            "flops": c["batch"] * c["vocab"] * 4}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_turn(c, s, sign):
    """The rotation as one complex factor for each token and pair."""
    a = s["pos"].double()[:, None] * s["freq"].double()
    return torch.polar(torch.ones_like(a), sign * a)[:, None, :]


def _exact_pairs(c, x):
    rot = c["rot"]
    if c["interleaved"]:
        return torch.view_as_complex(x[..., :rot].reshape(*x.shape[:-1], rot // 2, 2).contiguous())
    return torch.complex(x[..., :rot // 2], x[..., rot // 2:rot])


def _exact_turned(c, x, turn):
    z = _exact_pairs(c, x) * turn
    y = x.clone()
    if c["interleaved"]:
        y[..., :c["rot"]] = torch.view_as_real(z).flatten(-2)
    else:
        y[..., :c["rot"] // 2], y[..., c["rot"] // 2:c["rot"]] = z.real, z.imag
    return y


def _exact_norm(c, s):
    if not c["back"]:
        turn = _exact_turn(c, s, 1.0)
        found = {}
        for name, w in (("q", "qw"), ("k", "kw")):
            x = s[name].double()
            size = (x.square().sum(-1, keepdim=True) / c["dim"] + EPS).sqrt()
            found[name] = _exact_turned(c, x / size * s[w].double(), turn)
        return found
    turn = _exact_turn(c, s, -1.0)
    found = {}
    for name, w in (("q", "qw"), ("k", "kw")):
        x = s[name].double()
        size = (x.square().sum(-1, keepdim=True) / c["dim"] + EPS).sqrt()
        unit = x / size
        g = _exact_turned(c, s["d" + name].double(), turn)
        found["d" + name + "w"] = (g * unit).sum(0).sum(0)
        g = g * s[w].double()
        found["d" + name] = (g - unit * (g * unit).sum(-1, keepdim=True) / c["dim"]) / size
    return found


def _exact_cache(c, s):
    kind = _cache_type(c)
    found = {}
    for x, p, sc in (("k", "kp", "ks"), ("v", "vp", "vs")):
        heads, size = c["heads"], c["page"]
        # row of the flat cache that (token, head) lies in
        row = ((s["slots"] // size)[:, None] * heads + torch.arange(heads, device="cuda")) * size + (s["slots"] % size)[:, None]
        if kind not in TOP:
            found[x] = s[p].reshape(-1, c["dim"])[row].double() if c["read"] else s[x].double()
            continue
        if c["read"]:
            scale = s[sc].double()
            found[x] = s[p].double().reshape(-1, c["dim"])[row] * scale.reshape(-1)[row][..., None]
            found[sc] = scale
            continue
        y = s[x].double()
        top = y.abs().max(-1)[0]
        step = top / TOP[kind]
        unit = y / torch.where(step > 0, step, 1.0)[..., None]
        if kind == "i8":
            unit = torch.round(unit)
        else:
            # e4m3 has three bits after the first, from 2^-6 on; below that steps of 2^-9
            fine = torch.exp2(torch.floor(torch.log2(unit.abs().clamp(min=2.0 ** -6))) - 3)
            unit = torch.round(unit / fine) * fine
        found[x] = unit * step[..., None]
        scale = s[sc].double().reshape(-1)
        scale[row] = step
        found[sc] = scale.view(s[sc].shape)
    return found


def _exact_attend(c, s):
    group = c["q_heads"] // c["kv_heads"]
    out = torch.zeros(c["batch"], c["nodes"], c["q_heads"], c["dim"], device="cuda", dtype=torch.float64)
    lse = torch.full(out.shape[:3], -math.inf, device="cuda", dtype=torch.float64)
    for b in range(c["batch"]):
        ctx = int(s["lens"][b])
        nodes = int(s["count"][b]) if s["count"] is not None else c["nodes"]
        used = -(-(ctx + nodes) // c["page"])
        k, v = ([s[p][s["table"][b, :used].long()].double() * (s[sc][s["table"][b, :used].long()].double()[..., None] if s[sc] is not None else 1.0)
                 for p, sc in (("kp", "ks"), ("vp", "vs"))])
        k, v = (x.transpose(0, 1).reshape(c["kv_heads"], -1, c["dim"])[:, :ctx + nodes] for x in (k, v))
        bias = torch.zeros(nodes, ctx + nodes, device="cuda", dtype=torch.float64)
        if s["mask"] is None:
            bias[:, ctx:] = torch.triu(torch.full((nodes, nodes), -math.inf, device="cuda", dtype=torch.float64), 1)
        else:
            words = s["mask"][b, :nodes].tolist()
            hidden = torch.tensor([[not (w >> j) & 1 for j in range(nodes)] for w in words], device="cuda")
            bias[:, ctx:].masked_fill_(hidden, -math.inf)
        for h in range(c["kv_heads"]):
            q = s["q"][b, :nodes, h * group:(h + 1) * group].double().transpose(0, 1)          # (group, nodes, dim)
            x = q @ k[h].t().contiguous() * s["scale"] + bias
            out[b, :nodes, h * group:(h + 1) * group] = (torch.softmax(x, -1) @ v[h]).transpose(0, 1)
            lse[b, :nodes, h * group:(h + 1) * group] = torch.logsumexp(x, -1).t()
    return {"out": out, "lse": lse}


def _exact_verify(c, s):
    accepted = torch.zeros(c["batch"], dtype=torch.int32)
    tokens = torch.full((c["batch"], c["drafts"] + 1), -1, dtype=torch.int64)
    drafted, chance, count = s["drafted"].tolist(), s["u"].double().tolist(), s["count"].tolist()
    for b in range(c["batch"]):
        n = 0
        for d in drafted[b][:count[b]]:
            if not chance[b][n] * (float(s["q"][b, n, d]) if s["q"] is not None else 1.0) < float(s["p"][b, n, d]):
                break
            tokens[b, n] = d
            n += 1
        w = s["p"][b, n].double()
        if n < count[b]:
            if s["q"] is not None:
                w = w - s["q"][b, n]
            else:
                w[drafted[b][n]] -= 1.0
            w = torch.where(w > 0, w, 0.0)
            w = w if w.any() else s["p"][b, n].double()
        run = torch.cumsum(w, 0)
        accepted[b] = n
        tokens[b, n] = torch.searchsorted(run, run[-1] * s["r"][b].double(), right=True)
    return {"accepted": accepted, "tokens": tokens}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(case, s)
    if case["op"] == "cache":
        return _exact_cache(case, s)
    if case["op"] == "attend":
        return _exact_attend(case, s)
    return _exact_verify(case, s)
