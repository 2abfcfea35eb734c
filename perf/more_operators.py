"""Cases and plain forms of windowed attention and of attention over a shared prefix.

Four operators that stand beside the library's packed and paged attention:

  window        packed prompts of different lengths, each query against the last
                `window` tokens up to its own and the first `sinks` tokens of
                its sequence
  window_grad   its backward pass
  window_chunk  a chunk of new tokens per sequence (single tokens too) over the
                paged cache, with the same window and first tokens; blocks that
                have left the window are gone from the block table
  shared        a chunk of new tokens per sequence over the paged cache where
                groups of sequences share the blocks of a long prefix

`run` computes them from elementary torch operations in 32 bits or, where `own`
is true, with the library's calls.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
BLOCK = 16                        # tokens per cache block


# ---------------------------------------------------------------- cases
def listed():
    return [
        # Many short prompts in one call, one token to 200 each, a narrow window and
        # no first tokens: latency counts.
        dict(name="window_short", op="window", seqs=32, longest=200, lens=1, heads=16,
             kv_heads=16, d=64, dtype="bf16", window=64, sinks=0),
        # A prefill batch of a model with local layers: eight prompts up to 8192.
        dict(name="window_prompts", op="window", seqs=8, longest=8192, lens=2, heads=32,
             kv_heads=8, d=128, dtype="bf16", window=1024, sinks=4),
        # One long prompt, one key/value head, a wide window that starts inside a
        # tile, a whole tile of first tokens.
        dict(name="window_long", op="window", seqs=1, longest=16384, lens=3, heads=8, kv_heads=1,
             d=128, dtype="fp16", window=4000, sinks=128),
        # Training on short packed documents, d = 64.
        dict(name="window_grad_short", op="window_grad", seqs=16, longest=1024, lens=4, heads=16,
             kv_heads=4, d=64, dtype="bf16", window=256, sinks=0),
        # Training on packed documents up to 8192 tokens, grouped heads.
        dict(name="window_grad", op="window_grad", seqs=4, longest=8192, lens=5, heads=16,
             kv_heads=4, d=128, dtype="bf16", window=1024, sinks=4),
        # One new token of each of a few sequences, a narrow window: the shortest call.
        dict(name="window_step_few", op="window_chunk", seqs=4, longest=1, lens=6, context=2000,
             heads=32, kv_heads=8, dtype="bf16", window=128, sinks=4),
        # A decode step of 64 sequences far into streams of text.
        dict(name="window_step", op="window_chunk", seqs=64, longest=1, lens=7, context=131072,
             heads=32, kv_heads=8, dtype="bf16", window=4096, sinks=4),
        # Chunks of long prompts.
        dict(name="window_chunk", op="window_chunk", seqs=4, longest=2048, lens=8, context=32768,
             heads=32, kv_heads=8, dtype="bf16", window=4096, sinks=64),
        # A handful of requests behind one system prompt.
        dict(name="shared_few", op="shared", groups=1, seqs=8, longest=1, lens=9, prefix=1000,
             context=64, heads=32, kv_heads=8, dtype="bf16"),
        # A decode step of 64 requests behind one long document.
        dict(name="shared_step", op="shared", groups=1, seqs=64, longest=1, lens=10, prefix=8192,
             context=512, heads=32, kv_heads=8, dtype="bf16"),
        # Drafted tokens of requests in five groups, each with a prefix of its own.
        dict(name="shared_groups", op="shared", groups=5, seqs=96, longest=4, lens=11,
             prefix=4096, context=300, heads=24, kv_heads=8, dtype="bf16"),
        # A large batch of sampled continuations of one very long context.
        dict(name="shared_large", op="shared", groups=1, seqs=256, longest=1, lens=12,
             prefix=32768, context=2048, heads=32, kv_heads=8, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["window", "window_grad", "window_chunk", "shared"])
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * min(rng.choice([1, 2, 3, 4, 5, 6, 7, 8]), 32 // kv)
    case = dict(op=op, lens=rng.randrange(1 << 20), heads=heads, kv_heads=kv, dtype="bf16")
    if op == "shared":
        prefix, context = _log(rng, 1, 32768), _log(rng, 1, 2048)
        seqs, longest = _log(rng, 2, 256), min(_log(rng, 1, 64), context)
        # scores of the plain form, as many as the largest listed case has
        seqs = max(2, min(seqs, (1 << 28) // (longest * heads * prefix)))
        return dict(case, groups=rng.randint(1, min(6, seqs)), seqs=seqs, longest=longest,
                    prefix=prefix, context=context)
    case.update(window=_log(rng, 8, 8192), sinks=rng.choice([0, 0, 1, 4, 16, 100, 300]))
    if op == "window_chunk":
        longest = 1 if rng.random() < 0.3 else _log(rng, 1, 2048)
        context = _log(rng, longest, 131072)
        room = (1 << 31) // (heads * longest * min(context, case["window"] + longest))
        return dict(case, longest=longest, context=context,
                    seqs=max(1, min(_log(rng, 1, 96), room)))
    longest = _log(rng, 1 if op == "window" else 16, 8192)
    # heads x longest^2 x sequences of the plain form's scores
    room = (1 << 33 if op == "window" else 1 << 31) // (heads * longest * longest)
    return dict(case, seqs=max(1, min(_log(rng, 1, 64), room)), longest=longest,
                d=rng.choice([64, 128]),
                dtype=rng.choice(["bf16", "fp16"]) if op == "window" else "bf16")


def _lengths(case):
    """Sequence lengths: one of the longest, the others spread over the
    logarithm of 1 .. longest, in a mixed order."""
    r = random.Random(case["lens"])
    n = [case["longest"]] + [_log(r, 1, case["longest"]) for _ in range(case["seqs"] - 1)]
    r.shuffle(n)
    return n


def _contexts(case, lens):
    """Context lengths (shared: behind the prefix), each at least its chunk,
    one of them the longest."""
    r = random.Random(case["lens"] + 1)
    ctx = [max(n, r.randint(1, case["context"])) for n in lens]
    ctx[r.randrange(len(ctx))] = case["context"]
    return ctx


def _groups(case):
    """First sequence of each group (and the end), and the prefixes' lengths."""
    r = random.Random(case["lens"] + 2)
    cuts = sorted(r.sample(range(1, case["seqs"]), case["groups"] - 1))
    prefix = [_log(r, 1, case["prefix"]) for _ in range(case["groups"])]
    prefix[r.randrange(case["groups"])] = case["prefix"]
    return [0] + cuts + [case["seqs"]], prefix


def _pairs(first, n, window, sinks):
    """Visible pairs of n queries at positions first, first + 1, ..."""
    return sum(min(p + 1, window) + max(0, min(sinks, p + 1 - window))
               for p in range(first, first + n))


def _seen(first, n, window, sinks):
    """Keys that some query at positions first .. first + n - 1 sees."""
    low = max(0, first - window + 1)
    return first + n - low + min(sinks, low)


def work(case):
    h, hk = case["heads"], case["kv_heads"]
    lens = _lengths(case)
    t = sum(lens)
    if case["op"] in ("window", "window_grad"):
        d = case["d"]
        pairs = sum(_pairs(0, n, case["window"], case["sinks"]) for n in lens)
        qb, kb = t * h * d * 2, t * hk * d * 2
        if case["op"] == "window":
            return dict(bytes=2 * qb + 2 * kb + 4 * t * h, flops=4 * pairs * h * d)
        return dict(bytes=4 * qb + 4 * kb + 4 * t * h, flops=10 * pairs * h * d)
    ctx = _contexts(case, lens)
    if case["op"] == "window_chunk":
        at = [(c - n, n, case["window"], case["sinks"]) for n, c in zip(lens, ctx)]
        pairs, keys = sum(_pairs(*x) for x in at), sum(_seen(*x) for x in at)
    else:
        first, prefix = _groups(case)
        keys = sum(prefix) + sum(ctx)
        pairs = sum(n * c - n * (n - 1) // 2 for n, c in zip(lens, ctx))
        pairs += sum(p * sum(lens[a:b]) for p, a, b in zip(prefix, first, first[1:]))
    return dict(bytes=2 * t * h * 128 * 2 + 2 * keys * hk * 128 * 2 + 4 * keys // BLOCK,
                flops=4 * pairs * h * 128)


# ---------------------------------------------------------------- inputs
def _normal(g, dtype, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _offsets(lens):
    return torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32)


def _cache(g, st, nb):
    hk = st["case"]["kv_heads"]
    st["kc"] = _normal(g, torch.bfloat16, nb, hk, 16, BLOCK, 8)
    st["vc"] = _normal(g, torch.bfloat16, nb, hk, 128, BLOCK)


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    h, hk = case["heads"], case["kv_heads"]
    st = dict(case=case)
    lens = _lengths(case)
    t = sum(lens)
    st["cu"] = _offsets(lens)
    if case["op"] in ("window", "window_grad"):
        d = case["d"]
        # one projection's output, queries, keys and values side by side
        qkv = _normal(g, dt, t, h + 2 * hk, d)
        st["q"], st["k"], st["v"] = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
        if case["op"] == "window_grad":
            st["o"], st["lse"] = _window(st)
            st["do"] = _normal(g, dt, t, h, d)
        return st
    ctx = _contexts(case, lens)
    st["q"] = _normal(g, dt, t, h, 128)
    if case["op"] == "window_chunk":
        # Live blocks: those of the first tokens and those that the chunk's first
        # query still sees; the others have been given back.
        live = []
        for n, c in zip(lens, ctx):
            low = max(0, c - n - case["window"] + 1) // BLOCK
            keep = list(range(min(low, _blocks(min(case["sinks"], c)))))
            live.append(keep + list(range(low, _blocks(c))))
        nb = sum(len(x) for x in live) + 8
        _cache(g, st, nb)
        free = torch.randperm(nb, generator=g, device=DEV).int()
        st["bt"] = torch.full((len(lens), _blocks(max(ctx))), -1, device=DEV, dtype=torch.int32)
        at = 0
        for s, x in enumerate(live):
            st["bt"][s, torch.tensor(x, device=DEV)] = free[at:at + len(x)]
            at += len(x)
        st["ctx"] = torch.tensor(ctx, device=DEV, dtype=torch.int32)
        return st
    first, prefix = _groups(case)
    of = [i for i, (a, b) in enumerate(zip(first, first[1:])) for _ in range(a, b)]
    total = [prefix[i] + c for i, c in zip(of, ctx)]
    shared = [p // BLOCK for p in prefix]          # whole blocks of each prefix
    nb = sum(shared) + sum(_blocks(c) - shared[i] for i, c in zip(of, total)) + 8
    _cache(g, st, nb)
    free = torch.randperm(nb, generator=g, device=DEV).int()
    st["bt"] = torch.zeros((len(lens), _blocks(max(total))), device=DEV, dtype=torch.int32)
    at = 0
    for i, n in enumerate(shared):
        st["bt"][first[i]:first[i + 1], :n] = free[at:at + n]
        at += n
    for s, (i, c) in enumerate(zip(of, total)):
        n = _blocks(c) - shared[i]
        st["bt"][s, shared[i]:shared[i] + n] = free[at:at + n]
        at += n
    st["ctx"] = torch.tensor(total, device=DEV, dtype=torch.int32)
    st["groups"] = torch.tensor(first, device=DEV, dtype=torch.int32)
    st["prefix"] = torch.tensor(prefix, device=DEV, dtype=torch.int32)
    return st


# ---------------------------------------------------------------- one pass
def run(st):
    if own:
        return _run_own(st)
    return dict(window=_window, window_grad=_window_grad, window_chunk=_window_chunk,
                shared=_shared)[st["case"]["op"]](st)


def _run_own(st):
    import exact_attention_11_gb300 as fa
    case = st["case"]
    if case["op"] == "window":
        return fa.forward_packed_window(st["q"], st["k"], st["v"], st["cu"], case["window"],
                                        case["sinks"])
    if case["op"] == "window_grad":
        return fa.backward_packed_window(st["q"], st["k"], st["v"], st["o"], st["lse"], st["do"],
                                         st["cu"], case["window"], case["sinks"])
    if case["op"] == "window_chunk":
        return fa.paged_prefill_window(st["q"], st["kc"], st["vc"], st["bt"], st["ctx"], st["cu"],
                                       case["window"], case["sinks"])
    return fa.paged_prefill_shared(st["q"], st["kc"], st["vc"], st["bt"], st["ctx"], st["cu"],
                                   st["groups"], st["prefix"])


# ---------------------------------------------------------------- plain forms
def _heads(x, h):
    return x.repeat_interleave(h // x.shape[-3], dim=-3)


def _scores(q, k, see):
    """Scaled scores of q [.., n, d] and k [.., m, d], -inf where `see` is false."""
    s = (q @ k.transpose(-1, -2)) * q.shape[-1] ** -0.5
    return s.masked_fill_(~see, -math.inf)


def _softmax(s):
    """Weights, their sum and the log-sum-exp of each row; all 0 (and -inf) for a
    row that sees nothing."""
    m = s.amax(-1, keepdim=True)
    p = (s - m.clamp(min=torch.finfo(torch.float32).min)).exp_()
    l = p.sum(-1, keepdim=True)
    return p, l, (m + l.log()).squeeze(-1)


def _near(p, j, case):
    """Whether a query at position p sees key j."""
    return (j <= p) & ((j > p - case["window"]) | (j < case["sinks"]))


def _window(st):
    case = st["case"]
    t, h, d = st["q"].shape
    o = torch.empty(t, h, d, dtype=st["q"].dtype, device=DEV)
    lse = torch.empty(h, t, device=DEV)
    at = 0
    for n in _lengths(case):
        rows = slice(at, at + n)
        at += n
        i = torch.arange(n, device=DEV)
        q, k, v = (st[x][rows].float().transpose(0, 1) for x in "qkv")
        p, l, e = _softmax(_scores(q, _heads(k, h), _near(i[:, None], i, case)))
        o[rows] = ((p @ _heads(v, h)) / l).transpose(0, 1).to(o.dtype)
        lse[:, rows] = e
    return o, lse


def _window_grad(st):
    case = st["case"]
    t, h, d = st["q"].shape
    hk = case["kv_heads"]
    scale = d ** -0.5
    grads = [torch.empty_like(st[x], memory_format=torch.contiguous_format) for x in "qkv"]
    at = 0
    for n in _lengths(case):
        rows = slice(at, at + n)
        at += n
        i = torch.arange(n, device=DEV)
        q, k, v, o, do = (st[x][rows].float().transpose(0, 1) for x in ("q", "k", "v", "o", "do"))
        k, v = _heads(k, h), _heads(v, h)
        p = _scores(q, k, _near(i[:, None], i, case)).sub_(st["lse"][:, rows, None]).exp_()
        dv = p.transpose(-1, -2) @ do
        ds = (do @ v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
        dq = (ds @ k) * scale
        dk = (ds.transpose(-1, -2) @ q) * scale
        dk, dv = (x.unflatten(0, (hk, h // hk)).sum(1) for x in (dk, dv))
        for g, x in zip(grads, (dq, dk, dv)):
            g[rows] = x.transpose(0, 1).to(g.dtype)
    return tuple(grads)


def _rows(st):
    """Queries of each sequence side by side, [S, H, longest, d] in 32 bits (rows
    past a chunk's end repeat some other row), the numbers of new tokens
    [S, 1, 1, 1], and the place of each packed row."""
    cu, n = st["cu"].long(), st["case"]["longest"]
    at = cu[:-1, None] + torch.arange(n, device=DEV)
    q = st["q"][at.clamp(max=st["q"].shape[0] - 1)].float().transpose(1, 2)
    row = torch.arange(st["q"].shape[0], device=DEV)
    seq = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    return q, (cu[1:] - cu[:-1])[:, None, None, None], seq, row - cu[seq]


def _gather(st, table):
    """Keys and values of the blocks in table [.., blocks], in 32 bits:
    [.., Hk, tokens, d]."""
    b = table.long().clamp(min=0)
    k = st["kc"][b].float().movedim(-4, -5)          # [.., Hk, blocks, d/8, 16, 8]
    v = st["vc"][b].float().movedim(-3, -4)          # [.., Hk, blocks, d, 16]
    return (k.transpose(-3, -2).flatten(-2).flatten(-3, -2), v.transpose(-2, -1).flatten(-3, -2))


def _window_chunk(st):
    case = st["case"]
    h = case["heads"]
    q, lens, seq, pos = _rows(st)
    ctx = st["ctx"].long()[:, None, None, None]
    # Blocks of the first tokens, then of the window of the chunk's first query.
    ns = _blocks(case["sinks"])
    low = (ctx - lens - case["window"] + 1).clamp(min=0).flatten() // BLOCK
    most = (case["window"] + case["longest"]) // BLOCK + 2
    blk = torch.cat([torch.arange(ns, device=DEV).expand(low.shape[0], ns),
                     low[:, None] + torch.arange(most, device=DEV)], 1)
    # (a block of both is counted once, and a block past the table not at all)
    twice = torch.arange(ns + most, device=DEV) >= ns
    there = (blk < st["bt"].shape[1]) & ~(twice & (blk < ns))
    k, v = _gather(st, st["bt"].gather(1, blk.clamp(max=st["bt"].shape[1] - 1)))
    j = (blk[:, :, None] * BLOCK + torch.arange(BLOCK, device=DEV)).flatten(1)[:, None, None, :]
    p = ctx - lens + torch.arange(case["longest"], device=DEV)[:, None]
    see = _near(p, j, case) & (j < ctx) & there.repeat_interleave(BLOCK, 1)[:, None, None, :]
    w, l, _ = _softmax(_scores(q, _heads(k, h), see))
    return ((w @ _heads(v, h)) / l)[seq, :, pos].to(st["q"].dtype)


def _shared(st):
    case = st["case"]
    h, n = case["heads"], case["longest"]
    q, lens, seq, pos = _rows(st)
    first, prefix = _groups(case)
    whole = torch.tensor([p // BLOCK for p in prefix], device=DEV)
    sizes = torch.tensor([b - a for a, b in zip(first, first[1:])], device=DEV)
    skip = whole.repeat_interleave(sizes)            # blocks of each sequence's prefix
    # Each sequence's own blocks.
    own_blocks = _blocks(max(_contexts(case, _lengths(case))) + BLOCK - 1)
    blk = skip[:, None] + torch.arange(own_blocks, device=DEV)
    k, v = _gather(st, st["bt"].gather(1, blk.clamp(max=st["bt"].shape[1] - 1)))
    j = (blk[:, :, None] * BLOCK + torch.arange(BLOCK, device=DEV)).flatten(1)[:, None, None, :]
    ctx = st["ctx"].long()[:, None, None, None]
    p = torch.minimum(ctx - lens + torch.arange(n, device=DEV)[:, None], ctx - 1)
    s = _scores(q, _heads(k, h), j <= p)
    v = _heads(v, h)
    out = []
    for a, b, w in zip(first, first[1:], whole.tolist()):
        # The prefix's scores, all rows of the group against one set of keys.
        kp, vp = (_heads(x, h) for x in _gather(st, st["bt"][a, :w]))
        rows = q[a:b].transpose(0, 1).flatten(1, 2)                       # [H, rows, d]
        sp = (rows @ kp.transpose(-1, -2)) * 128 ** -0.5
        so = s[a:b].transpose(0, 1).flatten(1, 2)
        e, l, _ = _softmax(torch.cat([sp, so], -1))
        o = e[..., :w * BLOCK] @ vp
        o = o.unflatten(1, (b - a, n)).transpose(0, 1)
        own_e = e[..., w * BLOCK:].unflatten(1, (b - a, n)).transpose(0, 1)
        out.append((o + own_e @ v[a:b]) / l.unflatten(1, (b - a, n)).transpose(0, 1))
    return torch.cat(out)[seq, :, pos].to(st["q"].dtype)


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("window", "window_grad"):
        return _exact_packed(case, st)
    return _exact_paged(case, st)


def _parts(first, n, case, step=512):
    """Runs of at most `step` queries of positions first .. first + n - 1: their
    places in the chunk, the keys that any of them sees, and which see which."""
    for a in range(0, n, step):
        b = min(a + step, n)
        low = max(0, first + a - case["window"] + 1)
        keys = torch.cat([torch.arange(min(case["sinks"], low), device=DEV),
                          torch.arange(low, first + b, device=DEV)])
        back = torch.arange(first + a, first + b, device=DEV)[:, None] - keys
        yield slice(a, b), keys, (back >= 0) & ((back < case["window"]) | (keys < case["sinks"]))


def _attend64(q, k, v, see):
    """q [n, H, d], k and v [m, Hk, d], see [n, m]: output [n, H, d], log-sum-exp
    [H, n], weights [Hk, H / Hk, n, m]."""
    hk = k.shape[1]
    s = torch.einsum("nkgd,mkd->kgnm", q.unflatten(1, (hk, -1)), k) / math.sqrt(q.shape[-1])
    s.masked_fill_(~see, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = s.sub_(lse[..., None]).exp_()
    return torch.einsum("kgnm,mkd->nkgd", p, v).flatten(1, 2), lse.flatten(0, 1), p


def _exact_packed(case, st):
    grad, hk = case["op"] == "window_grad", case["kv_heads"]
    outs, at = [], 0
    for n in _lengths(case):
        q, k, v = (st[x][at:at + n].double() for x in "qkv")
        if grad:
            do = st["do"][at:at + n].double().unflatten(1, (hk, -1))
            dk, dv = torch.zeros_like(k), torch.zeros_like(v)
        rows = []
        at += n
        for part, keys, see in _parts(0, n, case):
            o, lse, p = _attend64(q[part], k[keys], v[keys], see)
            if not grad:
                rows.append((o, lse.t()))
                continue
            dp = torch.einsum("nkgd,mkd->kgnm", do[part], v[keys])
            ds = p * (dp - (dp * p).sum(-1, keepdim=True)) / math.sqrt(case["d"])
            rows.append((torch.einsum("kgnm,mkd->nkgd", ds, k[keys]).flatten(1, 2),))
            dk.index_add_(0, keys, torch.einsum("kgnm,nkgd->mkd", ds,
                                                q[part].unflatten(1, (hk, -1))))
            dv.index_add_(0, keys, torch.einsum("kgnm,nkgd->mkd", p, do[part]))
        rows = [torch.cat(x) for x in zip(*rows)]
        outs.append((rows[0], dk, dv) if grad else rows)
    outs = [torch.cat(x) for x in zip(*outs)]
    return tuple(outs) if grad else (outs[0], outs[1].t().contiguous())


def _exact_paged(case, st):
    wide = dict(window=1 << 40, sinks=0)
    at, outs = 0, []
    lens, ctx = _lengths(case), st["ctx"].tolist()
    for s, (n, c) in enumerate(zip(lens, ctx)):
        q = st["q"][at:at + n].double()
        at += n
        for part, keys, see in _parts(c - n, n, wide if case["op"] == "shared" else case):
            blk, off = st["bt"][s].long()[keys // BLOCK], keys % BLOCK
            k = st["kc"][blk, :, :, off].flatten(2).double()
            outs.append(_attend64(q[part], k, st["vc"][blk, :, :, off].double(), see)[0])
    return torch.cat(outs)
