"""Cases and plain forms of the packed-prompt, paged-chunk and query/key preparation operators.

Three operators (and the backward passes of two) that stand before and around
the library's attention calls in a model's layer:

  prep          RMS norm of the queries and keys of each head and the rotary
                position embedding, in one pass; into dense tensors (training)
                or with the keys and values written into the paged cache
                (serving); and its backward pass
  packed        attention over whole prompts of different lengths packed into
                one tensor, grouped key/value heads, causal or not; and its
                backward pass
  chunk         attention of a chunk of new tokens per sequence over the paged
                cache that already holds them and what came before

`run` computes them from elementary torch operations in 32 bits (angles in 64)
or, where `own` is true, with the library's calls.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BLOCK = 16                        # tokens per cache block


# ---------------------------------------------------------------- cases
def listed():
    return [
        # One new token of each of 64 sequences, far into long contexts: what a
        # decode step does before the paged decode.  Latency counts.
        dict(name="prep_step", op="prep", form="cache", tokens=64, heads=32, kv_heads=8, d=128,
             rot=128, layout="half", dtype="bf16", norm=True, far=131072, spread=1),
        # The prompt tokens of seven sequences, an odd count, half of each head
        # rotated, written into the cache.
        dict(name="prep_prompt", op="prep", form="cache", tokens=4099, heads=32, kv_heads=8,
             d=128, rot=64, layout="half", dtype="bf16", norm=True, far=4096, spread=0),
        # A training batch's queries and keys, interleaved pairs, fp16.
        dict(name="prep_train", op="prep", form="dense", tokens=16384, heads=16, kv_heads=16,
             d=64, rot=64, layout="pairs", dtype="fp16", norm=True, far=4096, spread=0),
        # Its gradient on grouped heads, with the norm weights' gradients.
        dict(name="prep_grad", op="prep", form="grad", tokens=8192, heads=32, kv_heads=8, d=128,
             rot=128, layout="half", dtype="bf16", norm=True, far=4096, spread=0),
        # A short fp32 batch's gradient (a test-size step).
        dict(name="prep_grad_small", op="prep", form="grad", tokens=257, heads=16, kv_heads=4,
             d=64, rot=32, layout="pairs", dtype="fp32", norm=True, far=1024, spread=0),
        # Many short prompts in one call, one token to 200 each.
        dict(name="packed_short", op="packed", form="forward", seqs=32, longest=200, lens=1,
             heads=16, kv_heads=16, d=64, dtype="bf16", causal=True),
        # An ordinary prefill batch: eight prompts up to 4096 tokens.
        dict(name="packed_prompts", op="packed", form="forward", seqs=8, longest=4096, lens=2,
             heads=32, kv_heads=8, d=128, dtype="bf16", causal=True),
        # One long prompt, one key/value head for all queries.
        dict(name="packed_long", op="packed", form="forward", seqs=1, longest=16384, lens=3,
             heads=8, kv_heads=1, d=128, dtype="fp16", causal=True),
        # Training on packed documents, d = 64, not causal (an encoder's step).
        dict(name="packed_grad_short", op="packed", form="grad", seqs=16, longest=1024, lens=4,
             heads=16, kv_heads=4, d=64, dtype="bf16", causal=False),
        # Training on packed documents up to 4096 tokens, causal, grouped heads.
        dict(name="packed_grad", op="packed", form="grad", seqs=4, longest=4096, lens=5,
             heads=16, kv_heads=4, d=128, dtype="bf16", causal=True),
        # A few drafted tokens of each sequence checked against long contexts:
        # few rows, memory bound.
        dict(name="chunk_draft", op="chunk", seqs=16, longest=6, lens=6, context=4096, heads=32,
             kv_heads=8, dtype="bf16"),
        # Chunks of long prompts prefilled over what the cache already holds.
        dict(name="chunk_prefill", op="chunk", seqs=4, longest=1024, lens=7, context=16384,
             heads=32, kv_heads=8, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prep", "packed", "chunk"])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    if op == "prep":
        form = rng.choice(["cache", "dense", "grad"])
        d = 128 if form == "cache" else rng.choice([64, 128, 256])
        group = min(group, 32 // kv)
        most = 8192 * 40 * 128 // (kv * (group + 1) * d)
        return dict(op=op, form=form, tokens=_log(rng, 1, min(16384, most)), heads=kv * group,
                    kv_heads=kv, d=d, rot=rng.choice([0, d // 4, d // 2, d]),
                    layout=rng.choice(["half", "pairs"]),
                    dtype="bf16" if form == "cache" else rng.choice(["bf16", "fp16", "fp32"]),
                    norm=rng.random() < 0.8, far=_log(rng, 1024, 1 << 20),
                    spread=rng.choice([0, 1]))
    if op == "packed":
        form = rng.choice(["forward", "grad"])
        group = min(group, 32 // kv)
        longest = _log(rng, 1, 4096)
        seqs = _log(rng, 1, 64)
        # the largest listed case of the form has heads x longest^2 x sequences
        # of 2^32 (forward) and 2^30 (gradient)
        room = (1 << 32 if form == "forward" else 1 << 30) // (kv * group * longest * longest)
        seqs = max(1, min(seqs, room))
        return dict(op=op, form=form, seqs=seqs, longest=longest, lens=rng.randrange(1 << 20),
                    heads=kv * group, kv_heads=kv, d=rng.choice([64, 128]),
                    dtype="bf16" if form == "grad" else rng.choice(["bf16", "fp16"]),
                    causal=rng.random() < 0.7)
    group = min(group, 32 // kv)
    longest = _log(rng, 1, 1024)
    context = _log(rng, longest, 16384)
    seqs = max(1, min(_log(rng, 1, 32), (1 << 31) // (kv * group * longest * context)))
    return dict(op=op, seqs=seqs, longest=longest, lens=rng.randrange(1 << 20), context=context,
                heads=kv * group, kv_heads=kv, dtype="bf16")


def _lengths(case):
    """Sequence lengths: one of the longest, the others spread over the
    logarithm of 1 .. longest, in a mixed order."""
    r = random.Random(case["lens"])
    n = [case["longest"]] + [_log(r, 1, case["longest"]) for _ in range(case["seqs"] - 1)]
    r.shuffle(n)
    return n


def _contexts(case, lens):
    """Context lengths, each at least its chunk, one of them the longest."""
    r = random.Random(case["lens"] + 1)
    ctx = [max(n, r.randint(1, case["context"])) for n in lens]
    ctx[r.randrange(len(ctx))] = case["context"]
    return ctx


def work(case):
    es = 4 if case["dtype"] == "fp32" else 2
    h, hk = case["heads"], case["kv_heads"]
    if case["op"] == "prep":
        d, t = case["d"], case["tokens"]
        qk = t * (h + hk) * d
        if case["form"] == "dense":
            return dict(bytes=2 * qk * es + t * 4, flops=10 * qk)
        if case["form"] == "cache":   # q, k, v in; q, k, v out
            return dict(bytes=2 * (qk + t * hk * d) * es + t * 12, flops=10 * qk)
        return dict(bytes=3 * qk * es + t * 4 + 2 * d * 4, flops=24 * qk)
    if case["op"] == "packed":
        d, lens = case["d"], _lengths(case)
        t = sum(lens)
        pairs = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in lens)
        qb, kb = t * h * d * es, t * hk * d * es
        if case["form"] == "forward":
            return dict(bytes=2 * qb + 2 * kb + 4 * t * h, flops=4 * pairs * h * d)
        return dict(bytes=4 * qb + 4 * kb + 4 * t * h, flops=10 * pairs * h * d)
    lens = _lengths(case)
    ctx = _contexts(case, lens)
    pairs = sum(n * c - n * (n - 1) // 2 for n, c in zip(lens, ctx))
    return dict(bytes=2 * sum(lens) * h * 128 * 2 + 2 * sum(ctx) * hk * 128 * 2
                + 4 * sum((c + BLOCK - 1) // BLOCK for c in ctx), flops=4 * pairs * h * 128)


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, dtype, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _frequencies(rot):
    """Rotary frequencies in 64 bits, base 10000."""
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    return 10000.0 ** (-2.0 * i / max(rot, 1))


def _offsets(lens):
    return torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]
    h, hk = case["heads"], case["kv_heads"]
    st = dict(case=case)
    if case["op"] == "prep":
        t, d = case["tokens"], case["d"]
        # one projection's output, queries, keys and values side by side
        qkv = _normal(g, dt, t, h + 2 * hk, d)
        st["q"], st["k"], st["v"] = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
        if case["spread"]:    # one token of each sequence, each at its own position
            st["pos"] = torch.randint(0, case["far"], (t,), generator=g, device=DEV).int()
        else:                 # runs of tokens of a few sequences
            run_len = max(1, t // 7)
            st["pos"] = (torch.arange(t, device=DEV) % run_len % case["far"]).int()
        st["freq"] = _frequencies(case["rot"])
        if case["norm"]:
            st["qw"] = (1 + 0.2 * _normal(g, torch.float32, d)).to(dt)
            st["kw"] = (1 + 0.2 * _normal(g, torch.float32, d)).to(dt)
        else:
            st["qw"] = st["kw"] = None
        if case["form"] == "cache":
            nb = max(1024, 2 * (t + BLOCK - 1) // BLOCK + 8)
            # what other tokens left there stays as it is
            st["kc"] = _normal(g, dt, nb, hk, d // 8, BLOCK, 8)
            st["vc"] = _normal(g, dt, nb, hk, d, BLOCK)
            if case["spread"]:    # each token in a block of its own
                blocks = torch.randperm(nb, generator=g, device=DEV)
                at = torch.arange(t, device=DEV)
                if t <= nb:
                    slots = blocks[at] * BLOCK + st["pos"] % BLOCK
                else:
                    slots = blocks[at // BLOCK] * BLOCK + at % BLOCK
            else:                 # runs fill scattered blocks in order
                blocks = torch.randperm(nb, generator=g, device=DEV)
                at = torch.arange(t, device=DEV) + 5
                slots = blocks[at // BLOCK] * BLOCK + at % BLOCK
            st["slots"] = slots.long()
        if case["form"] == "grad":
            st["dq"] = _normal(g, dt, t, h, d)
            st["dk"] = _normal(g, dt, t, hk, d)
        return st
    lens = _lengths(case)
    t = sum(lens)
    st["cu"] = _offsets(lens)
    if case["op"] == "packed":
        d = case["d"]
        qkv = _normal(g, dt, t, h + 2 * hk, d)
        st["q"], st["k"], st["v"] = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
        if case["form"] == "grad":
            st["o"], st["lse"] = _packed_forward(st)
            st["do"] = _normal(g, dt, t, h, d)
        return st
    ctx = _contexts(case, lens)
    mb = (max(ctx) + BLOCK - 1) // BLOCK
    nb = len(lens) * mb
    st["q"] = _normal(g, dt, t, h, 128)
    st["kc"] = _normal(g, dt, nb, hk, 16, BLOCK, 8)
    st["vc"] = _normal(g, dt, nb, hk, 128, BLOCK)
    st["bt"] = torch.randperm(nb, generator=g, device=DEV).view(len(lens), mb).int()
    st["ctx"] = torch.tensor(ctx, device=DEV, dtype=torch.int32)
    return st


# ---------------------------------------------------------------- one pass
def run(st):
    case = st["case"]
    if own:
        return _run_own(st)
    if case["op"] == "prep":
        if case["form"] == "grad":
            return _prep_grad(st)
        q, k = _prep(st, st["q"], st["qw"]), _prep(st, st["k"], st["kw"])
        if case["form"] == "dense":
            return q, k
        blk, off = st["slots"] // BLOCK, st["slots"] % BLOCK
        st["kc"][blk, :, :, off] = k.view(k.shape[0], k.shape[1], -1, 8)
        st["vc"][blk, :, :, off] = st["v"]
        return q, st["kc"], st["vc"]
    if case["op"] == "packed":
        return _packed_forward(st) if case["form"] == "forward" else _packed_grad(st)
    return _chunk(st)


def _run_own(st):
    import exact_attention_11_gb300 as fa
    case = st["case"]
    if case["op"] == "prep":
        pairs = case["layout"] == "pairs"
        if case["form"] == "dense":
            return fa.qk_norm_rope(st["q"], st["k"], st["pos"], st["freq"], st["qw"], st["kw"],
                                   interleaved=pairs)
        if case["form"] == "cache":
            q = fa.qk_norm_rope_cache(st["q"], st["k"], st["v"], st["pos"], st["freq"],
                                      st["slots"], st["kc"], st["vc"], st["qw"], st["kw"],
                                      interleaved=pairs)
            return q, st["kc"], st["vc"]
        return fa.qk_norm_rope_backward(st["dq"], st["dk"], st["q"], st["k"], st["pos"],
                                        st["freq"], st["qw"], st["kw"], interleaved=pairs)
    if case["op"] == "packed":
        if case["form"] == "forward":
            return fa.forward_packed(st["q"], st["k"], st["v"], st["cu"], causal=case["causal"])
        return fa.backward_packed(st["q"], st["k"], st["v"], st["o"], st["lse"], st["do"],
                                  st["cu"], causal=case["causal"])
    return fa.paged_prefill(st["q"], st["kc"], st["vc"], st["bt"], st["ctx"], st["cu"])


# ---------------------------------------------------------------- plain forms
EPS = 1e-6


def _angles(st):
    a = st["pos"].double()[:, None, None] * st["freq"]
    return a.cos().float(), a.sin().float()


def _split(x, case):
    """The two members of each rotated pair, and the rest of the head."""
    r = case["rot"]
    if case["layout"] == "pairs":
        return x[..., 0:r:2], x[..., 1:r:2], x[..., r:]
    return x[..., :r // 2], x[..., r // 2:r], x[..., r:]


def _join(a, b, rest, case):
    if case["layout"] == "pairs":
        return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)
    return torch.cat([a, b, rest], -1)


def _prep(st, x, w):
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w.float()
    c, s = _angles(st)
    a, b, rest = _split(y, st["case"])
    return _join(a * c - b * s, b * c + a * s, rest, st["case"]).to(x.dtype)


def _prep_grad(st):
    c, s = _angles(st)
    case = st["case"]

    def one(dy, x, w):
        a, b, rest = _split(dy.float(), case)
        g = _join(a * c + b * s, b * c - a * s, rest, case)
        if w is None:
            return g.to(x.dtype), None
        y, wf = x.float(), w.float()
        r = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS)
        gw = g * wf
        dx = r * (gw - y * r * r * (gw * y).mean(-1, keepdim=True))
        return dx.to(x.dtype), (g * y * r).sum((0, 1))

    dq, dqw = one(st["dq"], st["q"], st["qw"])
    dk, dkw = one(st["dk"], st["k"], st["kw"])
    return dq, dk, dqw, dkw


def _padded(x, cu, longest):
    """[T, H, d] -> fp32 [S, H, longest, d]; rows past a sequence's end repeat
    some other row and are masked by the callers."""
    at = cu[:-1, None].long() + torch.arange(longest, device=DEV)
    return x[at.clamp(max=x.shape[0] - 1)].float().transpose(1, 2)


def _places(cu, t):
    """Sequence and position of each packed row."""
    row = torch.arange(t, device=DEV, dtype=torch.int32)
    seq = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    return seq, row.long() - cu.long()[seq]


def _heads(x, h):
    return x.repeat_interleave(h // x.shape[1], dim=1)


def _visible(st):
    case, n = st["case"], st["case"]["longest"]
    i = torch.arange(n, device=DEV)
    lens = (st["cu"][1:] - st["cu"][:-1])[:, None, None, None]
    see = (i[None, :] < lens) & (i[:, None] < lens)
    return see & (i[None, :] <= i[:, None]) if case["causal"] else see


def _packed_forward(st):
    case = st["case"]
    t, h, d = st["q"].shape
    q = _padded(st["q"], st["cu"], case["longest"])
    k = _heads(_padded(st["k"], st["cu"], case["longest"]), h)
    v = _heads(_padded(st["v"], st["cu"], case["longest"]), h)
    s = (q @ k.transpose(-1, -2)) * d ** -0.5
    s = s.masked_fill_(~_visible(st), -math.inf)
    m = s.amax(-1, keepdim=True)
    p = (s - m).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p @ v) / l
    lse = (m + l.log()).squeeze(-1)
    seq, pos = _places(st["cu"], t)
    return o[seq, :, pos].to(st["q"].dtype), lse[seq, :, pos].t().contiguous()


def _packed_grad(st):
    case = st["case"]
    t, h, d = st["q"].shape
    hk = case["kv_heads"]
    n = case["longest"]
    q, do, o = (_padded(st[x], st["cu"], n) for x in ("q", "do", "o"))
    k = _heads(_padded(st["k"], st["cu"], n), h)
    v = _heads(_padded(st["v"], st["cu"], n), h)
    lse = _padded(st["lse"].t()[:, :, None], st["cu"], n)
    scale = d ** -0.5
    p = ((q @ k.transpose(-1, -2)) * scale - lse).exp_()
    p = p.masked_fill_(~_visible(st), 0.0)
    dv = p.transpose(-1, -2) @ do
    ds = (do @ v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    dq = (ds @ k) * scale
    dk = (ds.transpose(-1, -2) @ q) * scale
    dk, dv = (x.unflatten(1, (hk, h // hk)).sum(2) for x in (dk, dv))
    seq, pos = _places(st["cu"], t)
    return tuple(x[seq, :, pos].to(st["q"].dtype) for x in (dq, dk, dv))


def _chunk(st):
    case = st["case"]
    t, h, d = st["q"].shape
    s_, mb = st["bt"].shape
    bt = st["bt"].long()
    # [S, blocks, Hk, d/8, 16, 8] -> [S, Hk, tokens, d]
    k = st["kc"][bt].permute(0, 2, 1, 4, 3, 5).reshape(s_, -1, mb * BLOCK, d).float()
    v = st["vc"][bt].permute(0, 2, 1, 4, 3).reshape(s_, -1, mb * BLOCK, d).float()
    n = case["longest"]
    q = _padded(st["q"], st["cu"], n)
    lens = (st["cu"][1:] - st["cu"][:-1])[:, None, None, None]
    ctx = st["ctx"][:, None, None, None]
    last = ctx - lens + torch.arange(n, device=DEV)[:, None]
    see = torch.arange(mb * BLOCK, device=DEV) <= torch.minimum(last, ctx - 1)
    s = (q @ _heads(k, h).transpose(-1, -2)) * d ** -0.5
    s = s.masked_fill_(~see, -math.inf)
    p = (s - s.amax(-1, keepdim=True)).exp_()
    o = (p @ _heads(v, h)) / p.sum(-1, keepdim=True)
    seq, pos = _places(st["cu"], t)
    return o[seq, :, pos].to(st["q"].dtype)


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "prep":
        return _exact_prep(case, st)
    if case["op"] == "packed":
        return _exact_packed(case, st)
    return _exact_chunk(case, st)


def _rotation(case, st, sign):
    """A complex factor for every token and pair."""
    theta = sign * st["pos"].double().outer(st["freq"])
    return torch.polar(torch.ones_like(theta), theta)[:, None, :]


def _rotate64(x, case, factor):
    r = case["rot"]
    x = x.clone()
    even = slice(0, r, 2) if case["layout"] == "pairs" else slice(0, r // 2)
    odd = slice(1, r, 2) if case["layout"] == "pairs" else slice(r // 2, r)
    z = torch.complex(x[..., even].contiguous(), x[..., odd].contiguous()) * factor
    x[..., even], x[..., odd] = z.real, z.imag
    return x


def _exact_prep(case, st):
    turn = _rotation(case, st, 1.0)
    if case["form"] == "grad":
        back = _rotation(case, st, -1.0)
        out = []
        for x, dy, w in ((st["q"], st["dq"], st["qw"]), (st["k"], st["dk"], st["kw"])):
            g = _rotate64(dy.double(), case, back)
            if w is None:
                out.append((g, None))
                continue
            # y = w x / n with n = sqrt(mean x^2 + eps): dx = (w g - xh <w g, xh> / d) / n
            # where xh = x / n, and dw sums g xh
            x64 = x.double()
            n = ((x64 ** 2).sum(-1, keepdim=True) / case["d"] + EPS).sqrt()
            xh = x64 / n
            wg = w.double() * g
            out.append(((wg - xh * (wg * xh).sum(-1, keepdim=True) / case["d"]) / n,
                        torch.einsum("thd,thd->d", g, xh)))
        return out[0][0], out[1][0], out[0][1], out[1][1]

    def one(x, w):
        y = x.double()
        if w is not None:
            y = y / ((y ** 2).sum(-1, keepdim=True) / case["d"] + EPS).sqrt() * w.double()
        return _rotate64(y, case, turn)

    q, k = one(st["q"], st["qw"]), one(st["k"], st["kw"])
    if case["form"] == "dense":
        return q, k
    kc, vc = st["kc"].double(), st["vc"].double()
    nb, hk = kc.shape[:2]
    # flat index of (slot, head, c) in each cache
    blk, off = st["slots"] // BLOCK, st["slots"] % BLOCK
    c = torch.arange(128, device=DEV)
    head = (blk[:, None] * hk + torch.arange(hk, device=DEV))[:, :, None] * 128 * BLOCK
    kc.view(-1)[head + (c // 8 * BLOCK + off[:, None, None]) * 8 + c % 8] = k
    vc.view(-1)[head + c * BLOCK + off[:, None, None]] = st["v"].double()
    return q, kc, vc


def _softmax64(q, k, v, see):
    """q [H, n, d], k and v [Hk, m, d], see [n, m]: output, log-sum-exp, weights."""
    g = q.shape[0] // k.shape[0]
    s = torch.einsum("kgnd,kmd->kgnm", q.unflatten(0, (-1, g)), k) / math.sqrt(q.shape[-1])
    s = torch.where(see, s, torch.tensor(-math.inf, dtype=torch.float64, device=DEV))
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[..., None])
    return torch.einsum("kgnm,kmd->kgnd", p, v).flatten(0, 1), lse.flatten(0, 1), p


def _exact_packed(case, st):
    lens, at = _lengths(case), 0
    outs = []
    for n in lens:
        rows = slice(at, at + n)
        at += n
        i = torch.arange(n, device=DEV)
        see = i[:, None] >= i[None, :] if case["causal"] else torch.ones(n, n, device=DEV) > 0
        q, k, v = (st[x][rows].double().transpose(0, 1) for x in "qkv")
        if case["form"] == "forward":
            # head by key/value head, to bound the memory
            g = case["heads"] // case["kv_heads"]
            parts = [_softmax64(q[j * g:j * g + g], k[j:j + 1], v[j:j + 1], see)[:2]
                     for j in range(case["kv_heads"])]
            outs.append((torch.cat([p[0] for p in parts]).transpose(0, 1),
                         torch.cat([p[1] for p in parts])))
            continue
        do = st["do"][rows].double().transpose(0, 1)
        g = case["heads"] // case["kv_heads"]
        scale = 1 / math.sqrt(case["d"])
        dq, dk, dv = [], [], []
        for j in range(case["kv_heads"]):
            o, _, p = _softmax64(q[j * g:j * g + g], k[j:j + 1], v[j:j + 1], see)
            p, dj, qj = p[0], do[j * g:j * g + g], q[j * g:j * g + g]
            dp = dj @ v[j].t()
            ds = p * (dp - (dp * p).sum(-1, keepdim=True)) * scale
            dq.append(ds @ k[j])
            dk.append(torch.einsum("gnm,gnd->md", ds, qj))
            dv.append(torch.einsum("gnm,gnd->md", p, dj))
        outs.append((torch.cat(dq).transpose(0, 1), torch.stack(dk, 1), torch.stack(dv, 1)))
    if case["form"] == "forward":
        return torch.cat([o for o, _ in outs]), torch.cat([l for _, l in outs], 1)
    return tuple(torch.cat([x[i] for x in outs]) for i in range(3))


def _exact_chunk(case, st):
    lens = _lengths(case)
    ctx = _contexts(case, lens)
    outs, at = [], 0
    g = case["heads"] // case["kv_heads"]
    for s, (n, c) in enumerate(zip(lens, ctx)):
        tok = torch.arange(c, device=DEV)
        blk, off = st["bt"][s].long()[tok // BLOCK], tok % BLOCK
        q = st["q"][at:at + n].double().transpose(0, 1)
        see = tok[None, :] <= (c - n + torch.arange(n, device=DEV))[:, None]
        heads = []
        for j in range(case["kv_heads"]):
            k = st["kc"][blk, j, :, off].flatten(1).double()
            v = st["vc"][blk, j, :, off].double()
            heads.append(_softmax64(q[j * g:j * g + g], k[None], v[None], see)[0])
        outs.append(torch.cat(heads).transpose(0, 1))
        at += n
    return torch.cat(outs)
