"""Cases of rotary positions, causal prompt attention, tree attention over a paged cache and row moves within it.

Rows are bf16, 128 dims a head.  Four operators, as a text tower's prompt and answering steps run them:

rotary  Pairs of a head's first `dims` dims are turned by position x frequency and scaled by an amplitude: (a, b) ->
        A (a cos t - b sin t, b cos t + a sin t), t = p[axis of the pair] f_j.  Pairs are (j, j + dims/2), or (2j, 2j+1)
        where interleaved.  f_j = base^(-2j/dims), changed for long contexts: linear f/s; ntk, base s^(dims/(dims-2));
        parts, f (g + (1-g)/s) with g = clamp((L f/2pi - 1)/31, 0, 1) and A = 0.1 ln s + 1.  Outputs: q and k, or with
        `store` q and the cache whose slots took k and v.
causal  Packed prompts, grouped heads: row i of a prompt attends to its rows up to i; query head h reads key head
        h // (heads/kv_heads).  Outputs: o [S, H, 128], lse [H, S].
tree    Sequences with a context in pages and up to 64 drafted tokens behind it: a draft sees the context and the
        drafts of its mask (its ancestors and itself).  One draft is the plain single-token step.  Outputs: o, lse.
move    Rows of a cache copied to other slots, the sources of a group read before its destinations are written: drafts
        that were accepted move up, pages are forked.  Outputs: the cache's k and v.

With `own` unset the operators run in plain torch; with it set, through packed_varlen_non_gb300.h3attn."""
import math

import torch

own = False

SCALE = 128 ** -0.5

# Sixteen prompts of 488 to 3,440 tokens: the packed varlen workload of this repository.
VARLEN = "1400,2576,2400,488,3416,1512,3168,1600,1928,1248,3440,800,2088,1760,2328,2616"
# Two dozen short prompts (captions, audio prompts): 1 to 700 tokens.
RAGGED = "17,405,1,64,129,300,33,700,128,5,81,256,511,2,190,32,90,47,600,31,222,8,144,405"


def listed():
    return [
        # a decoding step of 32 sequences: one token each, far positions, into the cache; latency counts
        dict(name="rotary_step", op="rotary", tokens=32, heads=32, kv_heads=8, dims=128, interleaved=False, base=1e6,
             scaling="none", factor=1.0, axes=1, far=200000, store=True),
        # a prompt of 20,423 tokens, positions scaled by parts for a context four times as long
        dict(name="rotary_prompt", op="rotary", tokens=20423, heads=28, kv_heads=4, dims=128, interleaved=False, base=1e6,
             scaling="parts", factor=4.0, axes=1, far=0, store=False),
        # (t, h, w) positions on 64 of the dims, neighbouring pairs, stored as the step of a long prefill stores them
        dict(name="rotary_grid", op="rotary", tokens=5033, heads=21, kv_heads=21, dims=64, interleaved=True, base=10000.0,
             scaling="ntk", factor=2.0, axes=3, far=5000, store=True),
        # the smallest call: two tiny prompts
        dict(name="causal_tiny", op="causal", docs="64,80", heads=8, kv_heads=2),
        # two dozen short prompts, four query heads to a key head
        dict(name="causal_ragged", op="causal", docs=RAGGED, heads=32, kv_heads=8),
        # sixteen prompts, every head with keys of its own
        dict(name="causal_varlen", op="causal", docs=VARLEN, heads=21, kv_heads=21),
        # one long prompt, seven query heads to a key head
        dict(name="causal_long", op="causal", docs="20423", heads=28, kv_heads=4),
        # the single-token step: 32 sequences at 5,033 tokens, pages of 16
        dict(name="tree_tokens", op="tree", ctx=",".join(["5033"] * 32), drafts=",".join(["1"] * 32), heads=32, kv_heads=8,
             page=16, chain=True),
        # sixteen uneven sequences, trees of 16 drafts, pages of 64
        dict(name="tree_drafts", op="tree", ctx=VARLEN, drafts=",".join(["16"] * 16), heads=28, kv_heads=4, page=64,
             chain=False),
        # eight long sequences, full trees: 512 rows to a key head
        dict(name="tree_long", op="tree", ctx=",".join(["20423"] * 8), drafts=",".join(["64"] * 8), heads=64, kv_heads=8,
             page=128, chain=False),
        # the accepted drafts of 32 trees of 16 move up
        dict(name="move_accept", op="move", groups=32, width=16, page=16, kv_heads=8, fork=False),
        # 512 pages of 64 tokens are copied for forked sequences
        dict(name="move_fork", op="move", groups=512, width=64, page=64, kv_heads=8, fork=True),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "causal", "causal", "tree", "tree", "move"])
    kv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    if op == "rotary":
        axes = rng.choice([1, 1, 3])
        return dict(op=op, tokens=_between(rng, 1, 20000), heads=kv * group, kv_heads=kv, dims=rng.choice([16, 48, 64, 96, 128]),
                    interleaved=rng.random() < 0.5, base=rng.choice([10000.0, 5e5, 1e6]),
                    scaling=rng.choice(["none", "linear", "ntk", "parts"]), factor=rng.choice([2.0, 4.0, 8.0]), axes=axes,
                    far=_between(rng, 1, 1000000), store=rng.random() < 0.5)
    if op == "causal":
        total, lens = _between(rng, 1, 20000), []
        for _ in range(_between(rng, 1, 40)):
            lens.append(min(total, _between(rng, 1, 20000)))
            total -= lens[-1]
            if total <= 0:
                break
        if kv * group > 28:
            kv = 28 // group
        return dict(op=op, docs=",".join(map(str, lens)), heads=kv * group, kv_heads=kv)
    if op == "tree":
        left, ctx, drafts, chain = 100000, [], [], rng.random() < 0.5
        most = _between(rng, 1, 64)
        for _ in range(_between(rng, 1, 64)):
            ctx.append(min(left, _between(rng, 1, 20001) - 1))
            drafts.append(rng.randint(1, most))
            left -= ctx[-1]
            if left <= 0:
                break
        return dict(op=op, ctx=",".join(map(str, ctx)), drafts=",".join(map(str, drafts)), heads=kv * group, kv_heads=kv,
                    page=rng.choice([8, 16, 32, 48, 64, 128, 256]), chain=chain)
    page = rng.choice([8, 16, 32, 48, 64, 128])
    fork = rng.random() < 0.5
    return dict(op=op, groups=_between(rng, 1, 512 * 64 // page), width=page if fork else rng.randint(1, 64), page=page,
                kv_heads=kv, fork=fork)


def _ints(text):
    return [int(x) for x in text.split(",")]


def _rows(n, heads, gen, shift=None):
    """n rows x heads of normalised features: runs of 64 tokens share one of 32 topics, so that some keys matter more
    to a query than others."""
    proto = shift if shift is not None else torch.randn(32, heads, 128, generator=gen, device="cuda")
    topic = torch.randint(0, 32, (-(-n // 64),), generator=gen, device="cuda").repeat_interleave(64)[:n]
    x = proto[topic] + torch.randn(n, heads, 128, generator=gen, device="cuda")
    x *= torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    return x.to(torch.bfloat16)


def _qkv(n, heads, kv_heads, gen):
    """q, k and v out of one buffer, as a fused projection leaves them."""
    buf = torch.empty(n, heads + 2 * kv_heads, 128, dtype=torch.bfloat16, device="cuda")
    proto = torch.randn(32, kv_heads, 128, generator=gen, device="cuda")
    buf[:, :heads] = _rows(n, heads, gen, proto.repeat_interleave(heads // kv_heads, 1))
    buf[:, heads:heads + kv_heads] = _rows(n, kv_heads, gen, proto)
    buf[:, heads + kv_heads:] = torch.randn(n, kv_heads, 128, generator=gen, device="cuda")
    return buf[:, :heads], buf[:, heads:heads + kv_heads], buf[:, heads + kv_heads:]


def _pages(n_pages, page, kv_heads):
    """An empty cache: k and v, each [pages, tokens of a page, heads, 128]."""
    return [torch.zeros(n_pages, page, kv_heads, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    op, st = case["op"], dict(case=case)
    kv_heads = case["kv_heads"]
    if own:
        from packed_varlen_non_gb300 import h3attn

        st["h"] = h3attn
    if op == "rotary":
        n, heads = case["tokens"], case["heads"]
        st["q"], st["k"], st["v"] = _qkv(n, heads, kv_heads, gen)
        st["q_out"] = torch.empty(n, heads, 128, dtype=torch.bfloat16, device="cuda")
        # a sequence's positions from `far` on (step: scattered), or a 16-wide grid's in its place
        if case["axes"] == 3:
            i = torch.arange(n)
            pos = torch.stack([case["far"] + i // 512, i // 16 % 32, i % 16])
        elif case["store"]:
            pos = torch.randint(0, case["far"] + 1, (1, n), generator=host)
        else:
            pos = case["far"] + torch.arange(n)[None]
        st["pos"] = pos.to(torch.int32).cuda()
        if case["store"]:
            n_pages = -(-n // 16) + 3
            st["kc"], st["vc"] = _pages(n_pages, 16, kv_heads)
            st["slots"] = torch.randperm(16 * n_pages, generator=host)[:n].to(torch.int32).cuda()
        else:
            st["k_out"] = torch.empty(n, kv_heads, 128, dtype=torch.bfloat16, device="cuda")
        if own:
            st["rope"] = h3attn.h3attn_rope_init(
                case["dims"], case["base"], interleaved=case["interleaved"], scaling=case["scaling"], factor=case["factor"],
                original_len=32768, axes=[j % case["axes"] for j in range(case["dims"] // 2)])
            if case["store"]:
                st["cache"] = h3attn.Cache(st["kc"], st["vc"])
    elif op == "causal":
        lens, heads = _ints(case["docs"]), case["heads"]
        S = sum(lens)
        st["lens"] = lens
        st["q"], st["k"], st["v"] = _qkv(S, heads, kv_heads, gen)
        st["o"] = torch.empty(S, heads, 128, dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.empty(heads, S, dtype=torch.float32, device="cuda")
        if own:
            st["plan"] = h3attn.Plan([[(n, 1, 1, (0.0, 0.0, 0.0), (1.0, 0.0, 0.0))] for n in lens], heads)
            h3attn.h3attn_plan_set_causal(st["plan"].handle, kv_heads)
    elif op == "tree":
        ctx, drafts, heads, page = _ints(case["ctx"]), _ints(case["drafts"]), case["heads"], case["page"]
        S = sum(drafts)
        need = [-(-(c + t) // page) for c, t in zip(ctx, drafts)]
        n_pages, width = sum(need) + 2, max(need)
        # pages in the order in which a program that has run for a while hands them out
        free = torch.randperm(n_pages, generator=host)
        table, at = torch.full((len(ctx), width), -1, dtype=torch.int32), 0
        for b, m in enumerate(need):
            table[b, :m] = free[at:at + m]
            at += m
        st["ctx"], st["drafts"] = ctx, drafts
        st["kc"], st["vc"] = _pages(n_pages, page, kv_heads)
        proto = torch.randn(32, kv_heads, 128, generator=gen, device="cuda")
        for b in range(len(ctx)):
            n = ctx[b] + drafts[b]
            at = torch.arange(n)
            slot = (table[b][at // page].long() * page + at % page).cuda()
            st["kc"].view(-1, kv_heads, 128)[slot] = _rows(n, kv_heads, gen, proto)
            st["vc"].view(-1, kv_heads, 128)[slot] = torch.randn(n, kv_heads, 128, generator=gen, device="cuda").to(torch.bfloat16)
        st["q"] = _rows(S, heads, gen, proto.repeat_interleave(heads // kv_heads, 1))
        st["table"], st["lens"] = table.cuda(), torch.tensor(ctx, dtype=torch.int32, device="cuda")
        seen = []  # bit j of a draft's word: it sees draft j of its tree
        for t in drafts:
            words = [1]
            for i in range(1, t):
                parent = i - 1 if case["chain"] else int(torch.randint(max(0, i - 12), i, (1,), generator=host))
                words.append(words[parent] | 1 << i)
            seen += words[:t]
        st["mask"] = torch.tensor([w - (1 << 64) if w >> 63 else w for w in seen], device="cuda")
        st["o"] = torch.empty(S, heads, 128, dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.empty(heads, S, dtype=torch.float32, device="cuda")
        if own:
            st["plan"] = h3attn.Plan([[(t, 1, 1, (0.0, 0.0, 0.0), (1.0, 0.0, 0.0))] for t in drafts], heads)
            h3attn.h3attn_plan_set_tree(st["plan"].handle, kv_heads)
            st["cache"] = h3attn.Cache(st["kc"], st["vc"])
    else:
        groups, width, page = case["groups"], case["width"], case["page"]
        src = torch.full((groups, width), -1, dtype=torch.int32)
        dst = src.clone()
        if case["fork"]:  # page g of a random half into page g of the other half
            n_pages = 2 * groups
            where = torch.randperm(n_pages, generator=host).to(torch.int32)
            row = torch.arange(page, dtype=torch.int32)
            src[:], dst[:] = where[:groups, None] * page + row, where[groups:, None] * page + row
        else:
            # a tree of `width` drafts from a random row of its pages on; the accepted path is the root and nodes of
            # deeper levels, which lie behind the places that the path moves to
            each = -(-width // page) + 1
            n_pages = each * groups
            where = torch.randperm(n_pages, generator=host).view(groups, each)
            for g in range(groups):
                first = int(torch.randint(0, page, (1,), generator=host))
                n = int(torch.randint(1, (width + 1) // 2 + 1, (1,), generator=host))
                path = torch.cat([torch.zeros(1, dtype=torch.long),
                                  (n + torch.randperm(width - n, generator=host)[:n - 1]).sort().values])
                for line, at in ((src, first + path), (dst, first + torch.arange(n))):
                    line[g, :n] = (where[g][at // page] * page + at % page).to(torch.int32)
        st["kc"], st["vc"] = _pages(n_pages, page, kv_heads)
        for c in (st["kc"], st["vc"]):
            c.copy_(torch.randn(c.shape, generator=gen, device="cuda"))
        st["src"], st["dst"] = src.cuda(), dst.cuda()
        if own:
            st["cache"] = h3attn.Cache(st["kc"], st["vc"])
    return st


def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"rotary": _plain_rotary, "causal": _plain_causal, "tree": _plain_tree, "move": _plain_move}[op](st)
    h = st["h"]
    if op == "rotary":
        if case["store"]:
            h.h3attn_rotary_store(st["rope"], st["pos"], st["q"], st["q_out"], st["k"], st["v"], st["cache"], st["slots"])
            return st["q_out"], st["kc"], st["vc"]
        h.h3attn_rotary(st["rope"], st["pos"], st["q"], st["q_out"], st["k"], st["k_out"])
        return st["q_out"], st["k_out"]
    if op == "causal":
        h.h3attn_forward_causal(st["plan"].handle, st["q"], st["k"], st["v"], st["o"], SCALE, st["lse"])
        return st["o"], st["lse"]
    if op == "tree":
        h.h3attn_forward_tree(st["plan"].handle, st["q"], st["cache"], st["table"], st["lens"], st["o"], SCALE, st["lse"],
                              tree_mask=st["mask"])
        return st["o"], st["lse"]
    h.h3attn_cache_move(st["cache"], st["src"], st["dst"])
    return st["kc"], st["vc"]


def _plain_rotary(st):
    case = st["case"]
    d, s, axes = case["dims"], case["factor"], case["axes"]
    j = torch.arange(d // 2, dtype=torch.float64, device="cuda")
    base, amplitude = case["base"], 1.0
    if case["scaling"] == "ntk":
        base *= s ** (d / (d - 2))
    f = torch.exp(j * (-2.0 * math.log(base) / d))
    if case["scaling"] == "linear":
        f = f / s
    elif case["scaling"] == "parts":
        g = ((32768 * f / (2 * math.pi) - 1) / 31).clamp(0, 1)
        f, amplitude = f * (g + (1 - g) / s), 0.1 * math.log(s) + 1
    t = st["pos"].double()[torch.arange(d // 2, device="cuda") % axes].T * f  # [n, d/2]
    cos, sin = ((amplitude * x).float()[:, None] for x in (torch.cos(t), torch.sin(t)))

    def turn(x):
        y = x.float()
        a, b = (y[..., :d:2], y[..., 1:d:2]) if case["interleaved"] else (y[..., :d // 2], y[..., d // 2:d])
        lo, hi = a * cos - b * sin, b * cos + a * sin
        pairs = torch.stack([lo, hi], -1).flatten(-2) if case["interleaved"] else torch.cat([lo, hi], -1)
        return torch.cat([pairs, y[..., d:]], -1).to(torch.bfloat16)

    if not case["store"]:
        return turn(st["q"]), turn(st["k"])
    slots = st["slots"].long()
    for cache, rows in ((st["kc"], turn(st["k"])), (st["vc"], st["v"])):
        cache.view(-1, case["kv_heads"], 128)[slots] = rows
    return turn(st["q"]), st["kc"], st["vc"]


def _attend(q, k, v, hidden):
    """o and lse of rows q [H, n, 128] over keys k, v [Hkv, m, 128], the pairs of `hidden` [n, m] left out."""
    group = q.shape[0] // k.shape[0]
    k, v = (x.float().repeat_interleave(group, 0) for x in (k, v))
    s = torch.matmul(q.float(), k.transpose(-1, -2)).mul_(SCALE).masked_fill_(hidden, -math.inf)
    m = s.amax(-1, keepdim=True)
    e = s.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v)
    return torch.where(total > 0, o / total, torch.zeros_like(o)), (total.log() + m)[..., 0]


def _plain_causal(st):
    out, out_lse, at = torch.empty_like(st["o"]), torch.empty_like(st["lse"]), 0
    for n in st["lens"]:
        k, v = (st[x][at:at + n].permute(1, 0, 2) for x in ("k", "v"))
        for r in range(0, n, 4096):
            e = min(n, r + 4096)
            hidden = torch.arange(e, device="cuda") > torch.arange(r, e, device="cuda")[:, None]
            o, lse = _attend(st["q"][at + r:at + e].permute(1, 0, 2), k[:, :e], v[:, :e], hidden)
            out[at + r:at + e], out_lse[:, at + r:at + e] = o.permute(1, 0, 2).to(torch.bfloat16), lse
        at += n
    return out, out_lse


def _plain_tree(st):
    case, at = st["case"], 0
    out, out_lse = torch.empty_like(st["o"]), torch.empty_like(st["lse"])
    for b, (c, t) in enumerate(zip(st["ctx"], st["drafts"])):
        page = st["table"][b, :-(-(c + t) // case["page"])].long()
        k, v = (st[x][page].flatten(0, 1)[:c + t].permute(1, 0, 2) for x in ("kc", "vc"))
        hidden = torch.zeros(t, c + t, dtype=torch.bool, device="cuda")
        hidden[:, c:] = (st["mask"][at:at + t, None] >> torch.arange(t, device="cuda")) & 1 == 0
        o, lse = _attend(st["q"][at:at + t].permute(1, 0, 2), k, v, hidden)
        out[at:at + t], out_lse[:, at:at + t] = o.permute(1, 0, 2).to(torch.bfloat16), lse
        at += t
    return out, out_lse


def _plain_move(st):
    there = st["src"] >= 0
    src, dst = st["src"][there].long(), st["dst"][there].long()
    for cache in (st["kc"], st["vc"]):
        rows = cache.view(-1, st["case"]["kv_heads"], 128)
        rows[dst] = rows[src]
    return st["kc"], st["vc"]


def work(case):
    op, kv_heads = case["op"], case["kv_heads"]
    if op == "rotary":
        n, heads = case["tokens"], case["heads"]
        rows = heads + (2 if case["store"] else 1) * kv_heads
        return {"bytes": 512 * n * rows + 4 * n * (case["axes"] + case["store"]), "flops": 3 * n * (heads + kv_heads) * case["dims"]}
    if op == "causal":
        lens, heads = _ints(case["docs"]), case["heads"]
        return {"bytes": sum(lens) * (512 * (heads + kv_heads) + 4 * heads), "flops": 256 * heads * sum(n * (n + 1) for n in lens)}
    if op == "tree":
        ctx, drafts, heads = _ints(case["ctx"]), _ints(case["drafts"]), case["heads"]
        keys, S = sum(ctx) + sum(drafts), sum(drafts)
        return {"bytes": 512 * kv_heads * keys + S * (516 * heads + 8) + 4 * (len(ctx) + keys // case["page"]),
                "flops": 512 * heads * sum(t * (c + 1) for c, t in zip(ctx, drafts))}
    # (of a tree a quarter of the drafts is accepted on average)
    rows = case["groups"] * (case["width"] if case["fork"] else max(1, case["width"] // 4))
    return {"bytes": 1024 * kv_heads * rows + 8 * case["groups"] * case["width"], "flops": 0}


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rotary":
        d, s = case["dims"], case["factor"]
        pos = st["pos"].tolist()
        turn = []  # the angles of every token's pairs
        amplitude = 0.1 * math.log(s) + 1 if case["scaling"] == "parts" else 1.0
        for j in range(d // 2):
            base = case["base"] * (s ** (d / (d - 2)) if case["scaling"] == "ntk" else 1.0)
            f = base ** (-2.0 * j / d)
            if case["scaling"] == "linear":
                f /= s
            elif case["scaling"] == "parts":
                turns = 32768 * f / (2 * math.pi)  # of the pair over the original length
                g = 0.0 if turns < 1 else 1.0 if turns > 32 else (turns - 1) / 31
                f = g * f + (1 - g) * f / s
            turn.append([p * f for p in pos[j % case["axes"]]])
        z = amplitude * torch.polar(torch.ones(d // 2, case["tokens"], dtype=torch.float64), torch.tensor(turn, dtype=torch.float64))
        z = z.T.cuda()[:, None]

        def turned(x):
            y = x.double().clone()
            if case["interleaved"]:
                y[..., :d] = torch.view_as_real(torch.view_as_complex(y[..., :d].unflatten(-1, (-1, 2)).contiguous()) * z).flatten(-2)
            else:
                w = torch.complex(y[..., :d // 2], y[..., d // 2:d]) * z
                y[..., :d // 2], y[..., d // 2:d] = w.real, w.imag
            return y

        if not case["store"]:
            return turned(st["q"]), turned(st["k"])
        kc, vc = st["kc"].double(), st["vc"].double()
        kc.view(-1, case["kv_heads"], 128).index_copy_(0, st["slots"].long(), turned(st["k"]))
        vc.view(-1, case["kv_heads"], 128).index_copy_(0, st["slots"].long(), st["v"].double())
        return turned(st["q"]), kc, vc
    if op == "move":
        out = []
        for cache in (st["kc"], st["vc"]):
            rows = cache.double().view(-1, case["kv_heads"], 128)
            new = rows.clone()
            for a, b in zip(st["src"], st["dst"]):
                a, b = a[a >= 0].long(), b[b >= 0].long()
                new.index_copy_(0, b, rows.index_select(0, a))
            out.append(new.view(cache.shape))
        return tuple(out)
    heads, group = case["heads"], case["heads"] // case["kv_heads"]
    o = torch.zeros(st["o"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    if op == "causal":
        at = 0
        for n in st["lens"]:
            for h in range(heads):
                q, k, v = (st[x][at:at + n, y].double() for x, y in (("q", h), ("k", h // group), ("v", h // group)))
                for r in range(0, n, 2048):
                    e = min(n, r + 2048)
                    s = SCALE * (q[r:e] @ k[:e].T)
                    s += torch.full((e - r, e), -math.inf, dtype=torch.float64, device="cuda").triu(r + 1)
                    lse[h, at + r:at + e] = torch.logsumexp(s, -1)
                    o[at + r:at + e, h] = torch.softmax(s, -1) @ v[:e]
            at += n
        return o, lse
    at, table, masks = 0, st["table"].tolist(), st["mask"].tolist()
    for b, (c, t) in enumerate(zip(st["ctx"], st["drafts"])):
        slots = torch.tensor([table[b][p // case["page"]] * case["page"] + p % case["page"] for p in range(c + t)], device="cuda")
        k, v = (st[x].flatten(0, 1)[slots].double() for x in ("kc", "vc"))  # [keys, Hkv, 128]
        bias = torch.tensor([[0.0] * c + [0.0 if masks[at + i] >> j & 1 else -math.inf for j in range(t)] for i in range(t)],
                            dtype=torch.float64, device="cuda")
        for h in range(heads):
            s = SCALE * (st["q"][at:at + t, h].double() @ k[:, h // group].T) + bias
            lse[h, at:at + t] = torch.logsumexp(s, -1)
            o[at:at + t, h] = torch.softmax(s, -1) @ v[:, h // group]
        at += t
    return o, lse
