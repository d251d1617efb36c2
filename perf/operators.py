"""Cases of the block-sparse and shared-prefix attention operators, with their plain forms.

Three operators over a packed batch of documents (rows of q-hat, k-hat and v, bf16 [S, H, 128]):

select  Block scores and selection.  Each document is cut into query blocks of q_block rows and key tiles of 128
        rows.  score(h, i, j) = <mean of the q-hat rows of query block i, mean of the k-hat rows of key tile j>, the
        means rounded to 32 bits; a query block keeps the `keep` tiles of its document with the largest scores (ties
        to the lowest tile), the tiles that overlap it before all others where keep_own is set.  Outputs: the kept
        tiles in ascending order (int32 [H, NQ, keep], -1 behind them) and their number (int32 [H, NQ]).
sparse  Attention over the listed tiles: o_i = softmax_j(scale q_i.k_j) v_j over the keys j of the tiles listed for
        row i's query block and head; lse_i = ln sum_j exp(scale q_i.k_j).  An empty list gives o = 0, lse = -inf.
prefix  Attention of a batch that shares a prefix: row i of a document attends to the P prefix rows and to its own
        document.

With `own` unset the operators run in plain torch; with it set, through packed_varlen_non_gb300.h3attn."""
import math

import torch

own = False

SCALE = 128 ** -0.5
TILE = 128

# Sixteen documents of 488 to 3,440 tokens: the packed varlen workload of this repository.
VARLEN = "1400,2576,2400,488,3416,1512,3168,1600,1928,1248,3440,800,2088,1760,2328,2616"
# Two dozen short requests over one set of references (captions, audio prompts, small stills): 1 to 700 tokens.
RAGGED = "17,405,1,64,129,300,33,700,128,5,81,256,511,2,190,32,90,47,600,31,222,8,144,405"


def listed():
    return [
        # the scores of a 4,096-token video (8 x 16 x 32 grid), a quarter of its 32 key tiles kept
        dict(name="select_video", op="select", docs="4096", heads=21, q_block=512, keep=8, keep_own=True),
        # the 20,423-token render with six references, fine query blocks, a quarter of 160 tiles kept
        dict(name="select_ref2va", op="select", docs="20423", heads=21, q_block=256, keep=40, keep_own=False),
        # a packed training-like batch of sixteen documents: every document selects for itself
        dict(name="select_varlen", op="select", docs=VARLEN, heads=21, q_block=512, keep=8, keep_own=True),
        # the smallest call: two tiny latents, two heads; latency counts
        dict(name="sparse_tiny", op="sparse", docs="64,80", heads=2, q_block=256, keep=1, keep_own=True),
        # one video at a quarter of its pairs
        dict(name="sparse_video", op="sparse", docs="4096", heads=21, q_block=512, keep=8, keep_own=True),
        # the render at a quarter of its pairs, coarse query blocks
        dict(name="sparse_ref2va_q512", op="sparse", docs="20423", heads=21, q_block=512, keep=40, keep_own=True),
        # the render at an eighth of its pairs, fine query blocks
        dict(name="sparse_ref2va_q256", op="sparse", docs="20423", heads=21, q_block=256, keep=20, keep_own=True),
        # sixteen documents, eight tiles for each fine query block (the shorter documents keep all they have)
        dict(name="sparse_varlen", op="sparse", docs=VARLEN, heads=21, q_block=256, keep=8, keep_own=True),
        # thirty-two single queries over a 5,033-token audio prefix: the serving form, bound by reading the prefix
        dict(name="prefix_tokens", op="prefix", docs=",".join(["1"] * 32), heads=21, prefix=5033),
        # two dozen short requests that share six reference images (6 x 405 tokens)
        dict(name="prefix_ragged", op="prefix", docs=RAGGED, heads=21, prefix=2430),
        # three variants of one video request over the same six references
        dict(name="prefix_variants", op="prefix", docs="4096,4096,4096", heads=21, prefix=2430),
        # audio, references and a clip, each attending to a 12,960-token video context
        dict(name="prefix_long", op="prefix", docs="5033,2430,4096", heads=21, prefix=12960),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["select", "sparse", "sparse", "prefix", "prefix"])
    heads = rng.choice([1, 2, 5, 8, 16, 21])
    if op == "prefix":
        if rng.random() < 0.3:
            lens = [1] * _between(rng, 1, 128)  # single tokens
        else:
            n, left, lens = _between(rng, 1, 40), 10000, []
            for _ in range(n):
                lens.append(min(left, _between(rng, 1, 5000)))
                left -= lens[-1]
                if left <= 0:
                    break
        return dict(op=op, docs=",".join(map(str, lens)), heads=heads, prefix=_between(rng, 1, 12000))
    total, lens = _between(rng, 200, 20000), []
    for _ in range(_between(rng, 1, 16)):
        lens.append(min(total, _between(rng, 1, 20000)))
        total -= lens[-1]
        if total <= 0:
            break
    tiles = -(-max(lens) // TILE)
    return dict(op=op, docs=",".join(map(str, lens)), heads=heads, q_block=rng.choice([256, 512]),
                keep=min(40, rng.randint(1, max(1, tiles // 2))), keep_own=rng.random() < 0.5)


def _lens(case):
    return [int(x) for x in case["docs"].split(",")]


def _layout(lens, block):
    """(first row, end of the rows, document's first row, document's end) of every block of `block` rows."""
    out, at = [], 0
    for n in lens:
        out += [(at + r, min(at + r + block, at + n), at, at + n) for r in range(0, n, block)]
        at += n
    return out


def _rows(n, topics, proto, gain, gen, outlier=None):
    """n rows x H heads of normalised features, as a q/k RMSNorm leaves them: runs of 64 tokens share one of 32
    topics, so that some key tiles matter more to a query than others; `outlier` scales channels as in k."""
    x = proto[topics] + torch.randn(n, *proto.shape[1:], generator=gen, device="cuda")
    if outlier is not None:
        x *= outlier
    x *= torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    return (x * gain).to(torch.bfloat16)


def prepare(case, seed):
    lens, H = _lens(case), case["heads"]
    S = sum(lens)
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    proto = normal(32, H, 128)
    gain_q, gain_k = 1 + 0.1 * normal(128), 1 + 0.1 * normal(128)
    outlier = torch.exp(0.5 * normal(H, 128))
    P = case.get("prefix", 0)
    topic = torch.randint(0, 32, (-(-(S + P) // 64),), generator=gen, device="cuda").repeat_interleave(64)[:S + P]
    st = dict(case=case, lens=lens, S=S, H=H)
    st["q"] = _rows(S, topic[P:], proto, gain_q, gen)
    k = _rows(S + P, topic, proto, gain_k, gen, outlier)
    v = normal(S + P, H, 128).to(torch.bfloat16)
    st["k"], st["v"] = k[P:].contiguous(), v[P:].contiguous()
    if P:
        st["kp"], st["vp"] = k[:P].contiguous(), v[:P].contiguous()
    else:
        rows = _layout(lens, case["q_block"])
        st["blocks"] = torch.tensor(rows, device="cuda")  # [NQ, 4]
        NQ, keep = len(rows), case["keep"]
        st["idx"] = torch.empty(H, NQ, keep, dtype=torch.int32, device="cuda")
        st["cnt"] = torch.empty(H, NQ, dtype=torch.int32, device="cuda")
        st["tiles_per_doc"] = -(-max(lens) // TILE)
        if case["op"] == "sparse":
            # the lists that a selection step of the same block leaves behind
            idx, cnt = _plain_select(st)
            st["idx"].copy_(idx)
            st["cnt"].copy_(cnt)
    st["o"] = torch.empty(S, H, 128, dtype=torch.bfloat16, device="cuda")
    st["lse"] = torch.empty(H, S, dtype=torch.float32, device="cuda")
    if own:
        from packed_varlen_non_gb300 import h3attn

        st["h"] = h3attn
        st["plan"] = h3attn.Plan([[(n, 1, 1, (0.0, 0.0, 0.0), (1.0, 0.0, 0.0))] for n in lens], H)
        if P:
            h3attn.h3attn_plan_set_prefix(st["plan"].handle, P)
        else:
            h3attn.h3attn_plan_set_sparse(st["plan"].handle, case["q_block"], case["keep"])
    return st


def run(st):
    op = st["case"]["op"]
    if own:
        h, plan = st["h"], st["plan"].handle
        if op == "select":
            h.h3attn_block_select(plan, st["q"], st["k"], st["case"]["keep"], st["idx"], st["cnt"],
                                  keep_own=st["case"]["keep_own"])
            return st["idx"], st["cnt"]
        if op == "sparse":
            h.h3attn_forward_sparse(plan, st["q"], st["k"], st["v"], st["idx"], st["cnt"], st["o"], SCALE, st["lse"])
        else:
            h.h3attn_forward_prefix(plan, st["q"], st["k"], st["v"], st["kp"], st["vp"], st["o"], SCALE, st["lse"])
        return st["o"], st["lse"]
    if op == "select":
        return _plain_select(st)
    return _plain_sparse(st) if op == "sparse" else _plain_prefix(st)


def _block_rows(first, end, n):
    """Row numbers [B, n] of blocks that begin at `first`, and which of them lie before `end`."""
    at = first[:, None] + torch.arange(n, device="cuda")
    real = at < end[:, None]
    return torch.where(real, at, first[:, None]), real


def _block_means(x, first, end, n):
    at, real = _block_rows(first, end, n)
    total = (x[at].double() * real[:, :, None, None]).sum(1)  # [B, H, 128]
    return (total / real.sum(1)[:, None, None]).float().double()


def _plain_select(st):
    case = st["case"]
    q0, q1, d0, d1 = st["blocks"].unbind(1)
    # candidates: the tiles of each query block's document
    tile = torch.arange(st["tiles_per_doc"], device="cuda")
    there = tile < ((d1 - d0 + TILE - 1) // TILE)[:, None]  # [NQ, T]
    k0 = torch.where(there, d0[:, None] + tile * TILE, d0[:, None])
    # every document's tiles once: the mean of a tile is that of the tile beginning at its first row
    firsts, where = torch.unique(k0, return_inverse=True)
    ends = torch.empty_like(firsts).scatter_(0, where.flatten(), torch.minimum(k0 + TILE, d1[:, None]).flatten())
    qm = _block_means(st["q"], q0, q1, case["q_block"])
    km = _block_means(st["k"], firsts, ends, TILE)
    score = (qm[:, None] * km[where]).sum(-1).permute(2, 0, 1)  # [H, NQ, T]
    if case["keep_own"]:
        mine = there & (k0 < q1[:, None]) & (k0 + TILE > q0[:, None])
        score = score.masked_fill(mine, math.inf)
    score = score.masked_fill(~there, -math.inf)
    best = torch.sort(score, dim=-1, descending=True, stable=True).indices[:, :, :case["keep"]]
    cnt = torch.minimum(there.sum(1), torch.tensor(case["keep"], device="cuda"))
    best = torch.nn.functional.pad(best, (0, case["keep"] - best.shape[-1]))
    kept = torch.arange(case["keep"], device="cuda") < cnt[:, None]  # [NQ, keep]
    best = best.masked_fill(~kept, 1 << 30).sort(-1).values.masked_fill(~kept, -1)
    return best.int(), cnt.int().expand(st["H"], -1).contiguous()


def _softmax(s):
    """Unnormalised probabilities, their sums and the log-sum-exps of rows of scores; -inf is masked."""
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = s.sub_(m).exp_()
    total = e.sum(-1, keepdim=True)
    return e, total, (total.log() + m)[..., 0]


def _plain_sparse(st):
    case, S, H = st["case"], st["S"], st["H"]
    q0, q1, d0, d1 = st["blocks"].unbind(1)
    rows, real = _block_rows(q0, q1, case["q_block"])
    kept = torch.arange(case["keep"], device="cuda") < st["cnt"][..., None]  # [H, NQ, keep]
    key = (d0[:, None] + st["idx"].clamp(min=0) * TILE)[..., None] + torch.arange(TILE, device="cuda")
    seen = (key < d1[:, None, None]) & kept[..., None]
    key = torch.where(seen, key, 0).flatten(2)  # [H, NQ, keep * 128]
    seen = seen.flatten(2)[:, :, None]
    head = torch.arange(H, device="cuda")[:, None, None]
    q = st["q"][rows].permute(2, 0, 1, 3).float()  # [H, NQ, q_block, 128]
    s = torch.matmul(q, st["k"][key, head].float().transpose(-1, -2)).mul_(SCALE).masked_fill_(~seen, -math.inf)
    e, total, lse = _softmax(s)
    o = torch.matmul(e, st["v"][key, head].float())
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    out, out_lse = torch.empty(S, H, 128, device="cuda"), torch.empty(H, S, device="cuda")
    out[rows[real]] = o.permute(1, 2, 0, 3)[real]
    out_lse[:, rows[real]] = lse[:, real]
    return out.to(torch.bfloat16), out_lse


def _plain_prefix(st):
    doc = torch.arange(len(st["lens"]), device="cuda").repeat_interleave(torch.tensor(st["lens"], device="cuda"))
    q, k, v = (st[n].permute(1, 0, 2).float() for n in ("q", "k", "v"))
    kp, vp = (st[n].permute(1, 0, 2).float() for n in ("kp", "vp"))
    s = torch.empty(st["H"], st["S"], kp.shape[1] + st["S"], device="cuda")
    s[..., :kp.shape[1]] = torch.matmul(q, kp.transpose(-1, -2))
    s[..., kp.shape[1]:] = torch.matmul(q, k.transpose(-1, -2)).masked_fill_(doc[:, None] != doc, -math.inf)
    e, total, lse = _softmax(s.mul_(SCALE))
    o = torch.matmul(e, torch.cat([vp, v], 1)) / total
    return o.permute(1, 0, 2).to(torch.bfloat16), lse


def work(case):
    lens, H = _lens(case), case["heads"]
    S = sum(lens)
    row = H * 256  # bytes of one token's heads
    if case["op"] == "prefix":
        P = case["prefix"]
        return {"bytes": 4 * S * row + 2 * P * row + 4 * H * S, "flops": 512 * H * sum(n * (P + n) for n in lens)}
    blocks = [(n, -(-n // case["q_block"]), -(-n // TILE)) for n in lens]
    nq = sum(b for _, b, _ in blocks)
    lists = 4 * H * nq * (case["keep"] + 1)
    if case["op"] == "select":
        return {"bytes": 2 * S * row + lists, "flops": 2 * S * H * 128 + 256 * H * sum(b * t for _, b, t in blocks)}
    # the keys that a row sees: `keep` tiles, or its whole document where that has no more
    pairs = sum(n * min(n, case["keep"] * TILE) for n in lens)
    return {"bytes": 4 * S * row + 4 * H * S + lists, "flops": 512 * H * pairs}


def exact(case, seed):
    st = prepare(case, seed)
    lens, H, q = st["lens"], st["H"], st["q"].double()
    k, v = st["k"].double(), st["v"].double()
    if case["op"] == "select":
        idx = torch.full((H, len(st["blocks"]), case["keep"]), -1, dtype=torch.int32)
        cnt = torch.zeros(H, len(st["blocks"]), dtype=torch.int32)
        b = at = 0
        for n in lens:
            tiles = torch.stack([t.mean(0) for t in k[at:at + n].split(TILE)]).float().double()
            for r, block in zip(range(0, n, case["q_block"]), q[at:at + n].split(case["q_block"])):
                score = (tiles * block.mean(0).float().double()).sum(-1).cpu()  # [T, H]
                for h in range(H):
                    line = score[:, h].tolist()
                    if case["keep_own"]:
                        for t in range(r // TILE, -(-(r + len(block)) // TILE)):
                            line[t] = math.inf
                    best = sorted(sorted(range(len(line)), key=lambda t: -line[t])[:case["keep"]])
                    idx[h, b, :len(best)] = torch.tensor(best, dtype=torch.int32)
                    cnt[h, b] = len(best)
                b += 1
            at += n
        return idx, cnt
    o = torch.zeros(st["S"], H, 128, dtype=torch.float64, device="cuda")
    lse = torch.full((H, st["S"]), -math.inf, dtype=torch.float64, device="cuda")
    if case["op"] == "prefix":
        kp, vp, at = st["kp"].double(), st["vp"].double(), 0
        for n in lens:
            for h in range(H):
                keys, vals = (torch.cat([a[:, h], b[at:at + n, h]]) for a, b in ((kp, k), (vp, v)))
                s = SCALE * (q[at:at + n, h] @ keys.T)
                lse[h, at:at + n] = torch.logsumexp(s, -1)
                o[at:at + n, h] = torch.softmax(s, -1) @ vals
            at += n
        return o, lse
    idx, cnt = st["idx"].tolist(), st["cnt"].tolist()
    for b, (q0, q1, d0, d1) in enumerate(st["blocks"].tolist()):
        for h in range(H):
            at = [torch.arange(d0 + TILE * t, min(d0 + TILE * t + TILE, d1)) for t in idx[h][b][:cnt[h][b]]]
            if at:
                at = torch.cat(at).to("cuda")
                s = SCALE * (q[q0:q1, h] @ k[at, h].T)
                lse[h, q0:q1] = torch.logsumexp(s, -1)
                o[q0:q1, h] = torch.softmax(s, -1) @ v[at, h]
    return o, lse
