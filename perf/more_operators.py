"""Measured cases of the operators for positions and drafted tokens.

What a decode step of a rotary model with drafted tokens runs beside the FFN
block: the rotation of queries and keys by their positions (and its gradient),
keys and values rotated on their way into the 8-bit paged cache, the tree of
drafted tokens, attention for that tree over the cache, and the verification
of the drafted tokens.  Each has a plain form in elementary torch operations
(binary32, or 64 bits where 32 lose what matters) and a definition in 64 bits;
`own` selects this package's kernels instead.
"""
import math
import random

import torch

own = False

BLOCK = 16          # tokens that share one scale of the cache
MIN_EXP = -64       # smallest scale of the cache: 2^MIN_EXP
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}
BASE = 10000.0
NEAR = 4096         # positions that the scaled models were first trained on


def listed():
    return [
        # a decode step of 32 sequences, one token each: queries and keys of 32 + 8 heads, rotated where the projection left them
        dict(name="rotary_step", op="rotary", tokens=32, heads=40, dim=128, turned=128, pairs="half", scaling="none", factor=1.0,
             far=8191, dtype="f16"),
        # a prompt pass of a model stretched to 32 times its context, packed queries, keys and values
        dict(name="rotary_prompt", op="rotary", tokens=16001, heads=72, dim=128, turned=128, pairs="half", scaling="yarn",
             factor=32.0, far=131071, dtype="bf16"),
        # fine-tuning: the gradient of queries and keys whose leading quarter turns, neighbours in pairs
        dict(name="rotary_backward", op="rotary_grad", tokens=8190, heads=71, dim=64, turned=16, pairs="neighbours",
             scaling="linear", factor=4.0, far=16383, dtype="bf16"),
        # a decode step of 32 sequences: the token's query, key and value, into blocks that already hold tokens
        dict(name="append_step", op="append", seqs=32, lo=5, hi=8100, q=1, tree=False, heads=8, group=8, dim=128, turned=128,
             page=64, pairs="half", scaling="none", factor=1.0, dtype="f16"),
        # prompts of five requests (ragged) entering the cache of an 8192-wide model
        dict(name="append_prompt", op="append", seqs=5, lo=0, hi=0, q=6001, tree=False, heads=8, group=8, dim=128, turned=128,
             page=64, pairs="half", scaling="yarn", factor=8.0, dtype="bf16"),
        # the drafted tokens of a served batch: small trees
        dict(name="tree_step", op="tree", seqs=16, q=26, branch=4),
        # a large batch of the deepest and widest trees
        dict(name="tree_large", op="tree", seqs=512, q=256, branch=16),
        # one sequence of the 1024-wide layer (16 heads of 64), a chain of five drafted tokens
        dict(name="attend_chain", op="attend", seqs=1, lo=1537, hi=1537, q=5, branch=1, heads=16, group=1, dim=64, page=64,
             dtype="f16"),
        # a served batch of different lengths, trees of up to 26 tokens, 64 query heads on 8 kv heads
        dict(name="attend_trees", op="attend", seqs=16, lo=20, hi=8191, q=26, branch=4, heads=8, group=8, dim=128, page=64,
             dtype="bf16"),
        # one long document under a tree of 64: 128 query heads of 64 on 8 kv heads
        dict(name="attend_long", op="attend", seqs=1, lo=60011, hi=60011, q=64, branch=4, heads=8, group=16, dim=64, page=128,
             dtype="f16"),
        # a chain of four drafted tokens of one sequence against a small vocabulary
        dict(name="verify_one", op="verify", seqs=1, q=5, branch=1, vocab=50007, draft=True, dtype="f32"),
        # a served batch: trees of eight tokens against a large vocabulary
        dict(name="verify_batch", op="verify", seqs=64, q=8, branch=3, vocab=131072, draft=True, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rotary", "rotary_grad", "append", "tree", "attend", "attend", "verify", "verify"))
    pairs = rng.choice(("half", "neighbours"))
    scaling = rng.choice(("none", "linear", "ntk", "yarn"))
    factor = 1.0 if scaling == "none" else rng.choice((2.0, 4.0, 8.0, 32.0))
    if op in ("rotary", "rotary_grad"):
        dim, heads = rng.choice((64, 80, 96, 128, 256)), _log(rng, 1, 96)
        turned = rng.choice((dim, dim, dim // 2, dim // 4))
        return dict(op=op, tokens=_log(rng, 1, min(40000, (1 << 27) // (dim * heads))), heads=heads, dim=dim, turned=turned,
                    pairs=pairs, scaling=scaling, factor=factor, far=rng.choice((2047, 131071, 1048575)),
                    dtype=rng.choice(("f16", "bf16", "f32")))
    if op == "append":
        heads, dim, group = _log(rng, 1, 48), rng.choice((64, 96, 128, 256)), rng.choice((1, 2, 4, 5, 7, 8, 16))
        tokens = max(1, _log(rng, 1, (1 << 27) // (heads * dim * (group + 2))))
        tree = rng.random() < 0.4
        seqs = min(tokens, _log(rng, 1, 256))
        q = max(1, tokens // seqs)
        return dict(op=op, seqs=seqs, lo=0, hi=rng.choice((0, 40, 3000)), q=min(q, 256) if tree else q, tree=tree, heads=heads,
                    group=group, dim=dim, turned=rng.choice((dim, dim // 2)), page=rng.choice((16, 32, 64, 128)), pairs=pairs,
                    scaling=scaling, factor=factor, dtype=rng.choice(("f16", "bf16", "f32")))
    if op == "tree":
        return dict(op=op, seqs=_log(rng, 1, 512), q=_log(rng, 1, 256), branch=rng.choice((1, 2, 4, 16)))
    if op == "attend":
        heads, dim, group = _log(rng, 1, 32), rng.choice((64, 96, 128, 256)), rng.choice((1, 1, 2, 4, 5, 7, 8, 16))
        keys = _log(rng, 64, min(1 << 16, (1 << 27) // (heads * dim)))
        seqs = min(_log(rng, 1, 64), max(1, (1 << 27) // (heads * dim * keys)))
        q = rng.choice((2, 5, 8, 16, 26, 64, _log(rng, 3, 256)))
        while q > 2 and seqs * q * keys * heads * group * dim > 1 << 35:
            q //= 2
        return dict(op=op, seqs=seqs, lo=rng.choice((0, 1, keys // 2, keys)), hi=keys, q=q, branch=rng.choice((1, 2, 4, 16)),
                    heads=heads, group=group, dim=dim, page=rng.choice((16, 32, 64, 128)), dtype=rng.choice(("f16", "bf16")))
    vocab, q = _log(rng, 500, 150000), rng.choice((2, 3, 5, 8, 16, 33))
    return dict(op=op, seqs=_log(rng, 1, max(1, min(64, (1 << 26) // (q * vocab)))), q=q, branch=rng.choice((1, 1, 2, 4)),
                vocab=vocab, draft=rng.random() < 0.7, dtype=rng.choice(("f32", "f32", "bf16", "f16")))


def _spread(n, lo, hi):
    """n lengths between lo and hi, the longest among them, by a fixed rule."""
    return [hi if s == 0 else lo + int((hi - lo) * ((s * 0.6180339887498949) % 1.0)) for s in range(n)]


def _lengths(case):
    """Per sequence: tokens in the cache before the new ones, and new tokens.  `attend` counts the new ones among hi."""
    n, q = case["seqs"], case["q"]
    new = [q] * n if q <= 2 else [max(1, q - int(q * 0.5 * ((s * 0.7548776662466927) % 1.0))) for s in range(n)]
    if case["op"] in ("tree", "verify"):
        return [0] * n, new
    before = _spread(n, case["lo"], case["hi"])
    if case["op"] == "attend":
        before = [b - m for b, m in zip(before, new)]    # below 0: the first nodes have no place in the cache
    return before, new


def work(case):
    op = case["op"]
    if op == "tree":
        n = sum(_lengths(case)[1])
        return dict(bytes=4 * n * (2 + -(-case["q"] // 32)) + 4 * case["seqs"], flops=n * -(-case["q"] // 32))
    e = SIZE[case["dtype"]]
    if op in ("rotary", "rotary_grad"):
        n = case["tokens"] * case["heads"]
        return dict(bytes=2 * n * case["dim"] * e + 4 * case["tokens"], flops=3 * n * case["turned"])
    if op == "append":
        rows, D = sum(_lengths(case)[1]) * case["heads"], case["dim"]
        return dict(bytes=rows * (2 * (D * (e + 1) + 4 / BLOCK) + 2 * case["group"] * D * e),
                    flops=rows * (3 * case["turned"] * (case["group"] + 1) + 4 * D))
    if op == "attend":
        before, new = _lengths(case)
        keys = sum(max(0, b + m) for b, m in zip(before, new))
        pairs = sum(max(0, b) * m + m for b, m in zip(before, new))      # the cache, and at least itself
        rows = sum(new) * case["heads"] * case["group"]
        return dict(bytes=2 * keys * case["heads"] * (case["dim"] + 4 / BLOCK) + rows * (2 * case["dim"] * e + 4)
                    + 4 * sum(new) * -(-case["q"] // 32),
                    flops=4 * pairs * case["heads"] * case["group"] * case["dim"])
    # of each sequence the rows of the node where it ends, one element of both for each other node
    n = sum(_lengths(case)[1])
    both = 2 if case["draft"] else 1
    return dict(bytes=case["seqs"] * (both * case["vocab"] * e + 12 + 4 * case["q"]) + n * (12 + both * e),
                flops=4 * case["seqs"] * case["vocab"])


# ---- inputs -------------------------------------------------------------------

def _scale_of(amax):
    """Smallest power of two s >= 2^MIN_EXP with amax <= 448 s; exact in any precision."""
    m, e = torch.frexp(amax)                             # amax = m 2^e, m in [0.5, 1)
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(min=MIN_EXP)
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)))


def _pool(pages, heads, page, dim, gen):
    """A cache's content: codes uint8 [pages, heads, page, dim], scales [pages, heads, page / BLOCK]."""
    shape = (pages, heads, page // BLOCK, BLOCK, dim)
    x = torch.randn(shape, device="cuda", generator=gen)
    x *= torch.exp(0.5 * torch.randn(shape[:3] + (1, 1), device="cuda", generator=gen))
    s = _scale_of(x.abs().amax((3, 4)))
    codes = (x / s[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(pages, heads, page, dim)
    return codes, s


def _trees(case, seed):
    """Parent of each node, packed by sequence; a node hangs on one of the `branch` nodes before it."""
    rng = random.Random(seed)
    return [-1 if i == 0 else i - 1 - rng.randrange(min(i, case["branch"])) for m in _lengths(case)[1] for i in range(m)]


def _packed(case, seed):
    before, new = _lengths(case)
    i32 = dict(dtype=torch.int32, device="cuda")
    cu = [0]
    for m in new:
        cu.append(cu[-1] + m)
    st = dict(tokens=cu[-1], max_q=max(new), cu=torch.tensor(cu, **i32))
    if case["op"] != "append" or case["tree"]:
        tree = dict(case, branch=case.get("branch", 4))
        st["parent"] = torch.tensor(_trees(tree, seed), **i32)
    return st


def _cache_state(case, gen, seed):
    before, new = _lengths(case)
    st = _packed(case, seed)
    page, heads, dim = case["page"], case["heads"], case["dim"]
    need = [max(1, -(-max(0, b + m) // page)) for b, m in zip(before, new)]
    pages = sum(need) + 2
    order = torch.randperm(pages, device="cuda", generator=gen).int().cpu()
    table = torch.zeros(len(need), max(need), dtype=torch.int32)
    used = 0
    for s, n in enumerate(need):
        table[s, :n] = order[used:used + n]
        used += n
    st.update(table=table.cuda(), before=torch.tensor(before, dtype=torch.int32).cuda(),
              length=torch.tensor([max(0, b + m) for b, m in zip(before, new)], dtype=torch.int32).cuda())
    st["kc"], st["ks"] = _pool(pages, heads, page, dim, gen)
    st["vc"], st["vs"] = _pool(pages, heads, page, dim, gen)
    if own:
        import activation_sparse_rank_gb300 as pi
        st["cache"] = pi.KVCache.wrap(st["kc"], st["ks"], st["vc"], st["vs"])
    return st


def _frequencies(case):
    """Radians a position, 64 bits [turned / 2], and the factor on cosine and sine."""
    R, s, base = case["turned"], case["factor"], BASE
    i = torch.arange(R // 2, dtype=torch.float64, device="cuda")
    if case["scaling"] == "ntk" and R > 2:
        base *= s ** (R / (R - 2))
    f = torch.exp(-2.0 * i / R * math.log(base))
    if case["scaling"] == "linear":
        return f / s, 1.0
    if case["scaling"] != "yarn":
        return f, 1.0

    def dim_of(turns):                                   # where a frequency makes that many turns over NEAR positions
        return R * math.log(NEAR / (2 * math.pi * turns)) / (2 * math.log(BASE))
    lo, hi = max(0, math.floor(dim_of(32.0))), min(R - 1, math.ceil(dim_of(1.0)))
    ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
    return f * (1 - ramp) + f / s * ramp, 0.1 * math.log(s) + 1.0


def _turn_plan(case, st):
    if own:
        import activation_sparse_rank_gb300 as pi
        st["rope"] = pi.Rotary(case["turned"], base=BASE, interleaved=case["pairs"] == "neighbours",
                               scaling=None if case["scaling"] == "none" else case["scaling"], factor=case["factor"],
                               original_length=NEAR)
    else:
        st["freq"], st["mag"] = _frequencies(case)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    op = case["op"]

    def normal(*shape, std=1.0):
        return torch.empty(shape, device="cuda").normal_(0.0, std, generator=gen).to(DT[case["dtype"]])

    if op == "tree":
        st = _packed(case, seed)
    elif op in ("rotary", "rotary_grad"):
        T, H, D = case["tokens"], case["heads"], case["dim"]
        st = dict(pos=torch.randint(0, case["far"] + 1, (T,), device="cuda", generator=gen).int())
        if op == "rotary":                               # queries and keys of a packed projection, values behind them
            st["x"] = normal(T, H + max(1, H // 8), D, std=1.5)[:, :H]
        else:
            st["x"] = normal(T, H, D)
        _turn_plan(case, st)
    elif op == "append":
        st = _cache_state(case, gen, seed)
        T, H, D, G = st["tokens"], case["heads"], case["dim"], case["group"]
        qkv = normal(T, H * (G + 2), D)                  # as a packed projection leaves them
        st["q"], st["k"], st["v"] = qkv[:, :H * G], qkv[:, H * G:H * G + H], qkv[:, H * G + H:]
        st["pos"] = None
        if case["tree"]:                                 # a node's position is its depth behind the cache
            seq = torch.repeat_interleave(torch.arange(case["seqs"], device="cuda"), (st["cu"][1:] - st["cu"][:-1]).long())
            st["pos"] = st["before"][seq] + _depths(st, case)
        _turn_plan(case, st)
    elif op == "attend":
        st = _cache_state(case, gen, seed)
        st["q"] = normal(st["tokens"], case["heads"] * case["group"], case["dim"], std=1.5)
        st["mask"] = _tree(st, case)[0]                  # one tree for all layers of a step
        if own:
            st["ws"] = st["cache"].attention_workspace(st["q"].shape[1], st["tokens"], case["seqs"])
    else:
        st = _packed(case, seed)
        T, V, dt = st["tokens"], case["vocab"], DT[case["dtype"]]
        shape = (T, V)
        x = torch.empty(shape, device="cuda").normal_(0.0, 2.5, generator=gen)
        st["target"] = torch.softmax(x, 1).to(dt)
        x += torch.empty(shape, device="cuda").normal_(0.0, 0.6, generator=gen)
        q = torch.softmax(x, 1)
        up = _above(st, case).clamp(min=0)
        if case["draft"]:                                # siblings are drawn independently
            st["draft"] = q.to(dt)
            st["drawn"] = torch.cat([torch.multinomial(q[up[i:i + 64]], 1, generator=gen) for i in range(0, T, 64)])[:, 0].int()
        else:                                            # siblings are the likeliest tokens in turn
            st["draft"] = None
            first = torch.arange(T, device="cuda")
            rank = ((up[:, None] == up[None]) & (first[None] < first[:, None])).sum(1) % min(16, V)
            st["drawn"] = q.topk(min(16, V), 1).indices[up, rank].int()
        st["accept"] = torch.rand(T, device="cuda", generator=gen)
        st["sample"] = torch.rand(case["seqs"], device="cuda", generator=gen)
    st["case"] = dict(case)
    return st


# ---- plain forms ----------------------------------------------------------------

def _rotate(x, pos, freq, mag, turned, pairs, sign):
    """Binary32 rows turned by the angles, which are of 64 bits."""
    angle = pos.double()[:, None] * freq
    c, s = (angle.cos() * mag).float()[:, None], (angle.sin() * (sign * mag)).float()[:, None]
    y = x.float().clone()
    a, b = _pairs(y, turned, pairs)
    ta, tb = a * c - b * s, a * s + b * c
    a.copy_(ta)
    b.copy_(tb)
    return y


def _pairs(x, turned, pairs):
    if pairs == "half":
        return x[..., :turned // 2], x[..., turned // 2:turned]
    return x[..., 0:turned:2], x[..., 1:turned:2]


def _places(st):
    """Of every new token: position, page and offset in the page."""
    P = st["case"]["page"]
    cu = st["cu"].long()
    i = torch.arange(st["tokens"], device="cuda")
    s = torch.searchsorted(cu[1:], i, right=True)
    pos = st["before"].long()[s] + i - cu[s]
    return pos, st["table"].long()[s, pos // P], pos % P


def _write(x, codes, scales, page, off):
    n, H, P, D = codes.shape
    per = P // BLOCK
    block = page * per + off // BLOCK                               # [T]
    every, at = torch.unique(block, return_inverse=True)            # the blocks that are written
    x = x.float()
    amax = torch.zeros(len(every), H, device="cuda").index_reduce_(0, at, x.abs().amax(2), "amax")
    first = torch.full((len(every),), BLOCK, device="cuda").scatter_reduce_(0, at, off % BLOCK, "amin")
    pg, bk = every // per, every % per
    old, need = scales[pg, :, bk], _scale_of(amax)
    new = torch.where(first[:, None] == 0, need, torch.maximum(old, need))
    cells = codes.view(n, H, per, BLOCK, D)
    kept = cells[pg, :, bk]                                         # [blocks, H, BLOCK, D]
    again = kept.view(torch.float8_e4m3fn).float() * (old / new)[..., None, None]
    again = again.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    rows = torch.arange(BLOCK, device="cuda")[None] < first[:, None]
    cells[pg, :, bk] = torch.where(rows[:, None, :, None], again, kept)
    scales[pg, :, bk] = new
    q = (x / new[at][..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    codes[page, :, off] = q


def _above(st, case):
    """Row of each node's parent among all rows, -1 where it has none."""
    cu = st["cu"].long()
    i = torch.arange(st["tokens"], device="cuda")
    s = torch.searchsorted(cu[1:], i, right=True)
    up = st["parent"].long()
    return torch.where(up < 0, up, up + cu[s])


def _tree(st, case):
    """Bits of the nodes on the way to each node (itself among them), int32 [tokens, words], and its depth."""
    cu, T = st["cu"].long(), st["tokens"]
    words = -(-st["max_q"] // 32)
    i = torch.arange(T, device="cuda")
    local = i - cu[torch.searchsorted(cu[1:], i, right=True)]
    seen = local[:, None] == torch.arange(32 * words, device="cuda")
    up = _above(st, case)
    at, depth = up, torch.zeros_like(up)
    for _ in range(st["max_q"]):                                    # one step towards the root at a time
        there = at >= 0
        to = at.clamp(min=0)
        seen = seen | (there[:, None] & (local[to, None] == torch.arange(32 * words, device="cuda")))
        depth = depth + there
        at = torch.where(there, up[to], at)
    bits = (seen.view(T, words, 32).long() << torch.arange(32, device="cuda")).sum(2)
    return torch.where(bits >= 1 << 31, bits - (1 << 32), bits).int(), depth.int()


def _depths(st, case):
    up = _above(st, case)
    at, depth = up, torch.zeros_like(up)
    for _ in range(st["max_q"]):
        there = at >= 0
        depth = depth + there
        at = torch.where(there, up[at.clamp(min=0)], at)
    return depth.int()


def _attend(st):
    case = st["case"]
    S, H, G, D, P = case["seqs"], case["heads"], case["group"], case["dim"], case["page"]
    Q, L = st["max_q"], st["table"].shape[1] * P
    cu, length = st["cu"].long(), st["length"].long()
    n = cu[1:] - cu[:-1]
    i = torch.arange(Q, device="cuda")
    there = i[None] < n[:, None]                                    # [S, Q]
    rows_at = (cu[:-1, None] + i[None]).clamp(max=st["tokens"] - 1)
    q = st["q"].float()[rows_at]                                    # [S, Q, H G, D]
    q = q.view(S, Q, H, G, D).permute(0, 2, 3, 1, 4).reshape(S, H, G * Q, D)
    table = st["table"].long()

    def rows(codes, scales):                                        # [S, H, L, D]
        x = codes[table].view(torch.float8_e4m3fn).float()          # [S, pages, H, P, D]
        x *= scales[table].repeat_interleave(BLOCK, 3)[..., None]
        return x.permute(0, 2, 1, 3, 4).reshape(S, H, L, D)

    score = torch.matmul(q, rows(st["kc"], st["ks"]).transpose(2, 3)).view(S, H, G, Q, L) / math.sqrt(D)
    first = (length - n)[:, None, None]                             # place of the sequence's first node
    node = torch.arange(L, device="cuda")[None, None] - first       # [S, 1, L]
    word = st["mask"].long()[rows_at].gather(2, (node.clamp(0, Q - 1) // 32).expand(S, Q, L))
    bit = (word >> (node.clamp(0, Q - 1) % 32)) & 1
    keep = (node < 0) | ((bit == 1) & (node <= i[None, :, None]))
    keep &= torch.arange(L, device="cuda")[None, None] < length[:, None, None]
    score.masked_fill_(~keep[:, None, None], -math.inf)
    top = score.amax(4, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    score.sub_(top).exp_()
    total = score.sum(4, keepdim=True)
    out = torch.matmul(score.view(S, H, G * Q, L), rows(st["vc"], st["vs"])).view(S, H, G, Q, D)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    lse = (top + torch.log(total))[..., 0]
    out = out.permute(0, 3, 1, 2, 4).reshape(S, Q, H * G, D)[there]
    lse = lse.permute(0, 3, 1, 2).reshape(S, Q, H * G)[there]
    return out.to(DT[case["dtype"]]), lse


def _verify(st):
    """Nodes in order of index; w is what the target has left at the node that the sequence has come to, in 64 bits."""
    S, Q = st["case"]["seqs"], st["max_q"]
    cu = st["cu"].long()
    s, first, n = torch.arange(S, device="cuda"), cu[:-1], cu[1:] - cu[:-1]
    cur, count = torch.zeros_like(first), torch.zeros_like(first)
    path = torch.full((S, Q), -1, dtype=torch.int64, device="cuda")
    path[:, 0] = 0
    w, mass = st["target"][first].double(), torch.ones(S, dtype=torch.float64, device="cuda")
    for j in range(1, Q):
        row = (first + j).clamp(max=st["tokens"] - 1)
        child = (j < n) & (st["parent"].long()[row] == cur)
        x, u = st["drawn"].long()[row], st["accept"].double()[row]
        q = torch.ones_like(u) if st["draft"] is None else st["draft"][first + cur, x].double()
        yes = child & (u * q * mass < w[s, x])
        no = child & ~yes
        if st["draft"] is None:
            less = w.scatter(1, x[:, None], 0.0)
        else:
            less = (w - mass[:, None] * st["draft"][first + cur].double()).clamp(min=0)
        w = torch.where(no[:, None], less, w)
        mass = torch.where(no, w.sum(1), mass)
        cur, count = torch.where(yes, torch.full_like(cur, j), cur), count + yes
        path[s, count] = torch.where(yes, cur, path[s, count])
        w = torch.where(yes[:, None], st["target"][first + cur].double(), w)
        mass = torch.where(yes, torch.ones_like(mass), mass)
    upto = w.cumsum(1)
    none = upto[:, -1:] <= 0                                        # nothing left: the target itself
    upto = torch.where(none, st["target"][first + cur].double().cumsum(1), upto)
    token = (upto <= st["sample"].double()[:, None] * upto[:, -1:]).sum(1)
    return count.int(), path.int(), token.int()


def run(st):
    case, op = st["case"], st["case"]["op"]
    if own:
        import activation_sparse_rank_gb300 as pi
        if op == "rotary":
            return pi.rotary(st["x"], st["pos"], st["rope"])
        if op == "rotary_grad":
            return pi.rotary_backward(st["x"], st["pos"], st["rope"])
        if op == "append":
            q = st["cache"].append(st["k"], st["v"], st["table"], st["cu"], st["before"], st["rope"], positions=st["pos"],
                                   q=st["q"])
            return q, st["kc"].view(torch.float8_e4m3fn), st["ks"], st["vc"].view(torch.float8_e4m3fn), st["vs"]
        if op == "tree":
            return pi.draft_tree(st["parent"], st["cu"], st["max_q"])
        if op == "attend":
            return st["cache"].attention(st["q"], st["table"], st["cu"], st["length"], max_q=st["max_q"], tree=st["mask"],
                                         ws=st["ws"], want_lse=True)
        v = pi.verify_draft(st["target"], st["draft"], st["drawn"], st["parent"], st["cu"], st["accept"], st["sample"],
                            st["max_q"])
        return v.accepted, v.path, v.token
    if op in ("rotary", "rotary_grad"):
        y = _rotate(st["x"], st["pos"], st["freq"], st["mag"], case["turned"], case["pairs"], 1.0 if op == "rotary" else -1.0)
        return y.to(DT[case["dtype"]])
    if op == "append":
        place, page, off = _places(st)
        how = (place if st["pos"] is None else st["pos"], st["freq"], st["mag"], case["turned"], case["pairs"], 1.0)
        _write(_rotate(st["k"], *how), st["kc"], st["ks"], page, off)
        _write(st["v"], st["vc"], st["vs"], page, off)
        q = _rotate(st["q"], *how).to(DT[case["dtype"]])
        return q, st["kc"].view(torch.float8_e4m3fn), st["ks"], st["vc"].view(torch.float8_e4m3fn), st["vs"]
    if op == "tree":
        return _tree(st, case)
    if op == "attend":
        return _attend(st)
    return _verify(st)


# ---- definitions in 64 bits -------------------------------------------------------

def _e4m3(v):
    """v (float64) rounded to the nearest E4M3 value, ties to even, at most 448."""
    a = v.abs().clamp(max=448.0)
    _, e = torch.frexp(a)
    step = torch.ldexp(torch.ones_like(a), torch.clamp(e - 4, min=-9))
    return torch.copysign(torch.round(a / step) * step, v)


def _e4m3_value(codes):
    """The float64 value of each E4M3 bit pattern."""
    c = codes.to(torch.int64)
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, torch.ldexp(m, torch.full_like(e, -9)), torch.ldexp(8 + m, e - 10))
    return torch.where(c > 127, -v, v)


def _exact_turn(x, pos, case, back=False):
    """Pairs as complex numbers times magnitude e^(i angle)."""
    R, s = case["turned"], case["factor"]
    freq = []
    for i in range(R // 2):
        f = BASE ** (-2 * i / R)
        if case["scaling"] == "linear":
            f /= s
        elif case["scaling"] == "ntk" and R > 2:
            f = (BASE * s ** (R / (R - 2))) ** (-2 * i / R)
        elif case["scaling"] == "yarn":
            lo = max(0, math.floor(R * math.log(NEAR / (64 * math.pi)) / (2 * math.log(BASE))))
            hi = min(R - 1, math.ceil(R * math.log(NEAR / (2 * math.pi)) / (2 * math.log(BASE))))
            far = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f = f * (1 - far) + f / s * far
        freq.append(f)
    mag = 1 + math.log(s) / 10 if case["scaling"] == "yarn" else 1.0
    angle = pos.double()[:, None] * torch.tensor(freq, dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.full_like(angle, mag), -angle if back else angle)[:, None]
    x = x.double()
    if case["pairs"] == "half":
        z = torch.complex(x[..., :R // 2], x[..., R // 2:R]) * turn
        z = torch.cat((z.real, z.imag), -1)
    else:
        z = torch.view_as_real(torch.view_as_complex(x[..., :R].unflatten(-1, (-1, 2)).contiguous()) * turn).flatten(-2)
    return torch.cat((z, x[..., R:]), -1)


def _exact_append(st):
    case = st["case"]
    P, per = case["page"], case["page"] // BLOCK
    table, cu, before = st["table"].tolist(), st["cu"].tolist(), st["before"].tolist()
    pos = st["pos"]
    if pos is None:
        pos = torch.cat([torch.arange(b, b + cu[s + 1] - cu[s], device="cuda") for s, b in enumerate(before)])
    out = [_exact_turn(st["q"], pos, case)]
    for x, codes, scales in ((_exact_turn(st["k"], pos, case), st["kc"], st["ks"]), (st["v"].double(), st["vc"], st["vs"])):
        value, scale = _e4m3_value(codes), scales.double().clone()
        groups = {}                                                 # (tokens, first offset) -> rows and places
        for s in range(len(before)):
            p, end = before[s], before[s] + cu[s + 1] - cu[s]
            while p < end:
                m = min(end, (p // BLOCK + 1) * BLOCK) - p
                groups.setdefault((m, p % BLOCK), []).append((cu[s] + p - before[s], table[s][p // P], (p % P) // BLOCK))
                p += m
        for (m, at), places in groups.items():
            row, pg, bk = (torch.tensor(v, device="cuda") for v in zip(*places))
            new = x[row[:, None] + torch.arange(m, device="cuda")].transpose(1, 2)      # [n, H, m, D]
            s = torch.exp2(torch.ceil(torch.log2(new.abs().amax((2, 3)).clamp(min=2.0 ** -200) / 448)).clamp(min=MIN_EXP))
            off = bk[:, None] * BLOCK + torch.arange(at + m, device="cuda")
            if at:
                old = scale[pg, :, bk]
                s = torch.maximum(s, old)
                kept = value[pg[:, None], :, off[:, :at]].transpose(1, 2)
                new = torch.cat((kept * old[..., None, None], new), 2)
            value[pg[:, None], :, off] = _e4m3(new / s[..., None, None]).transpose(1, 2)
            scale[pg, :, bk] = s
        out += [value, scale]
    return tuple(out)


def _ways(st):
    """For each node of each sequence the nodes on its way, itself last."""
    cu, parent = st["cu"].tolist(), st["parent"].tolist()
    out = []
    for s in range(len(cu) - 1):
        ways = []
        for p in parent[cu[s]:cu[s + 1]]:
            ways.append((ways[p] if p >= 0 else []) + [len(ways)])
        out.append(ways)
    return out


def _exact_tree(st):
    mask, depth = [], []
    for ways in _ways(st):
        for way in ways:
            bits = sum(1 << j for j in way)
            words = [bits >> 32 * k & 0xffffffff for k in range(-(-st["max_q"] // 32))]
            mask.append([w - (1 << 32) if w >> 31 else w for w in words])
            depth.append(len(way) - 1)
    return torch.tensor(mask, dtype=torch.int32, device="cuda"), torch.tensor(depth, dtype=torch.int32, device="cuda")


def _exact_attend(st):
    case = st["case"]
    H, G, D, P = case["heads"], case["group"], case["dim"], case["page"]
    cu, length, table = st["cu"].tolist(), st["length"].tolist(), st["table"]
    out = torch.zeros(st["tokens"], H * G, D, dtype=torch.float64, device="cuda")
    lse = torch.full((st["tokens"], H * G), -math.inf, dtype=torch.float64, device="cuda")
    for s, (n, ways) in enumerate(zip(length, _ways(st))):
        m = cu[s + 1] - cu[s]
        if n == 0:
            continue
        pg = table[s, :-(-n // P)].long()
        hide = torch.ones(m, n, dtype=torch.bool)
        for i, way in enumerate(ways):
            hide[i, :max(0, n - m)] = False
            hide[i, [n - m + j for j in way if n - m + j >= 0]] = False
        hide = hide.cuda()
        seen = ~hide.all(1)
        for h in range(H):
            k, v = ((_e4m3_value(c[pg, h]) * z[pg, h].double().repeat_interleave(BLOCK, 1)[..., None]).reshape(-1, D)[:n]
                    for c, z in ((st["kc"], st["ks"]), (st["vc"], st["vs"])))
            q = st["q"][cu[s]:cu[s + 1], h * G:(h + 1) * G].double().transpose(0, 1)         # [G, m, D]
            a = (q @ k.T / math.sqrt(D)).masked_fill(hide, -math.inf)
            z = torch.logsumexp(a, 2)
            a = torch.exp(a - z[..., None])
            out[cu[s]:cu[s + 1], h * G:(h + 1) * G] = torch.where(seen[:, None, None], (a @ v).transpose(0, 1), 0.0)
            lse[cu[s]:cu[s + 1], h * G:(h + 1) * G] = z.T
    return out, lse


def _exact_verify(st):
    """Each sequence by itself: from node to node, at each the children in turn."""
    cu, parent, drawn = st["cu"].tolist(), st["parent"].tolist(), st["drawn"].tolist()
    accept, sample = st["accept"].tolist(), st["sample"].tolist()
    count, path, token = [], [], []
    for s in range(len(cu) - 1):
        way, done = [0], False
        while not done:
            node, done = way[-1], True
            left, mass = st["target"][cu[s] + node].double(), 1.0
            for j in range(node + 1, cu[s + 1] - cu[s]):
                if parent[cu[s] + j] != node:
                    continue
                x = drawn[cu[s] + j]
                q = st["draft"][cu[s] + node].double() if st["draft"] is not None else torch.zeros_like(left).index_fill(
                    0, torch.tensor([x], device="cuda"), 1.0)
                if accept[cu[s] + j] * q[x].item() * mass < left[x].item():
                    way.append(j)
                    done = False
                    break
                left = torch.relu(left - mass * q) if st["draft"] is not None else left * (1 - q)
                mass = left.sum().item()
        if mass == 0:
            left = st["target"][cu[s] + way[-1]].double()
        upto = torch.cumsum(left, 0)
        token.append(int(torch.searchsorted(upto, sample[s] * upto[-1], right=True)))
        count.append(len(way) - 1)
        path.append(way + [-1] * (st["max_q"] - len(way)))
    return tuple(torch.tensor(v, dtype=torch.int32, device="cuda") for v in (count, path, token))


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("rotary", "rotary_grad"):
        return _exact_turn(st["x"], st["pos"], case, op == "rotary_grad")
    if op == "append":
        return _exact_append(st)
    if op == "tree":
        return _exact_tree(st)
    if op == "attend":
        return _exact_attend(st) if case["seqs"] * case["heads"] <= 8192 else None
    return _exact_verify(st)
