"""Measured cases of the operators around the FFN block.

Four operators that a decode step runs beside the predictor-gated FFN:
the 8-bit key/value cache (written, read back), attention over it, layer norm
(forward and backward) and the log-probabilities of given tokens.  Each has a
plain form in elementary torch operations (binary32, rounded once at the end)
and a definition in 64 bits; `own` selects this package's kernels instead.
"""
import math

import torch

own = False

BLOCK = 16          # tokens that share one scale of the cache
MIN_EXP = -64       # smallest scale of the cache: 2^MIN_EXP
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}


def listed():
    return [
        # one decode step of 32 sequences of a 4096-wide model (32 heads of 128): one token each,
        # into blocks that already hold tokens
        dict(name="write_step", op="write", seqs=32, lo=5, hi=700, q=1, heads=32, dim=128, page=64, dtype="f16"),
        # prompts of five requests (ragged) entering the cache of an 8192-wide model with 8 kv heads
        dict(name="write_prompt", op="write", seqs=5, lo=0, hi=0, q=6001, heads=8, dim=128, page=64, dtype="bf16"),
        # cached prefixes of three requests read back to 16 bits, for a copy to another device or a prompt pass
        dict(name="read_prefix", op="read", seqs=3, lo=3, hi=90, q=20011, heads=8, dim=64, page=32, dtype="f16"),
        # the smallest decode step: one sequence of the 1024-wide layer (16 heads of 64)
        dict(name="attend_one", op="attend", seqs=1, lo=513, hi=513, q=1, heads=16, group=1, dim=64, page=64, dtype="f16"),
        # a served batch: 64 sequences of very different lengths, 64 query heads on 8 kv heads
        dict(name="attend_batch", op="attend", seqs=64, lo=1, hi=8191, q=1, heads=8, group=8, dim=128, page=64,
             dtype="bf16"),
        # one long document: 128 query heads of 64 on 8 kv heads, a single token
        dict(name="attend_long", op="attend", seqs=1, lo=130001, hi=130001, q=1, heads=8, group=16, dim=64, page=128,
             dtype="f16"),
        # a prompt in chunks: up to 512 new tokens a sequence over the cache that holds them and what came before
        dict(name="attend_chunk", op="attend", seqs=4, lo=2050, hi=8190, q=512, heads=8, group=8, dim=128, page=64,
             dtype="bf16"),
        # between the blocks of a decode step: residual plus the FFN's binary32 output, then the norm, 8 tokens
        dict(name="norm_step", op="norm", rows=8, dim=4096, dtype="f16", add=True),
        # the same over a long prompt of an 8192-wide model
        dict(name="norm_prompt", op="norm", rows=16384, dim=8192, dtype="bf16", add=False),
        # fine-tuning: the norm's gradient with respect to its input, weight and bias
        dict(name="norm_backward", op="norm_grad", rows=16001, dim=4096, dtype="bf16", add=True),
        # the tokens a decode step has just sampled: 16 rows of binary32 logits, five alternatives
        dict(name="score_step", op="score", rows=16, vocab=50007, top=5, dtype="f32"),
        # scoring of given texts: 2048 positions at once
        dict(name="score_text", op="score", rows=2048, vocab=131072, top=20, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("write", "read", "attend", "attend", "norm", "norm_grad", "score"))
    if op in ("write", "read"):
        heads, dim = _log(rng, 1, 96), rng.choice((64, 96, 128, 256))
        tokens = max(1, _log(rng, 1, (1 << 24) // (heads * dim)))      # rows of k and v in all
        seqs = min(tokens, _log(rng, 1, 256))
        return dict(op=op, seqs=seqs, lo=0, hi=rng.choice((0, 40, 300)), q=max(1, tokens // seqs), heads=heads, dim=dim,
                    page=rng.choice((16, 32, 64, 128)), dtype=rng.choice(("f16", "bf16", "f32")))
    if op == "attend":
        heads, dim, group = _log(rng, 1, 32), rng.choice((64, 96, 128, 256)), rng.choice((1, 1, 2, 4, 5, 7, 8, 16))
        keys = _log(rng, 64, min(1 << 17, (1 << 28) // (heads * dim)))
        seqs = min(_log(rng, 1, 96), max(1, (1 << 28) // (heads * dim * keys)))
        q = rng.choice((1, 1, 1, 1, 3, 8, _log(rng, 16, 400)))
        while q > 1 and seqs * q * keys * heads * group * dim > 1 << 36:
            q = max(1, q // 2)
        return dict(op=op, seqs=seqs, lo=rng.choice((0, 1, keys // 2, keys)), hi=keys, q=q, heads=heads, group=group,
                    dim=dim, page=rng.choice((16, 32, 64, 128)), dtype=rng.choice(("f16", "bf16")))
    if op in ("norm", "norm_grad"):
        dim = _log(rng, 64, 16384) if rng.random() < 0.5 else 8 * _log(rng, 8, 2048)
        return dict(op=op, rows=_log(rng, 1, min(40000, (1 << 26) // dim)), dim=dim,
                    dtype=rng.choice(("f16", "bf16", "f32")), add=rng.random() < 0.5)
    vocab = _log(rng, 500, 150000)
    return dict(op="score", rows=_log(rng, 1, min(20000, (1 << 27) // vocab)), vocab=vocab, top=rng.choice((0, 1, 5, 20, 32)),
                dtype=rng.choice(("f16", "bf16", "f32")))


def _spread(n, lo, hi):
    """n lengths between lo and hi, the longest among them, by a fixed rule."""
    return [hi if s == 0 else lo + int((hi - lo) * ((s * 0.6180339887498949) % 1.0)) for s in range(n)]


def _lengths(case):
    """Per sequence: tokens in the cache before the new ones, and new tokens.  A decode step has one new token of
    each sequence; `attend` counts the new ones among hi."""
    n, q = case["seqs"], case["q"]
    new = [q] * n if q <= 8 else [max(1, q - int(q * 0.5 * ((s * 0.7548776662466927) % 1.0))) for s in range(n)]
    before = _spread(n, case["lo"], case["hi"])
    if case["op"] == "attend":
        before = [b - m for b, m in zip(before, new)]    # below 0: rows with nothing to attend to
    return before, new


def _pairs(case):
    """(query, key) pairs a head has to compute, and keys read, over all sequences."""
    pairs = keys = 0
    for b, m in zip(*_lengths(case)):
        first = max(0, -b)                               # rows before it see nothing
        pairs += sum((b + first + 1, b + m)) * (m - first) // 2 if m > first else 0
        keys += max(0, b + m)
    return pairs, keys


def work(case):
    op, e = case["op"], SIZE[case["dtype"]]
    if op in ("write", "read"):
        rows = sum(_lengths(case)[1]) * case["heads"]
        return dict(bytes=2 * rows * (case["dim"] * (e + 1) + 4 / BLOCK), flops=4 * rows * case["dim"])
    if op == "attend":
        pairs, keys = _pairs(case)
        rows = sum(_lengths(case)[1]) * case["heads"] * case["group"]
        return dict(bytes=2 * keys * case["heads"] * (case["dim"] + 4 / BLOCK) + rows * (2 * case["dim"] * e + 4),
                    flops=4 * pairs * case["heads"] * case["group"] * case["dim"])
    if op == "norm":
        n = case["rows"] * case["dim"]
        return dict(bytes=n * (2 * e + (4 + e if case["add"] else 0)) + 8 * case["rows"] + 2 * e * case["dim"], flops=8 * n)
    if op == "norm_grad":
        n = case["rows"] * case["dim"]
        return dict(bytes=n * (3 * e + (e if case["add"] else 0)) + 8 * case["rows"] + (8 + e) * case["dim"], flops=14 * n)
    return dict(bytes=case["rows"] * (case["vocab"] * e + 16 + 8 * case["top"]), flops=6 * case["rows"] * case["vocab"])


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


def _cache_state(case, gen):
    before, new = _lengths(case)
    page, heads, dim = case["page"], case["heads"], case["dim"]
    need = [max(1, -(-max(0, b + m) // page)) for b, m in zip(before, new)]
    pages = sum(need) + 2
    st = dict(max_q=max(new), tokens=sum(new))
    order = torch.randperm(pages, device="cuda", generator=gen).int()
    table = torch.zeros(len(need), max(need), dtype=torch.int32)
    used, order = 0, order.cpu()
    for s, n in enumerate(need):
        table[s, :n] = order[used:used + n]
        used += n
    cu = torch.tensor([0] + new, dtype=torch.int64).cumsum(0).to(torch.int32)
    st.update(table=table.cuda(), cu=cu.cuda(), before=torch.tensor(before, dtype=torch.int32).cuda(),
              length=torch.tensor([max(0, b + m) for b, m in zip(before, new)], dtype=torch.int32).cuda())
    st["kc"], st["ks"] = _pool(pages, heads, page, dim, gen)
    st["vc"], st["vs"] = _pool(pages, heads, page, dim, gen)
    if own:
        import activation_sparse_rank_gb300 as pi
        st["cache"] = pi.KVCache.wrap(st["kc"], st["ks"], st["vc"], st["vs"])
    return st


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    op, dt = case["op"], DT[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        return torch.empty(shape, device="cuda").normal_(mean, std, generator=gen).to(dtype)

    if op in ("write", "read", "attend"):
        st = _cache_state(case, gen)
        T, H, D = st["tokens"], case["heads"], case["dim"]
        if op == "write":
            qkv = normal(T, 3 * H * D)                   # k and v as a packed projection leaves them
            st["k"], st["v"] = qkv[:, H * D:2 * H * D].view(T, H, D), qkv[:, 2 * H * D:].view(T, H, D)
        elif op == "attend":
            st["q"] = normal(T, H * case["group"], D, std=1.5)
            if own:
                st["ws"] = st["cache"].attention_workspace(st["q"].shape[1], T, case["seqs"])
    elif op in ("norm", "norm_grad"):
        R, D = case["rows"], case["dim"]
        st = dict(x=normal(R, D, mean=0.3, std=1.7), w=normal(D, mean=1.0, std=0.2), b=normal(D, std=0.2), add=None)
        if op == "norm":
            if case["add"]:
                st["add"] = normal(R, D, dtype=torch.float32)
        else:
            st["dy"], st["dsum"] = normal(R, D), normal(R, D) if case["add"] else None
            xf = st["x"].float()
            st["mean"] = xf.mean(1)
            st["rstd"] = torch.rsqrt((xf - st["mean"][:, None]).square().mean(1) + 1e-5)
    else:
        R, V = case["rows"], case["vocab"]
        x = torch.empty(R, V, device="cuda").normal_(0.0, 2.5, generator=gen)
        st = dict(targets=torch.randint(0, V, (R,), device="cuda", generator=gen).int())
        x.scatter_add_(1, st["targets"][:, None].long(), 6.0 * torch.rand(R, 1, device="cuda", generator=gen))
        st["logits"] = x.to(dt)
    st["case"] = dict(case)
    return st


# ---- plain forms ----------------------------------------------------------------

def _places(st):
    """Of every new token: sequence, page and offset in the page."""
    P = st["case"]["page"]
    cu = st["cu"].long()
    i = torch.arange(st["tokens"], device="cuda")
    s = torch.searchsorted(cu[1:], i, right=True)
    pos = st["before"].long()[s] + i - cu[s]
    return st["table"].long()[s, pos // P], pos % P


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


def _values(codes, scales):
    """The values a pool stands for, binary32 [pages, heads, page, dim]."""
    return codes.view(torch.float8_e4m3fn).float() * scales.repeat_interleave(BLOCK, 2)[..., None]


def _attend(st):
    case = st["case"]
    S, H, G, D, P = case["seqs"], case["heads"], case["group"], case["dim"], case["page"]
    Q, L = st["max_q"], st["table"].shape[1] * P
    cu, length = st["cu"].long(), st["length"].long()
    n = cu[1:] - cu[:-1]
    i = torch.arange(Q, device="cuda")
    there = i[None] < n[:, None]                                    # [S, Q]
    q = st["q"].float()[(cu[:-1, None] + i[None]).clamp(max=st["tokens"] - 1)]   # [S, Q, H G, D]
    q = q.view(S, Q, H, G, D).permute(0, 2, 3, 1, 4).reshape(S, H, G * Q, D)
    table = st["table"].long()

    def rows(codes, scales):                                        # [S, H, L, D]
        x = codes[table].view(torch.float8_e4m3fn).float()          # [S, pages, H, P, D]
        x *= scales[table].repeat_interleave(BLOCK, 3)[..., None]
        return x.permute(0, 2, 1, 3, 4).reshape(S, H, L, D)

    score = torch.matmul(q, rows(st["kc"], st["ks"]).transpose(2, 3)).view(S, H, G, Q, L) / math.sqrt(D)
    last = length[:, None] - n[:, None] + i[None]                   # a query sees the keys up to its own
    keep = torch.arange(L, device="cuda")[None, None] <= last[..., None]
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


def _norm(x, add, w, b, dt):
    total = None
    if add is not None:
        total = (x.float() + add.float()).to(dt)
        x = total
    x = x.float()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = torch.rsqrt(c.square().mean(1) + 1e-5)
    return (c * rstd[:, None] * w.float() + b.float()).to(dt), total, mean, rstd


def _norm_grad(st, dt):
    xh = (st["x"].float() - st["mean"][:, None]) * st["rstd"][:, None]
    dy = st["dy"].float()
    g = dy * st["w"].float()
    dx = (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True)) * st["rstd"][:, None]
    if st["dsum"] is not None:
        dx = dx + st["dsum"].float()
    return dx.to(dt), (dy * xh).sum(0), dy.sum(0)


def _score(x, targets, top):
    x = x.float()
    peak = x.amax(1, keepdim=True)
    z = x - peak
    e = z.exp()
    total = e.sum(1, keepdim=True)
    lse = (peak + total.log())[:, 0]
    entropy = total.log()[:, 0] - (e * z).sum(1) / total[:, 0]
    logp = x.gather(1, targets.long()[:, None])[:, 0] - lse
    if not top:
        return logp, entropy, lse
    bits = x.view(torch.int32).long()                               # an order of whole numbers: value, then lowest index
    key = torch.where(bits < 0, -(bits & 0x7fffffff), bits) * (1 << 31) + (x.shape[1] - 1 - torch.arange(x.shape[1], device="cuda"))
    at = key.topk(top, 1).indices
    return logp, entropy, lse, at.int(), x.gather(1, at) - lse[:, None]


def run(st):
    case, op = st["case"], st["case"]["op"]
    dt = DT[case["dtype"]]
    if own:
        import activation_sparse_rank_gb300 as pi
        if op == "write":
            st["cache"].write(st["k"], st["v"], st["table"], st["cu"], st["before"])
            return st["kc"].view(torch.float8_e4m3fn), st["ks"], st["vc"].view(torch.float8_e4m3fn), st["vs"]
        if op == "read":
            return st["cache"].read(st["table"], st["cu"], st["before"], st["tokens"], dtype=dt)
        if op == "attend":
            return st["cache"].attention(st["q"], st["table"], st["cu"], st["length"], max_q=st["max_q"], ws=st["ws"],
                                         want_lse=True)
        if op == "norm":
            y, total, mean, rstd = pi.layer_norm(st["x"], st["w"], st["b"], add=st["add"], want_stats=True)
            return dict(y=y, sum=total, mean=mean, rstd=rstd)
        if op == "norm_grad":
            return pi.layer_norm_backward(st["dy"], st["x"], st["w"], st["mean"], st["rstd"], d_sum=st["dsum"])
        r = pi.token_logprobs(st["logits"], st["targets"], top_k=case["top"])
        return (r.logprob, r.entropy, r.lse) + ((r.top_index, r.top_logprob) if case["top"] else ())
    if op == "write":
        page, off = _places(st)
        _write(st["k"], st["kc"], st["ks"], page, off)
        _write(st["v"], st["vc"], st["vs"], page, off)
        return st["kc"].view(torch.float8_e4m3fn), st["ks"], st["vc"].view(torch.float8_e4m3fn), st["vs"]
    if op == "read":
        page, off = _places(st)
        return tuple(
            (c[page, :, off].view(torch.float8_e4m3fn).float() * s[page, :, off // BLOCK][..., None]).to(dt)
            for c, s in ((st["kc"], st["ks"]), (st["vc"], st["vs"])))
    if op == "attend":
        return _attend(st)
    if op == "norm":
        y, total, mean, rstd = _norm(st["x"], st["add"], st["w"], st["b"], dt)
        return dict(y=y, sum=total, mean=mean, rstd=rstd)
    if op == "norm_grad":
        return _norm_grad(st, dt)
    return _score(st["logits"], st["targets"], case["top"])


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


def _exact_write(st):
    P, per = st["case"]["page"], st["case"]["page"] // BLOCK
    table, cu, before = st["table"].tolist(), st["cu"].tolist(), st["before"].tolist()
    out = []
    for x, codes, scales in ((st["k"], st["kc"], st["ks"]), (st["v"], st["vc"], st["vs"])):
        value, scale = _e4m3_value(codes), scales.double().clone()
        x = x.double()
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


def _exact_read(st):
    P = st["case"]["page"]
    table, cu, before = st["table"].tolist(), st["cu"].tolist(), st["before"].tolist()
    out = []
    for codes, scales in ((st["kc"], st["ks"]), (st["vc"], st["vs"])):
        rows = []
        for s in range(len(before)):
            pos = torch.arange(before[s], before[s] + cu[s + 1] - cu[s], device="cuda")
            pg = torch.tensor(table[s], device="cuda")[pos // P]
            rows.append(_e4m3_value(codes[pg, :, pos % P]) * scales.double()[pg, :, (pos % P) // BLOCK][..., None])
        out.append(torch.cat(rows))
    return tuple(out)


def _exact_attend(st):
    case = st["case"]
    H, G, D, P = case["heads"], case["group"], case["dim"], case["page"]
    cu, length, table = st["cu"].tolist(), st["length"].tolist(), st["table"]
    out = torch.zeros(st["tokens"], H * G, D, dtype=torch.float64, device="cuda")
    lse = torch.full((st["tokens"], H * G), -math.inf, dtype=torch.float64, device="cuda")
    for s, n in enumerate(length):
        m = cu[s + 1] - cu[s]
        if n == 0:
            continue
        pg = table[s, :-(-n // P)].long()
        for h in range(H):
            k, v = ((_e4m3_value(c[pg, h]) * z[pg, h].double().repeat_interleave(BLOCK, 1)[..., None]).reshape(-1, D)[:n]
                    for c, z in ((st["kc"], st["ks"]), (st["vc"], st["vs"])))
            hide = torch.arange(n, device="cuda")[None] > torch.arange(n - m, n, device="cuda")[:, None]
            seen = torch.arange(n - m, n, device="cuda") >= 0
            q = st["q"][cu[s]:cu[s + 1], h * G:(h + 1) * G].double().transpose(0, 1)         # [G, m, D]
            a = (q @ k.T / math.sqrt(D)).masked_fill(hide, -math.inf)
            z = torch.logsumexp(a, 2)
            a = torch.exp(a - z[..., None])
            out[cu[s]:cu[s + 1], h * G:(h + 1) * G] = torch.where(seen[:, None, None], (a @ v).transpose(0, 1), 0.0)
            lse[cu[s]:cu[s + 1], h * G:(h + 1) * G] = z.T
    return out, lse


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "write":
        return _exact_write(st)
    if op == "read":
        return _exact_read(st)
    if op == "attend":
        pairs, _ = _pairs(case)
        if 4 * pairs * case["heads"] * case["group"] * case["dim"] > 4e12 or case["seqs"] * case["heads"] > 8192:
            return None
        return _exact_attend(st)
    if op == "norm":
        x = st["x"].double()
        total = None
        if st["add"] is not None:
            total = x + st["add"].double()
            x = total.to(DT[case["dtype"]]).double()                # the norm is of the stored sum
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = (var + 1e-5) ** -0.5
        return dict(y=(x - mean[:, None]) * rstd[:, None] * st["w"].double() + st["b"].double(), sum=total, mean=mean,
                    rstd=rstd)
    if op == "norm_grad":
        n = case["dim"]
        dy, w, r = st["dy"].double(), st["w"].double(), st["rstd"].double()[:, None]
        xh = (st["x"].double() - st["mean"].double()[:, None]) * r
        a, c = (dy @ w)[:, None], ((dy * xh) @ w)[:, None]
        dx = r / n * (n * dy * w - a - xh * c)
        if st["dsum"] is not None:
            dx += st["dsum"].double()
        return dx, torch.einsum("td,td->d", dy, xh), dy.sum(0)
    x = st["logits"].double()
    p = torch.log_softmax(x, 1)
    lse = torch.logsumexp(x, 1)
    entropy = -(p.exp() * p).sum(1)
    logp = p[torch.arange(len(p), device="cuda"), st["targets"].long()]
    if not case["top"]:
        return logp, entropy, lse
    best = torch.topk(p, case["top"], 1).values                     # ties have one value, so their order says nothing
    return logp, entropy, lse, None, best
