"""Decoding with drafted trees on a one-layer rotary model: append, tree, attention, verification and
the accepted tokens' way into the cache, step after step, each against its definition."""
import numpy as np
import pytest
import torch

from oracle import operators as O
from tests.kv_helpers import batch, oracle_of
from tests.test_gpu_tree_attention import check

pytestmark = pytest.mark.gpu

HEADS, GROUP, DIM, PAGE, VOCAB, NODES = 2, 4, 64, 16, 997, 9
PARENT = [-1, 0, 0, 1, 1, 2, 3, 3, 6]


@pytest.fixture(scope="module")
def pi():
    import __graft_entry__
    __graft_entry__.build()
    import activation_sparse_rank_gb300 as pi
    return pi


def ints(v):
    return torch.tensor(np.asarray(v, np.int32), device="cuda")


class Model:
    """Queries, keys and values of a token by table; the next token's logits from the attention's output."""

    def __init__(self, dtype):
        g = torch.Generator().manual_seed(3)
        width = (GROUP + 2) * HEADS * DIM
        self.qkv = torch.randn(VOCAB, width, generator=g).to(dtype).cuda()
        self.out = (torch.randn(GROUP * HEADS * DIM, VOCAB, generator=g) * 0.06).cuda()
        self.bigram = torch.softmax(torch.randn(VOCAB, VOCAB, generator=g) * 1.5, 1).cuda()

    def heads(self, tokens):
        x = self.qkv[tokens.long()].view(-1, (GROUP + 2) * HEADS, DIM)
        return x[:, :GROUP * HEADS], x[:, GROUP * HEADS:(GROUP + 1) * HEADS], x[:, (GROUP + 1) * HEADS:]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("sequences", [1, 3])
def test_steps(pi, dtype, sequences):
    model, rope = Model(dtype), pi.Rotary(DIM, base=500.0)
    rng, gen = np.random.default_rng(sequences), torch.Generator("cuda").manual_seed(5)
    prompt = [37, 1, 64][:sequences]
    b = batch([0] * sequences, [n + 80 for n in prompt], PAGE)
    cache, table = pi.KVCache(b["pages"], HEADS, DIM, PAGE), b["dev"]["table"]
    texts = [list(rng.integers(0, VOCAB, n)) for n in prompt]
    # all but a prompt's last token; that one is the first tree's root
    new = [n - 1 for n in prompt]
    if sum(new):
        q, k, v = model.heads(ints([t for s in texts for t in s[:-1]]))
        cache.append(k, v, table, ints([0, *np.cumsum(new)]), ints([0] * sequences), rope, q=q)
    length = ints(new)
    cu = ints(np.arange(sequences + 1) * NODES)
    parent = ints(PARENT * sequences)
    accepted_in_all = 0
    for step in range(6):
        # a tree under the last token, every child drawn from the bigram table
        tokens = torch.zeros(sequences, NODES, dtype=torch.int64, device="cuda")
        tokens[:, 0] = ints([t[-1] for t in texts]).long()
        for i in range(1, NODES):
            tokens[:, i] = torch.multinomial(model.bigram[tokens[:, PARENT[i]]], 1, generator=gen)[:, 0]
        tokens = tokens.flatten().int()
        mask, depth = pi.draft_tree(parent, cu, NODES)
        q, k, v = model.heads(tokens)
        pos = length.repeat_interleave(NODES) + depth
        q = cache.append(k, v, table, cu, length, rope, positions=pos, q=q)
        full = length + NODES
        out, lse = cache.attention(q, table, cu, full, max_q=NODES, tree=mask, want_lse=True)
        bits, deep = O.draft_tree(PARENT * sequences, cu.cpu().numpy(), NODES)
        assert depth.tolist() == deep.tolist()
        check(cache, {"cu": cu.cpu().numpy(), "table": b["table"]}, q, out, lse, full.tolist(), bits)
        target = torch.softmax(out.float().view(sequences * NODES, -1) @ model.out, 1)
        draft = model.bigram[tokens.long()]
        a, u = (torch.rand(n, device="cuda", generator=gen) for n in (sequences * NODES, sequences))
        got = pi.verify_draft(target, draft, tokens, parent, cu, a, u, NODES)
        want = O.verify_draft(*(t.double().cpu().numpy() for t in (target, draft)), tokens.cpu().numpy(), PARENT * sequences,
                              cu.cpu().numpy(), *(t.double().cpu().numpy() for t in (a, u)), NODES)
        for g, w in zip(got, want):
            np.testing.assert_array_equal(g.cpu().numpy(), w)
        # the root and what was accepted, in a row, over the tree's place
        n = got.accepted + 1
        cu_kept = torch.zeros(sequences + 1, dtype=torch.int32, device="cuda")
        cu_kept[1:] = n.cumsum(0)
        rows = (got.path + cu[:-1, None])[got.path >= 0].long()
        cache.append(k[rows], v[rows], table, cu_kept, length, rope)
        length = length + n
        path = got.path.tolist()
        for s in range(sequences):
            texts[s] += [tokens[s * NODES + j].item() for j in path[s][1:] if j >= 0] + [got.token[s].item()]
        accepted_in_all += int(got.accepted.sum())
        assert cache.device_status() == 0
    assert accepted_in_all > 0
    # the cache holds the texts' turned keys and their values: a code is within 2^-4 of what it stands for, or half the
    # smallest step, 2^-10, of its block's scale; a block met again is rounded once more where its codes are smallest
    ref = oracle_of(cache)
    for s in range(sequences):
        n = int(length[s])
        assert n == len(texts[s]) - 1
        _, k, v = (t.double().cpu().numpy() for t in model.heads(ints(texts[s][:-1])))
        k, _ = O.rotary(k, np.arange(n), rope.inv_freq, 1.0, False)
        for which, x in ((0, k), (1, v)):
            held = ref.rows(which, b["table"][s], 0, n)
            scale = np.stack([ref.scale[which][b["table"][s][p // PAGE], :, p % PAGE // 16] for p in range(n)])
            assert (np.abs(held - x) <= 2.0 ** -4 * np.abs(x) + 2.0 ** -9 * scale[..., None]).all()


def test_a_step_in_one_graph(pi):
    """Tree, append, attention and verification captured together and replayed with new contents."""
    model, rope = Model(torch.float16), pi.Rotary(DIM)
    b = batch([40, 70], [NODES, NODES], PAGE)
    d = b["dev"]
    cache = pi.KVCache(b["pages"], HEADS, DIM, PAGE)
    start, parent = d["start"].clone(), ints(PARENT * 2)
    q, k, v = (t.clone() for t in model.heads(torch.randint(0, VOCAB, (2 * NODES,)).cuda()))
    drawn, a, u = ints(range(2 * NODES)), torch.rand(2 * NODES, device="cuda"), torch.rand(2, device="cuda")

    def step():
        mask, depth = pi.draft_tree(parent, d["cu"], NODES)
        seq = torch.arange(2, device="cuda").repeat_interleave(NODES)
        turned = cache.append(k, v, d["table"], d["cu"], start, rope, positions=start[seq] + depth, q=q)
        out = cache.attention(turned, d["table"], d["cu"], start + NODES, max_q=NODES, tree=mask)
        target = torch.softmax(out.float().view(2 * NODES, -1) @ model.out, 1)
        return (out, target, *pi.verify_draft(target, model.bigram[:2 * NODES], drawn, parent, d["cu"], a, u, NODES))
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = step()
    for seed in (1, 2):
        torch.manual_seed(seed)
        for t, new in zip((q, k, v), model.heads(torch.randint(0, VOCAB, (2 * NODES,)).cuda())):
            t.copy_(new)
        u.uniform_()
        a.uniform_()
        drawn.random_(0, VOCAB)
        codes = cache.k_codes.clone(), cache.k_scales.clone(), cache.v_codes.clone(), cache.v_scales.clone()
        g.replay()
        got = [t.clone() for t in kept]
        for t, old in zip((cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales), codes):
            t.copy_(old)
        for x, y in zip(got, step()):
            assert torch.equal(x, y)
