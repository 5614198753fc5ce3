"""The example decoder against a float64 restatement on the cached keys and values."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def decode():
    import __graft_entry__
    __graft_entry__.build()
    from examples import decode
    return decode


def plain(m, decode, ids, cu, start):
    """Logits of the new tokens in float64 but for the FFN, whose input is rounded
    as the layer's is and which is the layer's own call (its set of neurons
    belongs to the batch), with keys and values as the caches hold them."""
    D, H, K = decode.D, decode.HEADS, decode.DIM
    n = len(ids)
    cu, start = cu.tolist(), start.tolist()
    pos = torch.cat([torch.arange(cu[s + 1] - cu[s]) + start[s] for s in range(m.n_seqs)]).cuda()
    x = m.emb[ids].double() + m.pos[pos].double()

    def norm(x, i):
        w, b = m.norm[i]
        return torch.nn.functional.layer_norm(x, (D,), w.double(), b.double(), 1e-5)

    for i, (cache, ffn) in enumerate(zip(m.caches, m.ffn)):
        q = (norm(x, 2 * i) @ m.qkv[i].double().T).view(n, 3, H, K)[:, 0]
        a = torch.zeros(n, H, K, dtype=torch.float64, device="cuda")
        for s in range(m.n_seqs):
            r0, r1 = cu[s], cu[s + 1]
            if r0 == r1:
                continue
            total = start[s] + r1 - r0
            k, v = cache.read(m.table[s:s + 1], torch.tensor([0, total], dtype=torch.int32, device="cuda"),
                              torch.zeros(1, dtype=torch.int32, device="cuda"), total, dtype=torch.float32)
            z = torch.einsum("qhd,khd->hqk", q[r0:r1], k.double()) * K ** -0.5
            hide = torch.arange(total, device="cuda")[None] > torch.arange(start[s], total, device="cuda")[:, None]
            a[r0:r1] = torch.einsum("hqk,khd->qhd", z.masked_fill(hide, -torch.inf).softmax(-1), v.double())
        x = x + a.view(n, D) @ m.proj[i].double().T
        y = norm(x, 2 * i + 1).half()
        x = x + torch.cat([ffn.forward(p)[0] for p in y.split(128)]).double()
    return norm(x, 2 * len(m.caches)) @ m.emb.double().T


def test_against_plain(decode):
    """A ragged prompt, then single tokens.  Rounding to fp16 between the calls is
    2^-11 of each value, and a neuron whose logit is within it of 0 may change
    sides: 3% of the logits' norm covers some ten such roundings and one neuron
    in a thousand of the active ones."""
    m = decode.Decoder(sequences=3, vocab=1000, max_tokens=256)
    g = torch.Generator().manual_seed(3)
    for new in ([100, 0, 33], [1, 1, 1], [17, 70, 1]):
        cu = torch.tensor([0, *torch.tensor(new).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
        ids = torch.randint(0, 1000, (sum(new),), generator=g).cuda().int()
        start = m.length.clone()
        _, y = m.forward(ids, cu, max(new))
        got, want = m.logits(y).double(), plain(m, decode, ids, cu, start)
        assert (got - want).norm() < 0.03 * want.norm()
    m.check()
    assert m.length.tolist() == [118, 71, 35]


def test_generate_and_score(decode):
    """The chosen tokens' log-probabilities are those that scoring the whole text finds first in each row."""
    m = decode.Decoder(sequences=2, vocab=1000, max_tokens=128)
    cu = torch.tensor([0, 20, 27], dtype=torch.int32, device="cuda")
    ids = torch.randint(0, 1000, (27,), generator=torch.Generator().manual_seed(1)).cuda().int()
    tokens, logprob = m.generate(ids, cu, 20, steps=6)
    m.check()
    assert tokens.shape == (2, 6) and torch.isfinite(logprob).all() and (logprob <= 0).all()
    m.length.zero_()
    s = m.score(ids, cu, 20)
    assert torch.equal(tokens[:, 0], s.top_index[[19, 26], 0])
    _, y = m.forward(tokens[:, 0].contiguous(), torch.arange(3, dtype=torch.int32, device="cuda"), 1)
    want = m.logits(y).double().log_softmax(-1)
    # binary32 sums of 1000 terms and one exponential each: 1e-4 is generous
    assert (want.gather(1, tokens[:, 1:2].long())[:, 0] - logprob[:, 1]).abs().max() < 1e-4
    assert s.logprob[19] == 0 and s.logprob[26] == 0


def test_fit_norm(decode):
    """Twenty steps of the norm's gradient lower the loss, each of the first ones too."""
    m = decode.Decoder(sequences=1, vocab=1000, max_tokens=64)
    cu = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    ids = torch.randint(0, 1000, (41,), generator=torch.Generator().manual_seed(2)).cuda().int()
    x, _ = m.forward(ids[:40].contiguous(), cu, 40)
    losses = decode.fit_norm(m, x, ids[1:].contiguous())
    assert (losses[1:6] < losses[:5]).all() and losses[-1] < losses[0] - 0.05
