"""A small pre-norm decoder that stays on the GPU from token to token.

Random weights of the 1024-wide layer's shape (16 heads of 64, ReLU FFN of
4096 neurons behind its predictor).  Per layer: layer norm, projection (torch),
``KVCache.write``, ``KVCache.attention``, projection, the residual addition
with the next norm in one call, and ``Layer.forward``.  The last norm's rows
give logits; ``token_logprobs`` scores given texts and picks the next tokens.
``fit_norm`` adjusts the last norm to a text with ``layer_norm_backward``.

    python -m examples.decode
"""
from __future__ import annotations

import torch

import activation_sparse_rank_gb300 as pi
from workload import LayerSpec, make_layer

D, HEADS, DIM, FFN, PAGE = 1024, 16, 64, 4096, 64


class Decoder:
    """Weights, a key/value cache of each layer and one page table for all of them."""

    def __init__(self, layers=2, vocab=5000, sequences=4, max_tokens=512, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(*shape, generator=g) * std).to(device, torch.float16)

        self.device, self.n_seqs, self.max_tokens = device, sequences, max_tokens
        self.emb, self.pos = normal(vocab, D, std=0.05), normal(max_tokens, D, std=0.02)
        self.qkv = [normal(3 * D, D, std=D ** -0.5) for _ in range(layers)]
        self.proj = [normal(D, D, std=D ** -0.5) for _ in range(layers)]
        self.norm = [(1 + normal(D, std=0.05), normal(D, std=0.05)) for _ in range(2 * layers + 1)]
        spec = LayerSpec(d=D, ffn=FFN, rank=64, mean_f=0.1)
        self.ffn = [pi.Layer.from_dict({k: v.to(device) if torch.is_tensor(v) else v
                                        for k, v in make_layer(spec, base_seed=seed + 1, layer=i).items()})
                    for i in range(layers)]
        self.ffn_ws = self.ffn[0].workspace(pi.PI_MAX_BATCH)
        pages = -(-max_tokens // PAGE)
        self.caches = [pi.KVCache(sequences * pages, HEADS, DIM, PAGE, device) for _ in range(layers)]
        self.table = torch.randperm(sequences * pages, generator=g).to(device, torch.int32).view(sequences, pages)
        self.length = torch.zeros(sequences, dtype=torch.int32, device=device)      # tokens in the caches

    def forward(self, ids, cu, max_q):
        """The last norm's input (residual sum) and output for new tokens ids [n],
        packed by sequence (cu [sequences + 1]); at most max_q of any sequence."""
        n, start = ids.shape[0], self.length
        length = start + cu.diff()
        seq = torch.repeat_interleave(torch.arange(self.n_seqs, device=self.device), cu.diff(), output_size=n)
        x = self.emb[ids] + self.pos[torch.arange(n, device=self.device) - cu[seq] + start[seq]]
        y = pi.layer_norm(x, *self.norm[0])[0]
        for i, (cache, ffn) in enumerate(zip(self.caches, self.ffn)):
            q, k, v = torch.nn.functional.linear(y, self.qkv[i]).view(n, 3, HEADS, DIM).unbind(1)
            cache.write(k, v, self.table, cu, start)
            a = cache.attention(q, self.table, cu, length, max_q=max_q)
            a = torch.nn.functional.linear(a.view(n, D), self.proj[i])
            y, x, _, _ = pi.layer_norm(x, *self.norm[2 * i + 1], add=a)
            f = torch.cat([ffn.forward(part, ws=self.ffn_ws)[0] for part in y.split(pi.PI_MAX_BATCH)])
            y, x, _, _ = pi.layer_norm(x, *self.norm[2 * i + 2], add=f)
        self.length = length
        return x, y

    def logits(self, y):
        return torch.nn.functional.linear(y, self.emb)

    def score(self, ids, cu, max_q):
        """Log-probabilities of each new token given the ones before it, and the
        likeliest tokens after each position."""
        _, y = self.forward(ids, cu, max_q)
        last = torch.zeros_like(ids, dtype=torch.bool)
        last[cu[1:].long() - 1] = True
        target = torch.where(last, -1, ids.roll(-1)).to(torch.int32)                # nothing follows the last one yet
        return pi.token_logprobs(self.logits(y), target, top_k=5)

    def generate(self, ids, cu, max_q, steps):
        """`steps` tokens after each prompt, always the likeliest; [sequences, steps] and their log-probabilities."""
        scores = self.score(ids, cu, max_q)
        rows = cu[1:].long() - 1
        nxt, logprob = scores.top_index[rows, 0], scores.top_logprob[rows, 0]
        one = torch.arange(self.n_seqs + 1, dtype=torch.int32, device=self.device)
        out = [(nxt, logprob)]
        for _ in range(steps - 1):
            _, y = self.forward(nxt, one, 1)
            s = pi.token_logprobs(self.logits(y), top_k=1)
            nxt = s.top_index[:, 0]
            out.append((nxt, s.top_logprob[:, 0]))
        return torch.stack([t for t, _ in out], 1), torch.stack([p for _, p in out], 1)

    def check(self):
        """Raise if a kernel met a page or range that is not there."""
        for c, f in zip(self.caches, self.ffn):
            if c.device_status() or f.device_status():
                raise RuntimeError("a page, position or index out of range")


def fit_norm(model, x, target, steps=20, rate=0.5):
    """Fit the last norm's weight and bias to targets of residual rows x
    (gradient descent on the mean of -log p); returns the losses."""
    w, b = (t.float() for t in model.norm[-1])
    losses = []
    for _ in range(steps):
        y, _, mean, rstd = pi.layer_norm(x, w, b, want_stats=True)
        logits = model.logits(y)
        s = pi.token_logprobs(logits, target)
        losses.append(-s.logprob.mean())
        d_logits = torch.exp(logits.float() - s.lse[:, None])
        d_logits[torch.arange(len(target), device=x.device), target.long()] -= 1
        dy = (d_logits / len(target)).to(torch.float16) @ model.emb
        _, dw, db = pi.layer_norm_backward(dy, x, w, mean, rstd)
        w, b = w - rate * dw, b - rate * db
    return torch.stack(losses)


def main():
    model = Decoder()
    g = torch.Generator().manual_seed(7)
    new = [200, 1, 37, 90]
    cu = torch.tensor([0, *torch.tensor(new).cumsum(0).tolist()], dtype=torch.int32, device=model.device)
    ids = torch.randint(0, model.emb.shape[0], (sum(new),), generator=g).to(model.device, torch.int32)
    tokens, logprob = model.generate(ids, cu, max(new), steps=16)
    model.check()
    for s in range(model.n_seqs):
        print(f"sequence {s}: {new[s]} tokens, then {tokens[s].tolist()}  (mean log-probability {logprob[s].mean():.3f})")
    model.length.zero_()
    x, _ = model.forward(ids, cu, max(new))
    losses = fit_norm(model, x[:200], ids[1:201])
    print(f"norm fitted to sequence 0: loss {losses[0]:.3f} -> {losses[-1]:.3f}")


if __name__ == "__main__":
    main()
