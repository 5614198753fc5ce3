"""Drafted tokens without a GPU: refusals before any launch, and the oracle's own pins."""
import ctypes as C
import re
from pathlib import Path

import numpy as np
import pytest
import torch

from oracle import operators as O

ROOT = Path(__file__).resolve().parents[1]


@pytest.fixture(scope="module")
def pi():
    import __graft_entry__
    __graft_entry__._builder().build()
    import activation_sparse_rank_gb300 as pi
    return pi


def test_constant_matches_the_header(pi):
    text = (ROOT / "include" / "pi.h").read_text()
    assert int(re.search(r"#define\s+PI_MAX_TREE\s+([0-9]+)", text).group(1)) == pi.PI_MAX_TREE


def test_tree_abi_refusals(pi):
    p, odd = C.c_void_p(1 << 20), C.c_void_p((1 << 20) + 2)         # never dereferenced

    def call(parent=p, cu=p, seqs=2, n=5, q=4, mask=p, depth=p):
        return pi.lib.pi_draft_tree(parent, cu, seqs, n, q, mask, depth, None)

    for bad in (dict(parent=None), dict(cu=None), dict(seqs=-1), dict(n=-1), dict(mask=odd), dict(depth=odd), dict(cu=odd)):
        assert call(**bad) == 1, bad
    assert call(q=0) == 2 and call(q=257) == 2
    assert call(seqs=0) == 0 and call(n=0) == 0 and call(mask=None, depth=None) == 0


def test_verify_abi_refusals(pi):
    p, odd = C.c_void_p(1 << 20), C.c_void_p((1 << 20) + 2)

    def call(t=p, ts=100, d=p, ds=100, dt=2, vocab=100, x=p, parent=p, cu=p, seqs=2, n=5, q=4, a=p, u=p, acc=p, path=p, tok=p):
        return pi.lib.pi_verify_draft(t, ts, d, ds, dt, vocab, x, parent, cu, seqs, n, q, a, u, acc, path, tok, None)

    for bad in (dict(t=None), dict(ts=99), dict(ds=99), dict(dt=3), dict(vocab=0), dict(x=None), dict(parent=None), dict(cu=None),
                dict(seqs=-1), dict(n=-1), dict(a=None), dict(u=None), dict(acc=None), dict(path=None), dict(tok=None),
                dict(t=odd), dict(d=odd), dict(x=odd), dict(a=odd), dict(u=odd), dict(acc=odd), dict(path=odd), dict(tok=odd)):
        assert call(**bad) == 1, bad
    assert call(q=0) == 2 and call(q=257) == 2 and call(vocab=(1 << 21) + 1, ts=1 << 22, ds=1 << 22) == 2
    assert call(seqs=0) == 0


def test_host_tensors_are_refused(pi):
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError):
        pi.draft_tree(i, i)
    with pytest.raises(TypeError):
        pi.verify_draft(torch.zeros(3, 5), None, i, i, i, i.float(), i.float())


def test_oracle_of_a_tree():
    mask, depth = O.draft_tree([-1, 0, 0, 1, 5, -1, 9, 2], [0, 5, 8], 5)
    assert depth.tolist() == [0, 1, 1, 2, 0, 0, 0, 0]               # a parent at or behind its node is none
    assert [np.flatnonzero(m).tolist() for m in mask] == [[0], [0, 1], [0, 2], [0, 1, 3], [4], [0], [1], [2]]


def test_oracle_of_the_verification():
    p, q = np.array([[0.5, 0.25, 0.25, 0.0]] * 3), np.array([[0.25, 0.75, 0.0, 0.0]] * 3)
    chain = dict(drawn=[0, 1, 0], parent=[-1, 0, 1], cu=[0, 3], max_q=3)
    # 0.3 * 0.75 < 0.25 accepts token 1; 0.9 * 0.25 < 0.5 accepts token 0; then the target's own: 0.6 lies in token 1
    assert [v.tolist() for v in O.verify_draft(p, q, accept=[0, 0.3, 0.9], sample=[0.6], **chain)] == [[2], [[0, 1, 2]], [1]]
    # equality rejects: 0.25 = 1/3 * 0.75 in whole parts; what is left is (0.25, 0, 0.25, 0)
    half = dict(chain, drawn=[0, 0, 0])
    assert [v.tolist() for v in O.verify_draft(p, 2 * q, accept=[0, 1.0, 0], sample=[0.5], **half)] == [[0], [[0, -1, -1]], [2]]
    # two given children: the first is refused, the second takes W = 1 - 0.5 into account
    two = dict(drawn=[0, 0, 1], parent=[-1, 0, 0], cu=[0, 3], max_q=3)
    assert [v.tolist() for v in O.verify_draft(p, None, accept=[0, 0.5, 0.4], sample=[0.0], **two)] == [[1], [[0, 2, -1]], [0]]
    assert [v.tolist() for v in O.verify_draft(p, None, accept=[0, 0.5, 0.5], sample=[0.9], **two)] == [[0], [[0, -1, -1]], [2]]
    # nothing left (draft = target, refused): the target itself; an empty sequence; no distribution
    same = O.verify_draft(p, p, [0, 0], [-1, 0], [0, 2, 2], [0, 1.0], [0.8, 0.8], 2)
    assert [v.tolist() for v in same] == [[0, 0], [[0, -1], [-1, -1]], [2, -1]]
    assert O.verify_draft(0 * p, None, [0], [-1], [0, 1], [0], [0.5], 1)[2].tolist() == [-1]


def test_tree_attention_abi_refusals(pi):
    lib, fake = pi.lib, C.c_void_p(1 << 20)
    c = pi.binding.pi_kv_cache(4, 32, 2, 64, 1 << 20, 1 << 20, 1 << 20, 1 << 20, 1 << 20)
    tok = pi.binding.pi_kv_tokens(1, 300, 1 << 20, 1 << 20, 20)
    need = lib.pi_kv_attention_workspace_bytes(C.byref(c), 4, 300, 1)

    def attend(mask=fake, words=8, q=fake, st=(C.c_int64 * 2)(256, 64), heads=4, dt=0, max_q=3, n=need):
        return lib.pi_kv_tree_attention(C.byref(c), C.byref(tok), fake, max_q, mask, words, q, st, heads, dt, 0.125, fake, None,
                                        fake, n, None)

    for bad in (dict(mask=None), dict(mask=C.c_void_p((1 << 20) + 2)), dict(words=0), dict(q=None), dict(heads=3), dict(dt=2),
                dict(max_q=-1), dict(n=need - 1), dict(words=1, max_q=33)):
        assert attend(**bad) == 1, bad
    assert attend(max_q=257, words=9) == 2 and attend(max_q=0) == 0
