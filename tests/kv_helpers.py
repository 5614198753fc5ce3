"""Caches, page tables and ragged batches for the key/value cache's tests."""
import numpy as np
import torch

from oracle import operators as O

TORCH = {"float16": torch.float16, "bfloat16": torch.bfloat16, "float32": torch.float32}


def batch(start, new, page, seed=0, extra=3, device="cuda"):
    """A shuffled page table and row offsets for sequences with `start` tokens and `new` more."""
    rng = np.random.default_rng(seed)
    need = [max(1, -(-(s + n) // page)) for s, n in zip(start, new)]
    order = rng.permutation(sum(need) + extra)
    table = np.zeros((len(start), max(need)), np.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    dev = {k: torch.from_numpy(np.asarray(v, np.int32)).to(device) for k, v in
           dict(table=table, cu=cu, start=start, length=np.add(start, new)).items()}
    return dict(pages=sum(need) + extra, table=table, cu=cu, n=int(cu[-1]), dev=dev)


def random_cache(pi, pages, heads, dim, page, seed=0):
    """A KVCache with random codes (no NaN) and scales 2^-9 .. 2^-3, as a reused pool holds them."""
    g = torch.Generator().manual_seed(seed)
    c = pi.KVCache(pages, heads, dim, page)
    for codes, scales in ((c.k_codes, c.k_scales), (c.v_codes, c.v_scales)):
        x = torch.randn(codes.shape, generator=g) * 60
        codes.copy_(x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
        scales.copy_(torch.ldexp(torch.ones(scales.shape), torch.randint(-9, -2, scales.shape, generator=g)))
    return c


def oracle_of(c) -> O.CacheOracle:
    return O.CacheOracle(c.k_codes.cpu().numpy(), c.k_scales.cpu().numpy(), c.v_codes.cpu().numpy(),
                         c.v_scales.cpu().numpy())


def same_cache(c, ref: O.CacheOracle):
    """Every stored value and scale equal (codes of 0 and -0 alike)."""
    got = oracle_of(c)
    for which, name in ((0, "k"), (1, "v")):
        np.testing.assert_array_equal(got.scale[which], ref.scale[which], err_msg=name + " scales")
        np.testing.assert_array_equal(got.value[which], ref.value[which], err_msg=name + " values")
