"""The operators around the FFN block, as Python calls on torch tensors.

``KVCache`` (a paged key/value cache in E4M3 codes: ``write``, ``append``,
``read``, ``attention``), ``rotary`` with ``rotary_backward`` (positions by a
``Rotary``), ``draft_tree`` and ``verify_draft`` for drafted tokens,
``layer_norm`` with ``layer_norm_backward``, and ``token_logprobs``.  Argument checks and marshalling only; include/pi.h states
each operator's formula, limits and treatment of special values.

``stream`` is a torch stream (default: the current one).  Outputs and scratch
that the caller does not supply are allocated on the stream the call runs on;
inputs made on another stream have to be ordered before it by the caller, and
must not be freed before it has passed, as with every torch operator.

The calls are not known to autograd: an output never requires grad, whatever
the inputs do.  ``layer_norm_backward`` and ``rotary_backward`` are called by hand.
"""
from __future__ import annotations

import ctypes as C
import math
from fractions import Fraction
from functools import lru_cache
from typing import NamedTuple, Optional

import torch

from .binding import (PI_DT_BF16, PI_DT_F16, PI_DT_F32, PI_KV_BLOCK, PI_KV_MAX_PAGE, PI_MAX_ROTARY, PI_MAX_TOP_K, PI_MAX_TREE,
                      PiError, _check, lib, pi_kv_cache, pi_kv_tokens, pi_rotary)

__all__ = ["DraftVerdict", "KVCache", "Rotary", "TokenScores", "draft_tree", "layer_norm", "layer_norm_backward", "rotary",
           "rotary_backward", "token_logprobs", "verify_draft", "PI_KV_BLOCK", "PI_KV_MAX_PAGE", "PI_MAX_ROTARY",
           "PI_MAX_TOP_K", "PI_MAX_TREE"]

_DT = {torch.float16: PI_DT_F16, torch.bfloat16: PI_DT_BF16, torch.float32: PI_DT_F32}
_Stride2 = lru_cache(maxsize=256)(C.c_int64 * 2)     # the library only reads them, so calls may share one
_f32, _i32, _u8 = torch.float32, torch.int32, torch.uint8


def _dt(t: torch.Tensor, name: str) -> int:
    d = _DT.get(t.dtype)
    if d is None:
        raise TypeError(f"{name} must be float16, bfloat16 or float32, not {t.dtype}")
    return d


def _dev(t: torch.Tensor, device: Optional[torch.device], name: str) -> torch.device:
    """t is a CUDA tensor, on `device` if given."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    at = t.device
    if device is not None and at != device:
        raise ValueError(f"{name} is on {at}, not {device}")
    return at


def _whole(t: torch.Tensor, shape, dtype, device, name: str) -> torch.Tensor:
    """t is a contiguous CUDA tensor of this shape and type."""
    _dev(t, device, name)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _fits(t, shape, dtype, device) -> bool:
    """Whether _whole would pass (the short way through)."""
    return t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.device == device


_Tensor, _empty = torch.Tensor, torch.empty


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


# Calls of a decode step are short: the usual case (the current device and
# stream) asks for the stream's handle alone, without a stream object.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device   # a CUDA tensor exists: no set-up


def _on(device: torch.device, stream, fn, *args):
    """fn(stream handle, *args) with `device` current and allocations on the call's stream."""
    if stream is None:
        if _current_device() == device.index:
            return fn(_raw_stream(device.index), *args)
        with torch.cuda.device(device):
            return fn(_raw_stream(device.index), *args)
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    with torch.cuda.stream(stream):
        return fn(stream.cuda_stream, *args)


def _ws(ws: torch.Tensor, device) -> int:
    _dev(ws, device, "ws")
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    return ws.numel() * ws.element_size()


# 1 / (2 pi): frequencies as fractions of a turn are right to their last bit
_TURNS_PER_RADIAN = Fraction("0.1591549430918953357688837633725143620344596457404564487476673440588967976342")


def _frequencies(dim, base, scaling, factor, original_length, beta_fast, beta_slow, magnitude, inv_freq):
    """Radians a position of each pair, and the magnitude (see ``Rotary``)."""
    if dim < 2 or dim % 2 or dim > PI_MAX_ROTARY:
        raise ValueError(f"dim must be an even number up to {PI_MAX_ROTARY}, not {dim}")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"scaling must be None, 'linear', 'ntk' or 'yarn', not {scaling!r}")
    if not (1.0 < base < math.inf and 0.0 < factor < math.inf):
        raise ValueError(f"base must be above 1 and factor above 0, both finite, not {base} and {factor}")
    if inv_freq is not None:
        if scaling is not None:
            raise ValueError("inv_freq and scaling exclude each other")
        freq = [float(f) for f in inv_freq]
        if len(freq) != dim // 2 or not all(math.isfinite(f) for f in freq):
            raise ValueError(f"inv_freq must be {dim // 2} finite numbers")
    else:
        if scaling == "ntk" and dim > 2:
            base = base * factor ** (dim / (dim - 2))
        freq = [base ** (-2 * i / dim) for i in range(dim // 2)]
    if scaling == "linear":
        freq = [f / factor for f in freq]
    if scaling == "yarn":
        if original_length is None or original_length < 1 or not 0 < beta_slow <= beta_fast:
            raise ValueError("'yarn' needs original_length of at least 1 and 0 < beta_slow <= beta_fast")

        def pair_of(turns):                      # the pair that makes so many turns over original_length
            return dim * math.log(original_length / (2 * math.pi * turns)) / (2 * math.log(base))
        lo, hi = max(0, math.floor(pair_of(beta_fast))), min(dim - 1, math.ceil(pair_of(beta_slow)))
        ramp = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(dim // 2)]
        freq = [f * (1 - r) + f / factor * r for f, r in zip(freq, ramp)]
        if magnitude is None and factor > 1:
            magnitude = 0.1 * math.log(factor) + 1.0
    magnitude = 1.0 if magnitude is None else float(magnitude)
    if not math.isfinite(magnitude):
        raise ValueError("magnitude must be finite")
    return freq, magnitude


class Rotary:
    """Rotary positions: frequencies of the dim / 2 pairs of a head's first
    ``dim`` elements, kept on the device as exact fractions of a turn.

    Pair i is the elements (2i, 2i + 1) where ``interleaved``, else (i, i + dim / 2);
    it turns by base^(-2i / dim) radians a position.  ``scaling`` stretches the
    frequencies for contexts ``factor`` times longer:
      "linear"  every frequency divided by factor
      "ntk"     base raised by factor^(dim / (dim - 2)): the slowest pair is divided by factor, the fastest keeps its own
      "yarn"    pairs that make fewer than beta_slow turns over original_length positions are divided by factor, those of
                more than beta_fast keep their own, a ramp between; results times magnitude, by default 0.1 ln(factor) + 1
    ``inv_freq`` (dim / 2 numbers, radians a position) replaces all of these.
    ``magnitude`` multiplies the turned elements (default 1, but for "yarn").
    """

    def __init__(self, dim, base=10000.0, interleaved=False, scaling=None, factor=1.0, original_length=None, beta_fast=32.0,
                 beta_slow=1.0, magnitude=None, inv_freq=None, device="cuda"):
        freq, magnitude = _frequencies(dim, base, scaling, factor, original_length, beta_fast, beta_slow, magnitude, inv_freq)
        turns = [round(Fraction(f) * _TURNS_PER_RADIAN * (1 << 64)) % (1 << 64) for f in freq]
        self.dim, self.interleaved, self.magnitude, self.inv_freq = dim, bool(interleaved), magnitude, freq
        self.turns = torch.tensor([t - (1 << 64) if t >> 63 else t for t in turns], dtype=torch.int64, device=device)
        self.device = _dev(self.turns, None, "device")
        self._c = pi_rotary(dim, int(self.interleaved), magnitude, self.turns.data_ptr())
        self._ref = C.addressof(self._c)


def _heads3(t, device, name):
    """Strides of a [tokens, heads, head_dim] tensor with contiguous heads; those of single tokens and heads may be anything."""
    if not isinstance(t, _Tensor) or t.get_device() != device.index:
        _dev(t, device, name)
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim], got {tuple(shape)}")
    n, h, d = shape
    st, sh, sd = t.stride()
    if sd != 1 and d > 1 and n and h:                # without elements the strides may be anything
        raise ValueError(f"{name}: the elements of a head must be contiguous")
    return _Stride2(st if n > 1 else h * d, sh if h > 1 else d)


def _places(positions, n, device):
    if not _fits(positions, (n,), _i32, device):
        _whole(positions, (n,), _i32, device, "positions")


def _turn(x, positions, rope, out, inverse, stream, name):
    dev = rope.device
    xs = _heads3(x, dev, name)
    dt = _dt(x, name)
    n = x.shape[0]
    _places(positions, n, dev)
    if out is not None:
        if not isinstance(out, _Tensor) or out.shape != x.shape or out.dtype is not x.dtype:
            raise ValueError(f"the output must be {tuple(x.shape)} {x.dtype}")
        os = _heads3(out, dev, "the output")         # rows may lie apart, but not in one another
        d, (t, h) = x.shape[2], sorted(((os[0], n), (os[1], x.shape[1])))
        if x.numel() and (t[0] < d and t[1] > 1 or h[0] < (t[1] - 1) * t[0] + d and h[1] > 1):
            raise ValueError("the output's elements share memory")
        if out.data_ptr() == x.data_ptr() and (os[0], os[1]) != (xs[0], xs[1]):
            raise ValueError("the output begins where " + name + " does, with other strides")
    if stream is None and _current_device() == dev.index:
        return _rotary(_raw_stream(dev.index), x, xs, positions, rope, out, inverse, dt)
    return _on(dev, stream, _rotary, x, xs, positions, rope, out, inverse, dt)


def _rotary(handle, x, xs, positions, rope, out, inverse, dt):
    n, h, d = x.shape
    if out is None:
        out = _empty((n, h, d), dtype=x.dtype, device=rope.device)
        ys = _Stride2(h * d, d)
    else:
        ys = _heads3(out, rope.device, "the output")
    if h:
        _check(lib.pi_rotary_apply(rope._ref, positions.data_ptr(), n, h, d, x.data_ptr(), xs, out.data_ptr(), ys, dt, inverse,
                                   handle), "pi_rotary_apply")
    return out


def rotary(x, positions, rope, out=None, stream=None):
    """x [tokens, heads, head_dim] with the pairs of ``rope`` turned by positions
    (int32 [tokens]); elements past rope.dim as they are.  Queries and keys that lie
    side by side are one call.  ``out`` may be x (in place), or any tensor of x's shape
    and type with contiguous heads that shares no memory with x."""
    return _turn(x, positions, rope, out, 0, stream, "x")


def rotary_backward(dy, positions, rope, dx=None, stream=None):
    """Gradient of ``rotary`` with respect to x: dy turned the other way (times the
    magnitude as well).  ``dx`` may be dy."""
    return _turn(dy, positions, rope, dx, 1, stream, "dy")


class KVCache:
    """A paged key/value cache in E4M3 codes with one power-of-two scale for
    each PI_KV_BLOCK tokens of a head.

    Pages are [heads, page_size, head_dim] codes; a sequence's pages are the
    entries of its row of a page table (int32 [sequences, most pages]).  The
    four tensors and the table are plain torch tensors of the caller's to keep,
    copy or hand out: ``k_codes``, ``v_codes`` uint8 [pages, heads, page_size,
    head_dim] and ``k_scales``, ``v_scales`` float32 [pages, heads,
    page_size / PI_KV_BLOCK].
    """

    def __init__(self, n_pages: int, heads: int, head_dim: int, page_size: int = 64, device="cuda"):
        if page_size < 1 or page_size % PI_KV_BLOCK:
            raise ValueError(f"page_size must be a multiple of {PI_KV_BLOCK}, not {page_size}")
        codes = (n_pages, heads, page_size, head_dim)
        scales = (n_pages, heads, page_size // PI_KV_BLOCK)
        self._init(torch.zeros(codes, dtype=_u8, device=device), torch.ones(scales, dtype=_f32, device=device),
                   torch.zeros(codes, dtype=_u8, device=device), torch.ones(scales, dtype=_f32, device=device))

    @classmethod
    def wrap(cls, k_codes, k_scales, v_codes, v_scales) -> "KVCache":
        """A cache over tensors that exist already (shapes as above)."""
        self = cls.__new__(cls)
        self._init(k_codes, k_scales, v_codes, v_scales)
        return self

    def _init(self, k_codes, k_scales, v_codes, v_scales):
        device = _dev(k_codes, None, "k_codes")
        if k_codes.dim() != 4:
            raise ValueError("k_codes must be [pages, heads, page_size, head_dim]")
        pages, heads, page, dim = k_codes.shape
        if page % PI_KV_BLOCK:
            raise ValueError(f"page_size must be a multiple of {PI_KV_BLOCK}, not {page}")
        for t, n in ((k_codes, "k_codes"), (v_codes, "v_codes")):
            _whole(t, k_codes.shape, _u8, device, n)
        for t, n in ((k_scales, "k_scales"), (v_scales, "v_scales")):
            _whole(t, (pages, heads, page // PI_KV_BLOCK), _f32, device, n)
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.device, self.n_pages, self.heads, self.page_size, self.head_dim = device, pages, heads, page, dim
        self._index = device.index
        self._status = torch.zeros(1, dtype=_i32, device=device)
        self._c = pi_kv_cache(pages, page, heads, dim, k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(),
                              v_scales.data_ptr(), self._status.data_ptr())
        self._ref = C.addressof(self._c)
        self._scale = 1.0 / math.sqrt(dim)
        if lib.pi_kv_attention_workspace_bytes(self._ref, heads, 0, 0) == 0:
            raise PiError(2, "KVCache")

    def _tokens(self, page_table, cu, per_seq, name, n_tokens):
        dev = self.device
        _dev(page_table, dev, "page_table")
        if page_table.dtype is not _i32 or page_table.dim() != 2:
            raise ValueError("page_table must be an int32 [sequences, pages] tensor with contiguous rows")
        n, pages = page_table.shape
        stride, one = page_table.stride()
        if one != 1 and n and pages > 1:             # the stride of a single page, or of no row, may be anything
            raise ValueError("page_table must be an int32 [sequences, pages] tensor with contiguous rows")
        if not _fits(cu, (n + 1,), _i32, dev):
            _whole(cu, (n + 1,), _i32, dev, "cu_tokens")
        if not _fits(per_seq, (n,), _i32, dev):
            _whole(per_seq, (n,), _i32, dev, name)
        if pages == 0 and n:
            raise ValueError("page_table must have a page for each sequence at least")
        # a table of one row may carry any stride for it
        return pi_kv_tokens(n, n_tokens, cu.data_ptr(), page_table.data_ptr(), stride if n > 1 else pages, pages)

    def _rows(self, t, heads, name):
        """A [tokens, heads, head_dim] tensor with contiguous heads: its token and head strides."""
        if not isinstance(t, _Tensor) or t.get_device() != self._index:
            _dev(t, self.device, name)
        shape = t.shape
        if len(shape) != 3 or shape[1] != heads or shape[2] != self.head_dim:
            raise ValueError(f"{name} must be [tokens, {heads}, {self.head_dim}], got {tuple(shape)}")
        st, sh, sd = t.stride()
        if sd != 1 and shape[0] and heads:           # without elements the strides may be anything
            raise ValueError(f"{name}: the elements of a head must be contiguous")
        if shape[0] <= 1:                            # the stride of a single row may be anything, and no copy changes it
            st = heads * self.head_dim
        if heads == 1:
            sh = self.head_dim
        return _Stride2(st, sh)

    def write(self, k, v, page_table, cu_tokens, start, stream=None):
        """Quantise new tokens into the cache: row cu_tokens[s] + i of k and v
        [tokens, heads, head_dim] becomes position start[s] + i of sequence s."""
        ks, vs = self._rows(k, self.heads, "k"), self._rows(v, self.heads, "v")
        if v.shape != k.shape or v.dtype is not k.dtype:
            raise ValueError("k and v must have one shape and type")
        tok = self._tokens(page_table, cu_tokens, start, "start", k.shape[0])
        dt = _dt(k, "k")
        if stream is None and _current_device() == self._index:
            self._write(_raw_stream(self._index), tok, start, k, ks, v, vs, dt)
        else:
            _on(self.device, stream, self._write, tok, start, k, ks, v, vs, dt)

    def _write(self, handle, tok, start, k, ks, v, vs, dt):
        _check(lib.pi_kv_write(self._ref, C.addressof(tok), start.data_ptr(), k.data_ptr(), ks, v.data_ptr(), vs, dt,
                               handle), "pi_kv_write")

    def append(self, k, v, page_table, cu_tokens, start, rope, positions=None, q=None, q_out=None, stream=None):
        """``write`` with the keys turned by ``rope`` (rope.dim a multiple of 16) on the
        way, from binary32, and the same tokens' queries q [tokens, q_heads, head_dim]
        turned in the same launch.  Row cu_tokens[s] + i is turned by
        positions[cu_tokens[s] + i] (int32 [tokens]), by default start[s] + i; its place
        in the cache is start[s] + i either way.  Returns the turned queries, or None
        without q; q_out may be q itself (contiguous), and shares no other memory with q, k
        or v.  Rows of no sequence are left as they were (unset in a q_out made here).
        Drafted tokens that are refused and appended over leave the scale that they
        raised in a block begun before them."""
        ks, vs = self._rows(k, self.heads, "k"), self._rows(v, self.heads, "v")
        if v.shape != k.shape or v.dtype is not k.dtype:
            raise ValueError("k and v must have one shape and type")
        if not isinstance(rope, Rotary):
            raise TypeError("rope must be a Rotary")
        if rope.device != self.device:
            raise ValueError(f"rope is on {rope.device}, not {self.device}")
        tok = self._tokens(page_table, cu_tokens, start, "start", k.shape[0])
        dt = _dt(k, "k")
        qs = None
        if q is not None:
            qs = self._rows(q, q.shape[1] if q.dim() == 3 else 0, "q")
            if q.shape[0] != k.shape[0] or q.dtype is not k.dtype:
                raise ValueError("q must have k's tokens and type")
        elif q_out is not None:
            raise ValueError("q_out needs q")
        if positions is not None:
            _places(positions, k.shape[0], self.device)
        if stream is None and _current_device() == self._index:
            return self._append(_raw_stream(self._index), tok, start, k, ks, v, vs, dt, rope, positions, q, qs, q_out)
        return _on(self.device, stream, self._append, tok, start, k, ks, v, vs, dt, rope, positions, q, qs, q_out)

    def _append(self, handle, tok, start, k, ks, v, vs, dt, rope, positions, q, qs, q_out):
        heads = 0
        if q is not None:
            heads = q.shape[1]
            if q_out is None:
                q_out = _empty(q.shape, dtype=q.dtype, device=self.device)
            elif not _fits(q_out, q.shape, q.dtype, self.device):
                _whole(q_out, q.shape, q.dtype, self.device, "q_out")
        turns = heads and tok.n_tokens
        _check(lib.pi_kv_append(self._ref, C.addressof(tok), start.data_ptr(), rope._ref, _ptr(positions), k.data_ptr(), ks,
                                v.data_ptr(), vs, q.data_ptr() if turns else None, qs, heads if turns else 0,
                                q_out.data_ptr() if turns else None, dt, handle), "pi_kv_append")
        return q_out

    def read(self, page_table, cu_tokens, start, n_tokens, dtype=torch.float16, k=None, v=None, stream=None):
        """Positions start[s] .. of each sequence as (k, v) [n_tokens, heads, head_dim] of `dtype`."""
        if dtype not in _DT:
            raise TypeError(f"dtype must be float16, bfloat16 or float32, not {dtype}")
        tok = self._tokens(page_table, cu_tokens, start, "start", n_tokens)
        return _on(self.device, stream, self._read, tok, start, dtype, k, v)

    def _read(self, handle, tok, start, dtype, k, v):
        shape = (tok.n_tokens, self.heads, self.head_dim)
        k = torch.empty(shape, dtype=dtype, device=self.device) if k is None else _whole(k, shape, dtype, self.device, "k")
        v = torch.empty(shape, dtype=dtype, device=self.device) if v is None else _whole(v, shape, dtype, self.device, "v")
        _check(lib.pi_kv_read(self._ref, C.addressof(tok), start.data_ptr(), k.data_ptr(), v.data_ptr(), _DT[dtype],
                              handle), "pi_kv_read")
        return k, v

    def attention_workspace(self, q_heads: int, n_tokens: int, n_seqs: int) -> torch.Tensor:
        """Scratch for ``attention`` calls of up to this size; calls that overlap need separate ones."""
        n = lib.pi_kv_attention_workspace_bytes(self._ref, q_heads, n_tokens, n_seqs)
        if n == 0:
            raise PiError(1, "pi_kv_attention_workspace_bytes")
        return torch.empty(n, dtype=_u8, device=self.device)

    def attention(self, q, page_table, cu_tokens, length, max_q=None, sm_scale=None, causal=True, out=None, lse=None,
                  want_lse=False, ws=None, stream=None, tree=None):
        """Attention of each sequence's newest tokens q [tokens, q_heads, head_dim]
        (float16 or bfloat16) over its cache.  length[s] counts the tokens in the
        cache, the new ones among them.  max_q bounds the new tokens of any
        sequence and is best given: by default it is 1 where q has no more rows
        than there are sequences, else all of q's rows, and the kernels are
        chosen by it (single tokens and a long prompt: two calls).  Rows past max_q get 0 (lse -inf) and show in
        ``device_status``; rows of no sequence are left as they were (unset in
        an ``out`` made here).  Returns out, or (out, lse) with want_lse or an
        lse tensor.

        tree (``draft_tree``'s mask, int32 [tokens, words]): the new tokens are drafted
        ones, and one sees of them those whose bits its row has (up to itself), beside the
        cache before them.  max_q is then at most 32 words and PI_MAX_TREE, the default included.
        From 17 to 32 query rows a head the page table's width chooses the kernel: short
        sequences are faster under the columns that they use (page_table[:, :n])."""
        heads = q.shape[1] if q.dim() == 3 else 0
        qs = self._rows(q, heads, "q")
        if q.dtype is not torch.float16 and q.dtype is not torch.bfloat16:
            raise TypeError(f"q must be float16 or bfloat16, not {q.dtype}")
        tok = self._tokens(page_table, cu_tokens, length, "length", q.shape[0])
        scale = self._scale if sm_scale is None else sm_scale
        if tree is not None:
            words = tree.shape[1] if tree.dim() == 2 else 0
            if not _fits(tree, (tok.n_tokens, words), _i32, self.device):
                _whole(tree, (tok.n_tokens, words), _i32, self.device, "tree")
            if not causal:
                raise ValueError("tree is causal: a token sees none behind it")
            if max_q is None:
                max_q = min(tok.n_tokens, 32 * words, PI_MAX_TREE)
            if max_q > min(32 * words, PI_MAX_TREE) and tok.n_tokens:
                raise ValueError(f"max_q={max_q}: tree has bits for {32 * words}, {PI_MAX_TREE} at most")
        if max_q is None:
            max_q = 1 if tok.n_tokens <= tok.n_seqs else tok.n_tokens
        elif max_q == 0:
            max_q = 1                                # the library would leave every row as it is, unlooked at
        if stream is None and _current_device() == self._index:
            return self._attention(_raw_stream(self._index), tok, length, max_q, q, qs, scale, causal, out, lse, want_lse, ws, tree)
        return _on(self.device, stream, self._attention, tok, length, max_q, q, qs, scale, causal, out, lse, want_lse, ws, tree)

    def _attention(self, handle, tok, length, max_q, q, qs, scale, causal, out, lse, want_lse, ws, tree):
        dev, shape = self.device, q.shape
        if out is None:
            out = _empty(shape, dtype=q.dtype, device=dev)
        elif not _fits(out, shape, q.dtype, dev):
            _whole(out, shape, q.dtype, dev, "out")
        if lse is not None:
            _whole(lse, shape[:2], _f32, dev, "lse")
        elif want_lse:
            lse = _empty(shape[:2], dtype=_f32, device=dev)
        if ws is None:
            ws = self.attention_workspace(shape[1], tok.n_tokens, tok.n_seqs)
        if tree is not None and tok.n_tokens:
            _check(lib.pi_kv_tree_attention(self._ref, C.addressof(tok), length.data_ptr(), max_q, tree.data_ptr(), tree.shape[1],
                                            q.data_ptr(), qs, shape[1], _DT[q.dtype], scale, out.data_ptr(), _ptr(lse),
                                            ws.data_ptr(), _ws(ws, dev), handle), "pi_kv_tree_attention")
            return out if lse is None else (out, lse)
        _check(lib.pi_kv_attention(self._ref, C.addressof(tok), length.data_ptr(), max_q, q.data_ptr(), qs, shape[1],
                                   _DT[q.dtype], scale, 1 if causal else 0, out.data_ptr(), _ptr(lse), ws.data_ptr(),
                                   _ws(ws, dev), handle), "pi_kv_attention")
        return out if lse is None else (out, lse)

    def device_status(self, stream=None) -> int:
        """0 if no call met a bad page, position or token range since the last query, else the status code."""
        return _on(self.device, stream, lambda handle: int(lib.pi_kv_status(self._ref, handle)))


def _rows2d(x, name):
    """x as rows of its last dimension: (rows, d, elements between rows)."""
    d = x.shape[-1] if x.dim() else 0
    if x.dim() == 2 and (x.stride(1) == 1 or d == 1):
        return x.shape[0], d, x.stride(0) if x.shape[0] > 1 else d
    if x.dim() < 1 or not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous, or two-dimensional with contiguous rows")
    return x.numel() // d if d else 0, d, d


def layer_norm(x, weight=None, bias=None, eps=1e-5, add=None, y=None, sum=None, mean=None, rstd=None,
               want_stats=False, stream=None):
    """Layer norm of x over its last dimension; with ``add``, of x + add, which
    is stored in ``sum`` in x's type (``sum`` may be x).  Returns (y, sum, mean,
    rstd): sum is None without add, mean and rstd (float32, one a row) are None
    unless given or asked for with want_stats."""
    dev = _dev(x, None, "x")
    dt = _dt(x, "x")
    rows, d, stride = _rows2d(x, "x")
    w_dt = add_dt = 0
    w_ptr = b_ptr = add_ptr = None
    if weight is not None:
        w_dt, w_ptr = _dt(weight, "weight"), weight.data_ptr()
        if not _fits(weight, (d,), weight.dtype, dev):
            _whole(weight, (d,), weight.dtype, dev, "weight")
    if bias is not None:
        if weight is None:
            w_dt = _dt(bias, "bias")
        elif bias.dtype is not weight.dtype:
            raise TypeError("weight and bias must have one type")
        b_ptr = bias.data_ptr()
        if not _fits(bias, (d,), bias.dtype, dev):
            _whole(bias, (d,), bias.dtype, dev, "bias")
    if add is not None:
        add_dt, add_ptr = _dt(add, "add"), add.data_ptr()
        if not _fits(add, x.shape, add.dtype, dev):
            _whole(add, x.shape, add.dtype, dev, "add")
    elif sum is not None:
        raise ValueError("sum needs add")
    args = (x, stride, add_ptr, add_dt, w_ptr, b_ptr, w_dt, rows, d, dt, eps, y, sum, mean, rstd, want_stats, dev)
    if stream is None and _current_device() == dev.index:
        return _norm(_raw_stream(dev.index), *args)
    return _on(dev, stream, _norm, *args)


def _norm(handle, x, stride, add, add_dt, w, b, w_dt, rows, d, dt, eps, y, sum, mean, rstd, want_stats, dev):
    shape, dtype = x.shape, x.dtype
    if y is None:
        y = _empty(shape, dtype=dtype, device=dev)
    elif not _fits(y, shape, dtype, dev):
        _whole(y, shape, dtype, dev, "y")
    if add is not None or sum is not None:
        if sum is None:
            sum = _empty(shape, dtype=dtype, device=dev)
        elif not _fits(sum, shape, dtype, dev):
            _whole(sum, shape, dtype, dev, "sum")
    if mean is not None:
        _whole(mean, (rows,), _f32, dev, "mean")
    elif want_stats:
        mean = _empty(rows, dtype=_f32, device=dev)
    if rstd is not None:
        _whole(rstd, (rows,), _f32, dev, "rstd")
    elif want_stats:
        rstd = _empty(rows, dtype=_f32, device=dev)
    _check(lib.pi_layer_norm(x.data_ptr(), stride, add, add_dt, w, b, w_dt, rows, d, dt, eps, y.data_ptr(), _ptr(sum),
                             _ptr(mean), _ptr(rstd), handle), "pi_layer_norm")
    return y, sum, mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd, d_sum=None, dx=None, dweight=None, dbias=None, ws=None,
                        want_weight_grad=True, stream=None):
    """Gradient of ``layer_norm``: x is what was normed (``sum`` where something
    was added), mean and rstd as it returned them, d_sum the gradient that
    reaches ``sum`` another way.  Returns (dx, dweight, dbias); dx has x's type
    and may be dy, the other two are float32 (None without want_weight_grad)."""
    dev = _dev(x, None, "x")
    dt = _dt(x, "x")
    rows, d, stride = _rows2d(x, "x")
    for t, shape, dtype, name in ((dy, x.shape, x.dtype, "dy"), (mean, (rows,), _f32, "mean"), (rstd, (rows,), _f32, "rstd")):
        if not _fits(t, shape, dtype, dev):
            _whole(t, shape, dtype, dev, name)
    if d_sum is not None:
        _whole(d_sum, x.shape, x.dtype, dev, "d_sum")
    if weight is not None:
        _whole(weight, (d,), weight.dtype, dev, "weight")
    return _on(dev, stream, _norm_backward, dy, x, rows, d, stride, dt, weight, mean, rstd, d_sum, dx, dweight, dbias, ws,
               want_weight_grad)


def _norm_backward(handle, dy, x, rows, d, stride, dt, weight, mean, rstd, d_sum, dx, dweight, dbias, ws, want):
    dev = x.device
    dx = torch.empty(x.shape, dtype=x.dtype, device=dev) if dx is None else _whole(dx, x.shape, x.dtype, dev, "dx")
    if dweight is not None:
        _whole(dweight, (d,), _f32, dev, "dweight")
    elif want:
        dweight = torch.empty(d, dtype=_f32, device=dev)
    if dbias is not None:
        _whole(dbias, (d,), _f32, dev, "dbias")
    elif want:
        dbias = torch.empty(d, dtype=_f32, device=dev)
    if ws is None and (dweight is not None or dbias is not None):
        ws = torch.empty(lib.pi_layer_norm_backward_workspace_bytes(rows, d), dtype=_u8, device=dev)
    _check(lib.pi_layer_norm_backward(dy.data_ptr(), x.data_ptr(), stride, _ptr(weight),
                                      0 if weight is None else _dt(weight, "weight"), mean.data_ptr(), rstd.data_ptr(),
                                      _ptr(d_sum), rows, d, dt, dx.data_ptr(), _ptr(dweight), _ptr(dbias), _ptr(ws),
                                      0 if ws is None else _ws(ws, dev), handle), "pi_layer_norm_backward")
    return dx, dweight, dbias


class TokenScores(NamedTuple):
    """What ``token_logprobs`` returns; float32 [rows], top_* [rows, top_k]."""
    logprob: Optional[torch.Tensor]
    entropy: torch.Tensor
    lse: torch.Tensor
    top_index: Optional[torch.Tensor]
    top_logprob: Optional[torch.Tensor]


def token_logprobs(logits, targets=None, top_k=0, stream=None) -> TokenScores:
    """Log-probability of targets (int32 [rows]; below 0: padding, 0), entropy
    and log of the sum of exponentials of logits [rows, vocab], and its top_k
    tokens (int32 indices, log-probabilities), equal logits by lower index."""
    dev = _dev(logits, None, "logits")
    dt = _dt(logits, "logits")
    if logits.dim() != 2 or (logits.stride(1) != 1 and logits.shape[1] != 1 and logits.shape[0]):
        raise ValueError("logits must be [rows, vocab] with contiguous rows")
    rows, vocab = logits.shape
    if targets is not None and not _fits(targets, (rows,), _i32, dev):
        _whole(targets, (rows,), _i32, dev, "targets")
    if stream is None and _current_device() == dev.index:
        return _score(_raw_stream(dev.index), logits, rows, vocab, dt, targets, top_k)
    return _on(dev, stream, _score, logits, rows, vocab, dt, targets, top_k)


def _score(handle, logits, rows, vocab, dt, targets, top_k):
    dev = logits.device
    index = value = logprob = None
    entropy = _empty(rows, dtype=_f32, device=dev)
    lse = _empty(rows, dtype=_f32, device=dev)
    if targets is not None:
        logprob = _empty(rows, dtype=_f32, device=dev)
    if top_k > 0:
        index = _empty((rows, top_k), dtype=_i32, device=dev)
        value = _empty((rows, top_k), dtype=_f32, device=dev)
    _check(lib.pi_token_logprobs(
        logits.data_ptr(), logits.stride(0) if rows > 1 else vocab, dt, rows, vocab,
        targets.data_ptr() if targets is not None else None, top_k, logprob.data_ptr() if targets is not None else None,
        entropy.data_ptr(), lse.data_ptr(), index.data_ptr() if top_k > 0 else None,
        value.data_ptr() if top_k > 0 else None, handle), "pi_token_logprobs")
    return TokenScores(logprob, entropy, lse, index, value)


def _most_nodes(max_q, n):
    """max_q as given, or as few as there can be."""
    if max_q is None:
        if n > PI_MAX_TREE:
            raise ValueError(f"max_q must be given for more than {PI_MAX_TREE} nodes")
        return max(1, n)
    if not 1 <= max_q <= PI_MAX_TREE:
        raise ValueError(f"max_q must be 1 to {PI_MAX_TREE}, not {max_q}")
    return max_q


def _nodes(parent, cu_tokens, device):
    if parent.dim() != 1 or not _fits(parent, parent.shape, _i32, device):
        _whole(parent, (parent.numel(),), _i32, device, "parent")
    if cu_tokens.dim() != 1 or cu_tokens.shape[0] < 1:
        raise ValueError("cu_tokens must be int32 [sequences + 1]")
    if not _fits(cu_tokens, cu_tokens.shape, _i32, device):
        _whole(cu_tokens, cu_tokens.shape, _i32, device, "cu_tokens")
    return cu_tokens.shape[0] - 1, parent.shape[0]


def draft_tree(parent, cu_tokens, max_q=None, stream=None):
    """Trees of drafted tokens, packed by sequence: parent (int32 [tokens]) is the
    index in its sequence of the node that a node hangs on, or -1.  Returns (mask, depth): int32
    [tokens, ceil(max_q / 32)], bit j set for the nodes j of the sequence on a node's
    way from its root (itself among them), as ``KVCache.attention`` takes it, and int32
    [tokens], the nodes above it.  max_q bounds the nodes of any sequence, by default all nodes."""
    dev = _dev(parent, None, "parent")
    seqs, n = _nodes(parent, cu_tokens, dev)
    max_q = _most_nodes(max_q, n)
    if stream is None and _current_device() == dev.index:
        return _draft_tree(_raw_stream(dev.index), parent, cu_tokens, seqs, n, max_q, dev)
    return _on(dev, stream, _draft_tree, parent, cu_tokens, seqs, n, max_q, dev)


def _draft_tree(handle, parent, cu_tokens, seqs, n, max_q, dev):
    mask = _empty((n, (max_q + 31) // 32), dtype=_i32, device=dev)
    depth = _empty(n, dtype=_i32, device=dev)
    _check(lib.pi_draft_tree(parent.data_ptr(), cu_tokens.data_ptr(), seqs, n, max_q, mask.data_ptr(), depth.data_ptr(),
                             handle), "pi_draft_tree")
    return mask, depth


class DraftVerdict(NamedTuple):
    """What ``verify_draft`` returns; int32 [sequences], path [sequences, max_q]."""
    accepted: torch.Tensor
    path: torch.Tensor
    token: torch.Tensor


def _probs(t, shape, dtype, device, name):
    _dev(t, device, name)
    if t.dim() != 2 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must be [tokens, vocab]" + ("" if shape is None else f" as the target, {tuple(shape)}")
                         + f", got {tuple(t.shape)}")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must have the target's type, {dtype}")
    if t.stride(1) != 1 and t.shape[1] != 1 and t.shape[0]:
        raise ValueError(f"{name}: rows must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def verify_draft(target, draft, tokens, parent, cu_tokens, accept_u, sample_u, max_q=None, stream=None) -> DraftVerdict:
    """Which drafted tokens the target accepts, and the token that follows them.

    Nodes as in ``draft_tree``, each sequence's first node its last known token, with
    ``tokens`` (int32 [tokens]; that of the first node is not used).  Row r of target and draft
    (probabilities [tokens, vocab] of one type) says what follows node r; draft is None
    where the drafted tokens were chosen, not drawn.  accept_u (float32 [tokens]) and
    sample_u (float32 [sequences]) are uniform numbers in [0, 1).  Returns (accepted,
    path, token): how many drafted tokens were accepted, the nodes (0, the accepted
    ones, -1 behind them) and the next token.  max_q as in ``draft_tree``."""
    dev = _dev(target, None, "target")
    dt = _dt(target, "target")
    ts = _probs(target, None, None, dev, "target")
    qs = 0 if draft is None else _probs(draft, target.shape, target.dtype, dev, "draft")
    seqs, n = _nodes(parent, cu_tokens, dev)
    if target.shape[0] != n:
        raise ValueError(f"target has {target.shape[0]} rows for {n} nodes")
    for t, shape, dtype, name in ((tokens, (n,), _i32, "tokens"), (accept_u, (n,), _f32, "accept_u"),
                                  (sample_u, (seqs,), _f32, "sample_u")):
        if not _fits(t, shape, dtype, dev):
            _whole(t, shape, dtype, dev, name)
    max_q = _most_nodes(max_q, n)
    args = (target, ts, draft, qs, dt, tokens, parent, cu_tokens, seqs, n, max_q, accept_u, sample_u, dev)
    if stream is None and _current_device() == dev.index:
        return _verify(_raw_stream(dev.index), *args)
    return _on(dev, stream, _verify, *args)


def _verify(handle, target, ts, draft, qs, dt, tokens, parent, cu_tokens, seqs, n, max_q, accept_u, sample_u, dev):
    accepted = _empty(seqs, dtype=_i32, device=dev)
    path = _empty((seqs, max_q), dtype=_i32, device=dev)
    token = _empty(seqs, dtype=_i32, device=dev)
    _check(lib.pi_verify_draft(target.data_ptr(), ts, _ptr(draft), qs, dt, target.shape[1], tokens.data_ptr(), parent.data_ptr(),
                               cu_tokens.data_ptr(), seqs, n, max_q, accept_u.data_ptr(), sample_u.data_ptr(),
                               accepted.data_ptr(), path.data_ptr(), token.data_ptr(), handle), "pi_verify_draft")
    return DraftVerdict(accepted, path, token)
