"""Binding of the attention operators in include/sparseconv.h: attention of new positions over a paged
cache, rotary positions with the cache's update, copies of pages, and the norms around a block with its
residual sum.

As in sequence.py only arguments are marshalled here: the functions with the C names take the packed
argument structure; the others take torch tensors through the native binding (csrc/binding.cpp):
ValueError where a tensor does not fit, SparseConvError where the library refuses the call.  Nothing is
differentiable: a tensor that requires a gradient is refused unless gradients are off.

Activations are (batch, channels, positions) with contiguous positions and free batch and channel
strides, heads one after another along the channels; the ``_step`` functions take single positions,
(batch, channels) with any strides.  A cache is k_pages (pages, G, P, D) and v_pages (pages, G, D, P) for G heads of D dims and
pages of P positions, each page contiguous; table (batch, width) int32 names the pages of each sequence and past (batch,)
int32 says how many positions it has before the call.  Entries of the table outside the pool are no pages;
a sequence whose past is outside 0 .. width*P is idle (its outputs are 0 and nothing of it is written).
"""
from __future__ import annotations

import ctypes
import struct


from . import _check, _i32, _lib, _stream_ptr, _vp
from .sequence import _binding, _run

SC_ATT_OUT_F32, SC_ROT_INTERLEAVED, SC_NORM_CENTER = 1, 1, 1

# the C argument structures, field by field (pointers, 64-bit sizes and strides, floats, 32-bit sizes)
sc_paged_attention = struct.Struct("=10Q8q2f10iIi")
sc_cache_append = struct.Struct("=12Q13q12iIi")
sc_cache_copy = struct.Struct("=3Q3q4i")
sc_residual_norm = struct.Struct("=9Q11q2f4iIi")

for _name in ("sparseconv_paged_attention", "sparseconv_cache_append", "sparseconv_cache_copy", "sparseconv_residual_norm"):
    getattr(_lib, _name).restype = _i32
    getattr(_lib, _name).argtypes = [ctypes.c_char_p, _vp]
_lib.sparseconv_paged_attention_workspace.restype = _i32
_lib.sparseconv_paged_attention_workspace.argtypes = [ctypes.c_char_p, ctypes.POINTER(ctypes.c_int64)]


def sparseconv_paged_attention(args: bytes, stream=None) -> None:
    _check(_lib.sparseconv_paged_attention(args, _stream_ptr(stream)), "sparseconv_paged_attention")


def sparseconv_paged_attention_workspace(args: bytes) -> int:
    b = ctypes.c_int64()
    _check(_lib.sparseconv_paged_attention_workspace(args, ctypes.byref(b)), "sparseconv_paged_attention_workspace")
    return b.value


def sparseconv_cache_append(args: bytes, stream=None) -> None:
    _check(_lib.sparseconv_cache_append(args, _stream_ptr(stream)), "sparseconv_cache_append")


def sparseconv_cache_copy(args: bytes, stream=None) -> None:
    _check(_lib.sparseconv_cache_copy(args, _stream_ptr(stream)), "sparseconv_cache_copy")


def sparseconv_residual_norm(args: bytes, stream=None) -> None:
    _check(_lib.sparseconv_residual_norm(args, _stream_ptr(stream)), "sparseconv_residual_norm")


def paged_attention(q, k_pages, v_pages, table, past, *, lengths=None, scale=None, cap=0.0, window=0, slopes=None, prefix=None,
                    out=None, workspace=None, stream=None):
    """Attention of the new positions q (B, H*D, L) over a cache that holds them already; returns out (B, H*D, L).

    Head h reads the cache's head h // (H // G); position i of sequence b is its position past[b] + i.  Scores
    are scale * q.k (default D ** -0.5), through cap * tanh(s / cap) with a cap, minus slopes[h] times the
    distance (slopes (H,) float32).  Visible are the positions before the sequence's end that lie in its
    prefix (prefix (B,) int32), and those up to the query's own, with a window the last `window` of
    them; where nothing is visible out is 0.  lengths (B,) int32: positions past a sequence's length give 0.
    out may be float32 for 16-bit q, which keeps the weights in twice the bits.  workspace: a contiguous tensor, allocated where none is given."""
    return _run(_binding.paged_attention, "sparseconv_paged_attention", stream, q, k_pages, v_pages, table, past, lengths, prefix,
                slopes, scale, cap, window, out, workspace, 3)


def paged_attention_step(q, k_pages, v_pages, table, past, *, scale=None, cap=0.0, window=0, slopes=None, prefix=None, out=None,
                         workspace=None, stream=None):
    """The same for the next position of each sequence: q (B, H*D); returns out (B, H*D)."""
    return _run(_binding.paged_attention, "sparseconv_paged_attention", stream, q, k_pages, v_pages, table, past, None, prefix,
                slopes, scale, cap, window, out, workspace, 2)


_SIZES_ONLY = struct.Struct("=152x10i8x")  # sc_paged_attention with nothing but its sizes


def paged_attention_workspace(B, H, L, k_pages, width) -> int:
    """Bytes of workspace an attention of L new positions with a table of `width` pages needs (0: none)."""
    from .sequence import _TYPES
    pages, G, P, D = k_pages.shape
    return sparseconv_paged_attention_workspace(_SIZES_ONLY.pack(_TYPES[k_pages.dtype], B, H, G, D, L, P, width, pages, 0))


def cache_append(k, v, k_pages, v_pages, table, past, *, q=None, freqs=None, axes=None, positions=None, interleaved=False,
                 lengths=None, out=None, stream=None):
    """Writes the new positions' k and v (B, G*D, L) into the cache, k turned by its rotary positions; returns q (B, H*D, L)
    turned likewise, in the cache's type (None without q).

    freqs (pairs,) float64: the angle a position turns each pair by, in radians; the pairs are dims j and j + pairs
    of a head, or 2 j and 2 j + 1 if interleaved, and dims past 2 * pairs stay.  positions (B, n, L) int32: n coordinates of
    each position (default: one, its place in the sequence) and axes (pairs,) int32: the one that turns each
    pair (default: the first).  A float32 k may have a cache of any type, else the types are the same.  out may be q itself."""
    return _run(_binding.cache_append, "sparseconv_cache_append", stream, k, v, k_pages, v_pages, table, past, q, freqs, axes,
                positions, interleaved, lengths, out, 3)


def cache_append_step(k, v, k_pages, v_pages, table, past, *, q=None, freqs=None, axes=None, positions=None, interleaved=False,
                      out=None, stream=None):
    """The same for the next position of each sequence: k, v (B, G*D), q (B, H*D), positions (B, n, 1)."""
    return _run(_binding.cache_append, "sparseconv_cache_append", stream, k, v, k_pages, v_pages, table, past, q, freqs, axes,
                positions, interleaved, None, out, 2)


def cache_copy(pool, source, target, *, stream=None):
    """Copies page source[i] over page target[i] in every block of pool (blocks, pages, ...), whose pages are
    contiguous; returns pool.  source, target (n,) int32; a pair with an entry outside the pool is left out.  No page may be
    the target of two pairs, or of one and the source of another."""
    return _run(_binding.cache_copy, "sparseconv_cache_copy", stream, pool, source, target)


def residual_norm(x, y=None, *, weight=None, bias=None, post_weight=None, post_bias=None, gate=None, scale=1.0, eps=1e-6,
                  center=False, sum=None, out=None, stream=None):
    """The norms around a block: with the residual stream x (B, C, L) and the block's output y, r = x + scale * gate *
    post(y) and norm(r) * weight + bias; returns (r, norm).

    norm divides by the root of the mean square over the channels, after subtracting the mean if `center`; post
    is that norm with post_weight and post_bias, or y itself where there is no post_weight.  Weights and biases
    (C,) float32.  gate (B, C) or (B, C, L) of x's type.  Without y, r is x; without weight and out there is
    no second norm (None).  sum may be x itself and out y itself."""
    return _run(_binding.residual_norm, "sparseconv_residual_norm", stream, x, y, weight, bias, post_weight, post_bias, gate, scale,
                eps, center, sum, out, 3)


def residual_norm_step(x, y=None, *, weight=None, bias=None, post_weight=None, post_bias=None, gate=None, scale=1.0, eps=1e-6,
                       center=False, sum=None, out=None, stream=None):
    """The same for single positions: x, y (B, C), gate (B, C)."""
    return _run(_binding.residual_norm, "sparseconv_residual_norm", stream, x, y, weight, bias, post_weight, post_bias, gate, scale,
                eps, center, sum, out, 2)
