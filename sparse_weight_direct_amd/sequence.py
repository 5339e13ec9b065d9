"""Binding of the sequence operators in include/sparseconv.h: the short causal convolution, the
selective state space scan and the low-rank adapters, for prompts and for single positions.

As in the rest of the package only arguments are marshalled here.  The functions with the C
names take the packed argument structure; ``causal_conv``, ``causal_conv_step``,
``selective_scan``, ``selective_scan_step`` and ``adapter_apply`` take torch tensors through the
native binding (csrc/binding.cpp), which checks their types, shapes and strides and allocates what is
not given: ValueError where a tensor does not fit, SparseConvError where the library refuses the
call.  Nothing is differentiable: a tensor that requires a gradient is refused unless gradients are
off (torch.no_grad()).

Sequence tensors are (batch, channels, positions) with contiguous positions; batch and channel
strides are free, so slices of a projection's output are taken as they are.  The ``_step``
functions take single positions, (batch, channels) with any strides.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import LIB_PATH, SparseConvError, _check, _i32, _lib, _stream_ptr, _vp



class _NoBinding:
    """Stands for a binding that is missing or does not load: the rest of the package does not need it."""

    def __init__(self, why):
        self._why = why

    def __getattr__(self, name):
        raise ImportError(f"{name} needs _binding.so beside {LIB_PATH}, which is missing or does not load ({self._why}): build it "
                          "with `python -c 'import __graft_entry__ as g; g.build()'`")


try:
    from . import _binding
except ImportError as e:
    _binding = _NoBinding(str(e))

SC_F32, SC_BF16, SC_F16 = range(3)
SC_SEQ_SILU, SC_SEQ_SOFTPLUS = 1, 2
_TYPES = {torch.float32: SC_F32, torch.bfloat16: SC_BF16, torch.float16: SC_F16}

# the C argument structures, field by field (pointers, 64-bit sizes and strides, 32-bit sizes)
sc_causal_conv = struct.Struct("=8Q6q6iIi")
sc_selective_scan = struct.Struct("=14Q17q7iI")
sc_adapter = struct.Struct("=8Q7q8i")

for _name in ("sparseconv_causal_conv", "sparseconv_selective_scan", "sparseconv_adapter_apply"):
    getattr(_lib, _name).restype = _i32
    getattr(_lib, _name).argtypes = [ctypes.c_char_p, _vp]
for _name in ("sparseconv_selective_scan_workspace", "sparseconv_adapter_workspace"):
    getattr(_lib, _name).restype = _i32
    getattr(_lib, _name).argtypes = [ctypes.c_char_p, ctypes.POINTER(ctypes.c_int64)]


def sparseconv_causal_conv(args: bytes, stream=None) -> None:
    _check(_lib.sparseconv_causal_conv(args, _stream_ptr(stream)), "sparseconv_causal_conv")


def sparseconv_selective_scan(args: bytes, stream=None) -> None:
    _check(_lib.sparseconv_selective_scan(args, _stream_ptr(stream)), "sparseconv_selective_scan")


def sparseconv_selective_scan_workspace(args: bytes) -> int:
    b = ctypes.c_int64()
    _check(_lib.sparseconv_selective_scan_workspace(args, ctypes.byref(b)), "sparseconv_selective_scan_workspace")
    return b.value


def sparseconv_adapter_apply(args: bytes, stream=None) -> None:
    _check(_lib.sparseconv_adapter_apply(args, _stream_ptr(stream)), "sparseconv_adapter_apply")


def sparseconv_adapter_workspace(args: bytes) -> int:
    b = ctypes.c_int64()
    _check(_lib.sparseconv_adapter_workspace(args, ctypes.byref(b)), "sparseconv_adapter_workspace")
    return b.value


def _run(fn, where, stream, x, *args):
    """Call a function of the native binding (csrc/binding.cpp) on the current or the given stream; what
    it allocates belongs to that stream."""
    dev = x.get_device() if isinstance(x, torch.Tensor) else -1
    if dev < 0:
        raise ValueError("x must be a tensor on the GPU")
    if stream is None:
        r = fn(x, *args, _stream_ptr(None, dev))
    else:
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=dev) if stream else torch.cuda.default_stream(dev)
        with torch.cuda.stream(stream):
            r = fn(x, *args, stream.cuda_stream)
    if r.__class__ is int:
        raise SparseConvError(r, where)
    return r


def causal_conv(x, weight, bias=None, *, silu=True, lengths=None, slots=None, initial_state=None, final_state=None,
                out=None, stream=None):
    """Short causal convolution of each channel of x (B, D, L) with weight (D, K) float32 and
    bias (D,) float32, K <= 8, through SiLU unless silu is False; returns out (B, D, L).

    initial_state and final_state: pools (slots, D, K - 1) of x's type with the last K - 1 inputs
    of each sequence, read (default: zeros) and written (the same pool may be both).  slots
    (B,) int32: each sequence's slot (default: its number); one outside the pool is idle, its
    output 0.  lengths (B,) int32: positions past a sequence's length give 0 and leave the state
    alone."""
    return _run(_binding.causal_conv, "sparseconv_causal_conv", stream, x, weight, bias, silu, lengths, slots, initial_state,
                final_state, out, 3)


def causal_conv_step(x, state, weight, bias=None, *, silu=True, slots=None, out=None, stream=None):
    """The same for the next position of each sequence: x (B, D), state (slots, D, K - 1) updated
    in place; returns out (B, D)."""
    return _run(_binding.causal_conv, "sparseconv_causal_conv", stream, x, weight, bias, silu, None, slots, state, state, out, 2)


_SIZES_ONLY = struct.Struct("=248x7iI")  # sc_selective_scan with nothing but its sizes


def selective_scan_workspace(x, A, G, dtype=None) -> int:
    """Bytes of workspace a scan of x (B, D, L) with A (D, N) and G groups needs (0: none)."""
    nb, nd, L = x.shape
    return sparseconv_selective_scan_workspace(_SIZES_ONLY.pack(_TYPES[dtype or x.dtype], nb, nd, L, A.shape[1], G, nb, 0))


def selective_scan(x, dt, A, B, C, *, D=None, z=None, dt_bias=None, softplus=True, lengths=None, slots=None,
                   initial_state=None, final_state=None, out=None, workspace=None, stream=None):
    """Selective state space scan over x (B, D, L); returns out (B, D, L).

    dt: the raw time steps, like x; the step is softplus(dt + dt_bias), or dt + dt_bias with
    softplus=False.  A (D, N) float32; B and C (batch, groups, N, L) of x's type, channel d using
    group d // (D // groups).  D, dt_bias (D,) float32; z: the gate, like x (out is multiplied with
    silu(z)).  initial_state, final_state: pools (slots, D, N) float32; slots and lengths as for
    causal_conv.  workspace: a contiguous tensor of selective_scan_workspace(x, A, groups) bytes;
    allocated where none is given."""
    return _run(_binding.selective_scan, "sparseconv_selective_scan", stream, x, dt, A, B, C, D, z, dt_bias, softplus, lengths,
                slots, initial_state, final_state, out, workspace, 3)


def selective_scan_step(x, state, dt, A, B, C, *, D=None, z=None, dt_bias=None, softplus=True, slots=None, out=None,
                        stream=None):
    """The same for the next position of each sequence: x, dt, z (B, D), B and C (batch, groups, N),
    state (slots, D, N) float32 updated in place; returns out (B, D)."""
    return _run(_binding.selective_scan, "sparseconv_selective_scan", stream, x, dt, A, B, C, D, z, dt_bias, softplus, None,
                slots, state, state, out, None, 2)


def adapter_apply(x, down, up, index, *, scale=None, base=None, out=None, workspace=None, stream=None):
    """out[b] = base[b] + scale[r] * up[r] @ (down[r] @ x[b]) with r = index[b]: low-rank adapters of
    many requests beside a projection they share.

    x (B, C, L); base (B, M, L), the shared projection's output (default: zeros); down
    (adapters, R, C) and up (adapters, M, R) of x's type, contiguous; scale (adapters,) float32;
    index (B,) int32, no adapter where it is outside 0 .. adapters-1.  out may be base itself.
    workspace: a contiguous tensor, allocated where none is given."""
    return _run(_binding.adapter_apply, "sparseconv_adapter_apply", stream, x, down, up, index, scale, base, out, workspace)
