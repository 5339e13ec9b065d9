"""Binding of the sequence operators in include/sparseconv.h: the short causal convolution, the
selective state space scan and the low-rank adapters, for prompts and for single positions.

As in the rest of the package only arguments are marshalled here.  The functions with the C
names take the packed argument structure; ``causal_conv``, ``causal_conv_step``,
``selective_scan``, ``selective_scan_step`` and ``adapter_apply`` take torch tensors, check
their types, shapes and strides, and allocate what is not given.  Nothing is differentiable.

Sequence tensors are (batch, channels, positions) with contiguous positions; batch and channel
strides are free, so slices of a projection's output are taken as they are.  The ``_step``
functions take single positions, (batch, channels) with any strides.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import _check, _i32, _lib, _stream_ptr, _vp

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


def _bad(t, name, dtype, shape, how):
    got = f"{tuple(t.shape)} {t.dtype} on {t.device}, strides {t.stride()}" if isinstance(t, torch.Tensor) else repr(t)
    return ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on x's GPU, {how}: got {got}")


def _activation(t, name, dtype, dev, shape):
    """Strides of a tensor whose last axis is contiguous."""
    if t.dtype is dtype and t.get_device() == dev and t.shape == shape:
        st = t.stride()
        if st[-1] == 1 or shape[-1] <= 1:
            return st
    raise _bad(t, name, dtype, shape, "its last axis contiguous")


def _dense(t, name, dtype, dev, shape):
    """Address of a contiguous tensor; 0 for None."""
    if t is None:
        return 0
    if t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    raise _bad(t, name, dtype, shape, "contiguous")


def _states(t, name, dtype, dev, D, per):
    """(address, slots, slot stride) of a pool of states; zeros for None."""
    if t is None:
        return 0, 0, 0
    if t.dtype is dtype and t.get_device() == dev and t.dim() == 3 and t.shape[1:] == (D, per):
        st = t.stride()
        n = t.shape[0]
        if per == 0:
            return 0, n, 0
        if (st[2] == 1 or per == 1) and (st[1] == per or D == 1):
            return t.data_ptr(), n, st[0] if n > 1 else D * per
    raise _bad(t, name, dtype, ("slots", D, per), "each slot contiguous")


def _first_device(x):
    if not isinstance(x, torch.Tensor) or x.dtype not in _TYPES or not x.is_cuda:
        raise ValueError("x must be a float32, bfloat16 or float16 tensor on the GPU")
    return x.get_device()


def _empty(shape, dtype, dev, stream):
    """A new tensor that belongs to the stream the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _launch(fn, where, args, stream, dev):
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            _check(fn(args, _stream_ptr(stream, dev)), where)
    else:
        _check(fn(args, _stream_ptr(stream, dev)), where)


def _conv(x, xs, out, os_, B, D, L, weight, bias, silu, lengths, slots, initial_state, final_state, stream, dev):
    if weight.dim() != 2:
        raise ValueError(f"weight shape {tuple(weight.shape)} is not ({D}, taps)")
    K = weight.shape[1]
    dtype = x.dtype
    fp, fn, fs = _states(initial_state, "initial_state", dtype, dev, D, K - 1)
    lp, ln, ls = _states(final_state, "final_state", dtype, dev, D, K - 1)
    if fn != ln and initial_state is not None and final_state is not None:
        raise ValueError(f"initial_state has {fn} slots, final_state {ln}")
    _launch(_lib.sparseconv_causal_conv, "sparseconv_causal_conv",
            sc_causal_conv.pack(x.data_ptr(), out.data_ptr(), _dense(weight, "weight", torch.float32, dev, (D, K)),
                                _dense(bias, "bias", torch.float32, dev, (D,)), fp, lp,
                                _dense(lengths, "lengths", torch.int32, dev, (B,)),
                                _dense(slots, "slots", torch.int32, dev, (B,)), xs[0], xs[1], os_[0], os_[1], fs, ls,
                                _TYPES[dtype], B, D, L, K, fn or ln or B, SC_SEQ_SILU if silu else 0, 0),
            stream, dev)
    return out


def causal_conv(x, weight, bias=None, *, silu=True, lengths=None, slots=None, initial_state=None, final_state=None,
                out=None, stream=None):
    """Short causal convolution of each channel of x (B, D, L) with weight (D, K) float32 and
    bias (D,) float32, K <= 8, through SiLU unless silu is False; returns out (B, D, L).

    initial_state and final_state: pools (slots, D, K - 1) of x's type with the last K - 1 inputs
    of each sequence, read (default: zeros) and written (the same pool may be both).  slots
    (B,) int32: each sequence's slot (default: its number); one outside the pool is idle, its
    output 0.  lengths (B,) int32: positions past a sequence's length give 0 and leave the state
    alone."""
    dev = _first_device(x)
    if x.dim() != 3:
        raise ValueError(f"x must be (B, D, L), got {tuple(x.shape)}")
    shape = x.shape
    xs = _activation(x, "x", x.dtype, dev, shape)
    if out is None:
        out = _empty(shape, x.dtype, dev, stream)
    return _conv(x, xs, out, _activation(out, "out", x.dtype, dev, shape), *shape, weight, bias, silu, lengths, slots,
                 initial_state, final_state, stream, dev)


def causal_conv_step(x, state, weight, bias=None, *, silu=True, slots=None, out=None, stream=None):
    """The same for the next position of each sequence: x (B, D), state (slots, D, K - 1) updated
    in place; returns out (B, D)."""
    dev = _first_device(x)
    if x.dim() != 2:
        raise ValueError(f"x must be (B, D), got {tuple(x.shape)}")
    shape = x.shape
    if out is None:
        out = _empty(shape, x.dtype, dev, stream)
    elif out.dtype is not x.dtype or out.get_device() != dev or out.shape != shape:
        raise _bad(out, "out", x.dtype, shape, "strided")
    return _conv(x, x.stride(), out, out.stride(), *shape, 1, weight, bias, silu, None, slots, state, state, stream, dev)


def _scan(x, L, dt, A, B, C, D, z, dt_bias, softplus, lengths, slots, initial_state, final_state, out, workspace, stream,
          dev):
    """x, dt, z, out: (B, D, L), or (B, D) with L = 1; B, C: (B, G, N, L), or (B, G, N)."""
    dtype, shape = x.dtype, x.shape
    nb, nd = shape[0], shape[1]
    step = len(shape) == 2
    if A.dim() != 2:
        raise ValueError(f"A shape {tuple(A.shape)} is not ({nd}, states)")
    N = A.shape[1]
    if B.dim() != 4 - step:
        raise ValueError(f"B shape {tuple(B.shape)} is not (batch, groups, states{'' if step else ', positions'})")
    G = B.shape[1]
    bc = (nb, G, N) if step else (nb, G, N, L)
    if step:
        for t, name, sh in ((dt, "dt", shape), (z, "z", shape), (B, "B", bc), (C, "C", bc), (out, "out", shape)):
            if t is not None and (t.dtype is not dtype or t.get_device() != dev or t.shape != sh):
                raise _bad(t, name, dtype, sh, "strided")
        xs, ds, bs, cs = x.stride(), dt.stride(), B.stride(), C.stride()
        zs = z.stride() if z is not None else (0, 0)
    else:
        xs = _activation(x, "x", dtype, dev, shape)
        ds = _activation(dt, "dt", dtype, dev, shape)
        zs = _activation(z, "z", dtype, dev, shape) if z is not None else (0, 0)
        bs = _activation(B, "B", dtype, dev, bc)
        cs = _activation(C, "C", dtype, dev, bc)
    if out is None:
        out = _empty(shape, dtype, dev, stream)
        os_ = out.stride()
    else:
        os_ = out.stride() if step else _activation(out, "out", dtype, dev, shape)
    fp, fn, fs = _states(initial_state, "initial_state", torch.float32, dev, nd, N)
    lp, ln, ls = _states(final_state, "final_state", torch.float32, dev, nd, N)
    if fn != ln and initial_state is not None and final_state is not None:
        raise ValueError(f"initial_state has {fn} slots, final_state {ln}")
    sizes = (_TYPES[dtype], nb, nd, L, N, G, fn or ln or nb, SC_SEQ_SOFTPLUS if softplus else 0)
    wp = need = 0
    if not step:
        need = sparseconv_selective_scan_workspace(_SIZES_ONLY.pack(*sizes))
        if need:
            if workspace is None:
                workspace = _empty((need,), torch.uint8, dev, stream)
            elif not workspace.is_contiguous() or workspace.get_device() != dev:
                raise ValueError("workspace must be a contiguous tensor on x's GPU")
            wp, need = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    f32 = torch.float32
    _launch(_lib.sparseconv_selective_scan, "sparseconv_selective_scan",
            sc_selective_scan.pack(x.data_ptr(), dt.data_ptr(), z.data_ptr() if z is not None else 0, B.data_ptr(),
                                   C.data_ptr(), out.data_ptr(), _dense(A, "A", f32, dev, (nd, N)),
                                   _dense(D, "D", f32, dev, (nd,)), _dense(dt_bias, "dt_bias", f32, dev, (nd,)), fp, lp,
                                   _dense(lengths, "lengths", torch.int32, dev, (nb,)),
                                   _dense(slots, "slots", torch.int32, dev, (nb,)), wp, need, xs[0], xs[1], ds[0], ds[1],
                                   zs[0], zs[1], os_[0], os_[1], bs[0], bs[1], bs[2], cs[0], cs[1], cs[2], fs, ls, *sizes),
            stream, dev)
    return out


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
    dev = _first_device(x)
    if x.dim() != 3:
        raise ValueError(f"x must be (B, D, L), got {tuple(x.shape)}")
    return _scan(x, x.shape[2], dt, A, B, C, D, z, dt_bias, softplus, lengths, slots, initial_state, final_state, out,
                 workspace, stream, dev)


def selective_scan_step(x, state, dt, A, B, C, *, D=None, z=None, dt_bias=None, softplus=True, slots=None, out=None,
                        stream=None):
    """The same for the next position of each sequence: x, dt, z (B, D), B and C (batch, groups, N),
    state (slots, D, N) float32 updated in place; returns out (B, D)."""
    dev = _first_device(x)
    if x.dim() != 2:
        raise ValueError(f"x must be (B, D), got {tuple(x.shape)}")
    return _scan(x, 1, dt, A, B, C, D, z, dt_bias, softplus, None, slots, state, state, out, None, stream, dev)


_ADAPTER_SIZES = struct.Struct("=64x8x6q8i")


def adapter_apply(x, down, up, index, *, scale=None, base=None, out=None, workspace=None, stream=None):
    """out[b] = base[b] + scale[r] * up[r] @ (down[r] @ x[b]) with r = index[b]: low-rank adapters of
    many requests beside a projection they share.

    x (B, C, L); base (B, M, L), the shared projection's output (default: zeros); down
    (adapters, R, C) and up (adapters, M, R) of x's type, contiguous; scale (adapters,) float32;
    index (B,) int32, no adapter where it is outside 0 .. adapters-1.  out may be base itself.
    workspace: a contiguous tensor, allocated where none is given."""
    dev = _first_device(x)
    if x.dim() != 3 or down.dim() != 3 or up.dim() != 3:
        raise ValueError(f"x, down and up must have three axes, got {tuple(x.shape)}, {tuple(down.shape)}, {tuple(up.shape)}")
    dtype = x.dtype
    nb, nc, L = x.shape
    n, R = down.shape[0], down.shape[1]
    M = up.shape[1]
    shape = (nb, M, L)
    xs = _activation(x, "x", dtype, dev, (nb, nc, L))
    bs = _activation(base, "base", dtype, dev, shape) if base is not None else (0, 0)
    if out is None:
        out = _empty(shape, dtype, dev, stream)
    os_ = _activation(out, "out", dtype, dev, shape)
    tail = (xs[0], xs[1], bs[0], bs[1], os_[0], os_[1], _TYPES[dtype], nb, nc, M, L, R, n, 0)
    need = sparseconv_adapter_workspace(_ADAPTER_SIZES.pack(*tail))
    wp = 0
    if need:
        if workspace is None:
            workspace = _empty((need,), torch.uint8, dev, stream)
        elif not workspace.is_contiguous() or workspace.get_device() != dev:
            raise ValueError("workspace must be a contiguous tensor on x's GPU")
        wp, need = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _launch(_lib.sparseconv_adapter_apply, "sparseconv_adapter_apply",
            sc_adapter.pack(x.data_ptr(), base.data_ptr() if base is not None else 0, out.data_ptr(),
                            _dense(down, "down", dtype, dev, (n, R, nc)), _dense(up, "up", dtype, dev, (n, M, R)),
                            _dense(scale, "scale", torch.float32, dev, (n,)),
                            _dense(index, "index", torch.int32, dev, (nb,)), wp, need, *tail),
            stream, dev)
    return out
