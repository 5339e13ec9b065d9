"""A pruned state space layer for serving: packed sparse projections around a short causal
convolution and a selective scan, with low-rank adapters per request.

    x z   = in_proj u  (+ the request's adapter)      pruned 1x1 layer, (2 D, C)
    v     = silu(causal_conv(x))
    p b c = x_proj v                                  pruned 1x1 layer, (R + 2 N, D)
    y     = scan(v, dt_proj p, A, b, c, D, gate z)    pruned 1x1 layer, (D, R)
    out   = out_proj y  (+ the request's adapter)     pruned 1x1 layer, (C, D)

A sequence (B, C, L) is a batch of feature maps with H = 1 and W = L, so the projections are
ordinary handles: one set for prompts of `length` positions (shorter ones are padded on the right
and say so in `lengths`), one for single positions.  The states of all requests stay in two pools
of `slots` slots; a call names the slots of its sequences.  Everything runs on the current stream.
"""
from __future__ import annotations

import numpy as np
import torch

from . import Handle
from .sequence import adapter_apply, causal_conv, causal_conv_step, selective_scan, selective_scan_step


class Adapters:
    """Low-rank adapters of the layer's two outer projections: for each, ``down`` (adapters, R, inputs),
    ``up`` (adapters, outputs, R) and ``scale`` (adapters,), float32 on the GPU.  Either may be None."""

    def __init__(self, in_proj=None, out_proj=None):
        self.in_proj, self.out_proj = in_proj, out_proj


def _adapt(which, x, base, index):
    """base plus the requests' adapters, in place."""
    if which is not None:
        down, up, scale = which
        adapter_apply(x, down, up, index, scale=scale, base=base, out=base)
    return base


def _fits(which, u, B, inputs, outputs, index):
    """Refuses what adapter_apply would refuse of an adapter, before the call that uses it has written any state:
    the same call over no positions, and what such a call does not look at."""
    if which is None:
        return
    down, up, scale = which
    if index is None:
        raise ValueError("adapters need index, each request's adapter")
    adapter_apply(u.new_empty(B, inputs, 0), down, up, index, scale=scale, base=u.new_empty(B, outputs, 0))
    if down.data_ptr() % 16 or up.data_ptr() % 16:
        raise ValueError("an adapter's down and up must be 16-byte aligned")


class StateSpaceLayer:
    """in_proj (2 D, C), x_proj (R + 2 N, D), dt_proj (D, R), out_proj (C, D): pruned float32 weights
    on the host (zeros are not stored).  conv_weight (D, K), conv_bias (D,), A (D, N), skip (D,),
    dt_bias (D,): float32 on the GPU, contiguous (conv_bias, skip and dt_bias may be None).  A call that is
    refused leaves the states as they are."""

    def __init__(self, in_proj, x_proj, dt_proj, out_proj, conv_weight, conv_bias, A, skip, dt_bias, *, length: int,
                 slots: int):
        self.D, self.N = A.shape
        self.R = dt_proj.shape[1]
        self.C = in_proj.shape[1]
        shapes = dict(in_proj=(2 * self.D, self.C), x_proj=(self.R + 2 * self.N, self.D), dt_proj=(self.D, self.R),
                      out_proj=(self.C, self.D))
        weights = dict(in_proj=in_proj, x_proj=x_proj, dt_proj=dt_proj, out_proj=out_proj)
        for name, w in weights.items():
            if tuple(w.shape) != shapes[name]:
                raise ValueError(f"{name} shape {tuple(w.shape)} is not {shapes[name]}")
        params = dict(conv_weight=(conv_weight, (self.D, conv_weight.shape[-1])), conv_bias=(conv_bias, (self.D,)),
                      A=(A, (self.D, self.N)), skip=(skip, (self.D,)), dt_bias=(dt_bias, (self.D,)))
        for name, (t, shape) in params.items():
            if t is None and name in ("conv_bias", "skip", "dt_bias"):
                continue
            if tuple(t.shape) != shape or t.dtype != torch.float32 or t.device != A.device or not t.is_cuda or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous float32 tensor of shape {shape} on A's GPU")
        if not 1 <= conv_weight.shape[1] <= 8 or self.N > 256:
            raise ValueError("at most 8 taps of the convolution and 256 states")
        self.length = length
        self._prompt, self._token = ({n: Handle.from_dense(np.ascontiguousarray(w, np.float32)[:, :, None, None], 1, W, 1, 0)
                                      for n, w in weights.items()} for W in (length, 1))
        # detached: the layer has no gradient, and its operators refuse tensors that ask for one
        self.conv_weight, self.conv_bias, self.A, self.skip, self.dt_bias = (
            None if t is None else t.detach() for t, _ in params.values())
        dev = A.device
        self.conv_state = torch.zeros(slots, self.D, conv_weight.shape[1] - 1, device=dev)
        self.scan_state = torch.zeros(slots, self.D, self.N, device=dev)

    def prompt(self, u, slots, lengths=None, *, resume=False, adapters: Adapters | None = None, index=None):
        """u (B, C, length) -> (B, C, length).  slots, lengths (B,) int32; the sequences start anew, or
        with resume=True from their slots' states.  index (B,) int32: each request's adapter."""
        if u.dim() != 3 or u.shape[1:] != (self.C, self.length):
            raise ValueError(f"input shape {tuple(u.shape)} is not (B, {self.C}, {self.length})")
        a = adapters or Adapters()
        _fits(a.out_proj, u, u.shape[0], self.D, self.C, index)

        def project(name, x):
            return self._prompt[name].forward(x.contiguous().unsqueeze(2)).squeeze(2)

        xz = _adapt(a.in_proj, u, project("in_proj", u), index)
        v = causal_conv(xz[:, :self.D], self.conv_weight, self.conv_bias, lengths=lengths, slots=slots,
                        initial_state=self.conv_state if resume else None, final_state=self.conv_state)
        p = project("x_proj", v)
        b, c = (p[:, self.R + k * self.N:self.R + (k + 1) * self.N].unsqueeze(1) for k in range(2))
        y = selective_scan(v, project("dt_proj", p[:, :self.R]), self.A, b, c, D=self.skip, z=xz[:, self.D:],
                           dt_bias=self.dt_bias, lengths=lengths, slots=slots,
                           initial_state=self.scan_state if resume else None, final_state=self.scan_state)
        return _adapt(a.out_proj, y, project("out_proj", y), index)

    def step(self, u, slots, *, adapters: Adapters | None = None, index=None):
        """The next position of each sequence: u (B, C) -> (B, C)."""
        if u.dim() != 2 or u.shape[1] != self.C:
            raise ValueError(f"input shape {tuple(u.shape)} is not (B, {self.C})")
        a = adapters or Adapters()
        _fits(a.out_proj, u, u.shape[0], self.D, self.C, index)

        def project(name, x):
            return self._token[name].forward(x.contiguous()[:, :, None, None])[:, :, :, 0]

        xz = _adapt(a.in_proj, u.unsqueeze(2), project("in_proj", u), index)[:, :, 0]
        v = causal_conv_step(xz[:, :self.D], self.conv_state, self.conv_weight, self.conv_bias, slots=slots)
        p = project("x_proj", v)[:, :, 0]
        b, c = (p[:, self.R + k * self.N:self.R + (k + 1) * self.N].unsqueeze(1) for k in range(2))
        y = selective_scan_step(v, self.scan_state, project("dt_proj", p[:, :self.R])[:, :, 0], self.A, b, c, D=self.skip,
                                z=xz[:, self.D:], dt_bias=self.dt_bias, slots=slots)
        return _adapt(a.out_proj, y.unsqueeze(2), project("out_proj", y), index)[:, :, 0]
