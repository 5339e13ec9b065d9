"""A pruned attention layer for serving, and a stack of pruned layers that attend or scan.

    q k v = qkv_proj u  (+ the request's adapter)     pruned 1x1 layer, ((H + 2 G) D, C)
    q, k  = rotary positions; k, v into the cache
    y     = attention(q, cache)
    out   = out_proj y  (+ the request's adapter)     pruned 1x1 layer, (C, H D)

As in ssm.py a sequence (B, C, L) is a batch of feature maps with H = 1 and W = L: one set of handles
for prompts of `length` positions (shorter ones are padded on the right and say so in `lengths`), one for
single positions.  Keys and values stay in the pages of a PagePool (cache.py), in its type; a call takes
the table and the past that the pool's extend() gave for it.  Everything runs on the current stream.
"""
from __future__ import annotations

import numpy as np
import torch

from . import Handle
from .attention import (cache_append, cache_append_step, paged_attention, paged_attention_step, paged_attention_workspace, residual_norm,
                        residual_norm_step)
from .cache import PagePool
from .ssm import Adapters, StateSpaceLayer, _adapt, _fits


class AttentionLayer:
    """qkv_proj ((H + 2 G) D, C), out_proj (C, H D): pruned float32 weights on the host (zeros are not stored), G and D the
    pool's heads and dims.  layer: which of the pool's layers this one is.  freqs, axes, interleaved: rotary positions as in cache_append
    (freqs None: none); scale, cap, window, slopes: as in paged_attention.  What the operators would refuse of these is refused
    here.  A call that is refused has written, at most, positions of the cache past the sequences' `past`, which nobody sees."""

    def __init__(self, qkv_proj, out_proj, pool: PagePool, layer: int, *, length: int, freqs=None, axes=None, interleaved: bool = False,
                 scale: float | None = None, cap: float = 0.0, window: int = 0, slopes=None):
        self.G, self.D = pool.heads, pool.dims
        heads, rest = divmod(qkv_proj.shape[0], self.D)
        self.H, self.C = heads - 2 * self.G, qkv_proj.shape[1]
        if rest or self.H < 1 or self.H % self.G:
            raise ValueError(f"qkv_proj's {qkv_proj.shape[0]} rows are not (H + 2 * {self.G}) * {self.D} with H a multiple of {self.G}")
        if tuple(out_proj.shape) != (self.C, self.H * self.D):
            raise ValueError(f"out_proj shape {tuple(out_proj.shape)} is not {(self.C, self.H * self.D)}")
        if not 0 <= layer < pool.layers:
            raise ValueError(f"layer {layer} of a pool of {pool.layers}")
        self.length = length
        self.pool, self.k_pages, self.v_pages = pool, pool.k_pages(layer), pool.v_pages(layer)
        weights = dict(qkv_proj=qkv_proj, out_proj=out_proj)
        self._prompt, self._token = ({n: Handle.from_dense(np.ascontiguousarray(w, np.float32)[:, :, None, None], 1, W, 1, 0)
                                      for n, w in weights.items()} for W in (length, 1))
        self._rotary = dict(freqs=None if freqs is None else freqs.detach(), axes=axes, interleaved=interleaved)
        self._attend = dict(scale=scale, cap=cap, window=window, slopes=None if slopes is None else slopes.detach())
        self._fit = None  # sizes of a call that the operators take
        if self.k_pages.is_cuda:  # one idle sequence: everything is looked at, nothing of the cache is written
            table, past = (torch.full(s, -1, dtype=torch.int32, device=self.k_pages.device) for s in ((1, 1), (1,)))
            q, k = (self.k_pages.new_zeros(1, n * self.D) for n in (self.H, self.G))
            cache_append_step(k, k, self.k_pages, self.v_pages, table, past, q=q, **self._rotary)
            paged_attention_step(q, self.k_pages, self.v_pages, table, past, **self._attend)

    def _refuse(self, u, L, table, past, lengths, positions, prefix):
        """Refuses what the layer's operators would refuse of a call's arguments for L positions, before a stack has written any
        state: the same calls over no positions, and what such calls do not look at."""
        B, H, G, D = u.shape[0], self.H, self.G, self.D
        none = positions
        if isinstance(positions, torch.Tensor):
            if positions.dim() != 3 or positions.shape[2] != L or (L > 1 and positions.stride(2) != 1):
                raise ValueError(f"positions must be (B, axes, {L}) with contiguous positions: {tuple(positions.shape)}, strides {positions.stride()}")
            none = positions[:, :, :0]
        k = u.new_empty(B, G * D, 0)
        cache_append(k, k, self.k_pages, self.v_pages, table, past, positions=none, lengths=lengths, **self._rotary)
        paged_attention(u.new_empty(B, H * D, 0, dtype=self.k_pages.dtype), self.k_pages, self.v_pages, table, past, lengths=lengths,
                        prefix=prefix, **self._attend)
        sizes = B, L, table.shape[1]
        if sizes != self._fit:  # (the last that did)
            paged_attention_workspace(B, H, L, self.k_pages, table.shape[1])
            heads = H + 2 * G
            if B * L * heads * D >= 2 ** 32 if L < 16 else B * (-(-L // 64) + 1) * (-(-heads // 8) + 1) >= 2 ** 24:
                raise ValueError(f"{B} sequences of {L} positions are more than one cache_append takes")
            self._fit = sizes

    def _parts(self, qkv):
        q, k = self.H * self.D, (self.H + self.G) * self.D
        return qkv[:, :q], qkv[:, q:k], qkv[:, k:]

    def prompt(self, u, table, past, lengths=None, *, positions=None, prefix=None, adapters: Adapters | None = None, index=None):
        """u (B, C, length) -> (B, C, length): the positions past .. past + lengths - 1 of each sequence.  positions (B, n,
        length): their coordinates; prefix (B,): as in paged_attention; index (B,) int32: each request's adapter."""
        if u.dim() != 3 or u.shape[1:] != (self.C, self.length):
            raise ValueError(f"input shape {tuple(u.shape)} is not (B, {self.C}, {self.length})")
        a = adapters or Adapters()
        _fits(a.out_proj, u, u.shape[0], self.H * self.D, self.C, index)

        def project(name, x):
            return self._prompt[name].forward(x.contiguous().unsqueeze(2)).squeeze(2)

        q, k, v = self._parts(_adapt(a.in_proj, u, project("qkv_proj", u), index))
        q = cache_append(k, v, self.k_pages, self.v_pages, table, past, q=q, positions=positions, lengths=lengths, **self._rotary)
        y = paged_attention(q, self.k_pages, self.v_pages, table, past, lengths=lengths, prefix=prefix,
                            out=u.new_empty(q.shape, dtype=torch.float32), **self._attend)
        return _adapt(a.out_proj, y, project("out_proj", y), index)

    def step(self, u, table, past, *, positions=None, prefix=None, adapters: Adapters | None = None, index=None):
        """The next position of each sequence: u (B, C) -> (B, C)."""
        if u.dim() != 2 or u.shape[1] != self.C:
            raise ValueError(f"input shape {tuple(u.shape)} is not (B, {self.C})")
        a = adapters or Adapters()
        _fits(a.out_proj, u, u.shape[0], self.H * self.D, self.C, index)

        def project(name, x):
            return self._token[name].forward(x.contiguous()[:, :, None, None])[:, :, :, 0]

        q, k, v = self._parts(_adapt(a.in_proj, u.unsqueeze(2), project("qkv_proj", u), index)[:, :, 0])
        q = cache_append_step(k, v, self.k_pages, self.v_pages, table, past, q=q, positions=positions, **self._rotary)
        y = paged_attention_step(q, self.k_pages, self.v_pages, table, past, prefix=prefix,
                                 out=u.new_empty(q.shape, dtype=torch.float32), **self._attend)
        return _adapt(a.out_proj, y.unsqueeze(2), project("out_proj", y), index)[:, :, 0]


class HybridStack:
    """Layers one after another around a residual stream, attending or scanning, with a norm before each and one at the end:

        r_0 = x,  y_i = layer_i(norm(r_i) * weight[i]),  r_{i+1} = r_i + scale * post_i(y_i),  out = norm(r_n) * weight[n]

    layers: AttentionLayer and StateSpaceLayer, of the same channels and prompt length.  weights (n + 1, C) and post_weights (n, C; None: y
    as it is): float32 on the GPU.  A layer's sum and the next one's norm are one launch.  A call whose arguments are refused leaves
    the scanning layers' states as they are.  The stack passes its layers no adapters."""

    def __init__(self, layers, weights, *, post_weights=None, scale: float = 1.0, eps: float = 1e-6):
        self.layers = list(layers)
        n, C = len(self.layers), self.layers[0].C
        if any(x.C != C or x.length != self.layers[0].length for x in self.layers):
            raise ValueError("the layers differ in channels or prompt length")
        for name, t, rows in (("weights", weights, n + 1), ("post_weights", post_weights, n)):
            if t is not None and (tuple(t.shape) != (rows, C) or t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous float32 tensor of shape {(rows, C)} on the GPU")
        self.C, self.length, self.scale, self.eps = C, self.layers[0].length, scale, eps
        self.weights = weights.detach()
        self.post_weights = None if post_weights is None else post_weights.detach()
        for x in self.layers:
            if (x.scan_state if isinstance(x, StateSpaceLayer) else x.k_pages).device != weights.device:
                raise ValueError("the layers and the weights are on different GPUs")
        one = self.weights.new_zeros(1, C)  # scale, eps and the weights' device are looked at before any layer runs
        residual_norm_step(one, one.clone(), weight=self.weights[0], post_weight=None if self.post_weights is None else self.post_weights[0],
                           scale=scale, eps=eps)
        # the first layer that writes states, and the attending ones after it
        self._first = next((i for i, x in enumerate(self.layers) if isinstance(x, StateSpaceLayer)), n)
        self._late = [x for x in self.layers[self._first:] if isinstance(x, AttentionLayer)]

    def _run(self, x, norm, call, L, *args):
        _, h = norm(x, weight=self.weights[0], eps=self.eps)
        r = x
        for i, layer in enumerate(self.layers):
            if i == self._first:
                for late in self._late:
                    late._refuse(h, L, *args)
            y = call(layer, h)
            r, h = norm(r, y, weight=self.weights[i + 1], post_weight=None if self.post_weights is None else self.post_weights[i],
                        scale=self.scale, eps=self.eps, sum=None if r is x else r)  # the caller's x stays
        return h

    def prompt(self, x, slots, table, past, lengths=None, *, resume: bool = False, positions=None, prefix=None):
        """x (B, C, length) -> (B, C, length).  slots (B,) int32: of the scanning layers' states (which start anew, or with resume=True
        from there); table, past: of the attending layers' cache; lengths (B,) int32."""
        def call(layer, h):
            if isinstance(layer, StateSpaceLayer):
                return layer.prompt(h, slots, lengths, resume=resume)
            return layer.prompt(h, table, past, lengths, positions=positions, prefix=prefix)

        return self._run(x, residual_norm, call, self.length, table, past, lengths, positions, prefix)

    def step(self, x, slots, table, past, *, positions=None, prefix=None):
        """The next position of each sequence: x (B, C) -> (B, C)."""
        def call(layer, h):
            if isinstance(layer, StateSpaceLayer):
                return layer.step(h, slots)
            return layer.step(h, table, past, positions=positions, prefix=prefix)

        return self._run(x, residual_norm_step, call, 1, table, past, None, positions, prefix)
