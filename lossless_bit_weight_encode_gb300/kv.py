"""Paged key-value cache holders over the C ABI's w12_kv_* calls.

``KVPages`` keeps which page belongs to which request (one for all layers),
``KVStep`` is one step's tokens (``KVPages.plan`` fills it), ``KVCache`` is one
layer's keys and values.  A decoder layer's step, with q, k, v from a W12Group::

    pages.plan(lens, new_lens, step)              # once per step
    q = cache.store(q, k, v, step, rope=table)    # norm, rotation, cache write
    y = cache.attend(q, step)                     # input of the output product

Nothing here reads device memory on the host; a call whose buffers are all given
(``out=``, ``lse=``) allocates nothing, so that a step can be captured in a CUDA
graph after one ordinary call on the same stream.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os

import torch

from . import build, w12

_BF16, _I32, _I64, _F32 = torch.bfloat16, torch.int32, torch.int64, torch.float32
_workspaces = {}  # (device, stream handle) -> zeroed workspace of the attend calls on that stream
_outgrown = []  # smaller ones of before: a captured graph may still use them


def clear_workspaces():
    """Drop the attend calls' workspaces (after a TIMEOUT, which can leave their
    counters set; the next call makes a zeroed one).  Graphs captured with them
    must not be replayed any more."""
    _workspaces.clear()
    _outgrown.clear()


def _grow(index, st, size):
    """A zeroed workspace of at least ``size`` bytes for stream ``st``."""
    if torch.cuda.is_current_stream_capturing():
        raise RuntimeError("the workspace of this stream is not large enough yet: make one ordinary call of "
                           "this size on the stream before capturing, or pass workspace=")
    if (index, st) in _workspaces:
        _outgrown.append(_workspaces[index, st])
    ws = torch.zeros((size + (1 << 20) - 1) >> 20 << 20, dtype=torch.uint8, device=torch.device("cuda", index))
    _workspaces[index, st] = ws
    return ws


def _load_host():
    """The module that takes the calls from tensors to the C ABI."""
    path = build.KV_HOST_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"the paged cache's host module is not built ({path} missing): run "
                           "__graft_entry__.build()")
    loader = importlib.machinery.ExtensionFileLoader("kv_host", path)
    host = importlib.util.module_from_spec(importlib.util.spec_from_file_location("kv_host", loader=loader))
    loader.exec_module(host)
    lib = w12.lib()
    host.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
        lib.w12_kv_plan, lib.w12_kv_store, lib.w12_kv_read, lib.w12_kv_attend_workspace_size, lib.w12_kv_attend)),
        w12._check)
    return host


class _NotLoaded:
    """Stands for the module until the first call: the package is imported before the build too."""

    def __getattr__(self, name):
        global _host
        _host = _load_host()
        return getattr(_host, name)


_host = _NotLoaded()

_current_device = torch._C._cuda_getDevice
# handle of a device's current stream, without the stream object around it
_current_stream = torch._C._cuda_getCurrentRawStream


class _on:
    """The device and stream of a call that is not for the current ones: outputs
    are allocated for that stream.  ``stream`` as in w12.py: None (the current
    one), a torch stream or a handle."""

    def __init__(self, index, stream):
        self.index, self.stream, self.guards = index, stream, ()

    def __enter__(self):
        self.guards = (torch.cuda.device(self.index),)
        s = self.stream
        if s is not None:
            if isinstance(s, int):
                s = torch.cuda.ExternalStream(s, device=self.index) if s else torch.cuda.default_stream(self.index)
            self.guards += (torch.cuda.stream(s),)
        for g in self.guards:
            g.__enter__()

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)
        return False


def _need(ok, text):
    if not ok:
        raise ValueError(text)


def _ints(t, dtype, name, index):
    """Pointer of a contiguous 1-D integer tensor on CUDA device `index`."""
    if t.dtype is not dtype or t.dim() != 1 or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 1-D {dtype} tensor on CUDA device {index}")
    return t.data_ptr()


class KVStep:
    """One step of a batch: for request b, ``lens[b]`` cached tokens and the new
    tokens ``cu_new[b] : cu_new[b + 1]``; for every new token its ``position``
    and cache slot (-1: none).  ``tables`` [requests, max_blocks] holds the
    requests' pages.  ``tree`` (int32, bit j of a token's mask: it attends to new
    token j of its request) replaces the causal order among new tokens.  ``plan``
    numbers a request's new tokens one after the other; for a tree, write cached
    length + depth over ``positions`` before the store (rotation) and the attention
    (windows).
    ``max_new``: the most new tokens of a request, as far as is known.  What a
    call does not use may be None."""

    _kinds = {"lens": _I32, "cu_new": _I32, "positions": _I32, "slots": _I64, "tree": _I32}

    def __init__(self, tables=None, lens=None, cu_new=None, positions=None, slots=None, max_new=1, tree=None):
        self.tables, self.lens, self.cu_new = tables, lens, cu_new
        self.positions, self.slots = positions, slots
        self.max_new, self.tree = int(max_new), tree

    def __setattr__(self, name, value):
        # checked here, once, and not in every call of every layer
        if value is not None and name in self._kinds:
            _ints(value, self._kinds[name], name, self._one_device(value))
        elif value is not None and name == "tables":
            self._one_device(value)
            _need(value.dtype is _I32 and value.dim() == 2 and value.stride(1) == 1,
                  "tables must be an int32 CUDA tensor [requests, max_blocks] with contiguous rows")
        else:
            return object.__setattr__(self, name, value)
        object.__setattr__(self, "device", value.get_device())  # of its first array, and then of all
        object.__setattr__(self, name, value)

    def _one_device(self, t):
        _need(t.is_cuda and t.get_device() == self.__dict__.get("device", t.get_device()),
              "a step's arrays must be on one CUDA device")
        return t.get_device()


class KVPages:
    """Page tables of ``requests`` requests and the ring of free pages.

    ``tables`` int32 [requests, max_blocks]; ``owned`` int32 [requests]: pages
    each request holds; ``ring`` int32: free page numbers, of which
    ``ring[i % len]`` for head <= i < tail are free; ``ring_state`` int64
    {head, tail}.  ``KVPages.create`` starts with every page free."""

    def __init__(self, tables, owned, ring, ring_state, page_size):
        _need(tables.dtype is _I32 and tables.dim() == 2 and tables.stride(1) == 1 and tables.is_cuda,
              "tables must be an int32 CUDA tensor [requests, max_blocks] with contiguous rows")
        self._index = tables.get_device()
        _ints(owned, _I32, "owned", self._index)
        _ints(ring, _I32, "ring", self._index)
        _ints(ring_state, _I64, "ring_state", self._index)
        _need(owned.numel() == tables.shape[0] and ring.numel() >= 1 and ring_state.numel() == 2,
              "owned must have an entry per request, ring at least one and ring_state two")
        self.tables, self.owned, self.ring, self.ring_state = tables, owned, ring, ring_state
        self.page_size = int(page_size)

    @classmethod
    def create(cls, num_pages, page_size, requests, max_blocks, device=None):
        dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        return cls(torch.full((requests, max_blocks), -1, dtype=_I32, device=dev),
                   torch.zeros(requests, dtype=_I32, device=dev),
                   torch.arange(num_pages, dtype=_I32, device=dev),
                   torch.tensor([0, num_pages], dtype=_I64, device=dev), page_size)

    def step(self, tokens, max_new=1, tree=None):
        """A KVStep with buffers for up to ``tokens`` new tokens, for plan()."""
        dev = self.tables.device
        return KVStep(self.tables, None, torch.zeros(self.tables.shape[0] + 1, dtype=_I32, device=dev),
                      torch.zeros(tokens, dtype=_I32, device=dev),
                      torch.full((tokens,), -1, dtype=_I64, device=dev), max_new, tree)

    def plan(self, lens, new_lens, step, trim=False, owned_out=None, ring_state_out=None, stream=None):
        """Give the requests pages for ``new_lens`` (int32) more tokens behind
        ``lens`` (int32) cached ones and fill ``step``; ``trim`` takes back pages
        they no longer need.  ``owned`` and ``ring_state`` are updated in place
        unless outputs are given.  ``step`` refers to ``lens``, which must stay as
        it is until the step's attend calls have run.  A ring that runs out, or
        has no room for pages that trim gives back (those stay with their
        requests), is reported by w12_check_status."""
        if stream is not None or _current_device() != self._index:
            with _on(self._index, stream):
                return self.plan(lens, new_lens, step, trim, owned_out, ring_state_out)
        _host.plan(self, self._index, lens, new_lens, step, trim, owned_out, ring_state_out,
                   _current_stream(self._index))
        if step.lens is not lens:
            step.lens = lens
        if step.tables is not self.tables:
            step.tables = self.tables
        return step


class KVCache:
    """One layer's keys and values: ``k``, ``v`` [num_pages, kv_heads, page_size,
    head_dim] (any strides whose heads are contiguous rows of head_dim; a cache
    laid out as [page, token, head] is passed as its permuted view), BF16, or int8
    with ``scales`` fp32 [num_pages, kv_heads, page_size, 2] (key, value)."""

    def __init__(self, k, v, scales=None):
        _need(k.dim() == 4 and k.shape == v.shape and k.stride() == v.stride() and k.dtype == v.dtype,
              "k and v must be alike, [num_pages, kv_heads, page_size, head_dim]")
        _need(k.is_cuda and v.device == k.device and k.stride(3) == 1,
              "k and v must be CUDA tensors with contiguous rows")
        _need(k.dtype in (_BF16, torch.int8), "k and v must be BF16 or int8")
        _need((scales is None) == (k.dtype == _BF16), "an int8 cache needs scales, a BF16 cache has none")
        pages, heads, page, dim = k.shape
        if scales is not None:
            _need(scales.shape == (pages, heads, page, 2) and scales.dtype == _F32 and scales.is_contiguous()
                  and scales.device == k.device, "scales must be contiguous fp32 [num_pages, kv_heads, page_size, 2]")
        self.k, self.v, self.scales, self.device = k, v, scales, k.device
        self._index = k.get_device()
        self.kv_heads, self.page_size, self.head_dim = heads, page, dim
        # a dimension of one element has no stride that matters
        stride = [s if n > 1 else dim for n, s in zip(k.shape, k.stride())]
        self._c = w12.w12_kv_cache(k.data_ptr(), v.data_ptr(), None if scales is None else scales.data_ptr(), pages,
                                   stride[0], stride[1], stride[2], page, heads, dim,
                                   w12.KV_BF16 if scales is None else w12.KV_Q8)
        self._address = ctypes.addressof(self._c)
        self._scale = dim ** -0.5

    @classmethod
    def empty(cls, num_pages, page_size, kv_heads, head_dim, dtype="bf16", device=None):
        """A cache of uninitialised pages; dtype "bf16" or "q8"."""
        _need(dtype in ("bf16", "q8"), 'dtype must be "bf16" or "q8"')
        dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        shape = (num_pages, kv_heads, page_size, head_dim)
        t = _BF16 if dtype == "bf16" else torch.int8
        return cls(torch.empty(shape, dtype=t, device=dev), torch.empty(shape, dtype=t, device=dev),
                   None if dtype == "bf16" else torch.empty(shape[:3] + (2,), dtype=_F32, device=dev))

    def store(self, q, k, v, step, q_norm=None, k_norm=None, eps=1e-6, rope=None, interleaved=False, out=None,
              stream=None):
        """Norm (``q_norm``, ``k_norm``: BF16 [head_dim]) and rotation (``rope``:
        fp32 [positions, rot], cosines then sines) of q and k, k and v into the
        cache at step.slots.  Returns the new q, [tokens, heads, head_dim] (of
        ``out``, which may be q); q None: only k and v."""
        if stream is not None or _current_device() != self._index:
            with _on(self._index, stream):
                return self.store(q, k, v, step, q_norm, k_norm, eps, rope, interleaved, out)
        return _host.store(self._address, self._index, q, k, v, step, q_norm, k_norm, eps, rope, interleaved, out,
                           _current_stream(self._index))

    def read(self, slots, out=None, stream=None):
        """(k, v) BF16 [tokens, kv_heads, head_dim] of the cached rows at ``slots``
        (int64; zeros for -1).  ``out``: a pair to write to."""
        if stream is not None or _current_device() != self._index:
            with _on(self._index, stream):
                return self.read(slots, out)
        return _host.read(self._address, self._index, slots, out, _current_stream(self._index))

    def attend(self, q, step, scale=None, window=0, out=None, lse=None, workspace=None, stream=None):
        """Attention of the step's new tokens over their requests' cached ones
        (their own included).  ``scale`` defaults to head_dim ** -0.5; ``window``
        > 0: a token sees only that many last tokens, itself included (in a tree,
        by step.positions; where those are None, by the tokens' order).  ``lse``
        (fp32 [tokens, heads]) receives the log of the softmax sums.  Calls on one
        stream (of several threads too) share a workspace; ``workspace`` (uint8, zero-filled before its
        first use) takes its place, as a captured graph needs that is replayed
        beside other calls."""
        if stream is not None or _current_device() != self._index:
            with _on(self._index, stream):
                return self.attend(q, step, scale, window, out, lse, workspace)
        st = _current_stream(self._index)
        own = workspace is None
        return _host.attend(self._address, self._index, q, step, self._scale if scale is None else scale, window, out,
                            lse, _workspaces.get((self._index, st)) if own else workspace, _grow if own else None, st)
