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
# (device, stream handle) -> zeroed workspace of the attend calls on that stream;
# (device, stream handle, "shared") -> that of the ones with shared prefixes
_workspaces = {}
_outgrown = []  # smaller ones of before: a captured graph may still use them


def clear_workspaces():
    """Drop the attend calls' workspaces (after a TIMEOUT, which can leave their
    counters set; the next call makes a zeroed one).  Graphs captured with them
    must not be replayed any more."""
    _workspaces.clear()
    _outgrown.clear()


def _grow(index, st, size):
    """A zeroed workspace of at least ``size`` bytes for stream ``st``."""
    return _grow_for((index, st), index, size)


def _grow_shared(index, st, size):
    """The same for calls with shared prefixes, which leave other things in theirs.  Its size
    goes with the tokens: at least twice the last one, so that the smaller ones that are kept
    do not add up to more than it where a batch grows by degrees."""
    last = _workspaces.get((index, st, "shared"))
    return _grow_for((index, st, "shared"), index, size if last is None else max(size, 2 * last.numel()))


def _grow_for(key, index, size):
    if torch.cuda.is_current_stream_capturing():
        raise RuntimeError("the workspace of this stream is not large enough yet: make one ordinary call of "
                           "this size on the stream before capturing, or pass workspace=")
    if key in _workspaces:
        _outgrown.append(_workspaces[key])
    ws = torch.zeros((size + (1 << 20) - 1) >> 20 << 20, dtype=torch.uint8, device=torch.device("cuda", index))
    _workspaces[key] = ws
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
        lib.w12_kv_plan, lib.w12_kv_store, lib.w12_kv_read, lib.w12_kv_attend_workspace_size, lib.w12_kv_attend,
        lib.w12_kv_fork_workspace_size, lib.w12_kv_fork, lib.w12_kv_copy, lib.w12_kv_attend_shared_workspace_size, lib.w12_kv_attend_shared,
        lib.w12_beam_workspace_size, lib.w12_beam_select)), w12._check)
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
    ``max_new``: the most new tokens of a request, as far as is known.  ``prefix``
    (a KVPrefix): what groups of the requests share, which attend() then reads once for
    each group.  What a call does not use may be None."""

    _kinds = {"lens": _I32, "cu_new": _I32, "positions": _I32, "slots": _I64, "tree": _I32}

    def __init__(self, tables=None, lens=None, cu_new=None, positions=None, slots=None, max_new=1, tree=None,
                 prefix=None):
        self.tables, self.lens, self.cu_new = tables, lens, cu_new
        self.positions, self.slots = positions, slots
        self.max_new, self.tree, self.prefix = int(max_new), tree, prefix

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


class KVPrefix:
    """Groups of requests with a common prefix: group g has requests ``cu[g] : cu[g + 1]``
    (int32; together all requests), request b shares its first ``lens[b]`` (int32, whole pages,
    0: nothing, else the same in all of the group) tokens with its group; ``max_requests``: the
    most requests of a group, as far as is known.
    ``KVPages.fork`` fills ``lens``; for a prompt that was put in every request's table
    the caller does.  (With less than some 150 MB of keys and values, shared ones counted
    for each request, a step without a prefix is the shorter call, and so it is from some
    ten new tokens per request on, with an 8-bit cache some thirty.)
    A layer with a window takes a step without a prefix: a second KVStep of the same arrays."""

    def __init__(self, cu, lens, max_requests=1):
        _need(cu.is_cuda, "cu must be on a CUDA device")
        _ints(cu, _I32, "cu", cu.get_device())
        _ints(lens, _I32, "lens", cu.get_device())
        _need(cu.numel() >= 2, "cu must have an entry more than there are groups")
        self.cu, self.lens, self.max_requests = cu, lens, int(max_requests)

    @classmethod
    def create(cls, groups, members, device=None):
        """``groups`` groups of ``members`` requests each, which share nothing so far."""
        dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        return cls(torch.arange(groups + 1, dtype=_I32, device=dev) * members,
                   torch.zeros(groups * members, dtype=_I32, device=dev), members)


class KVCopies:
    """Pages to copy: the first ``rows[i]`` tokens (``rows`` None: all) of page ``src[i]`` to
    page ``dst[i]``; -1: none.  int32, as ``KVPages.fork`` writes them and ``KVCache.copy``
    takes them."""

    def __init__(self, src, dst, rows=None):
        _need(src.is_cuda, "src must be on a CUDA device")
        for name, t in (("src", src), ("dst", dst), ("rows", rows)):
            if t is not None:
                _ints(t, _I32, name, src.get_device())
                _need(t.numel() == src.numel(), "src, dst and rows must have as many entries")
        self.src, self.dst, self.rows = src, dst, rows

    @classmethod
    def empty(cls, requests, device=None):
        dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        none = lambda v: torch.full((requests,), v, dtype=_I32, device=dev)  # noqa: E731
        return cls(none(-1), none(-1), none(0))


class KVPages:
    """Page tables of ``requests`` requests and the ring of free pages.

    ``tables`` int32 [requests, max_blocks]; ``owned`` int32 [requests]: pages
    each request holds; ``ring`` int32: free page numbers, of which
    ``ring[i % len]`` for head <= i < tail are free; ``ring_state`` int64
    {head, tail}.  ``KVPages.create`` starts with every page free.  With ``shares`` (int32
    [num_pages]: the holders of each page less one, 0 of free ones) requests may share
    pages: ``fork``."""

    def __init__(self, tables, owned, ring, ring_state, page_size, shares=None):
        _need(tables.dtype is _I32 and tables.dim() == 2 and tables.stride(1) == 1 and tables.is_cuda,
              "tables must be an int32 CUDA tensor [requests, max_blocks] with contiguous rows")
        self._index = tables.get_device()
        _ints(owned, _I32, "owned", self._index)
        _ints(ring, _I32, "ring", self._index)
        _ints(ring_state, _I64, "ring_state", self._index)
        _need(owned.numel() == tables.shape[0] and ring.numel() >= 1 and ring_state.numel() == 2,
              "owned must have an entry per request, ring at least one and ring_state two")
        if shares is not None:
            _ints(shares, _I32, "shares", self._index)
            _need(ring.numel() >= shares.numel() >= 1, "ring must have as many entries as shares or more")
        self.tables, self.owned, self.ring, self.ring_state = tables, owned, ring, ring_state
        self.page_size, self.shares, self._ws, self._outgrown = int(page_size), shares, None, []

    @classmethod
    def create(cls, num_pages, page_size, requests, max_blocks, device=None, shared=False):
        dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        return cls(torch.full((requests, max_blocks), -1, dtype=_I32, device=dev),
                   torch.zeros(requests, dtype=_I32, device=dev),
                   torch.arange(num_pages, dtype=_I32, device=dev),
                   torch.tensor([0, num_pages], dtype=_I64, device=dev), page_size,
                   torch.zeros(num_pages, dtype=_I32, device=dev) if shared else None)

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
        requests), is reported by w12_check_status.  With ``shares`` there is no
        ``trim``: fork() takes back, for it knows who else holds a page."""
        if trim and self.shares is not None:
            raise ValueError("pages that requests share are taken back by fork(), not by trim")
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

    def fork(self, parents, lens, copies=None, prefix=None, lens_out=None, stream=None):
        """Request i goes on from request ``parents[i]`` (int32, -1: from none, it is empty
        then) as it was before the call, with the first ``lens[i]`` (int32) of its tokens.
        Full pages are shared; of requests that want the same partly filled page one keeps
        it and the others get pages of their own and an entry of ``copies`` (a KVCopies;
        None: a new one is made), which is returned: every layer's cache has to ``copy``
        it before the next store.  Pages that no request holds any more are free.
        ``lens_out`` (may be ``lens``) receives the tokens kept (0 where there is no parent),
        ``prefix.lens`` what the groups of ``prefix`` (a KVPrefix) share now."""
        if stream is not None or _current_device() != self._index:
            with _on(self._index, stream):
                return self.fork(parents, lens, copies, prefix, lens_out)
        if copies is None:
            copies = KVCopies.empty(self.tables.shape[0], self.tables.device)
        return _host.fork(self, self._index, parents, lens, copies, prefix, lens_out, self._ws, self._grow,
                          _current_stream(self._index))

    def _grow(self, index, st, size):
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("make one ordinary fork() of these pages before capturing one")
        if self._ws is not None:
            self._outgrown.append(self._ws)  # a captured graph may still use it
        self._ws = torch.zeros(size, dtype=torch.uint8, device=self.tables.device)
        return self._ws


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

    def copy(self, copies, others=(), stream=None):
        """Copy pages (``copies``: a KVCopies) inside this cache and, in the same launch,
        inside ``others``, caches of other layers that are laid out alike.  A page that is
        written to must not be another copy's."""
        if stream is not None or _current_device() != self._index:
            with _on(self._index, stream):
                return self.copy(copies, others)
        others = tuple(others)  # looked at twice: a generator has them once
        for c in others:
            _need(c._index == self._index, "the caches must be on one device")
        _host.copy(self._address, self._index, others, copies, _current_stream(self._index))

    def attend(self, q, step, scale=None, window=0, out=None, lse=None, workspace=None, stream=None):
        """Attention of the step's new tokens over their requests' cached ones
        (their own included).  ``scale`` defaults to head_dim ** -0.5; ``window``
        > 0: a token sees only that many last tokens, itself included (in a tree,
        by step.positions; where those are None, by the tokens' order).  ``lse``
        (fp32 [tokens, heads]) receives the log of the softmax sums.  Calls on one
        stream (of several threads too) share a workspace; ``workspace`` (uint8, zero-filled before its
        first use) takes its place, as a captured graph needs that is replayed
        beside other calls.  With ``step.prefix`` (no window then) the keys that a
        group of requests shares are read once for all of them; such calls have a workspace of
        their own, of 2 * tokens * heads * (4 * head_dim + 24) bytes (8192 tokens of 48 heads of
        128: 420 MB) and up to 80 MB more; it is kept for the stream and grows to twice its size
        or more."""
        if stream is not None or _current_device() != self._index:
            with _on(self._index, stream):
                return self.attend(q, step, scale, window, out, lse, workspace)
        st = _current_stream(self._index)
        grow = None
        if workspace is None:
            shared = getattr(step, "prefix", None) is not None
            workspace = _workspaces.get((self._index, st, "shared") if shared else (self._index, st))
            grow = _grow_shared if shared else _grow
        return _host.attend(self._address, self._index, q, step, self._scale if scale is None else scale, window, out,
                            lse, workspace, grow, st)
