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


import torch

from . import w12

_BF16, _I32, _I64, _F32 = torch.bfloat16, torch.int32, torch.int64, torch.float32
_workspaces = {}  # (device, stream handle) -> zeroed workspace of the attend calls on that stream




def clear_workspaces():
    """Drop the attend calls' workspaces (after a TIMEOUT, which can leave their
    counters set; the next call makes a zeroed one)."""
    _workspaces.clear()


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
        return _current_stream(self.index)

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


def _rows(t, dim, name, index, heads=None):
    """(pointer, token stride, tokens, heads) of [T, heads * dim] or
    [T, heads, dim] BF16 rows whose heads lie one after the other."""
    shape, stride = t.shape, t.stride()
    n = 0
    if len(shape) == 2:
        if stride[1] == 1 and shape[1] % dim == 0:
            n = shape[1] // dim
    elif len(shape) == 3 and shape[2] == dim and stride[2] == 1 and (stride[1] == dim or shape[1] == 1):
        n = shape[1]
    if n < 1 or t.dtype is not _BF16 or t.get_device() != index or (heads is not None and n != heads):
        raise ValueError(f"{name} must be BF16 [tokens, {heads or 'heads'} * {dim}] on CUDA device {index} with "
                         "contiguous heads")
    # one row has no stride that matters
    return t.data_ptr(), stride[0] if shape[0] > 1 else n * dim, shape[0], n


class KVStep:
    """One step of a batch: for request b, ``lens[b]`` cached tokens and the new
    tokens ``cu_new[b] : cu_new[b + 1]``; for every new token its ``position``
    and cache slot (-1: none).  ``tables`` [requests, max_blocks] holds the
    requests' pages.  ``tree`` (int32, bit j of a token's mask: it attends to new
    token j of its request) replaces the causal order among new tokens.
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
            _need(value.dtype is _I32 and value.dim() == 2 and value.stride(1) == 1,
                  "tables must be an int32 CUDA tensor [requests, max_blocks] with contiguous rows")
            self._one_device(value)
        object.__setattr__(self, name, value)

    def _one_device(self, t):
        _need(t.is_cuda and t.get_device() == self.__dict__.setdefault("device", t.get_device()),
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
        it is until the step's attend calls have run.  A ring that runs out is
        reported by w12_check_status."""
        if stream is None and _current_device() == self._index:
            return self._plan(lens, new_lens, step, trim, owned_out, ring_state_out, _current_stream(self._index))
        with _on(self._index, stream) as st:
            return self._plan(lens, new_lens, step, trim, owned_out, ring_state_out, st)

    def _plan(self, lens, new_lens, step, trim, owned_out, ring_state_out, st):
        tables, index = self.tables, self._index
        n, blocks = tables.shape
        if step.lens is not lens:
            step.lens = lens
        if step.tables is not tables:
            step.tables = tables
        cu, positions, slots, owned, state = step.cu_new, step.positions, step.slots, self.owned, self.ring_state
        tokens = slots.numel()
        if (step.device != index or lens.numel() != n or new_lens.numel() != n or cu.numel() != n + 1
                or positions.numel() != tokens):
            raise ValueError("lens, new_lens and step must be on the tables' device, with an entry per request")
        owned_p, state_p = owned.data_ptr(), state.data_ptr()
        owned_o, state_o = owned_p, state_p
        if owned_out is not None:
            owned_o = _ints(owned_out, _I32, "owned_out", index)
            _need(owned_out.numel() == n, "owned_out must have an entry per request")
        if ring_state_out is not None:
            state_o = _ints(ring_state_out, _I64, "ring_state_out", index)
            _need(ring_state_out.numel() == 2, "ring_state_out must have two entries")
        w12.w12_kv_plan(w12.w12_kv_plan_args(
            lens.data_ptr(), _ints(new_lens, _I32, "new_lens", index), owned_p, owned_o, tables.data_ptr(),
            tables.stride(0) if n > 1 else blocks, self.ring.data_ptr(), state_p, state_o, cu.data_ptr(),
            positions.data_ptr(), slots.data_ptr(), n, blocks, self.page_size, self.ring.numel(), tokens,
            1 if trim else 0), st)
        return step


class KVCache:
    """One layer's keys and values: ``k``, ``v`` [num_pages, kv_heads, page_size,
    head_dim] (any strides whose heads are contiguous rows of head_dim; a cache
    laid out as [page, token, head] is passed as its permuted view), BF16, or int8
    with ``scales`` fp32 [num_pages, kv_heads, page_size, 2] (key, value)."""

    def __init__(self, k, v, scales=None):
        _need(k.dim() == 4 and k.shape == v.shape and k.stride() == v.stride() and k.dtype == v.dtype,
              "k and v must be alike, [num_pages, kv_heads, page_size, head_dim]")
        _need(k.is_cuda and v.device == k.device and k.stride(3) == 1, "k and v must be CUDA tensors with contiguous rows")
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
        self._scale = dim ** -0.5
        self._ws_bytes = {}

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
        if stream is None and _current_device() == self._index:
            return self._store(q, k, v, step, q_norm, k_norm, eps, rope, interleaved, out, _current_stream(self._index))
        with _on(self._index, stream) as st:
            return self._store(q, k, v, step, q_norm, k_norm, eps, rope, interleaved, out, st)

    def _store(self, q, k, v, step, q_norm, k_norm, eps, rope, interleaved, out, st):
        dim, index = self.head_dim, self._index
        kp, ks, tokens, _ = _rows(k, dim, "k", index, self.kv_heads)
        vp, vs, nv, _ = _rows(v, dim, "v", index, self.kv_heads)
        slots = step.slots
        if slots is None or step.device != index or nv != tokens or slots.numel() != tokens:
            raise ValueError("k, v and step.slots must have as many tokens, on the cache's device")
        qp = qs = op = os_ = heads = rot = rows = rp = pp = 0
        if rope is not None:
            positions = step.positions
            if (rope.dtype is not _F32 or rope.dim() != 2 or not rope.is_contiguous() or rope.get_device() != index
                    or positions is None or positions.numel() != tokens):
                raise ValueError("rope must be a contiguous fp32 tensor [positions, rot] on the cache's device and "
                                 "step.positions have as many tokens as k")
            rows, rot = rope.shape
            rp, pp = rope.data_ptr(), positions.data_ptr()
        wq = self._weight(q_norm, "q_norm") if q_norm is not None else 0
        wk = self._weight(k_norm, "k_norm") if k_norm is not None else 0
        if q is not None:
            qp, qs, nq, heads = _rows(q, dim, "q", index)
            if out is None:
                out = torch.empty(q.shape, dtype=_BF16, device=self.device)
            op, os_, no, _ = _rows(out, dim, "out", index, heads)
            if nq != tokens or no != tokens:
                raise ValueError("q, out and k must have as many tokens")
        if tokens:
            w12.w12_kv_store(self._c, w12.w12_kv_store_args(qp, kp, vp, op, qs, ks, vs, os_, wq, wk, rp, pp,
                                                            slots.data_ptr(), rows, tokens, heads, rot,
                                                            1 if interleaved else 0, eps), st)
        return None if q is None else out if out.dim() == 3 else out.view(tokens, heads, dim)

    def _weight(self, w, name):
        if w.dtype is not _BF16 or w.dim() != 1 or w.numel() != self.head_dim or not w.is_contiguous() \
                or w.get_device() != self._index:
            raise ValueError(f"{name} must be contiguous BF16 [{self.head_dim}] on CUDA device {self._index}")
        return w.data_ptr()

    def read(self, slots, out=None, stream=None):
        """(k, v) BF16 [tokens, kv_heads, head_dim] of the cached rows at ``slots``
        (int64; zeros for -1).  ``out``: a pair to write to."""
        if stream is None and _current_device() == self._index:
            return self._read(slots, out, _current_stream(self._index))
        with _on(self._index, stream) as st:
            return self._read(slots, out, st)

    def _read(self, slots, out, st):
        sp, tokens = _ints(slots, _I64, "slots", self._index), slots.numel()
        shape = (tokens, self.kv_heads, self.head_dim)
        if out is None:
            k = torch.empty(shape, dtype=_BF16, device=self.device)
            v = torch.empty(shape, dtype=_BF16, device=self.device)
        else:
            k, v = out
            for t in out:
                _need(t.shape == shape and t.dtype is _BF16 and t.is_contiguous() and t.get_device() == self._index,
                      "out must be two contiguous BF16 tensors [tokens, kv_heads, head_dim]")
        if tokens:
            w12.w12_kv_read(self._c, sp, tokens, k.data_ptr(), v.data_ptr(), st)
        return k, v

    def workspace(self, args, key, st):
        """The zeroed workspace of the attend calls on stream ``st`` (shared by
        all caches), large enough for ``args``; ``key``: what its size depends on."""
        size = self._ws_bytes.get(key)
        if size is None:
            size = self._ws_bytes[key] = w12.w12_kv_attend_workspace_size(self._c, args)
        ws = _workspaces.get((self._index, st))
        if ws is None or ws.numel() < size:
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError("the workspace of this stream is not large enough yet: make one ordinary call of "
                                   "this size on the stream before capturing, or pass workspace=")
            ws = torch.zeros((size + (1 << 20) - 1) >> 20 << 20, dtype=torch.uint8, device=self.device)
            _workspaces[(self._index, st)] = ws
        return ws

    def attend(self, q, step, scale=None, window=0, out=None, lse=None, workspace=None, stream=None):
        """Attention of the step's new tokens over their requests' cached ones
        (their own included).  ``scale`` defaults to head_dim ** -0.5; ``window``
        > 0: a token sees only that many last tokens, itself included.  ``lse``
        (fp32 [tokens, heads]) receives the log of the softmax sums.  Calls on one
        stream share a workspace; ``workspace`` (uint8, zero-filled before its
        first use) takes its place, as a captured graph needs that is replayed
        beside other calls."""
        if stream is None and _current_device() == self._index:
            return self._attend(q, step, scale, window, out, lse, workspace, _current_stream(self._index))
        with _on(self._index, stream) as st:
            return self._attend(q, step, scale, window, out, lse, workspace, st)

    def _attend(self, q, step, scale, window, out, lse, workspace, st):
        dim, index = self.head_dim, self._index
        qp, qs, tokens, heads = _rows(q, dim, "q", index)
        tables, lens, cu, tree = step.tables, step.lens, step.cu_new, step.tree
        rows, blocks = tables.shape
        n = lens.numel()
        if step.device != index or rows != n or cu.numel() != n + 1:
            raise ValueError("step.tables, lens and cu_new must agree and be on the cache's device")
        tree_p = lse_p = 0
        if tree is not None:
            tree_p = tree.data_ptr()
            _need(tree.numel() >= tokens, "step.tree must have a mask per token")
        if lse is not None:
            if (lse.dtype is not _F32 or lse.shape != (tokens, heads) or not lse.is_contiguous()
                    or lse.get_device() != index):
                raise ValueError("lse must be contiguous fp32 [tokens, heads] on the cache's device")
            lse_p = lse.data_ptr()
        if out is None:
            out = torch.empty(q.shape, dtype=_BF16, device=self.device)
        op, os_, no, _ = _rows(out, dim, "out", index, heads)
        if no != tokens:
            raise ValueError("out and q must have as many tokens")
        if tokens == 0:
            return out
        args = w12.w12_kv_attend_args(
            qp, op, lse_p, qs, os_, tables.data_ptr(), tables.stride(0) if n > 1 else blocks, lens.data_ptr(),
            cu.data_ptr(), tree_p, n, blocks, tokens, heads, step.max_new, window, self._scale if scale is None else scale)
        ws = self.workspace(args, (n, tokens, heads, step.max_new, blocks), st) if workspace is None else workspace
        w12.w12_kv_attend(self._c, args, ws.data_ptr(), ws.numel() * ws.element_size(), st)
        return out
