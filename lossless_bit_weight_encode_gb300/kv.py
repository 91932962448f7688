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


class _on:
    """The device and stream a call runs on: outputs are allocated for that
    stream.  ``stream`` as in w12.py: None (the current one), a torch stream or
    a handle."""

    def __init__(self, tensor, stream):
        self.device = tensor.device.index
        self.stream = stream
        self.guards = ()

    def __enter__(self):
        if self.device != torch.cuda.current_device():
            self.guards = (torch.cuda.device(self.device),)
        if self.stream is not None:
            s = self.stream
            if isinstance(s, int):
                s = torch.cuda.ExternalStream(s, device=self.device) if s else torch.cuda.default_stream(self.device)
            self.guards += (torch.cuda.stream(s),)
        for g in self.guards:
            g.__enter__()
        return torch.cuda.current_stream(self.device).cuda_stream

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)
        return False


def _need(ok, text):
    if not ok:
        raise ValueError(text)


def _ints(t, dtype, name, device):
    """Pointer of a contiguous 1-D integer tensor."""
    if t.dtype != dtype or t.dim() != 1 or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 1-D {dtype} tensor on {device}")
    return t.data_ptr()


def _rows(t, dim, name, device, heads=None):
    """(pointer, token stride, heads) of [T, heads * dim] or [T, heads, dim]
    BF16 rows whose heads lie one after the other."""
    shape, stride = t.shape, t.stride()
    if len(shape) == 2:
        ok, n = stride[1] == 1 and shape[1] % dim == 0, shape[1] // dim
    else:
        ok = len(shape) == 3 and shape[2] == dim and stride[2] == 1 and (stride[1] == dim or shape[1] == 1)
        n = shape[1] if ok else 0
    if not ok or t.dtype != _BF16 or t.device != device or n < 1 or (heads is not None and n != heads):
        raise ValueError(f"{name} must be BF16 [tokens, {heads or 'heads'} * {dim}] on {device} with contiguous heads")
    # one row has no stride that matters
    return t.data_ptr(), stride[0] if shape[0] > 1 else n * dim, n


class KVStep:
    """One step of a batch: for request b, ``lens[b]`` cached tokens and the new
    tokens ``cu_new[b] : cu_new[b + 1]``; for every new token its ``position``
    and cache slot (-1: none).  ``tables`` [requests, max_blocks] holds the
    requests' pages.  ``tree`` (int32, bit j of a token's mask: it attends to new
    token j of its request) replaces the causal order among new tokens.
    ``max_new``: the most new tokens of a request, as far as is known.  What a
    call does not use may be None."""

    def __init__(self, tables=None, lens=None, cu_new=None, positions=None, slots=None, max_new=1, tree=None):
        self.tables, self.lens, self.cu_new = tables, lens, cu_new
        self.positions, self.slots = positions, slots
        self.max_new, self.tree = int(max_new), tree


class KVPages:
    """Page tables of ``requests`` requests and the ring of free pages.

    ``tables`` int32 [requests, max_blocks]; ``owned`` int32 [requests]: pages
    each request holds; ``ring`` int32: free page numbers, of which
    ``ring[i % len]`` for head <= i < tail are free; ``ring_state`` int64
    {head, tail}.  ``KVPages.create`` starts with every page free."""

    def __init__(self, tables, owned, ring, ring_state, page_size):
        dev = tables.device
        _need(tables.dtype == _I32 and tables.dim() == 2 and tables.stride(1) == 1 and tables.is_cuda,
              "tables must be an int32 CUDA tensor [requests, max_blocks] with contiguous rows")
        _ints(owned, _I32, "owned", dev)
        _ints(ring, _I32, "ring", dev)
        _ints(ring_state, _I64, "ring_state", dev)
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
        tables, dev = self.tables, self.tables.device
        n = tables.shape[0]
        _need(lens.numel() == n and new_lens.numel() == n, "lens and new_lens must have an entry per request")
        owned_out = self.owned if owned_out is None else owned_out
        ring_state_out = self.ring_state if ring_state_out is None else ring_state_out
        _need(owned_out.numel() == n and ring_state_out.numel() == 2, "owned_out or ring_state_out has another size")
        _need(step.cu_new.numel() == n + 1 and step.positions.numel() == step.slots.numel(),
              "step belongs to another number of requests")
        args = w12.w12_kv_plan_args(
            _ints(lens, _I32, "lens", dev), _ints(new_lens, _I32, "new_lens", dev), self.owned.data_ptr(),
            _ints(owned_out, _I32, "owned_out", dev), tables.data_ptr(), tables.stride(0) if n > 1 else tables.shape[1], self.ring.data_ptr(),
            self.ring_state.data_ptr(), _ints(ring_state_out, _I64, "ring_state_out", dev),
            _ints(step.cu_new, _I32, "cu_new", dev), _ints(step.positions, _I32, "positions", dev),
            _ints(step.slots, _I64, "slots", dev), n, tables.shape[1], self.page_size, self.ring.numel(),
            step.slots.numel(), 1 if trim else 0)
        with _on(tables, stream) as st:
            w12.w12_kv_plan(args, st)
        step.tables, step.lens = tables, lens
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
        self.kv_heads, self.page_size, self.head_dim = heads, page, dim
        # a dimension of one element has no stride that matters
        stride = [s if n > 1 else dim for n, s in zip(k.shape, k.stride())]
        self._c = w12.w12_kv_cache(k.data_ptr(), v.data_ptr(), None if scales is None else scales.data_ptr(), pages,
                                   stride[0], stride[1], stride[2], page, heads, dim,
                                   w12.KV_BF16 if scales is None else w12.KV_Q8)
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
        cache at step.slots.  Returns the new q (``out``, which may be q); q None:
        only k and v."""
        dim, dev = self.head_dim, self.device
        kp, ks, _ = _rows(k, dim, "k", dev, self.kv_heads)
        vp, vs, _ = _rows(v, dim, "v", dev, self.kv_heads)
        tokens = k.shape[0]
        _need(v.shape[0] == tokens and step.slots.numel() == tokens, "k, v and step.slots must have as many tokens")
        qp = qs = op = os_ = heads = 0
        rot = rows = rp = pp = 0
        if rope is not None:
            _need(rope.dtype == _F32 and rope.dim() == 2 and rope.is_contiguous() and rope.device == dev,
                  "rope must be a contiguous fp32 tensor [positions, rot]")
            _need(step.positions is not None and step.positions.numel() == tokens, "step.positions must have as many tokens")
            rows, rot = rope.shape
            rp, pp = rope.data_ptr(), _ints(step.positions, _I32, "step.positions", dev)
        for name, t in (("q_norm", q_norm), ("k_norm", k_norm)):
            if t is not None:
                _need(t.dtype == _BF16 and t.shape == (dim,) and t.is_contiguous() and t.device == dev,
                      f"{name} must be BF16 [{dim}]")
        sp = _ints(step.slots, _I64, "step.slots", dev)
        with _on(k, stream) as st:
            if q is not None:
                qp, qs, heads = _rows(q, dim, "q", dev)
                _need(q.shape[0] == tokens, "q and k must have as many tokens")
                if out is None:
                    out = torch.empty(q.shape, dtype=_BF16, device=dev)
                op, os_, n = _rows(out, dim, "out", dev, heads)
                _need(out.shape[0] == tokens, "out and q must have as many tokens")
            w12.w12_kv_store(self._c, w12.w12_kv_store_args(
                qp, kp, vp, op, qs, ks, vs, os_, None if q_norm is None else q_norm.data_ptr(),
                None if k_norm is None else k_norm.data_ptr(), rp, pp, sp, rows, tokens, heads, rot,
                1 if interleaved else 0, eps), st)
        return out if q is not None else None

    def read(self, slots, out=None, stream=None):
        """(k, v) BF16 [tokens, kv_heads, head_dim] of the cached rows at ``slots``
        (int64; zeros for -1).  ``out``: a pair to write to."""
        shape = (slots.numel(), self.kv_heads, self.head_dim)
        sp = _ints(slots, _I64, "slots", self.device)
        with _on(slots, stream) as st:
            if out is None:
                out = (torch.empty(shape, dtype=_BF16, device=self.device),
                       torch.empty(shape, dtype=_BF16, device=self.device))
            for t in out:
                _need(t.shape == shape and t.dtype == _BF16 and t.is_contiguous() and t.device == self.device,
                      "out must be two contiguous BF16 tensors [tokens, kv_heads, head_dim]")
            if shape[0]:
                w12.w12_kv_read(self._c, sp, shape[0], out[0].data_ptr(), out[1].data_ptr(), st)
        return out

    def workspace(self, args, st):
        """The zeroed workspace of the attend calls on stream ``st`` (shared by
        all caches), large enough for ``args``."""
        key = (args.requests, args.tokens, args.heads, args.max_new, args.max_blocks)
        size = self._ws_bytes.get(key)
        if size is None:
            size = self._ws_bytes[key] = w12.w12_kv_attend_workspace_size(self._c, args)
        ws = _workspaces.get((self.device.index, st))
        if ws is None or ws.numel() < size:
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError("the workspace of this stream is not large enough yet: make one ordinary call of "
                                   "this size on the stream before capturing, or pass workspace=")
            ws = torch.zeros((size + (1 << 20) - 1) >> 20 << 20, dtype=torch.uint8, device=self.device)
            _workspaces[(self.device.index, st)] = ws
        return ws

    def attend(self, q, step, scale=None, window=0, out=None, lse=None, workspace=None, stream=None):
        """Attention of the step's new tokens over their requests' cached ones
        (their own included).  ``scale`` defaults to head_dim ** -0.5; ``window``
        > 0: a token sees only that many last tokens, itself included.  ``lse``
        (fp32 [tokens, heads]) receives the log of the softmax sums.  Calls on one
        stream share a workspace; ``workspace`` (uint8, zero-filled before its
        first use) takes its place, as a captured graph needs that is replayed
        beside other calls."""
        dim, dev = self.head_dim, self.device
        qp, qs, heads = _rows(q, dim, "q", dev)
        tables, lens, tokens = step.tables, step.lens, q.shape[0]
        _need(tables.dtype == _I32 and tables.dim() == 2 and tables.stride(1) == 1 and tables.device == dev,
              "step.tables must be int32 [requests, max_blocks] with contiguous rows")
        n = lens.numel()
        _need(tables.shape[0] == n and step.cu_new.numel() == n + 1, "step.tables, lens and cu_new do not agree")
        tp = lp = 0
        if step.tree is not None:
            tp = _ints(step.tree, _I32, "step.tree", dev)
            _need(step.tree.numel() >= tokens, "step.tree must have a mask per token")
        if lse is not None:
            _need(lse.dtype == _F32 and lse.shape == (tokens, heads) and lse.is_contiguous() and lse.device == dev,
                  "lse must be contiguous fp32 [tokens, heads]")
            lp = lse.data_ptr()
        with _on(q, stream) as st:
            if out is None:
                out = torch.empty(q.shape, dtype=_BF16, device=dev)
            op, os_, _ = _rows(out, dim, "out", dev, heads)
            _need(out.shape[0] == tokens, "out and q must have as many tokens")
            if tokens == 0:
                return out
            args = w12.w12_kv_attend_args(
                qp, op, lp, qs, os_, tables.data_ptr(), tables.stride(0) if n > 1 else tables.shape[1],
                _ints(lens, _I32, "step.lens", dev), _ints(step.cu_new, _I32, "step.cu_new", dev), tp, n,
                tables.shape[1], tokens, heads, step.max_new, window, dim ** -0.5 if scale is None else scale)
            ws = self.workspace(args, st) if workspace is None else workspace
            w12.w12_kv_attend(self._c, args, ws.data_ptr(), ws.numel() * ws.element_size(), st)
        return out
