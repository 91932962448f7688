"""Beam search over the C ABI's w12_beam_select: which continuations of every request's
beams go on.

One step, with pages that requests share (kv.py) and logits from the LM head::

    beams.select(logits)                                   # tokens, parents, scores
    copies = pages.fork(beams.parents, lens, copies, prefix=step.prefix, lens_out=lens)
    caches[0].copy(copies, others=caches[1:])              # every layer's cache
    # beams.tokens are the next step's inputs
"""
from __future__ import annotations

import ctypes

import torch

from . import kv, w12


class Beams:
    """The beams of ``requests`` requests, ``beams`` (up to 32) each.

    ``select`` takes the beams' logits and leaves, for every request, in ``tokens``,
    ``parents`` (int32 [requests * beams]; rows of the logits, as ``KVPages.fork`` takes
    them) and ``scores`` (fp32 [requests, beams]) the best continuations that do not end with
    the token ``eos`` (None: none ends), and in ``cand_tokens``, ``cand_parents``,
    ``cand_scores`` ([requests, take]) the best ``take`` (2 * beams where not given, at most
    64) of all, best first: those that end among them are finished.  Where there are fewer,
    token and parent are -1 and the score -infinity.  A beam whose score is not finite does
    not go on: at first only each request's first one has a score (``reset``)."""

    def __init__(self, requests, beams, take=None, eos=None, device=None):
        dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.requests, self.beams = int(requests), int(beams)
        self.take = 2 * self.beams if take is None else int(take)
        self.eos = None if eos is None else int(eos)
        if self.requests < 1 or not 1 <= self.beams <= 32 or not 1 <= self.take <= 64:
            raise ValueError("requests must be at least 1, beams 1 to 32 and take 1 to 64")
        if self.eos is not None and self.eos < 0:
            raise ValueError("eos must be a token or None")
        ints = lambda *s: torch.full(s, -1, dtype=torch.int32, device=dev)  # noqa: E731
        self._tokens, self._parents = ints(self.requests * self.beams), ints(self.requests * self.beams)
        self._cand = (ints(self.requests, self.take), ints(self.requests, self.take),
                      torch.full((self.requests, self.take), float("-inf"), device=dev))
        self._scores = torch.empty(self.requests, self.beams, device=dev)
        self.reset()
        self._index = self._scores.get_device()
        self._ws, self._outgrown = None, []
        self._c = w12.w12_beam_args(None, 0, None, 0, self._scores.data_ptr(), self._scores.data_ptr(),
                                    self._tokens.data_ptr(), self._parents.data_ptr(),
                                    *(t.data_ptr() for t in self._cand), self.requests, self.beams, 0, self.take,
                                    -1 if self.eos is None else self.eos, w12.BEAM_BF16)
        self._address = ctypes.addressof(self._c)

    # written in place by every select: not to be replaced
    tokens = property(lambda self: self._tokens)
    parents = property(lambda self: self._parents)
    scores = property(lambda self: self._scores)
    cand_tokens = property(lambda self: self._cand[0])
    cand_parents = property(lambda self: self._cand[1])
    cand_scores = property(lambda self: self._cand[2])

    def reset(self):
        """The beginning of a search: one beam of each request, with score 0."""
        self._scores.fill_(float("-inf"))
        self._scores[:, 0] = 0.0

    def _grow(self, index, st, size):
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("the workspace is not large enough yet: make one ordinary call with this vocabulary "
                               "before capturing")
        if self._ws is not None:
            self._outgrown.append(self._ws)  # a captured graph may still use it
        self._ws = torch.zeros(size, dtype=torch.uint8, device=self._scores.device)
        return self._ws

    def select(self, logits, allowed=None, scores=None, stream=None):
        """One step: ``logits`` BF16 or fp32 [requests * beams, vocab] (or [requests, beams,
        vocab]).  ``allowed`` (int32 [requests * beams, ceil(vocab / 32)], or one line for
        all): bit v % 32 of word v / 32 is set for the tokens that count.  ``scores`` (fp32
        [requests, beams]): the scores so far in the place of ``self.scores``.  The results
        are written over those of the step before.  Calls of one holder on several streams
        have to be ordered."""
        if stream is not None or kv._current_device() != self._index:
            with kv._on(self._index, stream):
                return self.select(logits, allowed, scores)
        kv._host.select(self._address, self._index, logits, allowed, scores, self._ws, self._grow,
                        kv._current_stream(self._index))
