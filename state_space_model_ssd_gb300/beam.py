"""Beam search over cached states, over libssd.so: the choice of the beams that go on, and the move
of their states between the cache slots that the token steps work on:

    scores, parents, tokens = beam_select(logits, scores)
    slots = beam_reorder([state, window, ...], slots, parents)

With ``stream`` a call runs there, and what it allocates belongs to that stream.
"""

from __future__ import annotations

from . import layer
from .layer import _on

__all__ = ["beam_select", "beam_reorder"]


def beam_select(logits, scores, keep=None, finished=None, pad_token: int = 0, out=None, workspace=None,
                stream=None):
    """The ``keep`` (default: as many as there are beams, at most 64) best candidates of each batch
    row, best first: token t after beam i scores ``scores[i] + log_softmax(logits[i])[t]``.

    ``logits`` ``[batch, beams, vocab]`` float32 or bfloat16 (rows may be strided, e.g. a slice of a
    padded head), ``scores`` float32 ``[batch, beams]``.  ``finished`` (bool or uint8 ``[batch,
    beams]``): an ended beam goes on with ``pad_token`` alone, at its score.  Equal candidates come
    in the order of their beams, then tokens; those of one beam are ordered by their logits.  What is
    left out (tokens at -inf, beams whose score is not finite or whose logits hold a NaN, +inf or
    nothing but -inf) has the score -inf.  Returns ``(scores float32, parents int32, tokens int32)``,
    each ``[batch, keep]``; ``out`` may bring the three."""
    args = (logits, scores, keep, finished, pad_token, out, workspace)
    return layer._ext.beam_select(*args) if stream is None else _on(stream, layer._ext.beam_select, *args)


def beam_reorder(caches, slots, parents, out=None, stream=None):
    """Lets beam j of each batch row go on from the states of beam ``parents[j]`` and returns the
    new int32 ``[batch, beams]`` slots.

    ``caches``: a list of tensors ``[nslots, ...]`` of any type whose slots are contiguous, e.g. the
    scan's states and the convolution's windows of every layer, changed in place.  ``slots`` int32
    ``[batch, beams]``: each beam's slot; ``parents`` int32 of that shape, e.g. from
    ``beam_select``.  The first beam with a parent takes over its slot; the others take the slots
    of beams that nobody goes on from, and only their states are copied.  A beam whose parent lies
    outside the beams gets slot -1; slots outside the cache are passed on.  Slots must differ."""
    args = (caches, slots, parents, out)
    if stream is None:
        return layer._ext.beam_reorder(*args)
    if stream.device != slots.device:
        raise ValueError("stream is on %s, expected %s" % (stream.device, slots.device))
    return _on(stream, layer._ext.beam_reorder, *args)
