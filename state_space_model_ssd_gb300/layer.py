"""The operators around the scan in a layer of a language model, over libssd.so:

    (x, B, C), window = conv_forward(u, w, b, split=((H, P), (G, N), (G, N)))
    y, state = forward(x, raw_dt, B, C, delta_init)
    out, rstd = gated_norm_forward(y, z, w_gate)
    y_t = conv_decode_step(state, window, u_t, raw_t, w, b, positions, delta_init)
    n, h, stats = norm_forward(x, w_norm, b_norm, residual=h)

and their backward passes.  Activations are float32 or bfloat16 CUDA tensors; their rows may
be strided (a slice of the in-projection's output) as long as they are evenly spaced over all
leading dimensions, with neighbouring channels adjacent.
Weights and biases are float32 or bfloat16.  With ``stream`` the call runs there, and what it
allocates belongs to that stream.
"""

from __future__ import annotations

import ctypes
import os

from . import _lib

__all__ = ["conv_forward", "conv_backward", "conv_decode_step", "norm_forward", "norm_backward",
           "gated_norm_forward", "gated_norm_backward", "layer_status"]


def _load():
    """The binding: checks, allocation and the call into libssd.so."""
    global _ext
    if not os.path.exists(os.path.join(_lib.PKG, "_layer_ext.so")):
        raise RuntimeError("_layer_ext.so is not built; run state_space_model_ssd_gb300/build.py or "
                           "__graft_entry__.build()")
    import torch  # noqa: F401  (the binding is linked against its libraries)
    from . import _layer_ext
    _layer_ext.set_error(_lib.SSDError)
    _ext = _layer_ext
    return _ext


class _Unloaded:
    """In the binding's place until the first call."""

    def __getattr__(self, name):
        return getattr(_load(), name)


_ext = _Unloaded()
_KIND = {"layer": 0, "rms": 1}
_SILU = {"silu": True, None: False}


def _on(stream, f, *args):
    """``f`` with ``stream`` current: it launches there, and what it allocates belongs to it."""
    import torch
    for t in args:
        if isinstance(t, torch.Tensor):
            if stream.device != t.device:
                raise ValueError("stream is on %s, expected %s" % (stream.device, t.device))
            break
    with torch.cuda.stream(stream):
        return f(*args)


def _norm_kind(kind):
    k = _KIND.get(kind)
    if k is None:
        raise ValueError("kind must be 'layer' or 'rms'")
    return k


def _silu(activation):
    if activation not in _SILU:
        raise ValueError("activation must be 'silu' or None")
    return _SILU[activation]


# ------------------------------------------------------------------ convolution

def conv_forward(u, weight, bias=None, split=None, activation="silu", cu_seqlens=None,
                 positions=None, initial_state=None, final_state: bool = False, out=None,
                 final_state_out=None, stream=None):
    """Causal depthwise convolution over the tokens of each sequence, and its SiLU.

    ``u`` ``[batch, L, C]`` (rows may be strided), ``weight`` ``[C, width]`` (2 to 4 taps, the
    last one the current token's), ``bias`` ``[C]`` or None.  ``split`` names up to three
    pieces of the channels as sizes or shapes, e.g. ``((H, P), (G, N), (G, N))`` for the scan's
    x, B and C; the outputs are then a tuple of contiguous tensors ``[batch, L, *shape]``,
    otherwise one tensor.  ``cu_seqlens`` (int32 ``[nseq + 1]``, batch 1) packs sequences.
    ``initial_state`` ``[nseq, width, C]`` carries the tokens before each sequence: row ``p %
    width`` holds the one at position ``p``, ``positions`` (int32 ``[nseq]``, default 0) the
    position of each sequence's first token here.  Returns ``(outputs, final_state or None)``."""
    args = (u, weight, bias, split, _silu(activation), cu_seqlens, positions, initial_state,
            final_state, out, final_state_out)
    return _ext.conv_forward(*args) if stream is None else _on(stream, _ext.conv_forward, *args)


def conv_backward(u, weight, bias, dy, activation="silu", cu_seqlens=None, positions=None,
                  initial_state=None, d_final_state=None, d_initial_state: bool = False, out=None,
                  workspace=None, stream=None):
    """Backward of ``conv_forward``.  ``dy``: the gradient of the output, or a tuple of those of
    its pieces (contiguous, ``[batch, L, ...]``).  Returns a dict ``du, d_weight``, with a bias
    ``d_bias`` and with ``d_initial_state`` that too; ``out`` may bring any of them, and what it
    brings is written (``du`` may be strided, e.g. a slice of the in-projection's gradient;
    ``d_bias`` without a bias is refused)."""
    args = (u, weight, bias, dy, _silu(activation), cu_seqlens, positions, initial_state,
            d_final_state, d_initial_state, out, workspace)
    return _ext.conv_backward(*args) if stream is None else _on(stream, _ext.conv_backward, *args)


def conv_decode_step(state, conv_state, u, raw_dt, weight, bias, positions, delta_init: float,
                     ngroups: int = 1, slots=None, out=None, stream=None):
    """One token for each row of a batch: the convolution (SiLU) over the row of ``u``
    ``[batch, C]`` and the scan's step from it, in one launch.  The channels are x ``[H, P]``,
    B and C ``[ngroups, N]`` in that order.  ``state`` float32 ``[nslots, H, P, N]`` and
    ``conv_state`` ``[nslots, width, C]`` (as ``conv_forward`` leaves it) are updated in place.
    ``positions`` int32 ``[batch]``: the position of each row's token.  ``slots`` int32
    ``[batch]``: each row's cache slot (default: its index; the live rows' must differ); a row
    whose slot is negative or beyond the cache is padding, its y zero.  Returns y
    ``[batch, H, P]``."""
    args = (state, conv_state, u, raw_dt, weight, bias, positions, delta_init, ngroups, slots, out)
    return _ext.conv_decode_step(*args) if stream is None else _on(stream, _ext.conv_decode_step, *args)


# ------------------------------------------------------------------ norms

def norm_forward(x, weight, bias=None, residual=None, eps: float = 1e-5, kind: str = "layer",
                 out=None, residual_out=None, stats: bool = True, stream=None):
    """Norm of each row of ``x + residual`` (last dimension): ``kind`` "layer" subtracts the mean,
    "rms" does not.  ``residual`` has the shape of x and its type or float32.  Returns
    ``(y, h, stats)``: y in the type of x; h = x + residual in the residual's type (x itself
    without one); stats float32 ``[rows, 2]``, each row's mean and 1 / deviation, for the
    backward (None with ``stats=False``).  ``out=x`` and ``residual_out=residual`` work in place;
    ``residual_out`` without a residual is refused."""
    args = (x, weight, bias, residual, eps, _norm_kind(kind), out, residual_out, stats)
    return _ext.norm_forward(*args) if stream is None else _on(stream, _ext.norm_forward, *args)


def norm_backward(dy, h, weight, stats, dh=None, kind: str = "layer", bias: bool = True, out=None,
                  workspace=None, stream=None):
    """Backward of ``norm_forward``: ``dy`` the gradient of y, ``dh`` (optional) that of h, which
    arrives by the residual stream; ``h`` and ``stats`` as the forward returned them.  Returns a
    dict ``dx`` (in the type of dy), ``d_weight``, with ``bias`` ``d_bias``, and with ``dh`` or
    an h of another type ``d_residual`` (in the type of h; dx itself where the types agree).
    ``out`` may bring any of them, and what it brings is written (``dx`` may be strided)."""
    args = (dy, h, weight, stats, dh, _norm_kind(kind), bias, out, workspace)
    return _ext.norm_backward(*args) if stream is None else _on(stream, _ext.norm_backward, *args)


def gated_norm_forward(y, z, weight, eps: float = 1e-5, groups: int = 1, out=None, stream=None):
    """``y silu(z)`` normed by its root mean square in each of ``groups`` equal groups of the
    columns, times ``weight`` ``[D]``.  ``z`` ``[..., D]``; ``y`` the same, or with its columns
    as the scan leaves them, ``[..., H, P]`` with H P = D.  Returns ``(out, rstd)``: out in the
    shape of z, rstd float32 ``[rows, groups]`` for the backward."""
    args = (y, z, weight, eps, groups, out)
    return _ext.gated_norm_forward(*args) if stream is None else _on(stream, _ext.gated_norm_forward, *args)


def gated_norm_backward(dout, y, z, weight, rstd, groups: int = 1, out=None, workspace=None,
                        stream=None):
    """Backward of ``gated_norm_forward``.  Returns a dict ``dy`` (in the shape of y), ``dz``,
    ``d_weight``; ``out`` may bring any of them (dz may be strided, e.g. a slice of the
    in-projection's gradient)."""
    args = (dout, y, z, weight, rstd, groups, out, workspace)
    return _ext.gated_norm_backward(*args) if stream is None else _on(stream, _ext.gated_norm_backward, *args)


def layer_status(stream=None) -> int:
    """Waits for ``stream`` (default: the current one) and returns what the calls of this module
    have recorded on its device since the last query: 0, or the code of SSD_ERR_TIMEOUT if a
    kernel's bounded wait ran out (its outputs are then not valid)."""
    import torch
    v = ctypes.c_int32(0)
    s = torch.cuda.current_stream() if stream is None else stream
    with torch.cuda.device(s.device):  # the word is the current device's
        _lib.check(_lib.lib().ssd_layer_status(ctypes.c_void_p(s.cuda_stream), ctypes.byref(v)),
                   "ssd_layer_status")
    return int(v.value)
