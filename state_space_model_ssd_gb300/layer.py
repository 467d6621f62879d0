"""The operators around the scan in a layer of a language model, over libssd.so:

    (x, B, C), window = conv_forward(u, w, b, split=((H, P), (G, N), (G, N)))
    y, state = forward(x, raw_dt, B, C, delta_init)
    out, rstd = gated_norm_forward(y, z, w_gate)
    y_t = conv_decode_step(state, window, u_t, raw_t, w, b, positions, delta_init)
    n, h, stats = norm_forward(x, w_norm, b_norm, residual=h)

and their backward passes.  Activations are float32 or bfloat16 CUDA tensors; their rows may
be strided (a slice of the in-projection's output), with neighbouring channels adjacent.
Weights and biases are float32 or bfloat16.  With ``stream`` the call runs there, and what it
allocates belongs to that stream.
"""

from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import ConvProblem, GatedNormProblem, NormProblem, Problem, check

__all__ = ["conv_forward", "conv_backward", "conv_decode_step", "norm_forward", "norm_backward",
           "gated_norm_forward", "gated_norm_backward"]

_CODE = {torch.float32: _lib.DTYPE_F32, torch.bfloat16: _lib.DTYPE_BF16}
_KIND = {"layer": 0, "rms": 1}
_byref = ctypes.byref
_empty = torch.empty


def _ptr(t):
    return None if t is None else t.data_ptr()


class _on:
    """Makes ``device`` current, and ``stream`` when one is given: allocations inside belong
    to the stream that uses them.  ``raw`` is the stream's handle."""

    __slots__ = ("raw", "_guards")

    def __init__(self, device, stream):
        self._guards = ()
        if stream is not None:
            if stream.device != device:
                raise ValueError("stream is on %s, expected %s" % (stream.device, device))
            self._guards = (torch.cuda.stream(stream),)
        elif device.index != torch.cuda.current_device():
            self._guards = (torch.cuda.device(device),)

    def __enter__(self):
        for g in self._guards:
            g.__enter__()
        self.raw = torch.cuda.current_stream().cuda_stream
        return self

    def __exit__(self, *exc):
        for g in reversed(self._guards):
            g.__exit__(*exc)
        return False


def _code(t, name):
    c = _CODE.get(t.dtype)
    if c is None:
        raise TypeError("%s must be float32 or bfloat16, got %s" % (name, t.dtype))
    return c


def _check(t, name, device, dtype=None, shape=None):
    """A contiguous CUDA tensor on ``device`` of the given type and shape."""
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must be %s, got %s" % (name, list(shape), list(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _rows(t, name, device=None, dtype=None, shape=None):
    """The stride between the rows of ``t`` (its last dimension's vectors), which must be
    evenly spaced; the last dimension itself must be contiguous."""
    if device is None:
        if not t.is_cuda:
            raise ValueError("%s must be a CUDA tensor" % name)
    elif t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if shape is not None and t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, list(shape), list(t.shape)))
    if t.is_contiguous():
        return t.shape[-1]
    size, stride = t.shape, t.stride()
    if size[-1] > 1 and stride[-1] != 1:
        raise ValueError("%s: neighbouring channels must be adjacent" % name)
    step = None
    span = 1
    for n, s in zip(reversed(size[:-1]), reversed(stride[:-1])):
        if n == 1:
            continue
        if step is None:
            step = s
        elif s != span * step:
            raise ValueError("%s: rows must be evenly spaced" % name)
        span *= n
    if step is None:
        return size[-1]
    if step < size[-1]:
        raise ValueError("%s: rows overlap" % name)
    return step


def _params(weight, bias, device, shape):
    _check(weight, "weight", device, None, shape)
    code = _code(weight, "weight")
    if bias is not None:
        _check(bias, "bias", device, weight.dtype, shape[:1])
    return code


def _scratch(nbytes, device, workspace):
    if workspace is None:
        return _empty(nbytes, dtype=torch.uint8, device=device)
    if workspace.device != device:
        raise ValueError("workspace is on %s, expected %s" % (workspace.device, device))
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError("workspace too small: need %d bytes" % nbytes)
    return workspace


def _size(call, prob):
    n = ctypes.c_size_t(0)
    check(getattr(_lib.lib(), call)(_byref(prob), _byref(n)), call)
    return n.value


# ------------------------------------------------------------------ convolution

def _pieces(split, channels):
    """``split`` as a tuple of shapes, and their channel counts padded to three."""
    if split is None:
        return ((channels,),), (channels, 0, 0)
    shapes = tuple((s,) if isinstance(s, int) else tuple(s) for s in split)
    if not 1 <= len(shapes) <= 3:
        raise ValueError("split must name one to three pieces")
    sizes = []
    for s in shapes:
        n = 1
        for d in s:
            if d < 1:
                raise ValueError("split sizes must be positive")
            n *= d
        sizes.append(n)
    if sum(sizes) != channels:
        raise ValueError("split adds up to %d channels, u has %d" % (sum(sizes), channels))
    return shapes, tuple(sizes) + (0,) * (3 - len(sizes))


def _conv_problem(u, weight, bias, sizes, cu_seqlens, positions, initial_state, activation):
    dev = u.device
    if u.dim() != 3:
        raise ValueError("u must be [batch, L, channels]")
    stride = _rows(u, "u")
    batch, L, C = u.shape
    if weight.dim() != 2 or weight.shape[0] != C:
        raise ValueError("weight must be [channels, width]")
    width = weight.shape[1]
    wcode = _params(weight, bias, dev, (C, width))
    nseq = 0
    if cu_seqlens is not None:
        _check(cu_seqlens, "cu_seqlens", dev, torch.int32)
        nseq = cu_seqlens.numel() - 1
        if batch != 1:
            raise ValueError("packed sequences need batch == 1")
        if cu_seqlens.dim() != 1 or nseq < 1:
            raise ValueError("cu_seqlens must be [nseq + 1]")
    n = nseq or batch
    if positions is not None:
        _check(positions, "positions", dev, torch.int32, (n,))
    if initial_state is not None:
        _check(initial_state, "initial_state", dev, u.dtype, (n, width, C))
    if activation not in ("silu", None):
        raise ValueError("activation must be 'silu' or None")
    prob = ConvProblem(batch, L, stride, 0, sizes, width, nseq, _code(u, "u"), wcode,
                       activation is not None)
    return prob, n, width, C


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
    if u.dim() != 3:
        raise ValueError("u must be [batch, L, channels]")
    batch, L, C = u.shape
    shapes, sizes = _pieces(split, C)
    prob, n, width, _ = _conv_problem(u, weight, bias, sizes, cu_seqlens, positions, initial_state,
                                      activation)
    dev, dt = u.device, u.dtype
    with _on(dev, stream) as at:
        if out is None:
            outs = [_empty((batch, L) + s, dtype=dt, device=dev) for s in shapes]
        else:
            outs = [out] if split is None else list(out)
            if len(outs) != len(shapes):
                raise ValueError("out must hold %d tensors" % len(shapes))
            for o, s in zip(outs, shapes):
                _check(o, "out", dev, dt, (batch, L) + s)
        fs = final_state_out
        if fs is not None:
            _check(fs, "final_state_out", dev, dt, (n, width, C))
        elif final_state:
            fs = _empty((n, width, C), dtype=dt, device=dev)
        p = [o.data_ptr() for o in outs] + [None, None]
        st = _lib.lib().ssd_conv_forward(_byref(prob), u.data_ptr(), weight.data_ptr(), _ptr(bias),
                                         _ptr(cu_seqlens), _ptr(positions), _ptr(initial_state),
                                         p[0], p[1], p[2], _ptr(fs), at.raw)
    if st:
        check(st, "ssd_conv_forward")
    return (outs[0] if split is None else tuple(outs)), fs


def conv_backward(u, weight, bias, dy, activation="silu", cu_seqlens=None, positions=None,
                  initial_state=None, d_final_state=None, d_initial_state: bool = False, out=None,
                  workspace=None, stream=None):
    """Backward of ``conv_forward``.  ``dy``: the gradient of the output, or a tuple of those of
    its pieces (contiguous, ``[batch, L, ...]``).  Returns a dict ``du, d_weight``, with a bias
    ``d_bias`` and with ``d_initial_state`` that too; ``out`` may bring any of them (``du`` may
    be strided, e.g. a slice of the in-projection's gradient)."""
    if u.dim() != 3:
        raise ValueError("u must be [batch, L, channels]")
    batch, L, C = u.shape
    dev, dt = u.device, u.dtype
    dys = [dy] if isinstance(dy, torch.Tensor) else list(dy)
    shapes = []
    for d in dys:
        if d.dim() < 3 or d.shape[0] != batch or d.shape[1] != L:
            raise ValueError("dy must be [batch, L, ...]")
        _check(d, "dy", dev, dt)
        shapes.append(d.shape[2:])
    _, sizes = _pieces(shapes, C)
    prob, n, width, _ = _conv_problem(u, weight, bias, sizes, cu_seqlens, positions, initial_state,
                                      activation)
    if d_final_state is not None:
        _check(d_final_state, "d_final_state", dev, dt, (n, width, C))
    with _on(dev, stream) as at:
        g = {} if out is None else out
        if "du" not in g:
            g["du"] = _empty((batch, L, C), dtype=dt, device=dev)
        prob.du_stride = _rows(g["du"], "du", dev, dt, u.shape)
        if "d_weight" not in g:
            g["d_weight"] = _empty(weight.shape, dtype=weight.dtype, device=dev)
        _check(g["d_weight"], "d_weight", dev, weight.dtype, weight.shape)
        if bias is not None:
            if "d_bias" not in g:
                g["d_bias"] = _empty((C,), dtype=weight.dtype, device=dev)
            _check(g["d_bias"], "d_bias", dev, weight.dtype, (C,))
        d0 = None
        if d_initial_state:
            if "d_initial_state" not in g:
                g["d_initial_state"] = _empty((n, width, C), dtype=dt, device=dev)
            d0 = g["d_initial_state"]
            _check(d0, "d_initial_state", dev, dt, (n, width, C))
        ws = _scratch(_size("ssd_conv_workspace_size", prob), dev, workspace)
        p = [d.data_ptr() for d in dys] + [None, None]
        st = _lib.lib().ssd_conv_backward(
            _byref(prob), u.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(cu_seqlens),
            _ptr(positions), _ptr(initial_state), p[0], p[1], p[2], _ptr(d_final_state),
            g["du"].data_ptr(), g["d_weight"].data_ptr(), _ptr(g["d_bias"] if bias is not None else None),
            _ptr(d0), ws.data_ptr(), ws.numel() * ws.element_size(), at.raw)
    if st:
        check(st, "ssd_conv_backward")
    return g


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
    stride = _rows(u, "u")
    dev, dt = u.device, u.dtype
    if u.dim() != 2 or state.dim() != 4:
        raise ValueError("u must be [batch, channels], state [nslots, H, P, N]")
    batch, C = u.shape
    nslots, H, P, N = state.shape
    if C != H * P + 2 * ngroups * N:
        raise ValueError("u has %d channels, H P + 2 ngroups N is %d" % (C, H * P + 2 * ngroups * N))
    if weight.dim() != 2:
        raise ValueError("weight must be [channels, width]")
    width = weight.shape[1]
    wcode = _params(weight, bias, dev, (C, width))
    _check(state, "state", dev, torch.float32)
    _check(conv_state, "conv_state", dev, dt, (nslots, width, C))
    _check(raw_dt, "raw_dt", dev, torch.float32, (batch, H))
    _check(positions, "positions", dev, torch.int32, (batch,))
    if slots is not None:
        _check(slots, "slots", dev, torch.int32, (batch,))
    prob = Problem(batch, 1, H, P, N, ngroups, 64, 0, delta_init, _code(u, "u"))
    with _on(dev, stream) as at:
        if out is None:
            out = _empty((batch, H, P), dtype=dt, device=dev)
        else:
            _check(out, "out", dev, dt, (batch, H, P))
        st = _lib.lib().ssd_conv_decode_step(
            _byref(prob), width, wcode, nslots, stride, state.data_ptr(), conv_state.data_ptr(),
            u.data_ptr(), raw_dt.data_ptr(), weight.data_ptr(), _ptr(bias), positions.data_ptr(),
            _ptr(slots), out.data_ptr(), at.raw)
    if st:
        check(st, "ssd_conv_decode_step")
    return out


# ------------------------------------------------------------------ norms

def _norm_kind(kind):
    if kind not in _KIND:
        raise ValueError("kind must be 'layer' or 'rms'")
    return _KIND[kind]


def norm_forward(x, weight, bias=None, residual=None, eps: float = 1e-5, kind: str = "layer",
                 out=None, residual_out=None, stats: bool = True, stream=None):
    """Norm of each row of ``x + residual`` (last dimension): ``kind`` "layer" subtracts the mean,
    "rms" does not.  ``residual`` has the shape of x and its type or float32.  Returns
    ``(y, h, stats)``: y in the type of x; h = x + residual in the residual's type (x itself
    without one); stats float32 ``[rows, 2]``, each row's mean and 1 / deviation, for the
    backward (None with ``stats=False``).  ``out=x`` and ``residual_out=residual`` work in place."""
    dev, dt = x.device, x.dtype
    xs = _rows(x, "x")
    code, D = _code(x, "x"), x.shape[-1]
    wcode = _params(weight, bias, dev, (D,))
    n = x.numel() // D if D else 0
    rs, rdt, rcode = D, dt, code
    if residual is not None:
        rdt = residual.dtype
        rcode = _code(residual, "residual")
        rs = _rows(residual, "residual", dev, None, x.shape)
    k = _norm_kind(kind)
    with _on(dev, stream) as at:
        y = _empty(x.shape, dtype=dt, device=dev) if out is None else out
        h, hs = x, D
        if residual is not None:
            h = _empty(x.shape, dtype=rdt, device=dev) if residual_out is None else residual_out
            hs = _rows(h, "residual_out", dev, rdt, x.shape)
        ys = D if out is None else _rows(y, "out", dev, dt, x.shape)
        sv = _empty((n, 2), dtype=torch.float32, device=dev) if stats else None
        prob = NormProblem(n, xs, rs, hs, ys, D, k, code, rcode, wcode, eps)
        st = _lib.lib().ssd_norm_forward(
            _byref(prob), x.data_ptr(), _ptr(residual), weight.data_ptr(), _ptr(bias), y.data_ptr(),
            None if residual is None else h.data_ptr(), _ptr(sv), at.raw)
    if st:
        check(st, "ssd_norm_forward")
    return y, h, sv


def norm_backward(dy, h, weight, stats, dh=None, kind: str = "layer", bias: bool = True, out=None,
                  workspace=None, stream=None):
    """Backward of ``norm_forward``: ``dy`` the gradient of y, ``dh`` (optional) that of h, which
    arrives by the residual stream; ``h`` and ``stats`` as the forward returned them.  Returns a
    dict ``dx`` (in the type of dy), ``d_weight``, with ``bias`` ``d_bias``, and with ``dh`` or
    an h of another type ``d_residual`` (in the type of h; dx itself where the types agree)."""
    dev, dt = dy.device, dy.dtype
    ys = _rows(dy, "dy")
    code, D = _code(dy, "dy"), dy.shape[-1]
    hs = _rows(h, "h", dev, None, dy.shape)
    rdt, rcode = h.dtype, _code(h, "h")
    wcode = _params(weight, None, dev, (D,))
    n = dy.numel() // D if D else 0
    _check(stats, "stats", dev, torch.float32, (n, 2))
    rs = D if dh is None else _rows(dh, "dh", dev, rdt, dy.shape)
    k = _norm_kind(kind)
    with _on(dev, stream) as at:
        g = {} if out is None else out
        if "dx" not in g:
            g["dx"] = _empty(dy.shape, dtype=dt, device=dev)
        xs = _rows(g["dx"], "dx", dev, dt, dy.shape)
        dres = None
        if rdt != dt:
            if "d_residual" not in g:
                g["d_residual"] = _empty(dy.shape, dtype=rdt, device=dev)
            dres = g["d_residual"]
            _check(dres, "d_residual", dev, rdt, dy.shape)
        elif dh is not None:
            g["d_residual"] = g["dx"]
        if "d_weight" not in g:
            g["d_weight"] = _empty((D,), dtype=weight.dtype, device=dev)
        _check(g["d_weight"], "d_weight", dev, weight.dtype, (D,))
        if bias:
            if "d_bias" not in g:
                g["d_bias"] = _empty((D,), dtype=weight.dtype, device=dev)
            _check(g["d_bias"], "d_bias", dev, weight.dtype, (D,))
        prob = NormProblem(n, xs, rs, hs, ys, D, k, code, rcode, wcode, 0.0)
        ws = _scratch(_size("ssd_norm_workspace_size", prob), dev, workspace)
        st = _lib.lib().ssd_norm_backward(
            _byref(prob), dy.data_ptr(), h.data_ptr(), _ptr(dh), weight.data_ptr(), stats.data_ptr(),
            g["dx"].data_ptr(), _ptr(dres), g["d_weight"].data_ptr(),
            g["d_bias"].data_ptr() if bias else None, ws.data_ptr(), ws.numel() * ws.element_size(),
            at.raw)
    if st:
        check(st, "ssd_norm_backward")
    return g


def gated_norm_forward(y, z, weight, eps: float = 1e-5, groups: int = 1, out=None, stream=None):
    """``y silu(z)`` normed by its root mean square in each of ``groups`` equal groups of the
    columns, times ``weight`` ``[D]``.  ``z`` ``[..., D]``; ``y`` the same, or with its columns
    as the scan leaves them, ``[..., H, P]`` with H P = D.  Returns ``(out, rstd)``: out in the
    shape of z, rstd float32 ``[rows, groups]`` for the backward."""
    dev, dt = z.device, z.dtype
    zs = _rows(z, "z")
    code, D = _code(z, "z"), z.shape[-1]
    ys = _columns(y, "y", z, dev, dt)
    wcode = _params(weight, None, dev, (D,))
    n = z.numel() // D if D else 0
    with _on(dev, stream) as at:
        o = _empty(z.shape, dtype=dt, device=dev) if out is None else out
        os = D if out is None else _rows(o, "out", dev, dt, z.shape)
        rstd = _empty((n, groups), dtype=torch.float32, device=dev)
        prob = GatedNormProblem(n, ys, zs, os, D, D, D, groups, code, wcode, eps)
        st = _lib.lib().ssd_gated_norm_forward(_byref(prob), y.data_ptr(), z.data_ptr(),
                                               weight.data_ptr(), o.data_ptr(), rstd.data_ptr(),
                                               at.raw)
    if st:
        check(st, "ssd_gated_norm_forward")
    return o, rstd


def _columns(y, name, z, dev, dt):
    """The row stride of y, of z's shape or contiguous with z's last dimension split in two."""
    if y.shape == z.shape:
        return _rows(y, name, dev, dt)
    if (y.dim() != z.dim() + 1 or y.shape[:-2] != z.shape[:-1] or
            y.shape[-2] * y.shape[-1] != z.shape[-1]):
        raise ValueError("%s must be [..., D] as z, or [..., H, P] with H P = D" % name)
    _check(y, name, dev, dt)
    return z.shape[-1]


def gated_norm_backward(dout, y, z, weight, rstd, groups: int = 1, out=None, workspace=None,
                        stream=None):
    """Backward of ``gated_norm_forward``.  Returns a dict ``dy`` (in the shape of y), ``dz``,
    ``d_weight``; ``out`` may bring any of them (dz may be strided, e.g. a slice of the
    in-projection's gradient)."""
    dev, dt = z.device, z.dtype
    zs = _rows(z, "z")
    code, D = _code(z, "z"), z.shape[-1]
    ys = _columns(y, "y", z, dev, dt)
    os = _rows(dout, "dout", dev, dt, z.shape)
    wcode = _params(weight, None, dev, (D,))
    n = z.numel() // D if D else 0
    _check(rstd, "rstd", dev, torch.float32, (n, groups))
    with _on(dev, stream) as at:
        g = {} if out is None else out
        if "dy" not in g:
            g["dy"] = _empty(y.shape, dtype=dt, device=dev)
        elif g["dy"].shape != y.shape:
            raise ValueError("dy must have the shape of y")
        if "dz" not in g:
            g["dz"] = _empty(z.shape, dtype=dt, device=dev)
        if "d_weight" not in g:
            g["d_weight"] = _empty((D,), dtype=weight.dtype, device=dev)
        _check(g["d_weight"], "d_weight", dev, weight.dtype, (D,))
        dys = _columns(g["dy"], "dy", z, dev, dt)
        dzs = _rows(g["dz"], "dz", dev, dt, z.shape)
        prob = GatedNormProblem(n, ys, zs, os, dys, dzs, D, groups, code, wcode, 0.0)
        ws = _scratch(_size("ssd_gated_norm_workspace_size", prob), dev, workspace)
        st = _lib.lib().ssd_gated_norm_backward(
            _byref(prob), dout.data_ptr(), y.data_ptr(), z.data_ptr(), weight.data_ptr(),
            rstd.data_ptr(), g["dy"].data_ptr(), g["dz"].data_ptr(), g["d_weight"].data_ptr(),
            ws.data_ptr(), ws.numel() * ws.element_size(), at.raw)
    if st:
        check(st, "ssd_gated_norm_backward")
    return g
