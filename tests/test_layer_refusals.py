"""What the operators around the scan refuse, before anything is launched: sizes, types,
strides, missing and overlapping buffers (host checks; no GPU needed)."""

import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from state_space_model_ssd_gb300 import build, _lib
    build.build()
    return _lib.lib()


def at(mb):
    """A distinct, aligned, never dereferenced address."""
    return ctypes.c_void_p(mb << 20)


def _conv(**kw):
    from state_space_model_ssd_gb300 import _lib
    p = dict(batch=1, seqlen=10, u_stride=32, du_stride=32, split=(16, 8, 8), width=4, nseq=0, dtype=1,
             wdtype=0, activation=1)
    p.update(kw)
    return _lib.ConvProblem(*p.values())


BAD_CONV = [(dict(batch=0), 1), (dict(seqlen=-1), 1), (dict(u_stride=31), 1), (dict(du_stride=31), 1),
            (dict(split=(0, 16, 16)), 1), (dict(split=(16, 0, 16)), 1), (dict(split=(40, -8, 0)), 1),
            (dict(width=0), 1), (dict(width=1), 2), (dict(width=5), 2), (dict(batch=2, nseq=2), 1),
            (dict(dtype=2), 1), (dict(wdtype=-1), 1), (dict(activation=2), 1), (dict(seqlen=1 << 31), 2),
            (dict(batch=1 << 20, seqlen=1 << 20), 2)]


@pytest.mark.parametrize("kw,code", BAD_CONV)
def test_conv_problem(lib, kw, code):
    p = _conv(**kw)
    n = ctypes.c_size_t()
    assert lib.ssd_conv_workspace_size(ctypes.byref(p), ctypes.byref(n)) == code
    assert lib.ssd_conv_forward(ctypes.byref(p), at(1), at(2), None, None, None, None, at(3), at(4), at(5),
                                None, None) == code


def test_conv_buffers(lib):
    p = _conv()

    def fwd(u=at(1), w=at(2), cu=None, init=None, o=(at(3), at(4), at(5)), final=None, prob=p):
        return lib.ssd_conv_forward(ctypes.byref(prob), u, w, None, cu, None, init, *o, final, None)

    assert fwd(u=None) == 1 and fwd(w=None) == 1 and fwd(o=(at(3), None, at(5))) == 1
    assert fwd(cu=at(6)) == 1                                  # lengths for a dense batch
    assert fwd(prob=_conv(nseq=2)) == 1                        # packed without lengths
    assert fwd(u=ctypes.c_void_p((1 << 20) + 1)) == 3
    assert fwd(o=(at(1), at(4), at(5))) == 1                   # output over the input
    assert fwd(o=(ctypes.c_void_p((1 << 20) + 16), at(4), at(5))) == 1
    assert fwd(init=at(7), final=at(7)) == 1                   # the state in place
    n = ctypes.c_size_t()
    assert lib.ssd_conv_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0 and n.value >= 256

    def bwd(ws=at(9), nbytes=n.value, du=at(8), dw=at(10), db=None, prob=p, u=at(1)):
        return lib.ssd_conv_backward(ctypes.byref(prob), u, at(2), None, None, None, None, at(3), at(4), at(5),
                                     None, du, dw, db, None, ws, nbytes, None)

    assert bwd(ws=None) == 4 and bwd(nbytes=n.value - 1) == 4
    assert bwd(ws=ctypes.c_void_p((9 << 20) + 16)) == 3
    assert bwd(du=None) == 1 and bwd(dw=None) == 1 and bwd(db=at(11)) == 1   # d_bias without a bias
    assert bwd(du=at(1)) == 1 and bwd(du=at(3)) == 1
    assert bwd(prob=_conv(du_stride=0)) == 1


def _step(**kw):
    from state_space_model_ssd_gb300 import _lib
    p = dict(batch=3, seqlen=1, nheads=4, headdim=16, dstate=16, ngroups=1, chunk_size=64, nseq=0,
             delta_init=-4.6, dtype=1)
    p.update(kw)
    return _lib.Problem(*p.values())


def test_step(lib):
    C = 4 * 16 + 2 * 16

    def step(prob=_step(), width=4, wdt=0, nslots=3, stride=C, state=at(1), win=at(2), u=at(3), slots=None,
             y=at(7), raw=at(4), pos=at(6)):
        return lib.ssd_conv_decode_step(ctypes.byref(prob), width, wdt, nslots, stride, state, win, u, raw,
                                        at(5), None, pos, slots, y, None)

    assert step(prob=_step(seqlen=2)) == 1 and step(prob=_step(nseq=1)) == 1
    assert step(prob=_step(ngroups=3)) == 1 and step(prob=_step(delta_init=float("inf"))) == 1
    assert step(prob=_step(headdim=12), stride=200) == 2 and step(prob=_step(dstate=256), stride=1000) == 2
    assert step(width=5) == 2 and step(width=0) == 1 and step(wdt=7) == 1
    assert step(nslots=2) == 1                    # fewer slots than rows, and no slot list
    assert step(nslots=0, slots=at(8)) == 1 and step(stride=C - 1) == 1
    assert step(state=None) == 1 and step(pos=None) == 1 and step(raw=None) == 1
    assert step(state=ctypes.c_void_p((1 << 20) + 8)) == 3
    assert step(win=at(1)) == 1 and step(y=at(1)) == 1 and step(y=at(2)) == 1 and step(y=at(3)) == 1
    assert step(prob=_step(batch=65536), nslots=65536) == 2


def _norm(**kw):
    from state_space_model_ssd_gb300 import _lib
    p = dict(rows=4, x_stride=64, r_stride=64, h_stride=64, y_stride=64, dim=64, kind=0, dtype=1, rdtype=0,
             wdtype=0, eps=1e-5)
    p.update(kw)
    return _lib.NormProblem(*p.values())


BAD_NORM = [(dict(rows=-1), 1), (dict(dim=0), 1), (dict(kind=2), 1), (dict(dtype=3), 1), (dict(rdtype=3), 1),
            (dict(dtype=0, rdtype=1), 2), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
            (dict(x_stride=63), 1), (dict(r_stride=1), 1), (dict(rows=1 << 31), 2),
            (dict(dim=16392, x_stride=16392, r_stride=16392, h_stride=16392, y_stride=16392), 2),
            (dict(dim=8193, x_stride=8193, r_stride=8193, h_stride=8193, y_stride=8193), 2)]


@pytest.mark.parametrize("kw,code", BAD_NORM)
def test_norm_problem(lib, kw, code):
    p = _norm(**kw)
    n = ctypes.c_size_t()
    assert lib.ssd_norm_workspace_size(ctypes.byref(p), ctypes.byref(n)) == code
    assert lib.ssd_norm_forward(ctypes.byref(p), at(1), at(2), at(3), None, at(4), at(5), None, None) == code


def test_norm_buffers(lib):
    p = _norm()

    def fwd(x=at(1), r=at(2), y=at(4), h=at(5), st=None):
        return lib.ssd_norm_forward(ctypes.byref(p), x, r, at(3), None, y, h, st, None)

    assert fwd(x=None) == 1 and fwd(h=None) == 1 and fwd(r=None) == 1
    assert fwd(y=at(2)) == 1 and fwd(h=at(1)) == 1 and fwd(y=at(5)) == 1
    assert fwd(y=ctypes.c_void_p((1 << 20) + 2)) == 1          # not the same rows: overlapping ones
    assert fwd(st=ctypes.c_void_p((6 << 20) + 4)) == 3
    n = ctypes.c_size_t()
    assert lib.ssd_norm_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0

    def bwd(dx=at(6), dres=None, dw=at(7), ws=at(8), nb=n.value, dh=at(5), stats=at(9)):
        return lib.ssd_norm_backward(ctypes.byref(p), at(1), at(2), dh, at(3), stats, dx, dres, dw, None, ws,
                                     nb, None)

    assert bwd(ws=None) == 4 and bwd(nb=0) == 4 and bwd(dw=None) == 1 and bwd(stats=None) == 1
    assert bwd(dx=at(2)) == 1 and bwd(dx=at(5)) == 1 and bwd(dres=at(6)) == 1 and bwd(dres=at(1)) == 1


def _gated(**kw):
    from state_space_model_ssd_gb300 import _lib
    p = dict(rows=4, y_stride=64, z_stride=64, out_stride=64, dy_stride=64, dz_stride=64, dim=64, groups=2,
             dtype=1, wdtype=0, eps=1e-5)
    p.update(kw)
    return _lib.GatedNormProblem(*p.values())


@pytest.mark.parametrize("kw,code", [(dict(rows=-1), 1), (dict(groups=3), 1), (dict(groups=0), 1),
                                     (dict(dim=0), 1), (dict(dtype=5), 1), (dict(z_stride=63), 1),
                                     (dict(dz_stride=0), 1), (dict(eps=-1.0), 1), (dict(rows=1 << 30), 2)])
def test_gated_problem(lib, kw, code):
    p = _gated(**kw)
    n = ctypes.c_size_t()
    assert lib.ssd_gated_norm_workspace_size(ctypes.byref(p), ctypes.byref(n)) == code
    assert lib.ssd_gated_norm_forward(ctypes.byref(p), at(1), at(2), at(3), at(4), None, None) == code


def test_gated_buffers(lib):
    p = _gated()
    n = ctypes.c_size_t()
    assert lib.ssd_gated_norm_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0

    def bwd(dy=at(5), dz=at(6), dw=at(7), ws=at(8), nb=n.value):
        return lib.ssd_gated_norm_backward(ctypes.byref(p), at(1), at(2), at(3), at(4), at(9), dy, dz, dw, ws,
                                           nb, None)

    assert bwd(dy=None) == 1 and bwd(dw=None) == 1 and bwd(ws=None) == 4 and bwd(nb=1) == 4
    assert bwd(dy=at(6)) == 1 and bwd(dy=ctypes.c_void_p((1 << 20) + 2)) == 1
    assert lib.ssd_gated_norm_forward(ctypes.byref(p), at(1), at(2), None, at(4), None, None) == 1
    assert lib.ssd_gated_norm_forward(ctypes.byref(p), at(1), at(2), at(3), ctypes.c_void_p((1 << 20) + 2),
                                      None, None) == 1


def test_binding_refuses(lib):
    import torch
    import state_space_model_ssd_gb300 as ssd
    u, w = torch.zeros(1, 4, 16), torch.zeros(16, 4)
    with pytest.raises(ValueError):
        ssd.conv_forward(u, w)
    with pytest.raises(ValueError):
        ssd.conv_forward(u, w, split=(8, 4))
    with pytest.raises(ValueError):
        ssd.conv_decode_step(torch.zeros(1, 1, 8, 8), torch.zeros(1, 4, 24), torch.zeros(1, 24),
                             torch.zeros(1, 1), torch.zeros(24, 4), None, torch.zeros(1), -4.6)
    with pytest.raises(ValueError):
        ssd.norm_forward(torch.zeros(2, 8), torch.ones(8))
    with pytest.raises(ValueError):
        ssd.gated_norm_forward(torch.zeros(2, 8), torch.zeros(2, 8), torch.ones(8))


# ------------------------------------------------------------------ outputs over other buffers
# Every output over every other output and every input of a call is refused, but for the places
# that an output may take.  Addresses a MB apart; an overlap starts 32 bytes before the end of the
# other buffer, so that its whole extent counts.  Nothing is launched: a call that is not refused
# would be, so that without a GPU it ends in another status.

def _inside(mb, nbytes):
    return ctypes.c_void_p((mb << 20) + nbytes - 32)


def _refused(call, outs, ins, allowed=()):
    """``call(**addresses)``; outs and ins: name -> (MB, bytes of the buffer)."""
    every = dict(outs, **ins)
    for o in outs:
        for other, (mb, n) in every.items():
            if o != other:
                assert call(**{o: _inside(mb, n)}) == 1, (o, other)
                if (o, other) not in allowed:
                    assert call(**{o: at(mb)}) == 1, (o, other)


def test_conv_outputs_over_anything(lib):
    p = _conv(nseq=2)
    T, K, srows = 10, 4, 2 * 4

    def fwd(u=at(1), w=at(2), b=at(3), cu=at(4), pos=at(5), init=at(6), o0=at(7), o1=at(8), o2=at(9), final=at(10)):
        return lib.ssd_conv_forward(ctypes.byref(p), u, w, b, cu, pos, init, o0, o1, o2, final, None)

    ins = {"u": (1, T * 32 * 2), "w": (2, 32 * K * 4), "b": (3, 32 * 4), "cu": (4, 32), "pos": (5, 32),
           "init": (6, srows * 32 * 2)}
    # the shortest buffers (12 and 8 bytes) are hit by their first byte alone
    outs = {"o0": (7, T * 16 * 2), "o1": (8, T * 8 * 2), "o2": (9, T * 8 * 2), "final": (10, srows * 32 * 2)}
    _refused(fwd, outs, ins)

    n = ctypes.c_size_t()
    assert lib.ssd_conv_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0

    def bwd(u=at(1), w=at(2), b=at(3), cu=at(4), pos=at(5), init=at(6), d0=at(7), d1=at(8), d2=at(9), df=at(10),
            du=at(11), dw=at(12), db=at(13), di=at(14), ws=at(15)):
        return lib.ssd_conv_backward(ctypes.byref(p), u, w, b, cu, pos, init, d0, d1, d2, df, du, dw, db, di, ws,
                                     n.value, None)

    ins.update(d0=(7, T * 16 * 2), d1=(8, T * 8 * 2), d2=(9, T * 8 * 2), df=(10, srows * 32 * 2))
    outs = {"du": (11, T * 32 * 2), "dw": (12, 32 * K * 4), "db": (13, 32 * 4), "di": (14, srows * 32 * 2)}
    _refused(bwd, outs, dict(ins, ws=(15, n.value)))


def test_step_outputs_over_anything(lib):
    prob, C, K, n = _step(), 4 * 16 + 2 * 16, 4, 3

    def step(state=at(1), win=at(2), u=at(3), raw=at(4), w=at(5), b=at(6), pos=at(7), slots=at(8), y=at(9)):
        return lib.ssd_conv_decode_step(ctypes.byref(prob), K, 0, n, C, state, win, u, raw, w, b, pos, slots, y,
                                        None)

    _refused(step, {"state": (1, n * 4 * 16 * 16 * 4), "win": (2, n * K * C * 2), "y": (9, n * 64 * 2)},
             {"u": (3, n * C * 2), "raw": (4, n * 4 * 4), "w": (5, C * K * 4), "b": (6, C * 4), "pos": (7, 32),
              "slots": (8, 32)})


def test_norm_outputs_over_anything(lib):
    p, R, D = _norm(), 4, 64

    def fwd(x=at(1), r=at(2), w=at(3), b=at(4), y=at(5), h=at(6), st=at(7)):
        return lib.ssd_norm_forward(ctypes.byref(p), x, r, w, b, y, h, st, None)

    _refused(fwd, {"y": (5, R * D * 2), "h": (6, R * D * 4), "st": (7, R * 8)},
             {"x": (1, R * D * 2), "r": (2, R * D * 4), "w": (3, D * 4), "b": (4, D * 4)},
             allowed=[("y", "x"), ("h", "r")])
    # taken places do not hide what lies over them
    assert fwd(y=at(1), st=at(1)) == 1 and fwd(h=at(2), st=at(2)) == 1 and fwd(y=at(1), h=at(1)) == 1
    n = ctypes.c_size_t()
    assert lib.ssd_norm_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0

    def bwd(dy=at(1), h=at(2), dh=at(3), w=at(4), st=at(5), dx=at(6), dr=at(7), dw=at(8), db=at(9), ws=at(10)):
        return lib.ssd_norm_backward(ctypes.byref(p), dy, h, dh, w, st, dx, dr, dw, db, ws, n.value, None)

    _refused(bwd, {"dx": (6, R * D * 2), "dr": (7, R * D * 4), "dw": (8, D * 4), "db": (9, D * 4)},
             {"dy": (1, R * D * 2), "h": (2, R * D * 4), "dh": (3, R * D * 4), "w": (4, D * 4), "st": (5, R * 8),
              "ws": (10, n.value)}, allowed=[("dx", "dy"), ("dr", "dh")])
    assert bwd(dx=at(1), dr=at(1)) == 1 and bwd(dx=at(1), dw=at(1)) == 1 and bwd(dr=at(3), dx=at(3)) == 1
    same = _norm(rdtype=1)
    p = same
    assert bwd(dx=at(3), dr=at(3)) == 1 and bwd(dx=at(3), db=at(3)) == 1


def test_gated_norm_outputs_over_anything(lib):
    p, R, D, G = _gated(), 4, 64, 2

    def fwd(y=at(1), z=at(2), w=at(3), out=at(4), rstd=at(5)):
        return lib.ssd_gated_norm_forward(ctypes.byref(p), y, z, w, out, rstd, None)

    _refused(fwd, {"out": (4, R * D * 2), "rstd": (5, R * G * 4)},
             {"y": (1, R * D * 2), "z": (2, R * D * 2), "w": (3, D * 4)}, allowed=[("out", "y"), ("out", "z")])
    assert fwd(out=at(1), rstd=at(1)) == 1
    n = ctypes.c_size_t()
    assert lib.ssd_gated_norm_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0

    def bwd(do=at(1), y=at(2), z=at(3), w=at(4), rstd=at(5), dy=at(6), dz=at(7), dw=at(8), ws=at(9)):
        return lib.ssd_gated_norm_backward(ctypes.byref(p), do, y, z, w, rstd, dy, dz, dw, ws, n.value, None)

    _refused(bwd, {"dy": (6, R * D * 2), "dz": (7, R * D * 2), "dw": (8, D * 4)},
             {"do": (1, R * D * 2), "y": (2, R * D * 2), "z": (3, R * D * 2), "w": (4, D * 4), "rstd": (5, R * G * 4),
              "ws": (9, n.value)}, allowed=[(o, i) for o in ("dy", "dz") for i in ("do", "y", "z")])
    assert bwd(dy=at(1), dz=at(1)) == 1 and bwd(dy=at(2), dw=at(2)) == 1
    # the workspace over an input or an output
    assert bwd(ws=at(6)) == 1 and bwd(ws=at(1)) == 1


def test_an_empty_buffer_lies_over_nothing(lib):
    """No token at all: u and du of no bytes inside another buffer are no overlap (without a GPU
    the call then ends for want of a device)."""
    p = _conv(seqlen=0)
    n = ctypes.c_size_t()
    assert lib.ssd_conv_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0
    inside = _inside(6, 4 * 32 * 2)
    import torch
    if torch.cuda.is_available():
        pytest.skip("would be launched")
    assert lib.ssd_conv_backward(ctypes.byref(p), inside, at(2), None, None, None, at(6), inside, inside, inside,
                                 None, inside, at(12), None, at(14), at(15), n.value, None) == 5
