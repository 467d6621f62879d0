"""What linear attention and beam search refuse, before anything is launched (host checks)."""

import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from state_space_model_ssd_gb300 import build, _lib
    build.build()
    return _lib.lib()


def at(mb, off=0):
    """A distinct, aligned, never dereferenced address."""
    return ctypes.c_void_p((mb << 20) + off)


def _prob(**kw):
    from state_space_model_ssd_gb300 import _lib
    p = dict(batch=2, seqlen=8, q_stride=64, k_stride=32, v_stride=48, o_stride=96, dq_stride=64, dk_stride=32,
             dv_stride=48, nheads=4, ngroups=2, headdim=24, dstate=16, nseq=0, dtype=1, scale=0.25)
    p.update(kw)
    return _lib.LinAttnProblem(*p.values())


BAD = [(dict(batch=0), 1), (dict(seqlen=-1), 1), (dict(nheads=0), 1), (dict(ngroups=3), 1), (dict(ngroups=0), 1),
       (dict(headdim=0), 1), (dict(dstate=0), 1), (dict(nseq=-1), 1), (dict(nseq=2), 1), (dict(dtype=2), 1),
       (dict(scale=float("nan")), 1), (dict(q_stride=63), 1), (dict(k_stride=31), 1), (dict(v_stride=47), 1),
       (dict(o_stride=95), 1), (dict(headdim=129, v_stride=999, o_stride=999), 2),
       (dict(dstate=129, q_stride=999, k_stride=999), 2), (dict(seqlen=1 << 31), 2),
       (dict(batch=1 << 20, seqlen=1 << 20), 2)]


@pytest.mark.parametrize("kw,code", BAD)
def test_problem(lib, kw, code):
    n = ctypes.c_size_t()
    p = ctypes.byref(_prob(**kw))
    for bwd in (0, 1):
        assert lib.ssd_linear_attention_workspace_size(p, bwd, ctypes.byref(n)) == code
    assert lib.ssd_linear_attention_forward(p, at(1), at(2), at(3), at(4), None, None, at(5), None, at(6), 1 << 30,
                                            None) == code
    assert lib.ssd_linear_attention_backward(p, at(1), at(2), at(3), at(4), None, None, at(5), None, at(6), at(7),
                                             at(8), None, at(9), 1 << 30, None) == code


def test_forward_buffers(lib):
    def fwd(prob=_prob(), q=at(1), k=at(2), v=at(3), ld=at(4), cu=None, init=None, o=at(5), final=None, ws=at(6),
            n=1 << 30):
        return lib.ssd_linear_attention_forward(ctypes.byref(prob), q, k, v, ld, cu, init, o, final, ws, n, None)

    assert fwd(q=None) == 1 and fwd(k=None) == 1 and fwd(v=None) == 1 and fwd(ld=None) == 1 and fwd(o=None) == 1
    assert fwd(cu=at(7)) == 1 and fwd(prob=_prob(batch=1, nseq=2)) == 1
    assert fwd(q=at(1, 1)) == 3 and fwd(o=at(5, 1)) == 3 and fwd(init=at(7, 2)) == 3 and fwd(ld=at(4, 2)) == 3
    assert fwd(ws=at(6, 16)) == 3
    for x in (at(1), at(2), at(3), at(4)):
        assert fwd(o=x) == 1 and fwd(final=x) == 1
    assert fwd(final=at(5)) == 1 and fwd(init=at(7), final=at(7)) == 1 and fwd(init=at(5)) == 1
    # a long sequence needs a workspace, which counts as an output
    long = _prob(batch=1, seqlen=100000, nseq=2)
    size = ctypes.c_size_t()
    assert lib.ssd_linear_attention_workspace_size(ctypes.byref(long), 0, ctypes.byref(size)) == 0 and size.value
    assert fwd(prob=long, ws=None, cu=at(7)) == 4 and fwd(prob=long, n=size.value - 1, cu=at(7)) == 4
    far = dict(cu=at(7), q=at(100), k=at(200), v=at(300), o=at(400), ws=at(500))
    for x in ("q", "k", "v", "o"):
        assert fwd(prob=long, **{**far, "ws": far[x]}) == 1


def test_backward_buffers(lib):
    def bwd(prob=_prob(), q=at(1), k=at(2), v=at(3), ld=at(4), cu=None, init=None, do=at(5), dfinal=None, dq=at(6),
            dk=at(7), dv=at(8), d0=None, ws=at(900), n=1 << 30):
        return lib.ssd_linear_attention_backward(ctypes.byref(prob), q, k, v, ld, cu, init, do, dfinal, dq, dk, dv,
                                                 d0, ws, n, None)

    for x in ("q", "k", "v", "ld", "do", "dq", "dk", "dv"):
        assert bwd(**{x: None}) == 1, x
    assert bwd(prob=_prob(dq_stride=0)) == 1 and bwd(prob=_prob(dk_stride=31)) == 1
    assert bwd(prob=_prob(dv_stride=0)) == 1
    assert bwd(ws=None) == 4 and bwd(n=100) == 4 and bwd(ws=at(900, 16)) == 3     # shared heads: parts
    for out in ("dq", "dk", "dv", "d0"):
        for x in (at(1), at(2), at(3), at(4), at(5)):
            assert bwd(**{out: x}) == 1
        assert bwd(**{out: at(9), "init": at(9)}) == 1 and bwd(**{out: at(9), "dfinal": at(9)}) == 1
        assert bwd(**{out: at(900)}) == 1
    assert bwd(dq=at(7)) == 1 and bwd(dk=at(8)) == 1 and bwd(d0=at(6)) == 1
    assert bwd(dv=at(8, 1)) == 3 and bwd(d0=at(9, 2)) == 3


def test_slices_of_one_projection(lib):
    """Gradients that lie between one another's tokens are no overlap; those that do overlap are."""
    w = 64 + 32 + 48
    p = _prob(seqlen=0, dq_stride=w, dk_stride=w, dv_stride=w)
    p8 = _prob(dq_stride=w, dk_stride=w, dv_stride=w)

    def bwd(prob, dk, dv, dq=at(6), ws=None):
        return lib.ssd_linear_attention_backward(ctypes.byref(prob), at(1), at(2), at(3), at(4), None, None, at(5),
                                                 None, dq, dk, dv, None, ws, 0, None)

    # the workspace is looked at before the overlaps: without one the sound call ends there
    assert bwd(p8, at(6, 128), at(6, 192)) == 4
    n = 1 << 30
    for dk, dv in ((at(6, 126), at(6, 192)), (at(6, 128), at(6, 190)), (at(6, 128), at(6, 194))):
        assert lib.ssd_linear_attention_backward(ctypes.byref(p8), at(1), at(2), at(3), at(4), None, None, at(5),
                                                 None, at(6), dk, dv, None, at(900), n, None) == 1
    assert p.seqlen == 0


def test_step(lib):
    def step(prob=None, nslots=3, state=at(1), q=at(2), k=at(3), v=at(4), ld=at(5), slots=None, o=at(6), **kw):
        p = prob or _prob(**{**dict(seqlen=1), **kw})
        return lib.ssd_linear_attention_step(ctypes.byref(p), nslots, state, q, k, v, ld, slots, o, None)

    assert step(seqlen=2) == 1 and step(batch=1, nseq=1) == 1 and step(batch=0) == 1 and step(ngroups=3) == 1
    assert step(scale=float("inf")) == 1 and step(dtype=5) == 1 and step(nslots=0, slots=at(7)) == 1
    assert step(nslots=1) == 1                       # fewer slots than rows, and no slot list
    assert step(headdim=200, v_stride=999, o_stride=999) == 2 and step(batch=65536, nslots=65536) == 2
    assert step(q_stride=3) == 1 and step(o_stride=3) == 1
    for x in ("state", "q", "k", "v", "ld", "o"):
        assert step(**{x: None}) == 1, x
    assert step(state=at(1, 8)) == 3 and step(o=at(6, 1)) == 3 and step(slots=at(7, 2)) == 3
    for x in (at(1), at(2), at(3), at(4), at(5)):
        assert step(o=x) == 1
    assert step(state=at(2)) == 1 and step(slots=at(1)) == 1 and step(slots=at(6)) == 1


def _beam(**kw):
    from state_space_model_ssd_gb300 import _lib
    p = dict(batch=3, stride=100, beams=4, vocab=100, keep=8, pad_token=0, dtype=0)
    p.update(kw)
    return _lib.BeamProblem(*p.values())


BAD_BEAM = [(dict(batch=0), 1), (dict(stride=99), 1), (dict(beams=0), 1), (dict(vocab=0), 1), (dict(keep=0), 1),
            (dict(vocab=1, keep=5, stride=1), 1), (dict(pad_token=100), 1), (dict(pad_token=-1), 1), (dict(dtype=3), 1),
            (dict(beams=65), 2), (dict(keep=65), 2), (dict(vocab=(1 << 24) + 1, stride=1 << 25), 2),
            (dict(batch=20000), 2)]


@pytest.mark.parametrize("kw,code", BAD_BEAM)
def test_beam_problem(lib, kw, code):
    n = ctypes.c_size_t()
    p = ctypes.byref(_beam(**kw))
    assert lib.ssd_beam_select_workspace_size(p, ctypes.byref(n)) == code
    assert lib.ssd_beam_select(p, at(1), at(2), None, at(3), at(4), at(5), at(6), 1 << 30, None) == code


def test_beam_select_buffers(lib):
    n = ctypes.c_size_t()
    assert lib.ssd_beam_select_workspace_size(ctypes.byref(_beam()), ctypes.byref(n)) == 0

    def select(x=at(1), scores=at(2), finished=None, out=at(3), parents=at(4), tokens=at(5), ws=at(6), size=n.value):
        return lib.ssd_beam_select(ctypes.byref(_beam()), x, scores, finished, out, parents, tokens, ws, size, None)

    for x in ("x", "scores", "out", "parents", "tokens"):
        assert select(**{x: None}) == 1, x
    assert select(ws=None) == 4 and select(size=n.value - 1) == 4 and select(ws=at(6, 16)) == 3
    assert select(x=at(1, 2)) == 3 and select(tokens=at(5, 2)) == 3
    for o in ("out", "parents", "tokens", "ws"):
        assert select(**{o: at(1)}) == 1 and select(**{o: at(2)}) == 1 and select(**{o: at(7), "finished": at(7)}) == 1
    assert select(out=at(4)) == 1 and select(parents=at(5)) == 1 and select(tokens=at(6)) == 1


def test_beam_reorder(lib):
    def call(batch=2, beams=4, slots=at(1), parents=at(2), new=at(3), caches=(at(4), at(5)), nbytes=(64, 32),
             strides=(64, 48), nslots=8, n=None):
        m = len(caches)
        c = (ctypes.c_void_p * m)(*[x.value if x else None for x in caches])
        b, s = (ctypes.c_int64 * m)(*nbytes), (ctypes.c_int64 * m)(*strides)
        return lib.ssd_beam_reorder(batch, beams, slots, parents, new, m if n is None else n, c, b, s, nslots, None)

    assert call(batch=0) == 1 and call(beams=0) == 1 and call(nslots=0) == 1 and call(n=-1) == 1
    assert call(beams=65) == 2 and call(batch=65536) == 2
    for x in ("slots", "parents", "new"):
        assert call(**{x: None}) == 1
        assert call(**{x: at(7, 2)}) == 3
        assert call(**{x: at(4)}) == 1 and call(**{x: at(5, 48 * 7)}) == 1      # inside a cache
    assert call(caches=(at(4), None)) == 1 and call(nbytes=(-1, 32)) == 1 and call(strides=(64, 31)) == 1
    assert call(new=at(1)) == 1 and call(new=at(2)) == 1                        # slots in place


def test_python_binding_refuses(lib):
    import torch
    import state_space_model_ssd_gb300 as ssd
    z = torch.zeros
    with pytest.raises(ValueError, match="CUDA"):
        ssd.linear_attention_forward(z(1, 2, 1, 4), z(1, 2, 1, 4), z(1, 2, 1, 4), z(1))
    with pytest.raises(ValueError, match="CUDA"):
        ssd.linear_attention_backward(z(1, 2, 1, 4), z(1, 2, 1, 4), z(1, 2, 1, 4), z(1), z(1, 2, 1, 4))
    with pytest.raises(ValueError, match="CUDA"):
        ssd.linear_attention_step(z(1, 1, 4, 4), z(1, 1, 4), z(1, 1, 4), z(1, 1, 4), z(1))
    with pytest.raises(ValueError, match="CUDA"):
        ssd.beam_select(z(1, 2, 4), z(1, 2))
    with pytest.raises(ValueError, match="CUDA"):
        ssd.beam_reorder([], z(1, 2, dtype=torch.int32), z(1, 2, dtype=torch.int32))
    with pytest.raises(TypeError):
        ssd.beam_select(None, z(1, 2))
