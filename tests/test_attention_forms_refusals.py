"""Alignments that linear attention's step takes and refuses (host checks)."""

import ctypes

from test_attention_refusals import _prob, at, lib  # noqa: F401  (lib is the built library)


def test_states_of_a_step(lib):  # noqa: F811
    def step(dstate, state):
        p = _prob(seqlen=1, dstate=dstate, q_stride=99, k_stride=99, v_stride=99, o_stride=99)
        # the outputs over the queries: refused, but behind the alignment
        return lib.ssd_linear_attention_step(ctypes.byref(p), 3, state, at(2), at(3), at(4), at(5), None, at(2), None)

    assert step(16, at(1, 8)) == 3 and step(16, at(1, 16)) == 1
    assert step(21, at(1, 2)) == 3 and step(21, at(1, 4)) == 1
