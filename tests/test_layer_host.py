"""Host code of the operators around the scan that needs no GPU."""

import contextlib

import pytest


@pytest.fixture(scope="module")
def layer():
    from state_space_model_ssd_gb300 import build
    build.build()
    from state_space_model_ssd_gb300 import layer as m
    return m


def test_status_is_read_on_the_device_of_the_stream(layer, monkeypatch):
    """ssd_layer_status reads and clears the current device's word: that of the stream given."""
    import torch
    from state_space_model_ssd_gb300 import _lib
    words, current, reads = {0: 0, 1: 5}, [0], []

    class Lib:
        def ssd_layer_status(self, stream, out):
            reads.append((stream.value, current[0]))
            out._obj.value = words[current[0]]
            words[current[0]] = 0
            return 0

    @contextlib.contextmanager
    def device(d):
        before = current[0]
        current[0] = torch.device(d).index
        try:
            yield
        finally:
            current[0] = before

    class Stream:
        def __init__(self, index):
            self.device = torch.device("cuda", index)
            self.cuda_stream = 100 + index

    monkeypatch.setattr(_lib, "lib", lambda: Lib())
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream(current[0]))
    assert layer.layer_status() == 0
    assert words[1] == 5                              # the other device's word still stands
    assert layer.layer_status(stream=Stream(1)) == 5  # and is that of its own streams
    assert layer.layer_status(stream=Stream(1)) == 0
    assert reads == [(100, 0), (101, 1), (101, 1)] and current == [0]


def _python(code):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    return subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)


def test_package_names_need_neither_torch_nor_the_binding(layer):
    """``from state_space_model_ssd_gb300 import *`` needs what a call of the scan's C library needs;
    torch and the binding are looked for by the first call that takes tensors."""
    r = _python("""
import sys
sys.modules["torch"] = None
from state_space_model_ssd_gb300 import *
import state_space_model_ssd_gb300 as ssd
assert all(callable(globals()[n]) for n in ssd.__all__)
try:
    norm_forward(None, None)
except ImportError:
    print("torch is missing")
""")
    assert r.returncode == 0 and r.stdout == "torch is missing\n", r.stderr
    r = _python("""
import os
exists = os.path.exists
os.path.exists = lambda p: exists(p) and not str(p).endswith("_layer_ext.so")
from state_space_model_ssd_gb300 import *
for call in (lambda: norm_forward(None, None), lambda: conv_decode_step(*[None] * 8)):
    try:
        call()
    except RuntimeError as e:
        assert "not built" in str(e)
        print("not built")
""")
    assert r.returncode == 0 and r.stdout == "not built\n" * 2, r.stderr


@pytest.fixture(scope="module")
def ring(tmp_path_factory):
    """csrc/layer_ring.cuh, compiled for the host."""
    import ctypes
    import subprocess
    from state_space_model_ssd_gb300 import build
    d = tmp_path_factory.mktemp("ring")
    src, so = str(d / "ring.cpp"), str(d / "ring.so")
    with open(src, "w") as f:
        f.write('#include "layer_ring.cuh"\n'
                'extern "C" unsigned landed_parity(int p, int n, int s, unsigned q, int u) {\n'
                '    return ssd::layer::landed_parity(p, n, s, q, u);\n}\n')
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", build.CSRC, src, "-o", so], check=True)
    return ctypes.CDLL(so)


def test_a_thread_that_gave_up_waits_for_every_copy_on_its_way(ring):
    """A ring of barriers whose phase with parity q counts as complete once the barrier has left it.
    At every row whose wait can run out, the thread issues no more, walks on to its last row, and
    then waits: at each place, for the phase that is incomplete until its copy lands; at places
    without a copy on its way, for one that is complete."""
    for places in range(1, 9):
        for rows in range(1, 4 * places + 2):
            for row in range(rows):  # the wait for it runs out; the copies before it have landed
                sent = min(places + row, rows)
                issued = [len(range(p, sent, places)) for p in range(places)]
                landed = [len(range(p, row, places)) for p in range(places)]
                stage, parity = rows % places, rows // places & 1  # after the last row
                for p in range(places):
                    q = ring.landed_parity(p, places, stage, parity, rows - sent)
                    late = issued[p] - landed[p]
                    assert late in (0, 1)
                    assert ((landed[p] & 1) == q) == (late == 1), (places, rows, row, p)
                    assert issued[p] & 1 != q         # passes once every copy has landed
