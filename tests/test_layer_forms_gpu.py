"""The operators around the scan on the GPU, through the C ABI and the binding: forms that the
wider tests do not reach."""

import ctypes

import numpy as np
import pytest

import layer_ref as ref
from test_layer_ops_gpu import _dev, _strided, ssd  # noqa: F401  (ssd is the built package)

pytestmark = pytest.mark.gpu


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# rows and widths that take each way a row comes in: bulk copies, single vectors, pairs, elements
@pytest.mark.parametrize("R,D", [(37, 2560), (300, 512), (9, 64), (21, 34), (50, 97)])
@pytest.mark.parametrize("with_dh", [False, True])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_backward_without_d_residual(ssd, R, D, with_dh, kind):  # noqa: F811
    """ssd_norm_backward with bf16 rows, a float32 h and no d_residual (the final norm of a network
    has neither the stream's gradient nor a use for its own): dx, d_weight and d_bias are those of
    the call that asks for it, and right."""
    import torch
    from state_space_model_ssd_gb300 import _lib
    rng = np.random.default_rng(R + D)
    dy, dy64 = _dev(rng.standard_normal((R, D)), "bf16")
    h, h64 = _dev(rng.standard_normal((R, D)) + 0.5, "f32")
    dh, dh64 = _dev(rng.standard_normal((R, D)), "f32") if with_dh else (None, None)
    w, w64 = _dev(1 + 0.2 * rng.standard_normal(D), "f32")
    layer = kind == "layer"
    _, _, st = ref.norm(h64, w64, None, None, 1e-5, layer)
    stats = torch.from_numpy(st.astype(np.float32)).cuda()
    p = _lib.NormProblem(R, D, D, D, D, D, 0 if layer else 1, 1, 0, 0, 1e-5)
    n = ctypes.c_size_t()
    assert _lib.lib().ssd_norm_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0
    ws = torch.empty(n.value, dtype=torch.uint8, device="cuda")

    def call(dres):
        dx, dw, db = torch.empty_like(dy), torch.empty_like(w), torch.empty_like(w)
        assert _lib.lib().ssd_norm_backward(
            ctypes.byref(p), _p(dy), _p(h), _p(dh), _p(w), _p(stats), _p(dx), _p(dres), _p(dw), _p(db), _p(ws),
            n.value, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
        return dx, dw, db

    dres = torch.empty_like(h)
    without, full = call(None), call(dres)
    for a, b in zip(without, full):
        assert bool((a == b).all())
    dv, dw, db = ref.norm_bwd(dy64, h64, w64, stats.double().cpu().numpy(), dh64, layer)
    ref.assert_close(without[0], dv, "bf16", "dx")
    ref.assert_close(dres, dv, "f32", "d_residual")
    ref.assert_close(without[1], dw, "f32", "d_weight")
    ref.assert_close(without[2], db, "f32", "d_bias")
    # the binding's form of it
    g = ssd.norm_backward(dy, h, w, stats, dh=dh, kind=kind)
    assert bool((g["dx"] == full[0]).all()) and bool((g["d_residual"] == dres).all())
