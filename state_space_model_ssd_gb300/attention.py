"""Linear attention with a decay for each head, over libssd.so: a layer's mixer that keeps, like
the scan, a state ``[H, P, N]`` for each sequence,

    S_t = exp(log_decay[h]) S_{t-1} + v_t k_t^T,    o_t = scale S_t q_t,

in its chunked form for prompts and training, and one token at a time over cache slots:

    o, state = linear_attention_forward(q, k, v, log_decay, final_state=True)
    grads = linear_attention_backward(q, k, v, log_decay, do)
    o_t = linear_attention_step(state, q_t, k_t, v_t, log_decay, slots=slots)

q ``[batch, L, H, N]``, k ``[batch, L, G, N]`` and v ``[batch, L, G, P]`` are float32 or bfloat16
CUDA tensors, N and P up to 128; query heads share k and v in runs of H / G and have a state
each.  Tokens may be strided (slices of one projection's rows), their heads next to one another.
``log_decay`` float32 ``[H]``, zero or negative; it takes no gradient.  ``scale``: default
``N ** -0.5``.  With ``stream`` the call runs there, and what it allocates belongs to that stream.
"""

from __future__ import annotations

from . import layer
from .layer import _on

__all__ = ["linear_attention_forward", "linear_attention_backward", "linear_attention_step"]


def linear_attention_forward(q, k, v, log_decay, scale=None, cu_seqlens=None, initial_state=None,
                             final_state: bool = False, out=None, final_state_out=None, workspace=None,
                             stream=None):
    """``cu_seqlens`` (int32 ``[nseq + 1]``, batch 1) packs sequences; outputs (and gradients) of
    tokens before the first one or behind the last one are zero.  ``initial_state`` float32
    ``[nseq or batch, H, P, N]`` is what each sequence goes on from.  Returns
    ``(o, final_state or None)``: o ``[batch, L, H, P]`` in the type of q, the final states as the
    initial ones.

    bfloat16 calls with N and P 64 or 128, every row on 16 bytes, run on the tensor cores in blocks
    of 128 tokens: a NaN or an infinity in a token then reaches the outputs of all tokens of its
    sequence in its block.  The states are float32; where one meets q it is rounded to bfloat16, and
    so are the masked products of q and k, except of sequences within a block or in calls too small
    to fill the GPU, where two bfloat16 terms hold them.  bfloat16 calls of other sizes, or with rows
    off 16 bytes, take that way too, by copies in the workspace, from 16384 rows (of a head and
    token) on, unless they are so narrow that the copies were over four times as wide (or tensors do
    not start on 16 bytes and ``workspace`` is too small for copies).  Forwards of up to 16 tokens a
    sequence (a batch row, or all packed ones) are stepped through, and all other calls run on the
    plain cores, in float32."""
    args = (q, k, v, log_decay, scale, cu_seqlens, initial_state, final_state, out, final_state_out, workspace)
    return (layer._ext.linear_attention_forward(*args) if stream is None
            else _on(stream, layer._ext.linear_attention_forward, *args))


def linear_attention_backward(q, k, v, log_decay, do, scale=None, cu_seqlens=None, initial_state=None,
                              d_final_state=None, d_initial_state: bool = False, out=None,
                              workspace=None, stream=None):
    """Backward of ``linear_attention_forward`` for the gradient ``do`` of o and (optional)
    ``d_final_state`` of the final states.  Returns a dict ``dq, dk, dv`` and, with
    ``d_initial_state``, that too; ``out`` may bring any of them, and what it brings is written
    (tokens may be strided, e.g. slices of the projection's gradient).  Gradients of shared k and v
    are summed over their heads.  The same inputs give the same bits in every call."""
    args = (q, k, v, log_decay, do, scale, cu_seqlens, initial_state, d_final_state, d_initial_state, out,
            workspace)
    return (layer._ext.linear_attention_backward(*args) if stream is None
            else _on(stream, layer._ext.linear_attention_backward, *args))


def linear_attention_step(state, q, k, v, log_decay, scale=None, slots=None, out=None, stream=None):
    """One token for each row of a batch: q ``[batch, H, N]``, k ``[batch, G, N]``, v
    ``[batch, G, P]``.  ``state`` float32 ``[nslots, H, P, N]`` (on 16 bytes where N is a multiple of
    4) is updated in place.  ``slots``
    int32 ``[batch]``: each row's cache slot (default: its index; the live rows' must differ); a
    row whose slot is negative or beyond the cache is padding, its output zero.  Returns o
    ``[batch, H, P]``."""
    args = (state, q, k, v, log_decay, scale, slots, out)
    return (layer._ext.linear_attention_step(*args) if stream is None
            else _on(stream, layer._ext.linear_attention_step, *args))
