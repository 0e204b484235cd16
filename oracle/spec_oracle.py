"""Float64 CPU oracle for the speculative decoding step over the paged latent cache.

TEST INFRASTRUCTURE ONLY, like ``mla_oracle``: plain definitions in float64 NumPy, no
code shared with the CUDA path.
"""
from __future__ import annotations

import numpy as np


# ---------------------------------------------------------------------------
# Row append: norms, rotation
# ---------------------------------------------------------------------------
def rms_norm_ref(x: np.ndarray, weight, eps: float) -> np.ndarray:
    """x / sqrt(mean(x^2) + eps) * weight over the last axis; weight None leaves x as it is."""
    if weight is None:
        return x
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * weight


def rotate_ref(x: np.ndarray, cos_sin: np.ndarray, interleaved: bool) -> np.ndarray:
    """Pairs (2k, 2k+1), or (k, k+32), of the last 64 values as complex numbers times e^{i angle}.

    ``cos_sin`` [..., 64] (cos | sin) broadcasts against x [..., 64].
    """
    turn = cos_sin[..., :32] + 1j * cos_sin[..., 32:]
    z = (x[..., 0::2] + 1j * x[..., 1::2] if interleaved else x[..., :32] + 1j * x[..., 32:]) * turn
    out = np.empty(z.shape[:-1] + (64,))
    if interleaved:
        out[..., 0::2], out[..., 1::2] = z.real, z.imag
    else:
        out[..., :32], out[..., 32:] = z.real, z.imag
    return out


def rope_append_ref(q, kv, q_weight, kv_weight, eps, cos_sin, positions, interleaved):
    """(q_nope [N,H,128], q_pe [N,H,64], rows [N,576]) of N new tokens; q [N,H,192], kv [N,576]."""
    cs = cos_sin[positions]
    q = rms_norm_ref(q, q_weight, eps)
    rows = np.concatenate([rms_norm_ref(kv[:, :512], kv_weight, eps), rotate_ref(kv[:, 512:], cs, interleaved)], -1)
    return q[..., :128], rotate_ref(q[..., 128:], cs[:, None], interleaved), rows
