"""The gated linear recurrence, the normalisation and rotation of queries and keys, and the state-space-dual step on
torch tensors (include/ssm_scan.h).

As in api.py nothing is computed here, but for the rotation frequencies (a table a model makes once). The checks, the
allocations and the call itself are native (csrc/ssm_marshal.cpp): for tensors of a few thousand elements the GPU's part
takes 2 to 10 us, and Python's would take longer. Every tensor of a call is on one CUDA device; the call runs on torch's
current stream of that device, which need not be the current device.
"""
from __future__ import annotations

import math
from typing import Optional, Tuple

import torch

from . import _abi
from .api import _DISC


# ---- gated linear recurrence -------------------------------------------------------------------


def ssm_lru_num_states(L: int) -> int:
    """Saved states per channel of a sequence of L steps (the last axis of chunk_states)."""
    return _abi.load().ssm_lru_num_states(L)


def ssm_lru_fwd(x, r, i, lam, r_bias=None, i_bias=None, c: float = 8.0, h0=None, reset=None, lengths=None,
                out_dtype=None, save_states: bool = False, return_state: bool = False,
                out: Optional[torch.Tensor] = None):
    """Gated linear recurrence h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t + i_bias) x_t with
    a_t = exp(-c softplus(lam) sigmoid(r_t + r_bias)). x, r, i: (Bt, Dn, L), fp32 or bf16, the gates before
    their sigmoids; lam, r_bias, i_bias: (Dn,) fp32; h0: (Bt, Dn) fp32. ``reset`` ((Bt, L) bool or uint8) marks
    the steps that start a new sequence, ``lengths`` ((Bt,) int32) the live steps of each batch element (behind
    them out is 0). Returns ``out`` (every h_t), or a dict with ``out`` and, when asked, ``chunk_states`` (for
    ssm_lru_bwd) and ``h_last`` ((Bt, Dn) fp32, the state after the last live step). ``out``: a tensor to write
    to, no input's memory."""
    return _abi.marshal().lru_fwd(x, r, i, lam, r_bias, i_bias, c, h0, reset, lengths, out_dtype, save_states, return_state,
                                  out)


def ssm_lru_bwd(dout, x, r, i, lam, r_bias=None, i_bias=None, c: float = 8.0, h0=None, reset=None, lengths=None,
                chunk_states=None, dh_last=None, grad_dtype=None, workspace: Optional[torch.Tensor] = None):
    """Backward of ssm_lru_fwd. ``dout``: (Bt, Dn, L) of x's dtype; ``dh_last``: (Bt, Dn) fp32, the gradient
    arriving at h_last; ``chunk_states`` as saved by the forward (recomputed when not given). Returns a dict: dx,
    dr, di in ``grad_dtype`` (fp32 unless given), and in fp32 dlam, dr_bias / di_bias where the bias exists, and
    dh0 where h0 or dh_last does. ``workspace``: an optional uint8 tensor to use as scratch."""
    return _abi.marshal().lru_bwd(dout, x, r, i, lam, r_bias, i_bias, c, h0, reset, lengths, chunk_states, dh_last,
                                  grad_dtype, workspace)


def ssm_lru_step(x, r, i, lam, h, r_bias=None, i_bias=None, c: float = 8.0, out_dtype=None,
                 out: Optional[torch.Tensor] = None):
    """One token of the gated linear recurrence. x, r, i: (Bt, Dn); h: (Bt, Dn) fp32, read and updated in place.
    Returns the output (Bt, Dn)."""
    return _abi.marshal().lru_step(x, r, i, lam, h, r_bias, i_bias, c, out_dtype, out)


# ---- queries and keys --------------------------------------------------------------------------


def ssm_rope_inv_freq(rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                      original_length: int = 4096, turns_low: float = 1.0, turns_high: float = 32.0,
                      device=None) -> Tuple[torch.Tensor, float]:
    """(inv_freq, rot_scale) for ssm_qk_norm_rope_fwd: rot / 2 angles per position, fp64, base^(-2 j / rot),
    for contexts ``factor`` times as long as the ``original_length`` a model was trained on:

    - "none": unchanged; "linear": every angle divided by factor (interpolated positions);
    - "ntk": a larger base, base factor^(rot / (rot - 2)), so that the slowest pair is divided by factor and the fastest
      is unchanged;
    - "yarn": pairs that make fewer than turns_low turns over original_length are divided by factor, those
      with more than turns_high are unchanged, linear in the turns between; rot_scale = 0.1 ln(factor) + 1.
    """
    if rot <= 0 or rot % 2:
        raise ValueError("rot must be a positive even number")
    if scaling not in ("none", "linear", "ntk", "yarn"):
        raise ValueError("scaling must be 'none', 'linear', 'ntk' or 'yarn'")
    if not (base > 0 and factor >= 1 and turns_high > turns_low and original_length > 0):
        raise ValueError("base and original_length must be positive, factor >= 1, turns_high > turns_low")
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = float(base) ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    scale = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        turns = f * (original_length / (2.0 * math.pi))
        keep = ((turns - turns_low) / (turns_high - turns_low)).clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / factor)
        scale = 0.1 * math.log(factor) + 1.0
    return (f if device is None else f.to(device)), scale


_LAYOUTS = {"blhd": _abi.SSM_QK_STATE_LAST, "bhdl": _abi.SSM_QK_TIME_LAST}


def _layout(name: str) -> int:
    code = _LAYOUTS.get(name)
    if code is None:
        raise ValueError("layout must be 'blhd' or 'bhdl'")
    return code


def ssm_qk_norm_rope_fwd(q, k=None, q_weight=None, k_weight=None, inv_freq=None, positions=None, pos0: int = 0,
                         norm: bool = True, eps: float = 1e-6, interleaved: bool = False, rot_scale: float = 1.0,
                         layout: str = "blhd", out_dtype=None, out: Optional[Tuple] = None):
    """Normalise every head of q and k by its root mean square (times ``q_weight`` / ``k_weight``, (D,) fp32) and
    rotate it by position, in one pass; ``norm=False`` rotates alone, no ``inv_freq`` normalises alone.

    q: (Bt, L, Hq, D), k: (Bt, L, Hk, D) or None, fp32 or bf16; with ``layout="bhdl"`` (Bt, H, D, L), time
    innermost as the selective scan's B and C are (C.unsqueeze(1) is one head). Any strides but a dense last axis:
    slices of one projection need no copy. ``inv_freq`` ((rot / 2,) fp32 or fp64, see ssm_rope_inv_freq): the
    first rot elements of a head turn by position * inv_freq[j] in pairs (j, j + rot / 2), or (2 j, 2 j + 1) with
    ``interleaved``; cosine and sine are multiplied by ``rot_scale``. An ``eps`` below 2^-126 counts as 2^-126. ``positions``:
    (Bt, L) int32 or int64, or None for pos0 + t. ``out``: (q_out, k_out) to write to, q and k themselves or no
    input's memory (None in a place: allocated). Returns (q_out, k_out)."""
    q_out, k_out = (None, None) if out is None else out
    return _abi.marshal().qk_fwd(q, k, q_weight, k_weight, inv_freq, positions, pos0, norm, eps, interleaved, rot_scale,
                                 _layout(layout), out_dtype, q_out, k_out)


def ssm_qk_norm_rope_bwd(dq_out, q, dk_out=None, k=None, q_weight=None, k_weight=None, inv_freq=None, positions=None,
                         pos0: int = 0, norm: bool = True, eps: float = 1e-6, interleaved: bool = False,
                         rot_scale: float = 1.0, layout: str = "blhd", grad_dtype=None,
                         workspace: Optional[torch.Tensor] = None):
    """Backward of ssm_qk_norm_rope_fwd: q, k and the options are the forward's, dq_out / dk_out the gradients of
    its outputs (fp32 or bf16, both alike). Returns a dict: dq (and dk with k) in ``grad_dtype`` (fp32 unless
    given), dq_weight / dk_weight (fp32) where the weight exists."""
    return _abi.marshal().qk_bwd(dq_out, dk_out, q, k, q_weight, k_weight, inv_freq, positions, pos0, norm, eps, interleaved,
                                 rot_scale, _layout(layout), grad_dtype, workspace)


# ---- state-space-dual step ---------------------------------------------------------------------


def ssm_ssd_step(x, dt, A_log, B, C, h, D=None, dt_bias=None, delta_softplus: bool = True, out_dtype=None,
                 discretization: str = "zoh", out: Optional[torch.Tensor] = None):
    """One token of the state-space dual (ssm_ssd_fwd). x: (Bt, H, P); dt: (Bt, H); B, C: (Bt, N) shared by the
    heads, all bf16 or all fp32; A_log, D, dt_bias: (H,) fp32; h: (Bt, H, N, P) fp32, read and updated in place
    (ssm_ssd_fwd's h_last continues here). P and N up to 256. Returns y (Bt, H, P)."""
    if discretization not in _DISC:
        raise ValueError("discretization must be 'zoh' or 'euler'")
    return _abi.marshal().ssd_step(x, dt, A_log, B, C, h, D, dt_bias, delta_softplus, out_dtype, _DISC[discretization], out)
