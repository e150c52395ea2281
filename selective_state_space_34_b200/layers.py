"""PyTorch-facing marshalling of the gated linear recurrence, of the normalisation and rotation of
queries and keys, and of the state-space-dual step (include/ssm_scan.h).

As in api.py nothing is computed here, but for the rotation frequencies (a table a model makes once). Every
tensor of a call is on one CUDA device; the call runs on torch's current stream of that device, which need not be
the current device. Outputs and scratch are allocated with torch on that stream.
"""
from __future__ import annotations

import ctypes
import math
from typing import Dict, Optional, Tuple

import torch

from . import _abi
from .api import _DISC, _DT

_byref = ctypes.byref
_F32 = torch.float32


# The checks read each tensor once, in the order of the common mistakes' absence: a call of these operators can be
# shorter on the GPU than its checks are on the host.


def _first(name: str, t) -> Tuple[torch.dtype, int]:
    """(dtype, device index) of the call's leading tensor."""
    try:
        dev, dtype = t.get_device(), t.dtype
    except AttributeError:
        raise TypeError("%s must be a torch.Tensor" % name) from None
    if dev < 0:
        raise ValueError("%s must be a CUDA tensor (the library has no CPU path)" % name)
    if dtype not in _DT:
        raise TypeError("%s must be float32 or bfloat16" % name)
    return dtype, dev


def _refuse(name, t, dev, dtype, shape, dense=True):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.get_device() != dev:
        raise ValueError("%s must be a CUDA tensor on cuda:%d, got %s" % (name, dev, t.device))
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    raise ValueError("%s must be contiguous%s" % (name, "" if dense else " along its last axis"))


def _need(name, t, dev, dtype, shape) -> int:
    """The address of a dense tensor of this dtype and shape on device ``dev``."""
    try:
        if t.get_device() == dev and t.dtype is dtype and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(name, t, dev, dtype, shape)


def _maybe(name, t, dev, dtype, shape) -> Optional[int]:
    return None if t is None else _need(name, t, dev, dtype, shape)


def _out_type(name, dtype, default):
    if dtype is None:
        return default
    if dtype not in _DT:
        raise TypeError("%s must be float32 or bfloat16" % name)
    return dtype


def _like(t, dtype):
    """An uninitialised dense tensor of t's shape and device."""
    if t.dtype is dtype:
        return torch.empty_like(t, memory_format=torch.contiguous_format)
    return torch.empty_like(t, dtype=dtype, memory_format=torch.contiguous_format)


def _call(name: str, args, dev: int) -> None:
    """Run an entry point on the current stream of device ``dev``, which need not be the current device."""
    fn = getattr(_abi.load(), name)
    stream = torch._C._cuda_getCurrentRawStream(dev)
    if torch._C._cuda_getDevice() == dev:
        code = fn(_byref(args), stream)
    else:
        with torch.cuda.device(dev):
            code = fn(_byref(args), stream)
    if code:
        _abi.check(name, code)


def _scratch(need: int, dev: int, workspace: Optional[torch.Tensor]):
    """(tensor to hold on to, its first 256-byte boundary): the caller's workspace when that is large enough."""
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor on cuda:%d" % dev)
        base = workspace.data_ptr()
        at = (base + 255) & ~255
        if at + need <= base + workspace.numel() * workspace.element_size():
            return workspace, at
    ws = torch.empty(need + 256, dtype=torch.uint8, device=torch.device("cuda", dev))
    return ws, (ws.data_ptr() + 255) & ~255


# ---- gated linear recurrence -------------------------------------------------------------------


def ssm_lru_num_states(L: int) -> int:
    """Saved states per channel of a sequence of L steps (the last axis of chunk_states)."""
    return _abi.load().ssm_lru_num_states(L)


def _lru_args(a, x, r, i, lam, r_bias, i_bias, c, h0, reset, lengths):
    act, dev = _first("x", x)
    shape = x.shape
    if len(shape) != 3:
        raise ValueError("x must be (Bt, Dn, L)")
    Bt, Dn, L = shape
    of_dn = (Dn,)
    a.x = _need("x", x, dev, act, shape)
    a.r = _need("r", r, dev, act, shape)
    a.i = _need("i", i, dev, act, shape)
    a.lam = _need("lam", lam, dev, _F32, of_dn)
    if r_bias is not None:
        a.r_bias = _need("r_bias", r_bias, dev, _F32, of_dn)
    if i_bias is not None:
        a.i_bias = _need("i_bias", i_bias, dev, _F32, of_dn)
    if h0 is not None:
        a.h0 = _need("h0", h0, dev, _F32, (Bt, Dn))
    if reset is not None:
        dtype = getattr(reset, "dtype", torch.bool)
        if dtype not in (torch.bool, torch.uint8):
            raise TypeError("reset must be bool or uint8")
        a.reset = _need("reset", reset, dev, dtype, (Bt, L))
    if lengths is not None:
        a.lengths = _need("lengths", lengths, dev, torch.int32, (Bt,))
    a.Bt, a.Dn, a.L, a.c = Bt, Dn, L, c
    a.in_dtype = _DT[act]
    return act, dev, Bt, Dn, L


def ssm_lru_fwd(x, r, i, lam, r_bias=None, i_bias=None, c: float = 8.0, h0=None, reset=None, lengths=None,
                out_dtype=None, save_states: bool = False, return_state: bool = False,
                out: Optional[torch.Tensor] = None):
    """Gated linear recurrence h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t + i_bias) x_t with
    a_t = exp(-c softplus(lam) sigmoid(r_t + r_bias)). x, r, i: (Bt, Dn, L), fp32 or bf16, the gates before
    their sigmoids; lam, r_bias, i_bias: (Dn,) fp32; h0: (Bt, Dn) fp32. ``reset`` ((Bt, L) bool or uint8) marks
    the steps that start a new sequence, ``lengths`` ((Bt,) int32) the live steps of each batch element (behind
    them out is 0). Returns ``out`` (every h_t), or a dict with ``out`` and, when asked, ``chunk_states`` (for
    ssm_lru_bwd) and ``h_last`` ((Bt, Dn) fp32, the state after the last live step)."""
    a = _abi.LruArgs()
    act, dev, Bt, Dn, L = _lru_args(a, x, r, i, lam, r_bias, i_bias, c, h0, reset, lengths)
    od = _out_type("out_dtype", out_dtype, act)
    if out is None:
        out = _like(x, od)
        a.out = out.data_ptr()
    else:
        a.out = _need("out", out, dev, od, x.shape)
    a.out_dtype = _DT[od]
    res: Dict[str, torch.Tensor] = {"out": out}
    if save_states:
        st = res["chunk_states"] = torch.empty((Bt, Dn, ssm_lru_num_states(L)), dtype=_F32, device=x.device)
        a.chunk_states = st.data_ptr()
    if return_state:
        hl = res["h_last"] = torch.empty((Bt, Dn), dtype=_F32, device=x.device)
        a.h_last = hl.data_ptr()
    _call("ssm_lru_fwd", a, dev)
    return res if (save_states or return_state) else out


def ssm_lru_bwd(dout, x, r, i, lam, r_bias=None, i_bias=None, c: float = 8.0, h0=None, reset=None, lengths=None,
                chunk_states=None, dh_last=None, grad_dtype=None, workspace: Optional[torch.Tensor] = None):
    """Backward of ssm_lru_fwd. ``dout``: (Bt, Dn, L) of x's dtype; ``dh_last``: (Bt, Dn) fp32, the gradient
    arriving at h_last; ``chunk_states`` as saved by the forward (recomputed when not given). Returns a dict: dx,
    dr, di in ``grad_dtype`` (fp32 unless given), and in fp32 dlam, dr_bias / di_bias where the bias exists, and
    dh0 where h0 or dh_last does. ``workspace``: an optional uint8 tensor to use as scratch."""
    bw = _abi.LruBwdArgs()
    a = bw.fwd
    act, dev, Bt, Dn, L = _lru_args(a, x, r, i, lam, r_bias, i_bias, c, h0, reset, lengths)
    bw.dout = _need("dout", dout, dev, act, x.shape)
    if chunk_states is not None:
        a.chunk_states = _need("chunk_states", chunk_states, dev, _F32, (Bt, Dn, ssm_lru_num_states(L)))
    if dh_last is not None:
        bw.dh_last = _need("dh_last", dh_last, dev, _F32, (Bt, Dn))
    gd = _out_type("grad_dtype", grad_dtype, _F32)
    bw.grad_dtype = _DT[gd]
    grads = {"dx": _like(x, gd), "dr": _like(x, gd), "di": _like(x, gd), "dlam": _like(lam, _F32)}
    if r_bias is not None:
        grads["dr_bias"] = _like(lam, _F32)
    if i_bias is not None:
        grads["di_bias"] = _like(lam, _F32)
    if h0 is not None or dh_last is not None:
        grads["dh0"] = torch.empty((Bt, Dn), dtype=_F32, device=x.device)
    for n, g in grads.items():
        setattr(bw, n, g.data_ptr())
    need = _abi.load().ssm_lru_bwd_workspace_size(_byref(bw))
    if need:
        ws, bw.workspace = _scratch(need, dev, workspace)
        bw.workspace_bytes = need
    _call("ssm_lru_bwd", bw, dev)
    return grads


def ssm_lru_step(x, r, i, lam, h, r_bias=None, i_bias=None, c: float = 8.0, out_dtype=None,
                 out: Optional[torch.Tensor] = None):
    """One token of the gated linear recurrence. x, r, i: (Bt, Dn); h: (Bt, Dn) fp32, read and updated in place.
    Returns the output (Bt, Dn)."""
    act, dev = _first("x", x)
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("x must be (Bt, Dn)")
    Bt, Dn = shape
    of_dn = (Dn,)
    od = _out_type("out_dtype", out_dtype, act)
    if out is None:
        out = _like(x, od)
        to = out.data_ptr()
    else:
        to = _need("out", out, dev, od, shape)
    a = _abi.LruStepArgs(
        _need("x", x, dev, act, shape), _need("r", r, dev, act, shape), _need("i", i, dev, act, shape),
        _need("lam", lam, dev, _F32, of_dn), _maybe("r_bias", r_bias, dev, _F32, of_dn),
        _maybe("i_bias", i_bias, dev, _F32, of_dn), _need("h", h, dev, _F32, shape), to, Bt, Dn, c, _DT[act], _DT[od])
    _call("ssm_lru_step", a, dev)
    return out


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


def _heads(name, t, dev, dtype, shape, time):
    """(address, batch, head and row stride) of a (Bt, L, H, D) or, with time, (Bt, H, D, L) tensor whose last axis
    is dense."""
    try:
        st = t.stride()
        if t.get_device() == dev and t.dtype is dtype and t.shape == shape and (st[3] == 1 or shape[3] == 1):
            return (t.data_ptr(), st[0], st[1], st[2]) if time else (t.data_ptr(), st[0], st[2], st[1])
    except AttributeError:
        pass
    _refuse(name, t, dev, dtype, shape, False)


def _qk_args(a, q, k, q_weight, k_weight, inv_freq, positions, pos0, norm, eps, interleaved, rot_scale, layout):
    """Fill the inputs; returns (dtype, device, shape of q, shape of k or None, time innermost)."""
    act, dev = _first("q", q)
    code = _LAYOUTS.get(layout)
    if code is None:
        raise ValueError("layout must be 'blhd' or 'bhdl'")
    time = code == _abi.SSM_QK_TIME_LAST
    shape = q.shape
    if len(shape) != 4:
        raise ValueError("q must be 4-dimensional, got %s" % (tuple(shape),))
    if time:
        Bt, Hq, D, L = shape
    else:
        Bt, L, Hq, D = shape
    a.q, a.q_sb, a.q_sh, a.q_sr = _heads("q", q, dev, act, shape, time)
    k_shape = None
    if k is not None:
        try:
            Hk = k.shape[1 if time else 2]
        except (AttributeError, IndexError):
            raise TypeError("k must be a 4-dimensional torch.Tensor") from None
        k_shape = (Bt, Hk, D, L) if time else (Bt, L, Hk, D)
        a.k, a.k_sb, a.k_sh, a.k_sr = _heads("k", k, dev, act, k_shape, time)
        a.Hk = Hk
    elif k_weight is not None:
        raise ValueError("k_weight without k")
    if q_weight is not None:
        a.q_weight = _need("q_weight", q_weight, dev, _F32, (D,))
    if k_weight is not None:
        a.k_weight = _need("k_weight", k_weight, dev, _F32, (D,))
    if not norm and (q_weight is not None or k_weight is not None):
        raise ValueError("weights need norm=True")
    if inv_freq is not None:
        dtype = getattr(inv_freq, "dtype", _F32)
        if dtype is torch.float64:
            a.freq_f64 = 1
        elif dtype is not _F32:
            raise TypeError("inv_freq must be float32 or float64")
        fs = getattr(inv_freq, "shape", (0,))
        if len(fs) != 1:
            raise ValueError("inv_freq must be (rot / 2,)")
        if 2 * fs[0] > D:
            raise ValueError("inv_freq has %d pairs, more than the %d elements of a head hold" % (fs[0], D))
        a.inv_freq = _need("inv_freq", inv_freq, dev, dtype, fs)
        a.rot = 2 * fs[0]
    if positions is not None:
        dtype = getattr(positions, "dtype", torch.int64)
        if dtype is torch.int64:
            a.pos_i64 = 1
        elif dtype is not torch.int32:
            raise TypeError("positions must be int32 or int64")
        a.positions = _need("positions", positions, dev, dtype, (Bt, L))
    a.Bt, a.L, a.Hq, a.D, a.pos0 = Bt, L, Hq, D, pos0
    a.eps, a.rot_scale = eps, rot_scale
    a.layout, a.norm, a.interleaved, a.in_dtype = code, bool(norm), bool(interleaved), _DT[act]
    return act, dev, shape, k_shape, time


def ssm_qk_norm_rope_fwd(q, k=None, q_weight=None, k_weight=None, inv_freq=None, positions=None, pos0: int = 0,
                         norm: bool = True, eps: float = 1e-6, interleaved: bool = False, rot_scale: float = 1.0,
                         layout: str = "blhd", out_dtype=None, out: Optional[Tuple] = None):
    """Normalise every head of q and k by its root mean square (times ``q_weight`` / ``k_weight``, (D,) fp32) and
    rotate it by position, in one pass; ``norm=False`` rotates alone, no ``inv_freq`` normalises alone.

    q: (Bt, L, Hq, D), k: (Bt, L, Hk, D) or None, fp32 or bf16; with ``layout="bhdl"`` (Bt, H, D, L), time
    innermost as the selective scan's B and C are (C.unsqueeze(1) is one head). Any strides but a dense last axis:
    slices of one projection need no copy. ``inv_freq`` ((rot / 2,) fp32 or fp64, see ssm_rope_inv_freq): the
    first rot elements of a head turn by position * inv_freq[j] in pairs (j, j + rot / 2), or (2 j, 2 j + 1) with
    ``interleaved``; cosine and sine are multiplied by ``rot_scale``. ``positions``: (Bt, L) int32 or int64, or None
    for pos0 + t. ``out``: (q_out, k_out) to write to, possibly q and k themselves. Returns (q_out, k_out)."""
    a = _abi.QkArgs()
    act, dev, shape, k_shape, time = _qk_args(a, q, k, q_weight, k_weight, inv_freq, positions, pos0, norm, eps,
                                              interleaved, rot_scale, layout)
    od = _out_type("out_dtype", out_dtype, act)
    a.out_dtype = _DT[od]
    if out is None:
        q_out = _like(q, od)
        k_out = None if k is None else _like(k, od)
    else:
        q_out, k_out = out
    a.q_out, a.q_out_sb, a.q_out_sh, a.q_out_sr = _heads("q_out", q_out, dev, od, shape, time)
    if k is None:
        k_out = None
    else:
        a.k_out, a.k_out_sb, a.k_out_sh, a.k_out_sr = _heads("k_out", k_out, dev, od, k_shape, time)
    _call("ssm_qk_norm_rope_fwd", a, dev)
    return q_out, k_out


def ssm_qk_norm_rope_bwd(dq_out, q, dk_out=None, k=None, q_weight=None, k_weight=None, inv_freq=None, positions=None,
                         pos0: int = 0, norm: bool = True, eps: float = 1e-6, interleaved: bool = False,
                         rot_scale: float = 1.0, layout: str = "blhd", grad_dtype=None,
                         workspace: Optional[torch.Tensor] = None):
    """Backward of ssm_qk_norm_rope_fwd: q, k and the options are the forward's, dq_out / dk_out the gradients of
    its outputs (fp32 or bf16, both alike). Returns a dict: dq (and dk with k) in ``grad_dtype`` (fp32 unless
    given), dq_weight / dk_weight (fp32) where the weight exists."""
    if (k is None) != (dk_out is None):
        raise ValueError("k and dk_out come together")
    bw = _abi.QkBwdArgs()
    a = bw.fwd
    _, dev, shape, k_shape, time = _qk_args(a, q, k, q_weight, k_weight, inv_freq, positions, pos0, norm, eps,
                                            interleaved, rot_scale, layout)
    dd, _ = _first("dq_out", dq_out)
    gd = _out_type("grad_dtype", grad_dtype, _F32)
    bw.dq_out, a.q_out_sb, a.q_out_sh, a.q_out_sr = _heads("dq_out", dq_out, dev, dd, shape, time)
    dq = _like(q, gd)
    bw.dq, bw.dq_sb, bw.dq_sh, bw.dq_sr = _heads("dq", dq, dev, gd, shape, time)
    grads = {"dq": dq}
    if k is not None:
        bw.dk_out, a.k_out_sb, a.k_out_sh, a.k_out_sr = _heads("dk_out", dk_out, dev, dd, k_shape, time)
        dk = grads["dk"] = _like(k, gd)
        bw.dk, bw.dk_sb, bw.dk_sh, bw.dk_sr = _heads("dk", dk, dev, gd, k_shape, time)
    if q_weight is not None:
        g = grads["dq_weight"] = _like(q_weight, _F32)
        bw.dq_weight = g.data_ptr()
    if k_weight is not None:
        g = grads["dk_weight"] = _like(k_weight, _F32)
        bw.dk_weight = g.data_ptr()
    bw.dout_dtype, bw.grad_dtype = _DT[dd], _DT[gd]
    need = _abi.load().ssm_qk_norm_rope_bwd_workspace_size(_byref(bw))
    if need:
        ws, bw.workspace = _scratch(need, dev, workspace)
        bw.workspace_bytes = need
    _call("ssm_qk_norm_rope_bwd", bw, dev)
    return grads


# ---- state-space-dual step ---------------------------------------------------------------------


def ssm_ssd_step(x, dt, A_log, B, C, h, D=None, dt_bias=None, delta_softplus: bool = True, out_dtype=None,
                 discretization: str = "zoh", out: Optional[torch.Tensor] = None):
    """One token of the state-space dual (ssm_ssd_fwd). x: (Bt, H, P); dt: (Bt, H); B, C: (Bt, N) shared by the
    heads, all bf16 or all fp32; A_log, D, dt_bias: (H,) fp32; h: (Bt, H, N, P) fp32, read and updated in place
    (ssm_ssd_fwd's h_last continues here). P and N up to 256. Returns y (Bt, H, P)."""
    act, dev = _first("x", x)
    shape = x.shape
    if len(shape) != 3:
        raise ValueError("x must be (Bt, H, P)")
    if not isinstance(B, torch.Tensor) or len(B.shape) != 2:
        raise ValueError("B must be (Bt, N)")
    if discretization not in _DISC:
        raise ValueError("discretization must be 'zoh' or 'euler'")
    Bt, H, P = shape
    N = B.shape[1]
    of_h, of_n = (H,), (Bt, N)
    od = _out_type("out_dtype", out_dtype, act)
    if out is None:
        out = _like(x, od)
        to = out.data_ptr()
    else:
        to = _need("out", out, dev, od, shape)
    a = _abi.SsdStepArgs(
        _need("x", x, dev, act, shape), _need("dt", dt, dev, act, (Bt, H)), _maybe("dt_bias", dt_bias, dev, _F32, of_h),
        _need("A_log", A_log, dev, _F32, of_h), _need("B", B, dev, act, of_n), _need("C", C, dev, act, of_n),
        _maybe("D", D, dev, _F32, of_h), _need("h", h, dev, _F32, (Bt, H, N, P)), to, Bt, H, P, N, _DT[act], _DT[od],
        bool(delta_softplus), _DISC[discretization])
    _call("ssm_ssd_step", a, dev)
    return out
