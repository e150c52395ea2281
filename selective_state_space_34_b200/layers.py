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


def _act(name: str, t: torch.Tensor) -> torch.dtype:
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor (the library has no CPU path)" % name)
    if t.dtype not in _DT:
        raise TypeError("%s must be float32 or bfloat16" % name)
    return t.dtype


def _need(name, t, like, dtype, shape):
    """A dense CUDA tensor of this dtype and shape on the device of ``like``."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device != like.device:
        raise ValueError("%s must be a CUDA tensor on %s, got %s" % (name, like.device, t.device))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _maybe(name, t, like, dtype, shape):
    return None if t is None else _need(name, t, like, dtype, shape)


def _out_type(name, dtype, default):
    dtype = default if dtype is None else dtype
    if dtype not in _DT:
        raise TypeError("%s must be float32 or bfloat16" % name)
    return dtype


def _call(name: str, args, device) -> None:
    """Run an entry point on the device's current stream."""
    fn = getattr(_abi.load(), name)
    if device.index == torch.cuda.current_device():
        code = fn(_byref(args), torch.cuda.current_stream(device).cuda_stream)
    else:
        with torch.cuda.device(device):
            code = fn(_byref(args), torch.cuda.current_stream(device).cuda_stream)
    if code:
        _abi.check(name, code)


def _scratch(need: int, device, workspace: Optional[torch.Tensor]):
    """(tensor to hold on to, its first 256-byte boundary): the caller's workspace when that is large enough."""
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or workspace.device != device or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor on %s" % (device,))
        base = workspace.data_ptr()
        at = (base + 255) & ~255
        if at + need <= base + workspace.numel() * workspace.element_size():
            return workspace, at
    ws = torch.empty(need + 256, dtype=torch.uint8, device=device)
    return ws, (ws.data_ptr() + 255) & ~255


# ---- gated linear recurrence -------------------------------------------------------------------


def ssm_lru_num_states(L: int) -> int:
    return int(_abi.load().ssm_lru_num_states(int(L)))


def _lru_args(x, r, i, lam, r_bias, i_bias, c, h0, reset, lengths):
    act = _act("x", x)
    if x.dim() != 3:
        raise ValueError("x must be (Bt, Dn, L)")
    Bt, Dn, L = x.shape
    f32 = torch.float32
    a = _abi.LruArgs()
    a.x = _need("x", x, x, act, x.shape)
    a.r = _need("r", r, x, act, x.shape)
    a.i = _need("i", i, x, act, x.shape)
    a.lam = _need("lam", lam, x, f32, (Dn,))
    a.r_bias = _maybe("r_bias", r_bias, x, f32, (Dn,))
    a.i_bias = _maybe("i_bias", i_bias, x, f32, (Dn,))
    a.h0 = _maybe("h0", h0, x, f32, (Bt, Dn))
    if reset is not None:
        if isinstance(reset, torch.Tensor) and reset.dtype not in (torch.bool, torch.uint8):
            raise TypeError("reset must be bool or uint8")
        a.reset = _need("reset", reset, x, getattr(reset, "dtype", None), (Bt, L))
    a.lengths = _maybe("lengths", lengths, x, torch.int32, (Bt,))
    a.Bt, a.Dn, a.L, a.c = Bt, Dn, L, float(c)
    a.in_dtype = _DT[act]
    return a


def ssm_lru_fwd(x, r, i, lam, r_bias=None, i_bias=None, c: float = 8.0, h0=None, reset=None, lengths=None,
                out_dtype=None, save_states: bool = False, return_state: bool = False,
                out: Optional[torch.Tensor] = None):
    """Gated linear recurrence h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t + i_bias) x_t with
    a_t = exp(-c softplus(lam) sigmoid(r_t + r_bias)). x, r, i: (Bt, Dn, L), fp32 or bf16, the gates before
    their sigmoids; lam, r_bias, i_bias: (Dn,) fp32; h0: (Bt, Dn) fp32. ``reset`` ((Bt, L) bool or uint8) marks
    the steps that start a new sequence, ``lengths`` ((Bt,) int32) the live steps of each batch element (behind
    them out is 0). Returns ``out`` (every h_t), or a dict with ``out`` and, when asked, ``chunk_states`` (for
    ssm_lru_bwd) and ``h_last`` ((Bt, Dn) fp32, the state after the last live step)."""
    a = _lru_args(x, r, i, lam, r_bias, i_bias, c, h0, reset, lengths)
    Bt, Dn, L = x.shape
    od = _out_type("out_dtype", out_dtype, x.dtype)
    if out is None:
        out = torch.empty((Bt, Dn, L), dtype=od, device=x.device)
        a.out = out.data_ptr()
    else:
        a.out = _need("out", out, x, od, x.shape)
    a.out_dtype = _DT[od]
    res: Dict[str, torch.Tensor] = {"out": out}
    if save_states:
        st = torch.empty((Bt, Dn, ssm_lru_num_states(L)), dtype=torch.float32, device=x.device)
        a.chunk_states = st.data_ptr()
        res["chunk_states"] = st
    if return_state:
        hl = torch.empty((Bt, Dn), dtype=torch.float32, device=x.device)
        a.h_last = hl.data_ptr()
        res["h_last"] = hl
    _call("ssm_lru_fwd", a, x.device)
    return res if (save_states or return_state) else out


def ssm_lru_bwd(dout, x, r, i, lam, r_bias=None, i_bias=None, c: float = 8.0, h0=None, reset=None, lengths=None,
                chunk_states=None, dh_last=None, grad_dtype=None, workspace: Optional[torch.Tensor] = None):
    """Backward of ssm_lru_fwd. ``dout``: (Bt, Dn, L) of x's dtype; ``dh_last``: (Bt, Dn) fp32, the gradient
    arriving at h_last; ``chunk_states`` as saved by the forward (recomputed when not given). Returns a dict: dx,
    dr, di in ``grad_dtype`` (fp32 unless given), and in fp32 dlam, dr_bias / di_bias where the bias exists, and
    dh0 where h0 or dh_last does. ``workspace``: an optional uint8 tensor to use as scratch."""
    bw = _abi.LruBwdArgs()
    bw.fwd = _lru_args(x, r, i, lam, r_bias, i_bias, c, h0, reset, lengths)
    Bt, Dn, L = x.shape
    dev = x.device
    f32 = torch.float32
    bw.dout = _need("dout", dout, x, x.dtype, x.shape)
    bw.fwd.chunk_states = _maybe("chunk_states", chunk_states, x, f32, (Bt, Dn, ssm_lru_num_states(L)))
    bw.dh_last = _maybe("dh_last", dh_last, x, f32, (Bt, Dn))
    gd = _out_type("grad_dtype", grad_dtype, f32)
    bw.grad_dtype = _DT[gd]
    grads = {n: torch.empty((Bt, Dn, L), dtype=gd, device=dev) for n in ("dx", "dr", "di")}
    grads["dlam"] = torch.empty((Dn,), dtype=f32, device=dev)
    if r_bias is not None:
        grads["dr_bias"] = torch.empty((Dn,), dtype=f32, device=dev)
    if i_bias is not None:
        grads["di_bias"] = torch.empty((Dn,), dtype=f32, device=dev)
    if h0 is not None or dh_last is not None:
        grads["dh0"] = torch.empty((Bt, Dn), dtype=f32, device=dev)
    for n, g in grads.items():
        setattr(bw, n, g.data_ptr())
    need = int(_abi.load().ssm_lru_bwd_workspace_size(_byref(bw)))
    if need:
        ws, bw.workspace = _scratch(need, dev, workspace)
        bw.workspace_bytes = need
    _call("ssm_lru_bwd", bw, dev)
    return grads


def ssm_lru_step(x, r, i, lam, h, r_bias=None, i_bias=None, c: float = 8.0, out_dtype=None,
                 out: Optional[torch.Tensor] = None):
    """One token of the gated linear recurrence. x, r, i: (Bt, Dn); h: (Bt, Dn) fp32, read and updated in place.
    Returns the output (Bt, Dn)."""
    act = _act("x", x)
    if x.dim() != 2:
        raise ValueError("x must be (Bt, Dn)")
    shape = x.shape
    Bt, Dn = shape
    f32 = torch.float32
    a = _abi.LruStepArgs()
    a.x = _need("x", x, x, act, shape)
    a.r = _need("r", r, x, act, shape)
    a.i = _need("i", i, x, act, shape)
    a.lam = _need("lam", lam, x, f32, (Dn,))
    a.r_bias = _maybe("r_bias", r_bias, x, f32, (Dn,))
    a.i_bias = _maybe("i_bias", i_bias, x, f32, (Dn,))
    a.h = _need("h", h, x, f32, shape)
    od = _out_type("out_dtype", out_dtype, act)
    if out is None:
        out = torch.empty((Bt, Dn), dtype=od, device=x.device)
        a.out = out.data_ptr()
    else:
        a.out = _need("out", out, x, od, shape)
    a.Bt, a.Dn, a.c, a.in_dtype, a.out_dtype = Bt, Dn, float(c), _DT[act], _DT[od]
    _call("ssm_lru_step", a, x.device)
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


def _strides(name, t, time):
    """(batch, head, row) strides of a (Bt, L, H, D) or, with time, (Bt, H, D, L) tensor whose last axis is dense."""
    if t.shape[3] > 1 and t.stride(3) != 1:
        raise ValueError("%s must be contiguous along its last axis" % name)
    s = t.stride()
    return (s[0], s[1], s[2]) if time else (s[0], s[2], s[1])


def _heads(name, t, like, dtype, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device != like.device:
        raise ValueError("%s must be a CUDA tensor on %s, got %s" % (name, like.device, t.device))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.dim() != 4 or (shape is not None and t.shape != shape):
        raise ValueError("%s must be %s, got %s" % (name, "4-dimensional" if shape is None else tuple(shape),
                                                    tuple(t.shape)))


def _qk_args(q, k, q_weight, k_weight, inv_freq, positions, pos0, norm, eps, interleaved, rot_scale, layout):
    act = _act("q", q)
    if layout not in _LAYOUTS:
        raise ValueError("layout must be 'blhd' or 'bhdl'")
    time = layout == "bhdl"
    _heads("q", q, q, act)
    a = _abi.QkArgs()
    if time:
        Bt, Hq, D, L = q.shape
    else:
        Bt, L, Hq, D = q.shape
    Hk = 0
    if k is not None:
        _heads("k", k, q, act)
        Hk = k.shape[1 if time else 2]
        if k.shape != ((Bt, Hk, D, L) if time else (Bt, L, Hk, D)):
            raise ValueError("k must have q's shape but for its heads")
        a.k = k.data_ptr()
        a.k_sb, a.k_sh, a.k_sr = _strides("k", k, time)
    elif k_weight is not None:
        raise ValueError("k_weight without k")
    a.q = q.data_ptr()
    a.q_sb, a.q_sh, a.q_sr = _strides("q", q, time)
    if not norm and (q_weight is not None or k_weight is not None):
        raise ValueError("weights need norm=True")
    a.q_weight = _maybe("q_weight", q_weight, q, torch.float32, (D,))
    a.k_weight = _maybe("k_weight", k_weight, q, torch.float32, (D,))
    if inv_freq is not None:
        if isinstance(inv_freq, torch.Tensor) and inv_freq.dtype not in (torch.float32, torch.float64):
            raise TypeError("inv_freq must be float32 or float64")
        if getattr(inv_freq, "ndim", 1) != 1:
            raise ValueError("inv_freq must be (rot / 2,)")
        a.inv_freq = _need("inv_freq", inv_freq, q, getattr(inv_freq, "dtype", None), getattr(inv_freq, "shape", None))
        a.freq_f64 = inv_freq.dtype == torch.float64
        a.rot = 2 * inv_freq.shape[0]
        if a.rot > D:
            raise ValueError("inv_freq has %d pairs, more than the %d elements of a head hold" % (inv_freq.shape[0], D))
    if positions is not None:
        if isinstance(positions, torch.Tensor) and positions.dtype not in (torch.int32, torch.int64):
            raise TypeError("positions must be int32 or int64")
        a.positions = _need("positions", positions, q, getattr(positions, "dtype", None), (Bt, L))
        a.pos_i64 = positions.dtype == torch.int64
    a.Bt, a.L, a.Hq, a.Hk, a.D, a.pos0 = Bt, L, Hq, Hk, D, int(pos0)
    a.eps, a.rot_scale = float(eps), float(rot_scale)
    a.layout, a.norm, a.interleaved, a.in_dtype = _LAYOUTS[layout], bool(norm), bool(interleaved), _DT[act]
    return a, time


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
    a, time = _qk_args(q, k, q_weight, k_weight, inv_freq, positions, pos0, norm, eps, interleaved, rot_scale, layout)
    od = _out_type("out_dtype", out_dtype, q.dtype)
    a.out_dtype = _DT[od]
    if out is None:
        q_out = torch.empty(q.shape, dtype=od, device=q.device)
        k_out = None if k is None else torch.empty(k.shape, dtype=od, device=q.device)
    else:
        q_out, k_out = out
        _heads("q_out", q_out, q, od, q.shape)
        if k is not None:
            _heads("k_out", k_out, q, od, k.shape)
    a.q_out = q_out.data_ptr()
    a.q_out_sb, a.q_out_sh, a.q_out_sr = _strides("q_out", q_out, time)
    if k is not None:
        a.k_out = k_out.data_ptr()
        a.k_out_sb, a.k_out_sh, a.k_out_sr = _strides("k_out", k_out, time)
    _call("ssm_qk_norm_rope_fwd", a, q.device)
    return q_out, (None if k is None else k_out)


def ssm_qk_norm_rope_bwd(dq_out, q, dk_out=None, k=None, q_weight=None, k_weight=None, inv_freq=None, positions=None,
                         pos0: int = 0, norm: bool = True, eps: float = 1e-6, interleaved: bool = False,
                         rot_scale: float = 1.0, layout: str = "blhd", grad_dtype=None,
                         workspace: Optional[torch.Tensor] = None):
    """Backward of ssm_qk_norm_rope_fwd: q, k and the options are the forward's, dq_out / dk_out the gradients of
    its outputs (fp32 or bf16, both alike). Returns a dict: dq (and dk with k) in ``grad_dtype`` (fp32 unless
    given), dq_weight / dk_weight (fp32) where the weight exists."""
    bw = _abi.QkBwdArgs()
    if (k is None) != (dk_out is None):
        raise ValueError("k and dk_out come together")
    a, time = _qk_args(q, k, q_weight, k_weight, inv_freq, positions, pos0, norm, eps, interleaved, rot_scale, layout)
    dd = _act("dq_out", dq_out)
    gd = _out_type("grad_dtype", grad_dtype, torch.float32)
    dev = q.device
    _heads("dq_out", dq_out, q, dd, q.shape)
    a.q_out_sb, a.q_out_sh, a.q_out_sr = _strides("dq_out", dq_out, time)
    bw.dq_out = dq_out.data_ptr()
    grads = {"dq": torch.empty(q.shape, dtype=gd, device=dev)}
    bw.dq_sb, bw.dq_sh, bw.dq_sr = _strides("dq", grads["dq"], time)
    if k is not None:
        _heads("dk_out", dk_out, q, dd, k.shape)
        a.k_out_sb, a.k_out_sh, a.k_out_sr = _strides("dk_out", dk_out, time)
        bw.dk_out = dk_out.data_ptr()
        grads["dk"] = torch.empty(k.shape, dtype=gd, device=dev)
        bw.dk_sb, bw.dk_sh, bw.dk_sr = _strides("dk", grads["dk"], time)
    for n, w in (("dq_weight", q_weight), ("dk_weight", k_weight)):
        if w is not None:
            grads[n] = torch.empty(w.shape, dtype=torch.float32, device=dev)
    for n, g in grads.items():
        setattr(bw, n, g.data_ptr())
    bw.fwd = a
    bw.dout_dtype, bw.grad_dtype = _DT[dd], _DT[gd]
    need = int(_abi.load().ssm_qk_norm_rope_bwd_workspace_size(_byref(bw)))
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
    act = _act("x", x)
    if x.dim() != 3:
        raise ValueError("x must be (Bt, H, P)")
    if not isinstance(B, torch.Tensor) or B.dim() != 2:
        raise ValueError("B must be (Bt, N)")
    Bt, H, P = x.shape
    N = B.shape[1]
    f32 = torch.float32
    a = _abi.SsdStepArgs()
    a.x = _need("x", x, x, act, x.shape)
    a.dt = _need("dt", dt, x, act, (Bt, H))
    a.dt_bias = _maybe("dt_bias", dt_bias, x, f32, (H,))
    a.A_log = _need("A_log", A_log, x, f32, (H,))
    a.B = _need("B", B, x, act, (Bt, N))
    a.C = _need("C", C, x, act, (Bt, N))
    a.D = _maybe("D", D, x, f32, (H,))
    a.h = _need("h", h, x, f32, (Bt, H, N, P))
    od = _out_type("out_dtype", out_dtype, act)
    if out is None:
        out = torch.empty((Bt, H, P), dtype=od, device=x.device)
        a.out = out.data_ptr()
    else:
        a.out = _need("out", out, x, od, x.shape)
    if discretization not in _DISC:
        raise ValueError("discretization must be 'zoh' or 'euler'")
    a.Bt, a.H, a.P, a.N = Bt, H, P, N
    a.in_dtype, a.out_dtype = _DT[act], _DT[od]
    a.delta_softplus, a.discretization = bool(delta_softplus), _DISC[discretization]
    _call("ssm_ssd_step", a, x.device)
    return out
