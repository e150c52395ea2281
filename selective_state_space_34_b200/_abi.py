"""ctypes mirror of include/ssm_scan.h. Declarations only: every computation happens in the CUDA
library. Loading fails loudly when the library has not been built; there is no fallback."""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libssm_scan.so")

SSM_F32, SSM_BF16 = 0, 1
SSM_ZOH, SSM_EULER = 0, 1
SSM_SCAN_LANES, SSM_SCAN_CHUNKED = 0, 1
SSM_SSD_AUTO, SSM_SSD_THREE_PASS, SSM_SSD_FUSED = 0, 1, 2
SSM_QK_STATE_LAST, SSM_QK_TIME_LAST = 0, 1
SSM_STATE_CHUNK = 16
SSM_NOALLOC_SCRATCH_BYTES = 72 << 20
SSM_ERR_TIMEOUT = 8

STATUS = {
    0: "SSM_OK", 1: "SSM_ERR_NULL", 2: "SSM_ERR_SHAPE", 3: "SSM_ERR_ALIGN", 4: "SSM_ERR_DTYPE",
    5: "SSM_ERR_UNSUPPORTED", 6: "SSM_ERR_CUDA", 7: "SSM_ERR_WORKSPACE", 8: "SSM_ERR_TIMEOUT",
}


class FwdArgs(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p), ("dt", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p),
        ("A_log", ctypes.c_void_p), ("B", ctypes.c_void_p), ("C", ctypes.c_void_p),
        ("D", ctypes.c_void_p), ("z", ctypes.c_void_p), ("conv_w", ctypes.c_void_p),
        ("conv_b", ctypes.c_void_p), ("out", ctypes.c_void_p), ("chunk_states", ctypes.c_void_p),
        ("u_out", ctypes.c_void_p),
        ("Bt", ctypes.c_int64), ("Dn", ctypes.c_int64), ("N", ctypes.c_int64), ("L", ctypes.c_int64),
        ("K", ctypes.c_int32), ("in_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
        ("delta_softplus", ctypes.c_int32),
        ("h0", ctypes.c_void_p), ("conv_hist", ctypes.c_void_p), ("h_last", ctypes.c_void_p),
        ("conv_hist_out", ctypes.c_void_p), ("discretization", ctypes.c_int32),
        ("n_segments", ctypes.c_int32), ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t), ("scan_form", ctypes.c_int32),
    ]


class BwdArgs(ctypes.Structure):
    _fields_ = [
        ("fwd", FwdArgs), ("dout", ctypes.c_void_p), ("chunk_states", ctypes.c_void_p),
        ("dx", ctypes.c_void_p), ("ddt", ctypes.c_void_p), ("dz", ctypes.c_void_p),
        ("dA_log", ctypes.c_void_p), ("dB", ctypes.c_void_p), ("dC", ctypes.c_void_p),
        ("dD", ctypes.c_void_p), ("ddt_bias", ctypes.c_void_p), ("dconv_w", ctypes.c_void_p),
        ("dconv_b", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t), ("timing_events", ctypes.c_void_p),
        ("dh_last", ctypes.c_void_p), ("dh0", ctypes.c_void_p), ("dconv_hist", ctypes.c_void_p),
    ]


class StepArgs(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p), ("dt", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p),
        ("A_log", ctypes.c_void_p), ("B", ctypes.c_void_p), ("C", ctypes.c_void_p),
        ("D", ctypes.c_void_p), ("z", ctypes.c_void_p), ("conv_w", ctypes.c_void_p),
        ("conv_b", ctypes.c_void_p), ("h", ctypes.c_void_p), ("conv_hist", ctypes.c_void_p),
        ("out", ctypes.c_void_p), ("Bt", ctypes.c_int64), ("Dn", ctypes.c_int64),
        ("N", ctypes.c_int64), ("K", ctypes.c_int32), ("in_dtype", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32), ("delta_softplus", ctypes.c_int32),
        ("discretization", ctypes.c_int32),
    ]


class SsdArgs(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p), ("dt", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p),
        ("A_log", ctypes.c_void_p), ("B", ctypes.c_void_p), ("C", ctypes.c_void_p),
        ("D", ctypes.c_void_p), ("h0", ctypes.c_void_p), ("y", ctypes.c_void_p),
        ("h_last", ctypes.c_void_p),
        ("Bt", ctypes.c_int64), ("H", ctypes.c_int64), ("L", ctypes.c_int64), ("P", ctypes.c_int64),
        ("N", ctypes.c_int64),
        ("in_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
        ("delta_softplus", ctypes.c_int32), ("discretization", ctypes.c_int32),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("timing_events", ctypes.c_void_p), ("form", ctypes.c_int32),
    ]


_P, _I64, _I32, _F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float


def _fields(*groups):
    """(names, type) groups as a ctypes field list."""
    return [(n, t) for names, t in groups for n in names.split()]


class LruArgs(ctypes.Structure):
    _fields_ = _fields(("x r i lam r_bias i_bias h0 reset lengths out chunk_states h_last", _P), ("Bt Dn L", _I64),
                       ("c", _F32), ("in_dtype out_dtype", _I32))


class LruBwdArgs(ctypes.Structure):
    _fields_ = _fields(("fwd", LruArgs), ("dout dh_last dx dr di dlam dr_bias di_bias dh0", _P), ("grad_dtype", _I32),
                       ("workspace", _P), ("workspace_bytes", ctypes.c_size_t))


class LruStepArgs(ctypes.Structure):
    _fields_ = _fields(("x r i lam r_bias i_bias h out", _P), ("Bt Dn", _I64), ("c", _F32), ("in_dtype out_dtype", _I32))


class QkArgs(ctypes.Structure):
    _fields_ = _fields(("q k q_weight k_weight inv_freq positions q_out k_out", _P),
                       ("q_sb q_sh q_sr k_sb k_sh k_sr q_out_sb q_out_sh q_out_sr k_out_sb k_out_sh k_out_sr", _I64),
                       ("Bt L Hq Hk D rot pos0", _I64), ("eps rot_scale", _F32),
                       ("layout norm interleaved freq_f64 pos_i64 in_dtype out_dtype", _I32))


class QkBwdArgs(ctypes.Structure):
    _fields_ = _fields(("fwd", QkArgs), ("dq_out dk_out dq dk", _P), ("dq_sb dq_sh dq_sr dk_sb dk_sh dk_sr", _I64),
                       ("dq_weight dk_weight", _P), ("dout_dtype grad_dtype", _I32), ("workspace", _P),
                       ("workspace_bytes", ctypes.c_size_t))


class SsdStepArgs(ctypes.Structure):
    _fields_ = _fields(("x dt dt_bias A_log B C D h out", _P), ("Bt H P N", _I64),
                       ("in_dtype out_dtype delta_softplus discretization", _I32))


# (name, restype, argtypes) of every exported function in include/ssm_scan.h
SIGNATURES = [
    ("ssm_num_state_chunks", ctypes.c_int64, [ctypes.c_int64]),
    ("ssm_scan_fwd", ctypes.c_int, [ctypes.POINTER(FwdArgs), ctypes.c_void_p]),
    ("ssm_fwd_workspace_size", ctypes.c_size_t, [ctypes.POINTER(FwdArgs)]),
    ("ssm_bwd_workspace_size", ctypes.c_size_t, [ctypes.POINTER(BwdArgs)]),
    ("ssm_workspace_size", ctypes.c_size_t, [ctypes.POINTER(FwdArgs), ctypes.c_int32]),
    ("ssm_scan_bwd", ctypes.c_int, [ctypes.POINTER(BwdArgs), ctypes.c_void_p]),
    ("ssm_scan_bwd_noalloc", ctypes.c_int, [ctypes.POINTER(BwdArgs), ctypes.c_void_p]),
    ("ssm_scan_step", ctypes.c_int, [ctypes.POINTER(StepArgs), ctypes.c_void_p]),
    ("ssm_ssd_workspace_size", ctypes.c_size_t, [ctypes.POINTER(SsdArgs)]),
    ("ssm_ssd_fwd", ctypes.c_int, [ctypes.POINTER(SsdArgs), ctypes.c_void_p]),
    ("ssm_ssd_check", ctypes.c_int, [ctypes.POINTER(SsdArgs), ctypes.c_void_p]),
    ("ssm_ssd_step", ctypes.c_int, [ctypes.POINTER(SsdStepArgs), ctypes.c_void_p]),
    ("ssm_lru_num_states", ctypes.c_int64, [ctypes.c_int64]),
    ("ssm_lru_fwd", ctypes.c_int, [ctypes.POINTER(LruArgs), ctypes.c_void_p]),
    ("ssm_lru_bwd_workspace_size", ctypes.c_size_t, [ctypes.POINTER(LruBwdArgs)]),
    ("ssm_lru_bwd", ctypes.c_int, [ctypes.POINTER(LruBwdArgs), ctypes.c_void_p]),
    ("ssm_lru_step", ctypes.c_int, [ctypes.POINTER(LruStepArgs), ctypes.c_void_p]),
    ("ssm_qk_norm_rope_fwd", ctypes.c_int, [ctypes.POINTER(QkArgs), ctypes.c_void_p]),
    ("ssm_qk_norm_rope_bwd_workspace_size", ctypes.c_size_t, [ctypes.POINTER(QkBwdArgs)]),
    ("ssm_qk_norm_rope_bwd", ctypes.c_int, [ctypes.POINTER(QkBwdArgs), ctypes.c_void_p]),
    ("ssm_wait_selftest", ctypes.c_int, [ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p]),
    ("ssm_conv1d_silu", ctypes.c_int,
     [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
      ctypes.c_int64, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
      ctypes.c_void_p]),
    ("ssm_status_string", ctypes.c_char_p, [ctypes.c_int]),
    ("ssm_last_cuda_error", ctypes.c_int, []),
]

_lib = None


def load():
    """Load libssm_scan.so and declare its signatures. Raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                "libssm_scan.so is not built (expected at %s); run "
                "`python -m selective_state_space_34_b200.build`" % LIB_PATH)
        lib = ctypes.CDLL(LIB_PATH)
        for name, res, args in SIGNATURES:
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


_native = None


def marshal():
    """The native marshalling module (csrc/ssm_marshal.cpp). Raises if it is not built; there is no other path."""
    global _native
    if _native is None:
        load()
        try:
            from . import _marshal
        except ImportError as e:
            raise ImportError("_marshal.so is not built or does not match this torch (%s); run "
                              "`python -m selective_state_space_34_b200.build`" % e) from e
        from .build import built_for
        if _marshal.BUILT_FOR != built_for():
            raise ImportError("_marshal.so is built for %s, this is %s; run `python -m selective_state_space_34_b200.build`"
                              % (_marshal.BUILT_FOR, built_for()))
        _native = _marshal
    return _native


class SSMError(RuntimeError):
    def __init__(self, fn: str, code: int):
        lib = load()
        msg = lib.ssm_status_string(code).decode()
        if code == 6:
            msg += " (cudaError %d)" % lib.ssm_last_cuda_error()
        super().__init__("%s: %s" % (fn, msg))
        self.code = code


def check(fn: str, code: int) -> None:
    if code != 0:
        raise SSMError(fn, code)
