"""Calls of the layers' operators from several host threads at once: the interpreter's lock is released around a launch."""
import ctypes
import threading

import pytest
import torch

import selective_state_space_34_b200 as ssm
from selective_state_space_34_b200 import _abi
from test_gpu_qk import freq, inputs

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _arguments(t, D, L, out, inv_freq):
    """The C arguments of a time-innermost forward of one head of t["q"] into out."""
    a = _abi.QkArgs()
    a.q, a.q_out, a.inv_freq, a.positions = (v.data_ptr() for v in (t["q"], out, inv_freq, t["positions"]))
    a.q_weight = t["q_weight"].data_ptr()
    a.q_sb = a.q_out_sb = a.q_sh = a.q_out_sh = D * L
    a.q_sr = a.q_out_sr = L
    a.Bt, a.L, a.Hq, a.Hk, a.D, a.rot, a.eps, a.rot_scale = 1, L, 1, 0, D, D, 1e-6, 1.0
    a.layout, a.norm, a.pos_i64, a.freq_f64 = _abi.SSM_QK_TIME_LAST, 1, 1, int(inv_freq.dtype == torch.float64)
    a.in_dtype = a.out_dtype = _abi.SSM_BF16 if t["q"].dtype == BF else _abi.SSM_F32
    return a


@pytest.mark.parametrize("dtype", [BF, F32])
def test_threads_do_not_fail_each_others_launches(dtype):
    """Head sizes that run one kernel with different amounts of shared memory (eight and sixteen warps a block), four threads
    on streams of their own that call the library in close loops."""
    lib, L, calls = _abi.load(), 24, []
    for D in (136, 384, 200, 512):
        t, f = inputs(1, L, 1, 0, D, dtype, True, seed=D), freq(D)
        kw = dict(q_weight=t["q_weight"], inv_freq=f, positions=t["positions"], layout="bhdl")
        want, _ = ssm.ssm_qk_norm_rope_fwd(t["q"], None, **kw)
        out = torch.zeros_like(want)
        calls.append((_arguments(t, D, L, out, f), out, want, (t, f)))
    torch.cuda.synchronize()
    failed = []

    def work(j):
        stream = torch.cuda.Stream()
        handle, args = ctypes.c_void_p(stream.cuda_stream), ctypes.byref(calls[j][0])
        for k in range(20000):
            status = lib.ssm_qk_norm_rope_fwd(args, handle)
            if status:
                failed.append((j, k, status, lib.ssm_last_cuda_error()))
                break
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(j,)) for j in range(len(calls))]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not failed
    assert all(torch.equal(out, want) for _, out, want, _ in calls)


@pytest.mark.parametrize("sizes", [(3, 16, 8, 12), (20, 64, 33, 48)])
def test_threads_of_the_chunked_scan(sizes):
    """The same of the scan's chunked layout, whose shared memory goes by the number of states."""
    lib, Bt, Dn, L, calls = _abi.load(), 1, 16, 64, []
    g = torch.Generator().manual_seed(0)
    n = lambda *s: torch.randn(s, generator=g).cuda()  # noqa: E731
    for N in sizes:
        t = {"x": n(Bt, Dn, L), "dt": n(Bt, Dn, L), "A_log": n(Dn, N), "B": n(Bt, N, L), "C": n(Bt, N, L)}
        want = ssm.ssm_scan_fwd(*t.values(), scan_form="chunked")
        out = torch.zeros_like(want)
        a = _abi.FwdArgs()
        for k, v in dict(t, out=out).items():
            setattr(a, k, v.data_ptr())
        a.Bt, a.Dn, a.N, a.L, a.delta_softplus = Bt, Dn, N, L, 1
        a.in_dtype = a.out_dtype = _abi.SSM_F32
        a.scan_form = _abi.SSM_SCAN_CHUNKED
        calls.append((a, out, want, t))
    torch.cuda.synchronize()
    failed = []

    def work(j):
        stream = torch.cuda.Stream()
        handle, args = ctypes.c_void_p(stream.cuda_stream), ctypes.byref(calls[j][0])
        for k in range(20000):
            status = lib.ssm_scan_fwd(args, handle)
            if status:
                failed.append((j, k, status, lib.ssm_last_cuda_error()))
                break
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(j,)) for j in range(len(calls))]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not failed
    assert all(torch.equal(out, want) for _, out, want, _ in calls)
