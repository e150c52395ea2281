"""What the binding of the recurrence, of queries and keys and of the dual step refuses, on CUDA tensors; and that a refused
call leaves its buffers alone."""
import pytest
import torch

import selective_state_space_34_b200 as ssm
from selective_state_space_34_b200 import _abi

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def refused(error, match, fn, *a, **kw):
    with pytest.raises(error, match=match):
        fn(*a, **kw)


def test_recurrence():
    x = torch.zeros(2, 4, 16, dtype=BF, device="cuda")
    lam, h = torch.zeros(4, device="cuda"), torch.zeros(2, 4, device="cuda")
    f = ssm.ssm_lru_fwd
    refused(TypeError, "float32 or bfloat16", f, x.half(), x, x, lam)
    refused(TypeError, "r must be torch.bfloat16", f, x, x.float(), x, lam)
    refused(TypeError, "i must be a torch.Tensor", f, x, x, None, lam)
    refused(ValueError, "r must be", f, x, x[..., :8].contiguous(), x, lam)
    refused(ValueError, "contiguous", f, x.transpose(0, 1), x, x, lam)
    refused(ValueError, "i must be contiguous", f, x, x, torch.zeros(2, 4, 32, dtype=BF, device="cuda")[..., ::2], lam)
    refused(ValueError, "lam must be", f, x, x, x, lam[:3])
    refused(ValueError, "lam must be a CUDA tensor on cuda:0, got cpu", f, x, x, x, lam.cpu())
    refused(TypeError, "lam must be torch.float32", f, x, x, x, lam.double())
    refused(ValueError, "h0 must be", f, x, x, x, lam, h0=h.t())
    refused(TypeError, "reset must be bool", f, x, x, x, lam, reset=torch.zeros(2, 16, device="cuda"))
    refused(ValueError, "reset must be", f, x, x, x, lam, reset=torch.zeros(2, 15, dtype=torch.bool, device="cuda"))
    refused(TypeError, "lengths must be torch.int32", f, x, x, x, lam, lengths=torch.zeros(2, dtype=torch.int64, device="cuda"))
    refused(TypeError, "out_dtype", f, x, x, x, lam, out_dtype=torch.float16)
    refused(TypeError, "out must be torch.float32", f, x, x, x, lam, out_dtype=F32, out=torch.empty_like(x))
    refused(ValueError, r"\(Bt, Dn, L\)", f, x[0], x, x, lam)
    for c in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(_abi.SSMError, match="ssm_lru_fwd") as e:
            f(x, x, x, lam, c=c)
        assert e.value.code == 5
    b = ssm.ssm_lru_bwd
    refused(TypeError, "dout must be torch.bfloat16", b, x.float(), x, x, x, lam)
    refused(ValueError, "chunk_states must be", b, x, x, x, x, lam, chunk_states=torch.zeros(2, 4, 3, device="cuda"))
    refused(ValueError, "dh_last must be", b, x, x, x, x, lam, dh_last=h[:1])
    refused(ValueError, "workspace", b, x, x, x, x, lam, workspace=torch.zeros(4096, dtype=torch.uint8))
    s = ssm.ssm_lru_step
    refused(TypeError, "h must be torch.float32", s, x[..., 0].contiguous(), x[..., 0].contiguous(), x[..., 0].contiguous(), lam,
            h.bfloat16())
    refused(ValueError, "x must be", s, x, x, x, lam, h)
    assert not bool(h.any())


def test_workspace_of_the_caller():
    x = torch.randn(3, 40, 700, device="cuda").to(BF)
    lam = torch.full((40,), -4.0, device="cuda")
    want = ssm.ssm_lru_bwd(x, x, x, x, lam)
    for n in (64, 1 << 20):  # too small: an allocation of the call's own; large enough: used
        ws = torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda")
        got = ssm.ssm_lru_bwd(x, x, x, x, lam, workspace=ws)
        assert all(torch.equal(got[k], want[k]) for k in want)
        assert bool((ws != 0x5A).any()) == (n > 64)


def test_queries_and_keys():
    q, k = torch.zeros(2, 5, 4, 64, dtype=BF, device="cuda"), torch.zeros(2, 5, 2, 64, dtype=BF, device="cuda")
    w, freq = torch.ones(64, device="cuda"), torch.ones(32, device="cuda")
    f = ssm.ssm_qk_norm_rope_fwd
    refused(ValueError, "layout", f, q, k, layout="lbhd")
    refused(TypeError, "k must be torch.bfloat16", f, q, k.float())
    refused(ValueError, "k must be", f, q, k[:, :4])
    refused(ValueError, "4-dimensional", f, q[0])
    refused(ValueError, "last axis", f, q.transpose(2, 3), None)
    refused(ValueError, "weights need norm", f, q, k, q_weight=w, norm=False)
    refused(ValueError, "k_weight without k", f, q, k_weight=w)
    refused(ValueError, "q_weight must be", f, q, k, q_weight=w[:32])
    refused(ValueError, "33 pairs", f, q, k, inv_freq=torch.ones(33, device="cuda"))
    refused(TypeError, "inv_freq", f, q, k, inv_freq=freq.half())
    refused(TypeError, "positions must be int", f, q, k, inv_freq=freq, positions=torch.zeros(2, 5, device="cuda"))
    refused(ValueError, "positions must be", f, q, k, inv_freq=freq, positions=torch.zeros(5, dtype=torch.int64, device="cuda"))
    refused(TypeError, "q_out must be", f, q, k, out=(q.float(), k))
    refused(TypeError, "k_out must be", f, q, k, out=(torch.empty_like(q), [0]))
    mine = torch.empty_like(q)
    got = f(q, k, out=(mine, None))  # None: allocated by the call
    assert got[0] is mine and got[1].shape == k.shape
    with pytest.raises(_abi.SSMError) as e:  # every batch element would be written to one place
        f(q, None, out=(q[:1].expand(2, 5, 4, 64), None))
    assert e.value.code == 2
    for eps in (-1.0, float("nan")):
        with pytest.raises(_abi.SSMError) as e:
            f(q, k, eps=eps)
        assert e.value.code == 5
    with pytest.raises(_abi.SSMError) as e:
        f(torch.zeros(1, 1, 1, 513, device="cuda"))
    assert e.value.code == 5
    b = ssm.ssm_qk_norm_rope_bwd
    refused(ValueError, "come together", b, q, q, None, k)
    refused(TypeError, "dk_out must be", b, q, q, k.float(), k)
    refused(ValueError, "dq_out must be", b, q[:1], q)


def test_dual_step():
    x, dt = torch.zeros(2, 3, 16, dtype=BF, device="cuda"), torch.zeros(2, 3, dtype=BF, device="cuda")
    A, B, h = torch.zeros(3, device="cuda"), torch.zeros(2, 8, dtype=BF, device="cuda"), torch.ones(2, 3, 8, 16, device="cuda")
    s = ssm.ssm_ssd_step
    refused(ValueError, "discretization", s, x, dt, A, B, B, h, discretization="tustin")
    refused(ValueError, "B must be", s, x, dt, A, B[0], B, h)
    refused(TypeError, "C must be torch.bfloat16", s, x, dt, A, B, B.float(), h)
    refused(ValueError, "h must be", s, x, dt, A, B, B, h.transpose(2, 3))
    refused(TypeError, "h must be torch.float32", s, x, dt, A, B, B, h.double())
    refused(ValueError, "dt must be", s, x, dt[:1], A, B, B, h)
    big = torch.zeros(1, 1, 257, device="cuda")
    with pytest.raises(_abi.SSMError) as e:
        s(big, torch.zeros(1, 1, device="cuda"), A[:1], torch.zeros(1, 4, device="cuda"), torch.zeros(1, 4, device="cuda"),
          torch.zeros(1, 1, 4, 257, device="cuda"))
    assert e.value.code == 5
    assert bool((h == 1).all())
