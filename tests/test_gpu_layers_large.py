"""The layers' operators on the plans that large work runs: one warp a row over many chunks, weight gradients of many blocks, offsets past
2^31."""
import pytest
import torch

import layer_bounds
import layer_refs as ref
import selective_state_space_34_b200 as ssm
from test_gpu_lru import compare, inputs as lru_inputs, options
from test_gpu_qk import freq, inputs as qk_inputs

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _poisoned():
    ref.poison_shared()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("Bt,Dn,L,packed", [(2, 640, 1500, True), (2, 640, 1500, False), (1, 1200, 2047, True), (5, 250, 1024, True)])
def test_recurrence_of_one_warp_a_row(Bt, Dn, L, packed, dtype):
    """1184 rows and more: every row is one warp's, over up to nine chunks, with resets, lengths and both types of gradient."""
    t = lru_inputs(Bt, Dn, L, dtype, seed=L)
    kw = options(t, ("r_bias", "i_bias", "h0") + (("reset", "lengths") if packed else ()))
    args = (t["x"], t["r"], t["i"], t["lam"])
    want = layer_bounds.lru(*args, dout=t["dout"], dh_last=t["dh_last"], **kw)
    f = ssm.ssm_lru_fwd(*args, save_states=True, return_state=True, **kw)
    compare(f, want, ref.HALF[dtype])
    for grad in (F32, BF):
        g = ssm.ssm_lru_bwd(t["dout"], *args, chunk_states=f["chunk_states"], dh_last=t["dh_last"], grad_dtype=grad, **kw)
        compare(g, want, None, ref.HALF[grad])


@pytest.mark.parametrize("dtype,dout", [(BF, F32), (F32, F32), (BF, BF)])
@pytest.mark.parametrize("time,case", [
    (False, (2, 20000, 6, 2, 32, 32)), (False, (1, 30011, 5, 0, 40, 24)), (False, (3, 9001, 4, 1, 33, 18)), (False, (2, 4096, 8, 2, 128, 128)),
    (True, (4, 40000, 1, 1, 16, 16)), (True, (2, 24008, 2, 1, 48, 32)), (True, (1, 30001, 2, 1, 20, 20)), (True, (3, 8203, 1, 1, 40, 40))])
def test_weight_gradients_of_many_blocks(time, case, dtype, dout):
    """dw against float64 with a bound of the kernels' own chains: 128 EPS for a row's share; a group of lanes adds its rows, a quarter more than an
    even cut of them over 296 blocks of at least eight groups; a block its 256 groups at most; the last sum 10 shares and 5 exchanges. The
    bound is far below dw itself, so that shares lost or added twice show."""
    Bt, L, Hq, Hk, D, rot = case
    t = qk_inputs(Bt, L, Hq, Hk, D, dtype, time, seed=D, dout=dout)
    kw = dict(inv_freq=freq(rot), positions=t["positions"], interleaved=D == 40, layout="bhdl" if time else "blhd")
    g = ssm.ssm_qk_norm_rope_bwd(t["dq_out"], t["q"], t["dk_out"], t["k"], q_weight=t["q_weight"], k_weight=t["k_weight"], grad_dtype=BF, **kw)
    for side, H in (("q", Hq), ("k", Hk)):
        if not H:
            continue
        want = ref.qk(t[side], t[side + "_weight"], kw["inv_freq"], t["positions"], True, 1e-6, D == 40, 1.0, time, t["d%s_out" % side])
        v, b = want["dw"]
        rows = Bt * L * H
        absolute = b / ((128.0 + rows) * ref.EPS)  # the sum over rows of the terms' absolute values
        bound = (128.0 + 1.25 * rows / (296 * 8) + 256 + 16) * ref.EPS * absolute
        assert float(bound.max()) < 0.05 * float(v.square().mean().sqrt())
        ref.check("d%s_weight" % side, g["d%s_weight" % side], v, bound + ref.EPS * v.abs())


@pytest.mark.parametrize("time", [False, True])
def test_queries_and_keys_past_32_bits(time):
    """The last elements of tensors of more than 2^31 are those of a call on them alone, bit for bit."""
    n, D = 40, 128
    if time:
        shape, D = (2, 2, 16, 2 ** 25 + n), 16
    else:
        shape = (1, 2 ** 21 + n, 8, D)
    L = shape[3] if time else shape[1]
    q = torch.empty(shape, dtype=BF, device="cuda").normal_()
    assert q.numel() > 2 ** 31
    last = (lambda v: v[-1:, -1:, :, L - n:].contiguous()) if time else (lambda v: v[:, L - n:].contiguous())  # noqa: E731
    kw = dict(q_weight=torch.linspace(0.5, 1.5, D).cuda(), inv_freq=freq(D, torch.float64), layout="bhdl" if time else "blhd")
    out, _ = ssm.ssm_qk_norm_rope_fwd(q, None, **kw)
    small, _ = ssm.ssm_qk_norm_rope_fwd(last(q), None, pos0=L - n, **kw)
    assert torch.equal(last(out), small)
    del out
    g = ssm.ssm_qk_norm_rope_bwd(q, q, grad_dtype=BF, **kw)["dq"]
    s = ssm.ssm_qk_norm_rope_bwd(last(q), last(q), grad_dtype=BF, pos0=L - n, **kw)["dq"]
    assert torch.equal(last(g), s)


def test_recurrence_backward_past_32_bits():
    """Rows beyond 2^31 elements against the same rows in tensors of their own, as many as take the same plan."""
    Dn, L, rows = 4104, 524288, 1184
    x = torch.empty(1, Dn, L, dtype=BF, device="cuda").normal_()
    lam = torch.linspace(-6.0, -2.0, Dn).cuda()
    reset = torch.zeros(1, L, dtype=torch.bool, device="cuda")
    reset[0, ::1000] = True
    g = ssm.ssm_lru_bwd(x, x, x, x, lam, reset=reset, grad_dtype=BF)
    last = x[:, -rows:].contiguous()
    s = ssm.ssm_lru_bwd(last, last, last, last, lam[-rows:].contiguous(), reset=reset, grad_dtype=BF)
    for k in ("dx", "dr", "di"):
        assert torch.equal(g[k][:, -rows:], s[k]), k
    assert torch.equal(g["dlam"][-rows:], s["dlam"])


def test_dual_step_past_32_bits():
    Bt, H, P, N, n = 1032, 64, 128, 256, 8
    h = torch.empty(Bt, H, N, P, device="cuda").normal_()
    assert h.numel() > 2 ** 31
    x, dt = torch.randn(Bt, H, P, device="cuda").to(BF), torch.randn(Bt, H, device="cuda").to(BF)
    B, C = (torch.randn(Bt, N, device="cuda").to(BF) for _ in range(2))
    A_log = torch.linspace(0.0, 2.0, H).cuda()
    own = [v[-n:].clone() for v in (x, dt, B, C, h)]
    y = ssm.ssm_ssd_step(x, dt, A_log, B, C, h)
    z = ssm.ssm_ssd_step(own[0], own[1], A_log, own[2], own[3], own[4])
    assert torch.equal(y[-n:], z) and torch.equal(h[-n:], own[4])
