"""Gradients of the gated linear recurrence where a gate or a decay is extreme, against float64 with bounds from the derivative's own terms
(layer_bounds): decays next to 1, gates held open, channels that forget at once."""
import pytest
import torch

import layer_bounds
import layer_refs as ref
import selective_state_space_34_b200 as ssm
from test_gpu_lru import compare, inputs, options

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
# rows that share warps; one warp a row, two chunks; four and eight warps; one again, three chunks
SIZES = [(2, 18, 40), (1, 18, 300), (1, 18, 700), (1, 18, 1100), (2, 1188, 700)]


@pytest.fixture(autouse=True)
def _poisoned():
    ref.poison_shared()


def run_and_check(t, names, grad=F32):
    kw = options(t, names)
    args = (t["x"], t["r"], t["i"], t["lam"])
    want = layer_bounds.lru(*args, dout=t["dout"], dh_last=t["dh_last"], **kw)
    f = ssm.ssm_lru_fwd(*args, save_states=True, return_state=True, **kw)
    compare(f, want, ref.HALF[t["x"].dtype])
    g = ssm.ssm_lru_bwd(t["dout"], *args, chunk_states=f["chunk_states"], dh_last=t["dh_last"], grad_dtype=grad, **kw)
    compare(g, want, None, ref.HALF[grad])
    return want


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("Bt,Dn,L", SIZES)
def test_decays_next_to_one(Bt, Dn, L, dtype):
    """softplus(lam) from 1e-26 down to denormals and to 0: finite, and the formula's values but for what 1e-36 in y adds."""
    t = inputs(Bt, Dn, L, dtype, seed=L)
    slow = torch.tensor([-60.0, -75.0, -80.0, -85.0, -87.0, -90.0, -91.0, -92.0, -95.0, -100.0, -103.0, -103.5, -104.0, -200.0])
    t["lam"] = slow.repeat(Dn // len(slow) + 1)[:Dn].cuda()
    want = run_and_check(t, ("r_bias", "i_bias", "h0"))
    assert all(bool(v.isfinite().all()) for v, _ in want.values())
    assert float(want["dr"][1].abs().max()) < 1e-12  # the bound tells a value of 1 from 0


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("bias", [6.0, 12.0, 20.0])
@pytest.mark.parametrize("Bt,Dn,L", SIZES[:2])
def test_gates_held_open(Bt, Dn, L, bias, dtype):
    """1 - r and 1 - g keep their digits: dr and di carry them as factors."""
    t = inputs(Bt, Dn, L, dtype, seed=L)
    t["r_bias"], t["i_bias"] = t["r_bias"] + bias, t["i_bias"] + bias
    t["lam"] = torch.linspace(-7.0, -4.0, Dn).cuda()
    run_and_check(t, ("r_bias", "i_bias", "h0"))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("Bt,Dn,L", SIZES)
def test_channels_that_forget_at_once(Bt, Dn, L, packed, dtype):
    """Decays from 0.6 down to e^-60 a step, some gates open: what is left of the gradient of the decay is of the size of the decay
    itself, not of the input's rounding."""
    t = inputs(Bt, Dn, L, dtype, seed=L + 1)
    t["lam"] = torch.linspace(-3.0, 7.5, Dn).cuda()
    t["r_bias"] = torch.linspace(-2.0, 4.0, Dn).flip(0).roll(Dn // 3).cuda()
    run_and_check(t, ("r_bias", "i_bias", "h0") + (("reset", "lengths") if packed else ()))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("Bt,Dn,L", SIZES)
def test_nan_stays_in_a_sequence_that_forgets(Bt, Dn, L, dtype):
    """Factors that underflow are no cuts: a NaN reaches the end of its own packed sequence forwards, and its start backwards, and no
    further, whether or not a sequence starts in the same chunk."""
    t = inputs(Bt, Dn, L, dtype, seed=L)
    t["lam"] = torch.linspace(-1.0, 7.0, Dn).cuda()
    t["r_bias"] = torch.full((Dn,), 2.0, device="cuda")
    starts = sorted({0, L // 7, L // 7 + 3, L // 2, L // 2 + 1, L - 2})
    reset = torch.zeros(Bt, L, dtype=torch.bool, device="cuda")
    reset[:, starts] = True
    args = lambda x: (x, t["r"], t["i"], t["lam"], t["r_bias"])  # noqa: E731
    clean = ssm.ssm_lru_fwd(*args(t["x"]), reset=reset, save_states=True)
    g0 = ssm.ssm_lru_bwd(t["dout"], *args(t["x"]), reset=reset, chunk_states=clean["chunk_states"])
    step = torch.arange(L, device="cuda")
    for lo, hi in zip(starts, starts[1:] + [L]):
        for at in {lo, (lo + hi) // 2, hi - 1}:
            x, d = t["x"].clone(), t["dout"].clone()
            x[..., at] = d[..., at] = float("nan")
            out = ssm.ssm_lru_fwd(*args(x), reset=reset)
            ours = (step >= at) & (step < hi)
            assert bool(out[..., ours].isnan().all()) and torch.equal(out[..., ~ours], clean["out"][..., ~ours]), (lo, hi, at)
            g = ssm.ssm_lru_bwd(d, *args(t["x"]), reset=reset, chunk_states=clean["chunk_states"])
            ours = (step >= lo) & (step <= at)
            for k in ("dx", "di", "dr"):
                assert bool(g[k][..., ours].isnan().all()) and torch.equal(g[k][..., ~ours], g0[k][..., ~ours]), (k, lo, hi, at)
