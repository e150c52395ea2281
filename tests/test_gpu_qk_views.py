"""Views of queries and keys that users' programs make: axes of length 1 with any stride."""
import pytest
import torch

import layer_refs as ref
import selective_state_space_34_b200 as ssm
from test_gpu_qk import freq, inputs

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _poisoned():
    ref.poison_shared()


@pytest.mark.parametrize("axis", [0, 1, 2])
@pytest.mark.parametrize("D", [64, 80])
def test_strides_of_axes_of_length_one_do_not_matter(axis, D):
    """A view whose only batch element, token or head has an odd stride runs as the dense tensor does: the same bits (element by element
    the sums would be added up in another order)."""
    shape = [3, 40, 4]
    shape[axis] = 1
    t = inputs(shape[0], shape[1], shape[2], 0, D, BF, dout=F32)
    kw = dict(q_weight=t["q_weight"], inv_freq=freq(D), positions=t["positions"])

    def view(v):
        strides = list(v.stride())
        strides[axis] = 7
        return v.as_strided(v.shape, strides)

    want, _ = ssm.ssm_qk_norm_rope_fwd(t["q"], None, out_dtype=F32, **kw)
    out = torch.zeros_like(want)
    ssm.ssm_qk_norm_rope_fwd(view(t["q"]), None, out_dtype=F32, out=(view(out), None), **kw)
    assert torch.equal(out, want)
    g = ssm.ssm_qk_norm_rope_bwd(t["dq_out"], t["q"], **kw)
    h = ssm.ssm_qk_norm_rope_bwd(view(t["dq_out"]), view(t["q"]), **kw)
    assert all(torch.equal(g[n], h[n]) for n in g)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("time,D", [(False, 64), (False, 33), (False, 80), (True, 16), (True, 33), (True, 200)])
def test_rows_whose_squares_are_subnormal(time, D, dtype):
    """An eps of 0 counts as 2^-126: rows of 1e-20 and of zeros have finite results and gradients, those of the formula with that eps.
    (Squares of 1e-40 are off by 2^-150 each and in their sum: 2^-23 of an eps of 2^-126, inside the bounds' 64 and 128 EPS.)"""
    t = inputs(2, 24, 2, 1, D, dtype, time, seed=D)
    for n in ("q", "k"):
        t[n] = (t[n].float() * 1e-20).to(dtype)
        ref.qk_rows(t[n], time)[:, 3] = 0.0
    f = freq(D // 2 * 2)
    kw = dict(q_weight=t["q_weight"], k_weight=t["k_weight"], inv_freq=f, positions=t["positions"], layout="bhdl" if time else "blhd")
    out = ssm.ssm_qk_norm_rope_fwd(t["q"], t["k"], out_dtype=F32, eps=0.0, **kw)
    g = ssm.ssm_qk_norm_rope_bwd(t["dq_out"], t["q"], t["dk_out"], t["k"], eps=0.0, **kw)
    for side, o in zip("qk", out):
        want = ref.qk(t[side], t[side + "_weight"], f, t["positions"], True, 2.0 ** -126, False, 1.0, time, t["d%s_out" % side])
        for name, got, (v, b) in ((side + "_out", o, want["out"]), ("d" + side, g["d" + side], want["d"]),
                                  ("d%s_weight" % side, g["d%s_weight" % side], want["dw"])):
            ref.check(name, got, v, b + ref.EPS * v.abs() + 1e-37)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("time,D", [(False, 64), (False, 33), (False, 80), (True, 16), (True, 33), (True, 200)])
def test_frequencies_that_are_no_numbers(time, D, interleaved, dtype):
    """A NaN or infinite frequency makes its pair's elements NaN, both ways, and leaves the others' bits as they are."""
    t = inputs(2, 24, 2, 1, D, dtype, time, seed=D)
    rot = D // 2 * 2
    f = freq(rot)
    kw = dict(positions=t["positions"], interleaved=interleaved, layout="bhdl" if time else "blhd", norm=False)
    axis = 2 if time else 3
    for bad in (float("nan"), float("inf"), -float("inf")):
        j = rot // 4
        e = f.clone()
        e[j] = bad
        pair = [2 * j, 2 * j + 1] if interleaved else [j, j + rot // 2]
        rest = torch.tensor([n for n in range(D) if n not in pair], device="cuda")
        pair = torch.tensor(pair, device="cuda")
        results = []
        for inv_freq in (f, e.double() if bad > 0 else e):
            g = ssm.ssm_qk_norm_rope_bwd(t["dq_out"], t["q"], t["dk_out"], t["k"], inv_freq=inv_freq, **kw)
            results.append(list(ssm.ssm_qk_norm_rope_fwd(t["q"], t["k"], inv_freq=inv_freq, **kw)) + [g["dq"], g["dk"]])
        for good, got in zip(*results):
            assert bool(got.index_select(axis, pair).isnan().all())
            assert torch.equal(got.index_select(axis, rest), good.index_select(axis, rest))


def test_outputs_without_room_leave_no_memory_behind():
    """The keys' output does not fit the device: the call fails as torch's allocations do, and the queries' output, made before, is freed."""
    q = torch.zeros(1, 1 << 16, 1, 64, dtype=BF, device="cuda")
    k = q[:, :, :1].expand(1, 1 << 16, 1 << 20, 64)  # 8 TiB of results
    with pytest.raises(torch.OutOfMemoryError):
        ssm.ssm_qk_norm_rope_fwd(q, k, inv_freq=freq(64))
    before = torch.cuda.memory_allocated()
    for _ in range(3):
        with pytest.raises(torch.OutOfMemoryError):
            ssm.ssm_qk_norm_rope_fwd(q, k, inv_freq=freq(64))
    assert torch.cuda.memory_allocated() == before
