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
