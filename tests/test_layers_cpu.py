"""Host-side checks of the recurrence's, the queries' and keys' and the dual step's entry points that need no GPU:
struct layouts, the documented status codes (only invalid or empty arguments are passed), the binding's refusals and the
rotation frequencies."""
import ctypes
import math

import pytest
import torch

import layer_refs as ref
import selective_state_space_34_b200 as ssm
from selective_state_space_34_b200 import _abi, build
from test_abi_cpu import _header_fields


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _abi.load()


@pytest.mark.parametrize("struct,cls,size", [
    ("ssm_lru_args", "LruArgs", 12 * 8 + 3 * 8 + 4 + 2 * 4 + 4),
    ("ssm_lru_bwd_args", "LruBwdArgs", 136 + 9 * 8 + 8 + 8 + 8),
    ("ssm_lru_step_args", "LruStepArgs", 8 * 8 + 2 * 8 + 4 + 2 * 4 + 4),
    ("ssm_qk_args", "QkArgs", 8 * 8 + 12 * 8 + 7 * 8 + 2 * 4 + 7 * 4 + 4),
    ("ssm_qk_bwd_args", "QkBwdArgs", 256 + 4 * 8 + 6 * 8 + 2 * 8 + 2 * 4 + 8 + 8),
    ("ssm_ssd_step_args", "SsdStepArgs", 9 * 8 + 4 * 8 + 4 * 4),
])
def test_struct_layout(struct, cls, size):
    ct = getattr(_abi, cls)
    assert [f[0] for f in ct._fields_] == _header_fields(struct)
    assert ctypes.sizeof(ct) == size


def _set(a, names, base=0x10000, **kw):
    for j, n in enumerate(names.split()):
        setattr(a, n, base * (j + 1))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _lru(**kw):
    return _set(_abi.LruArgs(), "x r i lam out", **{**dict(Bt=2, Dn=8, L=32, c=8.0, in_dtype=1, out_dtype=1), **kw})


def test_lru_codes(lib):
    f = lambda **kw: lib.ssm_lru_fwd(ctypes.byref(_lru(**kw)), None)  # noqa: E731
    assert lib.ssm_lru_fwd(None, None) == 1
    assert [f(**{n: None}) for n in ("x", "r", "i", "lam", "out")] == [1] * 5
    assert f(Bt=-1) == 2 and f(Dn=0) == 2 and f(L=-1) == 2 and f(Bt=1 << 40, Dn=1 << 30) == 2
    assert f(x=0x10001) == 3 and f(out=0x10001) == 3 and f(h0=0x10002) == 3 and f(lengths=0x10002) == 3
    assert f(in_dtype=2) == 4 and f(out_dtype=-1) == 4
    assert f(c=0.0) == 5 and f(c=-8.0) == 5 and f(c=math.nan) == 5 and f(c=math.inf) == 5
    assert f(Bt=0, x=None) == 0 and f(L=0, out=None) == 0
    assert lib.ssm_lru_num_states(0) == 0 and lib.ssm_lru_num_states(-4) == 0
    assert [lib.ssm_lru_num_states(n) for n in (1, 249, 250, 256, 505, 506)] == [1, 1, 2, 2, 2, 3]


def test_lru_backward_codes(lib):
    def bw(fwd=None, **kw):
        a = _set(_abi.LruBwdArgs(), "dout dx dr di dlam", base=0x100000, **kw)
        a.fwd = _lru(**(fwd or {}))
        return a

    f = lambda *p, **kw: lib.ssm_lru_bwd(ctypes.byref(bw(*p, **kw)), None)  # noqa: E731
    size = lambda *p, **kw: lib.ssm_lru_bwd_workspace_size(ctypes.byref(bw(*p, **kw)))  # noqa: E731
    assert lib.ssm_lru_bwd(None, None) == 1 and lib.ssm_lru_bwd_workspace_size(None) == 0
    assert f(dout=None) == 1 and f({"x": None}) == 1
    assert f(grad_dtype=9) == 4 and f(dx=0x100001) == 3 and f(dlam=0x100002) == 3
    assert f({"out": None}) == 7  # the output is not an argument of the backward; no workspace
    # one state a row (32 steps), 16 rows, and one array of row sums
    assert size() == 256 + 256 and size({"chunk_states": 0x900000}) == 256
    assert size({"chunk_states": 0x900000, "Bt": 1}) == 0
    assert size({"chunk_states": 0x900000}, dlam=None) == 0
    assert size({"chunk_states": 0x900000}, dr_bias=0x800000, di_bias=0x810000) == 3 * 256
    assert f(workspace=0x900010, workspace_bytes=512) == 7 and f(workspace=0x900100, workspace_bytes=511) == 7
    assert size({"L": 0}) == 0 and size({"c": -1.0}) == 0


def test_lru_step_codes(lib):
    def f(**kw):
        a = _set(_abi.LruStepArgs(), "x r i lam h out", **{**dict(Bt=2, Dn=8, c=8.0, in_dtype=1, out_dtype=1), **kw})
        return lib.ssm_lru_step(ctypes.byref(a), None)

    assert lib.ssm_lru_step(None, None) == 1 and f(h=None) == 1 and f(out=None) == 1
    assert f(Dn=0) == 2 and f(Bt=-1) == 2 and f(h=0x10002) == 3 and f(x=0x10001) == 3
    assert f(in_dtype=7) == 4 and f(c=0.0) == 5 and f(Bt=0, x=None) == 0


def _qk(**kw):
    base = dict(Bt=2, L=6, Hq=4, Hk=2, D=64, rot=64, eps=1e-6, rot_scale=1.0, norm=1, in_dtype=1, out_dtype=1,
                q_sb=6 * 256, q_sh=64, q_sr=256, q_out_sb=6 * 256, q_out_sh=64, q_out_sr=256,
                k_sb=6 * 128, k_sh=64, k_sr=128, k_out_sb=6 * 128, k_out_sh=64, k_out_sr=128)
    return _set(_abi.QkArgs(), "q k inv_freq q_out k_out", **{**base, **kw})


def test_qk_codes(lib):
    f = lambda **kw: lib.ssm_qk_norm_rope_fwd(ctypes.byref(_qk(**kw)), None)  # noqa: E731
    assert lib.ssm_qk_norm_rope_fwd(None, None) == 1
    assert [f(**{n: None}) for n in ("q", "k", "inv_freq", "q_out", "k_out")] == [1] * 5
    assert f(D=0) == 2 and f(rot=3) == 2 and f(rot=66) == 2 and f(rot=-2) == 2 and f(Hq=-1) == 2 and f(L=-1) == 2
    assert f(Bt=1 << 40, L=1 << 40) == 2 and f(Hq=1 << 25) == 2
    assert f(D=513) == 5 and f(layout=2) == 5 and f(eps=-1.0) == 5 and f(eps=math.nan) == 5
    assert f(norm=0, q_weight=0x80000) == 5
    assert f(q=0x10001) == 3 and f(k_out=0x10001) == 3 and f(inv_freq=0x10004, freq_f64=1) == 3
    assert f(positions=0x10004, pos_i64=1) == 3 and f(q_weight=0x10002) == 3
    assert f(in_dtype=3) == 4 and f(out_dtype=3) == 4
    assert f(Bt=0, q=None) == 0 and f(L=0) == 0 and f(Hq=0, Hk=0, q=None) == 0
    # outputs that overlap themselves: repeated, or heads inside each other
    assert f(q_out_sb=0) == 2 and f(q_out_sh=63) == 2 and f(k_out_sr=-128) == 2 and f(q_out_sr=192) == 2


def test_qk_backward_codes(lib):
    def bw(fwd=None, **kw):
        base = dict(dq_sb=6 * 256, dq_sh=64, dq_sr=256, dk_sb=6 * 128, dk_sh=64, dk_sr=128, dout_dtype=1, grad_dtype=0)
        a = _set(_abi.QkBwdArgs(), "dq_out dk_out dq dk", base=0x100000, **{**base, **kw})
        a.fwd = _qk(**(fwd or {}))
        return a

    f = lambda *p, **kw: lib.ssm_qk_norm_rope_bwd(ctypes.byref(bw(*p, **kw)), None)  # noqa: E731
    size = lambda *p, **kw: lib.ssm_qk_norm_rope_bwd_workspace_size(ctypes.byref(bw(*p, **kw)))  # noqa: E731
    assert lib.ssm_qk_norm_rope_bwd(None, None) == 1 and lib.ssm_qk_norm_rope_bwd_workspace_size(None) == 0
    assert f(dq_out=None) == 1 and f(dk_out=None) == 1 and f({"q": None}) == 1
    assert f(dout_dtype=5) == 4 and f(grad_dtype=5) == 4 and f(dq=0x100002) == 3
    assert f(dq_sh=32) == 2 and f({"norm": 0}, dq_weight=0x900000) == 5
    assert size() == 0 and size(dq_weight=0x900000) > 0
    assert f(dq_weight=0x900000) == 7 and f(dq_weight=0x900000, workspace=0x900010, workspace_bytes=1 << 30) == 7
    assert size({"L": 0}, dq_weight=0x900000) == 0 and f({"L": 0}) == 0


def test_ssd_step_codes(lib):
    def f(**kw):
        a = _set(_abi.SsdStepArgs(), "x dt A_log B C h out", **{**dict(Bt=2, H=3, P=64, N=64, in_dtype=1, out_dtype=1), **kw})
        return lib.ssm_ssd_step(ctypes.byref(a), None)

    assert lib.ssm_ssd_step(None, None) == 1
    assert [f(**{n: None}) for n in ("x", "dt", "A_log", "B", "C", "h", "out")] == [1] * 7
    assert f(H=0) == 2 and f(Bt=-1) == 2 and f(P=0) == 2 and f(Bt=1 << 40, H=1 << 30) == 2
    assert f(P=257) == 5 and f(N=257) == 5 and f(discretization=2) == 5
    assert f(h=0x10002) == 3 and f(x=0x10001) == 3 and f(in_dtype=4) == 4 and f(Bt=0, x=None) == 0


def test_binding_refuses_cpu_tensors_and_wrong_options():
    x = torch.zeros(1, 2, 8)
    with pytest.raises(ValueError, match="CUDA"):
        ssm.ssm_lru_fwd(x, x, x, torch.zeros(2))
    with pytest.raises(ValueError, match="CUDA"):
        ssm.ssm_lru_bwd(x, x, x, x, torch.zeros(2))
    with pytest.raises(ValueError, match="CUDA"):
        ssm.ssm_lru_step(x[..., 0], x[..., 0], x[..., 0], torch.zeros(2), torch.zeros(1, 2))
    with pytest.raises(ValueError, match="CUDA"):
        ssm.ssm_qk_norm_rope_fwd(torch.zeros(1, 2, 3, 4))
    with pytest.raises(ValueError, match="CUDA"):
        ssm.ssm_qk_norm_rope_bwd(torch.zeros(1, 2, 3, 4), torch.zeros(1, 2, 3, 4))
    with pytest.raises(ValueError, match="CUDA"):
        ssm.ssm_ssd_step(x, x[..., 0], torch.zeros(2), x[0], x[0], torch.zeros(1, 2, 8, 8))
    with pytest.raises(TypeError):
        ssm.ssm_lru_fwd(None, x, x, torch.zeros(2))
    for bad in (dict(rot=3), dict(rot=0), dict(rot=8, scaling="x"), dict(rot=8, factor=0.5), dict(rot=8, base=-1.0),
                dict(rot=8, turns_low=4.0, turns_high=4.0)):
        with pytest.raises(ValueError):
            ssm.ssm_rope_inv_freq(**bad)


def test_rotation_frequencies():
    f, s = ssm.ssm_rope_inv_freq(8, 10000.0)
    assert s == 1.0 and f.dtype == torch.float64
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-14, atol=0)
    lin, _ = ssm.ssm_rope_inv_freq(8, scaling="linear", factor=4.0)
    assert torch.equal(lin, f / 4)
    ntk, _ = ssm.ssm_rope_inv_freq(8, scaling="ntk", factor=4.0)
    assert ntk[0] == f[0] and math.isclose(float(ntk[-1]), float(f[-1]) / 4, rel_tol=1e-12)
    yarn, s = ssm.ssm_rope_inv_freq(8, scaling="yarn", factor=4.0, original_length=4096)
    assert math.isclose(s, 0.1 * math.log(4.0) + 1)
    # turns over 4096 tokens: 652, 65, 6.5, 0.65 -- unchanged, unchanged, between, divided
    assert yarn[0] == f[0] and yarn[1] == f[1] and math.isclose(float(yarn[3]), float(f[3]) / 4, rel_tol=1e-12)
    keep = (4096 * 0.01 / (2 * math.pi) - 1) / 31
    assert math.isclose(float(yarn[2]), 0.01 * (keep + (1 - keep) / 4), rel_tol=1e-9)


def test_reference_recurrence_against_autograd():
    """The reference's hand-written gradients against float64 autograd of the recurrence."""
    g = torch.Generator().manual_seed(0)
    n = lambda *s: torch.randn(s, generator=g).double()  # noqa: E731
    Bt, Dn, L = 2, 3, 9
    p = {"x": n(Bt, Dn, L), "r": n(Bt, Dn, L), "i": n(Bt, Dn, L), "lam": n(Dn) - 3, "r_bias": n(Dn), "i_bias": n(Dn),
         "h0": n(Bt, Dn)}
    reset = torch.rand(Bt, L, generator=g) < 0.3
    lengths = torch.tensor([9, 5], dtype=torch.int32)
    dout, dh = n(Bt, Dn, L), n(Bt, Dn)
    want = ref.lru(**p, reset=reset, lengths=lengths, dout=dout, dh_last=dh)
    q = {k: v.clone().requires_grad_() for k, v in p.items()}
    h, loss = q["h0"], 0.0
    for t in range(L):
        a = torch.exp(-8.0 * torch.nn.functional.softplus(q["lam"]) * torch.sigmoid(q["r"][..., t] + q["r_bias"]))
        new = a * h * (~reset[:, t, None]) + torch.sqrt(1 - a * a) * torch.sigmoid(q["i"][..., t] + q["i_bias"]) * q["x"][..., t]
        live = (t < lengths)[:, None]
        loss = loss + (torch.where(live, new, 0 * new) * dout[..., t]).sum()
        h = torch.where(live, new, h)
    (loss + (h * dh).sum()).backward()
    for k in p:
        assert torch.allclose(want["d" + k][0], q[k].grad, rtol=1e-9, atol=1e-11), k


def test_reference_rows_against_autograd():
    g = torch.Generator().manual_seed(0)
    for interleaved, time in ((False, False), (True, True)):
        v = torch.randn(2, 3, 4, 6, generator=g).double().requires_grad_()
        w = torch.randn(6, generator=g).double().requires_grad_()
        f = torch.tensor([1.0, 0.3]).double()
        L = 6 if time else 3
        pos = torch.randint(0, 1000, (2, L), generator=g)
        if time:
            w = torch.randn(4, generator=g).double().requires_grad_()
        d = torch.randn(2, 3, 4, 6, generator=g).double()
        rows = v.permute(0, 3, 1, 2) if time else v
        n = rows / torch.sqrt((rows ** 2).mean(-1, keepdim=True) + 1e-3) * w
        angle = pos.double()[:, :, None, None] * f
        z = torch.view_as_complex(n[..., :4].unflatten(-1, (2, 2)).contiguous()) if interleaved else \
            torch.complex(n[..., 0:2], n[..., 2:4])
        z = z * torch.polar(torch.full_like(angle, 1.5), angle)
        o = torch.view_as_real(z).flatten(-2) if interleaved else torch.cat([z.real, z.imag], -1)
        o = torch.cat([o, n[..., 4:]], -1)
        o = o.permute(0, 2, 3, 1) if time else o
        (o * d).sum().backward()
        want = ref.qk(v.detach(), w.detach(), f, pos, True, 1e-3, interleaved, 1.5, time, d)
        assert torch.allclose(want["out"][0], o.detach(), rtol=1e-11)
        assert torch.allclose(want["d"][0], v.grad, rtol=1e-9, atol=1e-11)
        assert torch.allclose(want["dw"][0], w.grad, rtol=1e-9, atol=1e-11)
