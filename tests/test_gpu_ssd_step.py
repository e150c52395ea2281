"""The state-space-dual step against float64, continuing ssm_ssd_fwd; and the new operators run together as
recurrent layers use them: normalised and rotated B and C in front of the scan and the dual, the gated recurrence behind."""
import ctypes

import pytest
import torch

import layer_refs as ref
import selective_state_space_34_b200 as ssm
from selective_state_space_34_b200 import _abi
from test_gpu_guard import GuardedTorch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _poisoned():
    ref.poison_shared()


def inputs(Bt, H, P, N, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0: torch.randn(s, generator=g) * std  # noqa: E731
    t = {"x": n(Bt, H, P), "dt": n(Bt, H), "B": n(Bt, N, std=0.3), "C": n(Bt, N, std=0.3)}
    t = {k: v.to(dtype).cuda() for k, v in t.items()}
    t.update(A_log=torch.log(torch.rand(H, generator=g) * 15 + 1).cuda(), D=n(H).cuda(), dt_bias=(n(H) - 3).cuda(),
             h=n(Bt, H, N, P).cuda())
    return t


@pytest.mark.parametrize("dtype,out_dtype", [(F32, F32), (BF, BF), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("Bt,H,P,N", [(1, 1, 1, 1), (2, 3, 64, 128), (1, 24, 64, 64), (3, 2, 33, 7), (2, 5, 96, 33),
                                      (1, 2, 256, 256), (40, 9, 16, 20), (2, 2, 250, 3)])
def test_step(Bt, H, P, N, dtype, out_dtype):
    for euler, soft, extra in ((False, True, True), (True, True, False), (False, False, True)):
        t = inputs(Bt, H, P, N, dtype, seed=P)
        if not soft:
            t["dt"].abs_()
            t["dt_bias"].abs_()
        kw = dict(D=t["D"], dt_bias=t["dt_bias"]) if extra else {}
        want = ref.ssd_step(t["x"], t["dt"], t["A_log"], t["B"], t["C"], t["h"], softplus_on=soft, euler=euler, **kw)
        y = ssm.ssm_ssd_step(t["x"], t["dt"], t["A_log"], t["B"], t["C"], t["h"], delta_softplus=soft,
                             discretization="euler" if euler else "zoh", out_dtype=out_dtype, **kw)
        assert y.dtype == out_dtype
        v, b = want["out"]
        ref.check("out", y, v, b + ref.HALF[out_dtype] * (v.abs() + b) + 1e-37)
        v, b = want["h"]
        ref.check("h", t["h"], v, b + ref.EPS * v.abs() + 1e-37)


def test_state_off_the_vector_boundary():
    t = inputs(2, 3, 64, 16, BF)
    buf = torch.empty(t["h"].numel() + 1, device="cuda")
    h = buf[1:].view(t["h"].shape).copy_(t["h"])
    a = ssm.ssm_ssd_step(t["x"], t["dt"], t["A_log"], t["B"], t["C"], t["h"])
    b = ssm.ssm_ssd_step(t["x"], t["dt"], t["A_log"], t["B"], t["C"], h)
    assert torch.equal(h, t["h"])  # every state element is its own
    assert torch.allclose(a.float(), b.float(), rtol=2.0 ** -7, atol=1e-5)


def test_dual_layer_prefill_and_decode_with_rotated_states():
    """C and B normalised and rotated in front of the dual, a prompt in one call and 5 tokens by steps, against
    the recurrence with complex decay a_t e^{i w_j} that the rotation stands for (pairs of states)."""
    Bt, H, L, P, N, steps = 2, 3, 200, 64, 64, 5
    T = L + steps
    g = torch.Generator().manual_seed(0)
    n = lambda *s, std=1.0: torch.randn(s, generator=g) * std  # noqa: E731
    x, dt = n(Bt, H, T, P).to(BF).cuda(), n(Bt, H, T).to(BF).cuda()
    B, C = n(Bt, T, 1, N).to(BF).cuda(), n(Bt, T, 1, N).to(BF).cuda()
    wq, wk = (0.3 + 0.05 * n(N)).cuda(), (0.3 + 0.05 * n(N)).cuda()
    A_log, D, bias = torch.log(torch.rand(H, generator=g) * 4 + 1).cuda(), n(H).cuda(), (n(H) - 3).cuda()
    f, scale = ssm.ssm_rope_inv_freq(N, scaling="yarn", factor=4.0, device="cuda")
    kw = dict(q_weight=wq, k_weight=wk, inv_freq=f, rot_scale=scale)
    Cr, Br = ssm.ssm_qk_norm_rope_fwd(C[:, :L], B[:, :L], **kw)
    y, h = ssm.ssm_ssd_fwd(x[:, :, :L].contiguous(), dt[:, :, :L].contiguous(), A_log, Br[:, :, 0], Cr[:, :, 0], D=D,
                           dt_bias=bias, return_state=True, out_dtype=F32)
    ys = [y]
    for t in range(L, T):
        Ct, Bt_ = ssm.ssm_qk_norm_rope_fwd(C[:, t:t + 1], B[:, t:t + 1], pos0=t, **kw)
        ys.append(ssm.ssm_ssd_step(x[:, :, t].contiguous(), dt[:, :, t].contiguous(), A_log, Bt_[:, 0, 0], Ct[:, 0, 0], h,
                                   D=D, dt_bias=bias, out_dtype=F32)[:, :, None])
    got = ref.d64(torch.cat(ys, 2))
    # complex form: s_t = a_t s_{t-1} e^{-i w} + beta b_t x_t, y = Re(conj(c) s) scale^2, of unrotated c, b
    unit = lambda v, w: (v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6) * w)[:, :, 0]  # noqa: E731
    b64, c64 = unit(ref.d64(B), ref.d64(wk)), unit(ref.d64(C), ref.d64(wq))
    z = lambda v: torch.complex(v[..., :N // 2], v[..., N // 2:])  # noqa: E731
    bz, cz = z(b64), z(c64)
    w = f.cpu()
    back = torch.polar(torch.ones_like(w), -w)
    delta = ref.softplus(ref.d64(dt) + ref.d64(bias)[:, None])
    rate = torch.exp(ref.d64(A_log))[:, None]
    a, beta = torch.exp(-delta * rate), -torch.expm1(-delta * rate) / rate
    s = torch.zeros(Bt, H, N // 2, P, dtype=torch.complex128)
    absolute = torch.zeros(Bt, H, P).double()
    xs = ref.d64(x)
    for t in range(T):
        s = a[:, :, t, None, None] * back[:, None] * s + (beta[:, :, t, None] * bz[:, None, t])[..., None] * xs[:, :, t, None]
        # the same over absolute values: |c| . |b| bounds every term of the sum over states
        absolute = a[:, :, t, None] * absolute + (beta[:, :, t] * (bz[:, t].abs().max(-1).values)[:, None])[..., None] * xs[:, :, t].abs()
        want = (cz.conj()[:, None, t, :, None] * s).real.sum(2) * scale ** 2 + ref.d64(D)[:, None] * xs[:, :, t]
        bound = cz[:, t].abs().sum(-1)[:, None, None] * absolute * scale ** 2
        # B and C rounded to bf16 once each (2^-8 both), two more roundings of a term in the dual (2^-7). D is added to the
        # score of a step with itself, which the dual rounds to bf16: 2^-8 of D x, inside the same factor.
        bound = bound + (ref.d64(D)[:, None] * xs[:, :, t]).abs()
        ref.check("y[%d]" % t, got[:, :, t], want, (2.0 ** -6 + 2.0 ** -10) * bound + 1e-5 * want.abs() + 1e-6)


def test_training_chain_through_scan_and_recurrence():
    """Forward and backward of: (C, B) normalised and rotated -> selective scan -> gated recurrence, fp32,
    against float64 autograd of the same formulas."""
    Bt, Dn, N, L = 2, 6, 8, 70
    g = torch.Generator().manual_seed(0)
    n = lambda *s, std=1.0: torch.randn(s, generator=g) * std  # noqa: E731
    p = {"u": n(Bt, Dn, L), "dt": n(Bt, Dn, L, std=0.5), "A_log": torch.log(torch.arange(1, N + 1).float()).repeat(Dn, 1),
         "B": n(Bt, 1, N, L), "C": n(Bt, 1, N, L), "wB": 1 + 0.1 * n(N), "wC": 1 + 0.1 * n(N), "r": n(Bt, Dn, L),
         "i": n(Bt, Dn, L), "lam": n(Dn) - 4}
    w = n(Bt, Dn, L)
    f, _ = ssm.ssm_rope_inv_freq(N, 100.0)
    c = {k: v.cuda().contiguous() for k, v in p.items()}
    kw = dict(q_weight=c["wC"], k_weight=c["wB"], inv_freq=f.cuda(), interleaved=True, layout="bhdl")
    Cr, Br = ssm.ssm_qk_norm_rope_fwd(c["C"], c["B"], **kw)
    scan = (c["u"], c["dt"], c["A_log"], Br[:, 0], Cr[:, 0])
    s = ssm.ssm_scan_fwd(*scan, save_states=True)
    l = ssm.ssm_lru_fwd(s["out"], c["r"], c["i"], c["lam"], save_states=True)
    gl = ssm.ssm_lru_bwd(w.cuda(), s["out"], c["r"], c["i"], c["lam"], chunk_states=l["chunk_states"])
    gs = ssm.ssm_scan_bwd(gl["dx"], *scan, chunk_states=s["chunk_states"])
    gq = ssm.ssm_qk_norm_rope_bwd(gs["dC"].unsqueeze(1), c["C"], gs["dB"].unsqueeze(1), c["B"], **kw)
    q = {k: v.double().requires_grad_() for k, v in p.items()}

    def turned(v, weight):
        v = v[:, 0] / torch.sqrt((v[:, 0] ** 2).mean(1, keepdim=True) + 1e-6) * weight[:, None]
        angle = f[:, None] * torch.arange(L).double()
        a, b = v[:, 0::2], v[:, 1::2]
        return torch.stack([a * torch.cos(angle) - b * torch.sin(angle), b * torch.cos(angle) + a * torch.sin(angle)], 2).flatten(1, 2)

    B, C = turned(q["B"], q["wB"]), turned(q["C"], q["wC"])
    delta, A = torch.nn.functional.softplus(q["dt"]), -torch.exp(q["A_log"])
    h, hl = torch.zeros(Bt, Dn, N).double(), torch.zeros(Bt, Dn).double()
    outs = []
    for t in range(L):
        bar = torch.exp(delta[..., t, None] * A)
        h = bar * h + (bar - 1) / A * B[:, None, :, t] * q["u"][..., t, None]
        y = (h * C[:, None, :, t]).sum(-1)
        a = torch.exp(-8.0 * torch.nn.functional.softplus(q["lam"]) * torch.sigmoid(q["r"][..., t]))
        hl = a * hl + torch.sqrt(1 - a * a) * torch.sigmoid(q["i"][..., t]) * y
        outs.append(hl)
    out = torch.stack(outs, -1)
    (out * w.double()).sum().backward()
    near = lambda k, got, want: ref.check(k, got, want.detach(), 1e-4 * want.detach().abs().max() + 1e-3 * want.detach().abs())  # noqa: E731
    near("out", l["out"], out)
    for k, v in (("u", gs["dx"]), ("dt", gs["ddt"]), ("A_log", gs["dA_log"]), ("B", gq["dk"]), ("C", gq["dq"]),
                 ("wB", gq["dk_weight"]), ("wC", gq["dq_weight"]), ("r", gl["dr"]), ("i", gl["di"]), ("lam", gl["dlam"])):
        near("d" + k, v, q[k].grad)


def test_recurrent_layer_prefill_then_decode():
    """Padded prompts through the gated recurrence, then tokens by steps: each row continues from its own end."""
    Bt, Dn, L, steps = 3, 40, 90, 4
    g = torch.Generator().manual_seed(6)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    x, r, i = (n(Bt, Dn, L + steps).to(BF).cuda() for _ in range(3))
    lam = (n(Dn) - 4).cuda()
    lengths = torch.tensor([L, 1, 37], dtype=torch.int32, device="cuda")
    cut = [v[..., :L].contiguous() for v in (x, r, i)]
    f = ssm.ssm_lru_fwd(*cut, lam, lengths=lengths, return_state=True)
    h = f["h_last"]
    tail = [v[..., L:] for v in (x, r, i)]
    outs = [ssm.ssm_lru_step(*(v[..., t].contiguous() for v in tail), lam, h, out_dtype=F32) for t in range(steps)]
    for b in range(Bt):
        m = int(lengths[b])
        row = [torch.cat([v[b:b + 1, :, :m], v[b:b + 1, :, L:]], -1) for v in (x, r, i)]
        v, e = ref.lru(*row, lam)["out"]
        ref.check("row %d" % b, torch.stack(outs, -1)[b:b + 1], v[..., m:], (e + ref.EPS * v.abs())[..., m:])


def _guarded(fn):
    """Run fn(allocator) twice over memory filled with two patterns, every buffer between guard bands: no byte outside a
    buffer changes, every output element is written, and nothing read differs with the pattern."""
    results = []
    for fill in (0xA5, 0x5A):
        g = GuardedTorch(fill)
        outs = fn(g)
        torch.cuda.synchronize()
        g.check()
        results.append([v.clone() for v in outs])
    assert all(torch.equal(a, b) for a, b in zip(*results))


def _fill(g, args, inputs, outputs, **numbers):
    """Copies of the inputs and fresh outputs ({name: (shape, dtype)}) in guarded buffers, their addresses in args."""
    made = {}
    for k, v in inputs.items():
        if v is not None:
            made[k] = g.empty(tuple(v.shape), dtype=v.dtype, device="cuda")
            made[k].copy_(v)
    for k, (shape, dtype) in outputs.items():
        made[k] = g.empty(tuple(shape), dtype=dtype, device="cuda")
    for k, v in made.items():
        setattr(args, k, v.data_ptr())
    for k, v in numbers.items():
        setattr(args, k, v)
    return made


def _run(g, name, args, size=None):
    lib = _abi.load()
    if size is not None:
        need = getattr(lib, size)(ctypes.byref(args))
        if need:
            args.workspace = g.empty((need,), dtype=torch.uint8, device="cuda").data_ptr()
            args.workspace_bytes = need
            assert args.workspace % 256 == 0
    _abi.check(name, getattr(lib, name)(ctypes.byref(args), torch.cuda.current_stream().cuda_stream))


CODE = {F32: _abi.SSM_F32, BF: _abi.SSM_BF16}


@pytest.mark.parametrize("Bt,Dn,L,dtype", [(2, 5, 517, BF), (1, 3, 4100, F32), (3, 2, 9, BF), (2, 3, 70, F32)])
def test_guard_bands_of_the_recurrence(Bt, Dn, L, dtype):
    from test_gpu_lru import inputs as lru_inputs

    t = lru_inputs(Bt, Dn, L, dtype)
    names = ("x", "r", "i", "lam", "r_bias", "i_bias", "h0", "lengths", "reset")

    def fn(g):
        a = _abi.LruArgs()
        n = dict(Bt=Bt, Dn=Dn, L=L, c=8.0, in_dtype=CODE[dtype], out_dtype=CODE[dtype])
        ns = ssm.ssm_lru_num_states(L)
        m = _fill(g, a, {k: t[k] for k in names}, {"out": ((Bt, Dn, L), dtype), "h_last": ((Bt, Dn), F32)}, **n)
        # states: rows that start a group early use one more than others, so only the bands are checked
        st = g.empty((Bt * Dn * ns * 4,), dtype=torch.uint8, device="cuda")
        a.chunk_states = st.data_ptr()
        _run(g, "ssm_lru_fwd", a)
        b = _abi.LruBwdArgs()
        b.fwd = a
        outs = {k: ((Bt, Dn, L), dtype) for k in ("dx", "dr", "di")}
        outs.update({k: ((Dn,), F32) for k in ("dlam", "dr_bias", "di_bias")}, dh0=((Bt, Dn), F32))
        w = _fill(g, b, {"dout": t["dout"], "dh_last": t["dh_last"]}, outs, grad_dtype=CODE[dtype])
        _run(g, "ssm_lru_bwd", b, "ssm_lru_bwd_workspace_size")
        b.fwd.chunk_states = None  # recomputed into the workspace
        _run(g, "ssm_lru_bwd", b, "ssm_lru_bwd_workspace_size")
        return [m["out"], m["h_last"]] + [w[k] for k in outs]

    _guarded(fn)


@pytest.mark.parametrize("Bt,L,Hq,Hk,D,rot,time", [
    (2, 37, 3, 1, 80, 48, False), (1, 21, 2, 2, 33, 18, False), (1, 5, 2, 1, 128, 128, False), (2, 72, 1, 1, 16, 16, True),
    (1, 45, 2, 1, 66, 20, True), (1, 24, 1, 1, 130, 64, True), (1, 9, 2, 1, 300, 300, True)])
@pytest.mark.parametrize("interleaved", [0, 1])
def test_guard_bands_of_queries_and_keys(Bt, L, Hq, Hk, D, rot, time, interleaved):
    from test_gpu_qk import freq, inputs as qk_inputs

    t = qk_inputs(Bt, L, Hq, Hk, D, BF, time)
    shape = {"q": t["q"].shape, "k": t["k"].shape}

    def strides(H):
        return dict(sb=L * H * D, sh=D * L if time else D, sr=L if time else H * D)

    def fn(g):
        n = dict(Bt=Bt, L=L, Hq=Hq, Hk=Hk, D=D, rot=rot, eps=1e-6, rot_scale=1.0, norm=1, interleaved=interleaved, pos_i64=1,
                 layout=int(time), in_dtype=1, out_dtype=1)
        for side, H in (("q", Hq), ("k", Hk)):
            for k, v in strides(H).items():
                n["%s_%s" % (side, k)] = n["%s_out_%s" % (side, k)] = v
        a = _abi.QkArgs()
        ins = {k: t[k] for k in ("q", "k", "q_weight", "k_weight", "positions")}
        m = _fill(g, a, dict(ins, inv_freq=freq(rot)), {"q_out": (shape["q"], BF), "k_out": (shape["k"], BF)}, **n)
        _run(g, "ssm_qk_norm_rope_fwd", a)
        b = _abi.QkBwdArgs()
        b.fwd = a
        n = dict(dout_dtype=1, grad_dtype=0)
        for side, H in (("q", Hq), ("k", Hk)):
            n.update({"d%s_%s" % (side, k): v for k, v in strides(H).items()})
        outs = {"dq": (shape["q"], F32), "dk": (shape["k"], F32), "dq_weight": ((D,), F32), "dk_weight": ((D,), F32)}
        w = _fill(g, b, {"dq_out": t["dq_out"], "dk_out": t["dk_out"]}, outs, **n)
        _run(g, "ssm_qk_norm_rope_bwd", b, "ssm_qk_norm_rope_bwd_workspace_size")
        return [m["q_out"], m["k_out"]] + [w[k] for k in outs]

    _guarded(fn)


@pytest.mark.parametrize("Bt,H,P,N", [(2, 5, 96, 33), (1, 2, 250, 7), (3, 1, 33, 64)])
def test_guard_bands_of_the_steps(Bt, H, P, N):
    t = inputs(Bt, H, P, N, BF)

    def fn(g):
        a = _abi.SsdStepArgs()
        m = _fill(g, a, t, {"out": ((Bt, H, P), BF)}, Bt=Bt, H=H, P=P, N=N, in_dtype=1, out_dtype=1, delta_softplus=1)
        _run(g, "ssm_ssd_step", a)
        s = _abi.LruStepArgs()
        x = {k: t["x"][:, 0].contiguous() for k in ("x", "r", "i")}
        x.update(lam=t["A_log"].new_full((P,), -4.0), h=t["h"][:, 0, 0].contiguous())
        k = _fill(g, s, x, {"out": ((Bt, P), BF)}, Bt=Bt, Dn=P, c=8.0, in_dtype=1, out_dtype=1)
        _run(g, "ssm_lru_step", s)
        return [m["out"], m["h"], k["out"], k["h"]]

    _guarded(fn)
