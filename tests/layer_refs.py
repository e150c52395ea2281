"""float64 references of the gated linear recurrence, of query/key normalisation with rotation and of the
state-space-dual step, each with a bound on what the kernels' roundings can add, derived term by term.

eps = 2^-24 is half a step of fp32. The bounds carry the rounding errors of the kernels' formulas forward with
absolute values in the place of every term, so cancellation is covered:

  * sigmoid: 20 eps relative (the exponent's rounding, up to 8 eps for |argument| <= 8, hardware exp2 and
    reciprocal at 4 and 2 eps, the products).
  * la = log decay: that plus two products, KL = 24 eps; a absolutely a |la| KL + eps or less; e^la - 1 and with it
    1 - a^2 to KL + 8 relative, m = sqrt(1 - a^2) to half of that; b = m g x to KB = 45.
  * a step of the recurrence adds the errors of a (relative to a |h|, |h| the recurrence over |b|), of b and 2 eps
    for its own rounding; the tree that composes a chunk adds at most 5 shuffle levels, 8 elements and 16 warps.
"""
import torch

EPS = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: EPS}  # half a step of a result's rounding, relative


def poison_shared():
    """Leave NaN in the shared memory of every SM (a call over NaN whose staging buffers and tables fill 70 KB of it), so
    that a kernel which reads shared memory before writing it shows."""
    import selective_state_space_34_b200 as ssm
    q = torch.full((1, 4000, 4, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    w = torch.full((512,), float("nan"), device="cuda")
    f = torch.full((256,), float("nan"), device="cuda")
    ssm.ssm_qk_norm_rope_bwd(q, q, q_weight=w, inv_freq=f)


def d64(t):
    return None if t is None else t.detach().double().cpu()


def sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def softplus(v):
    return torch.log1p(torch.exp(-v.abs())) + v.clamp(min=0)


def check(name, got, ref, bound):
    got, ref = d64(got), ref
    assert got.shape == ref.shape, (name, tuple(got.shape), tuple(ref.shape))
    off = (got - ref).abs() - bound
    bad = ~(off <= 0)
    if bool(bad.any()):
        at = tuple(int(v[0]) for v in torch.where(bad))
        raise AssertionError("%s: %d of %d outside the bound; at %s got %r, reference %r, bound %r"
                             % (name, int(bad.sum()), bad.numel(), at, got[at].item(), ref[at].item(),
                                bound[at].item()))


def lru(x, r, i, lam, r_bias=None, i_bias=None, c=8.0, h0=None, reset=None, lengths=None, dout=None, dh_last=None):
    """Outputs and, with dout, gradients of the recurrence, as {name: (value, bound before the last rounding)}."""
    KL, KB, KG = 24.0, 45.0, 110.0
    x, r, i, lam = d64(x), d64(r), d64(i), d64(lam)
    Bt, Dn, L = x.shape
    rb = torch.zeros(Dn).double() if r_bias is None else d64(r_bias)
    ib = torch.zeros(Dn).double() if i_bias is None else d64(i_bias)
    h = torch.zeros(Bt, Dn).double() if h0 is None else d64(h0)
    cut = torch.zeros(Bt, L).bool() if reset is None else reset.cpu().bool()
    n = torch.full((Bt,), L) if lengths is None else lengths.cpu().long().clamp(0, L)
    rr, g = sigmoid(r + rb[:, None]), sigmoid(i + ib[:, None])
    rate = c * softplus(lam)[:, None]
    la = -rate * rr
    a = torch.exp(la)
    m = torch.sqrt(-torch.expm1(2 * la))
    b = m * g * x
    out, before, Hs, Es = (torch.zeros(Bt, Dn, L).double() for _ in range(4))
    H, E = h.abs(), torch.zeros_like(h)  # the recurrence over absolute values; the error bound
    da = a * la.abs() * KL + 1.0         # absolute error of a, in eps
    for t in range(L):
        live = (t < n)[:, None]
        k = torch.where(cut[:, t, None], 0.0, 1.0).double()
        E_new = k * (a[..., t] * E + EPS * (da[..., t] + 2.0 * a[..., t]) * H) + EPS * KB * b[..., t].abs()
        H_new = k * a[..., t] * H + b[..., t].abs()
        # a step of nothing but zeros where a is cut off must not carry 0 * inf
        prev = torch.where(cut[:, t, None], torch.zeros_like(h), h)
        h_new = a[..., t] * prev + b[..., t]
        before[..., t] = prev
        h, H, E = torch.where(live, h_new, h), torch.where(live, H_new, H), torch.where(live, E_new, E)
        out[..., t], Hs[..., t], Es[..., t] = (torch.where(live, v, torch.zeros_like(v)) for v in (h, H, E))
    tree = 32.0 * EPS
    Es = Es + tree * Hs
    got = {"out": (out, Es), "h_last": (h, E + tree * H)}
    if dout is None:
        return got
    dout = d64(dout)
    p = torch.zeros(Bt, Dn).double() if dh_last is None else d64(dh_last)
    P, F = p.abs(), torch.zeros_like(p)
    lm, LM, EL = (torch.zeros(Bt, Dn, L).double() for _ in range(3))
    for t in reversed(range(L)):
        live = (t < n)[:, None]
        v, V = dout[..., t] + p, dout[..., t].abs() + P
        G = F + EPS * V
        lm[..., t], LM[..., t], EL[..., t] = (torch.where(live, w, torch.zeros_like(w)) for w in (v, V, G))
        keep = ~cut[:, t, None]
        zero = torch.zeros_like(v)
        p = torch.where(live, torch.where(keep, a[..., t] * v, zero), p)
        P_new = torch.where(keep, a[..., t] * V, zero)
        F = torch.where(live, torch.where(keep, a[..., t] * G + EPS * (da[..., t] + a[..., t]) * V, zero), F)
        P = torch.where(live, P_new, P)
    EL = EL + tree * LM
    on = (torch.arange(L) < n[:, None])[:, None, :].expand_as(x)
    z = lambda v: torch.where(on, v, torch.zeros_like(v))  # noqa: E731
    mg = m * g
    dx, di = z(lm * mg), z(lm * mg * x * (1 - g))
    q = z(lm * (a * before - g * x * a * a / m) * la)
    T = la.abs() * Hs + (la / m ** 2 * b).abs()  # |la h| + |rho b|
    # the errors of a product: of lambda, and KG eps of the other factors (1 - g: absolutely KG eps of 1)
    e_dx = z(EL * mg + KG * EPS * LM * mg)
    e_di = z((EL + KG * EPS * LM) * mg * x.abs() * (1 - g) + KG * EPS * LM * mg * x.abs())
    e_q = z(EL * T + LM * (la.abs() * Es + KG * EPS * T))
    dr = q * (1 - rr)
    e_dr = z(e_q * (1 - rr) + KG * EPS * LM * T)
    adds = EPS * (L / 32.0 + 40.0 + Bt)  # roundings of the sums over time and batch
    total = lambda v, e: (v.sum((0, 2)), (e + adds * v.abs()).sum((0, 2)))  # noqa: E731
    fac = sigmoid(lam) / softplus(lam)
    sq, eq = total(q, e_q)
    got.update(dx=(dx, e_dx), di=(di, e_di), dr=(dr, e_dr), dlam=(sq * fac, (eq + 8 * EPS * sq.abs()) * fac),
               dr_bias=total(dr, e_dr), di_bias=total(di, e_di), dh0=(p, F + tree * P))
    return got


def qk_rows(v, time):
    """(Bt, L, H, D) view of either layout."""
    return v.permute(0, 3, 1, 2) if time else v


def turned(v, cos, sin, rot, interleaved):
    v = v.clone()
    if rot:
        i, j = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
        p, q = v[..., i].clone(), v[..., j].clone()
        v[..., i], v[..., j] = p * cos - q * sin, q * cos + p * sin
    return v


def _pair_sum(v, rot, interleaved, scale):
    """Per element, scale (v_p + v_q) of its pair; v where it is not rotated."""
    v = v.clone()
    i, j = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    s = (v[..., i] + v[..., j]) * abs(scale)
    v[..., i] = s
    v[..., j] = s
    return v


def qk(v, weight, inv_freq, positions, norm, eps, interleaved, rot_scale, time, dout=None):
    """One side: {"out": (value, bound)} and with dout "d" and "dw". KF covers the normalisation (a sum of at
    most 512 positive squares in at most 48 serial roundings, halved by the root) and the angle (16 eps);
    KR the same for the backward's two products and its mean."""
    KF, KR = 64.0, 128.0
    rows = qk_rows(d64(v), time)
    Bt, L, H, D = rows.shape
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    w = torch.ones(D).double() if weight is None else d64(weight)
    s = 1.0 / torch.sqrt((rows * rows).mean(-1, keepdim=True) + eps) if norm else torch.ones(Bt, L, H, 1).double()
    n = rows * s * w
    if rot:
        angle = positions.cpu().double()[:, :, None, None] * d64(inv_freq)
        cos, sin = torch.cos(angle) * rot_scale, torch.sin(angle) * rot_scale
    else:
        cos = sin = None
    back = (lambda u: u.permute(0, 2, 3, 1)) if time else (lambda u: u)
    wide = (lambda u: _pair_sum(u.abs(), rot, interleaved, rot_scale)) if rot else (lambda u: u.abs())
    got = {"out": (back(turned(n, cos, sin, rot, interleaved)), back(KF * EPS * wide(n)))}
    if dout is None:
        return got
    d = qk_rows(d64(dout), time)
    u = turned(d, cos, None if sin is None else -sin, rot, interleaved)
    U = wide(d)
    unit = rows * s
    if norm:
        got["dw"] = ((u * unit).sum((0, 1, 2)), ((KR + Bt * L * H) * EPS * U * unit.abs()).sum((0, 1, 2)))
        dv = s * (u * w - unit * (u * w * unit).mean(-1, keepdim=True))
        e = KR * EPS * s * (U * w.abs() + unit.abs() * (U * w.abs() * unit.abs()).mean(-1, keepdim=True))
    else:
        dv, e = u, KR * EPS * U
    got["d"] = (back(dv), back(e))
    return got


def ssd_step(x, dt, A_log, B, C, h, D=None, dt_bias=None, softplus_on=True, euler=False):
    """{"out", "h"}: 40 eps for the factors (softplus, exp, expm1, their products; the exponent's own
    rounding is relative to it, |delta A| eps), N + 8 roundings of the readout's sum."""
    x, dt, A_log, B, C, h = (d64(v) for v in (x, dt, A_log, B, C, h))
    H = x.shape[1]
    v = dt + (0 if dt_bias is None else d64(dt_bias))
    delta = softplus(v) if softplus_on else v
    rate = torch.exp(A_log)
    a = torch.exp(-delta * rate)[..., None, None]
    beta = delta if euler else -torch.expm1(-delta * rate) / rate
    add = (beta[..., None] * B[:, None, :])[..., None] * x[:, :, None, :]
    new = a * h + add
    big = a * h.abs() + add.abs()
    e = EPS * (40.0 + 8.0 * (delta * rate).abs()[..., None, None]) * big
    Cc = C[:, None, :, None]
    skip = torch.zeros(H).double() if D is None else d64(D)
    y = (new * Cc).sum(2) + skip[:, None] * x
    ey = (e * Cc.abs()).sum(2) + EPS * (C.shape[1] + 8.0) * ((big * Cc.abs()).sum(2) + (skip[:, None] * x).abs())
    return {"out": (y, ey), "h": (new, e)}
