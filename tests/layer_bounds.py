"""float64 gradients of the gated linear recurrence with bounds built from the terms of the derivative itself, and a bound on sums of
weight gradients by the length of the kernels' chains; EPS = 2^-24 is half a step of fp32.

Relative errors of the recurrence's factors, in EPS, each carried into the next:

  * t = -v log2 e (v = raw + bias): the product's own rounding |v|, that of bias log2 e |bias|, that of the constant (|raw| + |bias|) / 2;
    e^-v = exp2(t) adds 4 (hardware exp2: 2^-22). KE = |v| + |raw| / 2 + 1.5 |bias| + 5.
  * sigmoid = 1 / (1 + e^-v), 1 - sigmoid = e^-v sigmoid: sums, products and the reciprocal shared by two gates add 12. KR = KE + 12.
  * y = -log decay = rate r: rate = c softplus 5, a product, a fused one 1 each. KY = KR + 8.
  * n = 1 - a: its slope in y is at most 1 relative, the polynomial 4, or 2^-22 of exp2 on n >= 0.39: KN = KY + 12. a = e^-y: absolutely n KN + 1, or
    relatively y KY and the exponent's roundings: KA = y (KY + 2) + 6. The smaller holds.
  * s = n + n a: twice n's, 2; m = s / sqrt(s): half of s's and 4. KM = KN + 6.  b = m g x: KB = KM + KR + 3.  1 / s: 2 KN + 8.
  * a step adds its rounding (2 of a |h|); the tree that composes a chunk 5 shuffle levels, 8 elements, 16 warps: 32 in all.

y is y + 1e-36 in the kernels, so that a decay of 1 has a root: m moves by sqrt(2e-36) at most, the other term of the gradient of y, y a^2 b / s =
a^2 g x y / sqrt(s), by sqrt(1e-36 / 2). With a rate of 0 or a denormal these are all there is, and they carry their own factors' errors: the sum of the
K above, below 4000 EPS < 2^-12 for arguments of up to 60, so that 1 + 2^-10 under the roots covers them.
"""
import torch

from layer_refs import EPS, d64, sigmoid, softplus

TINY = 1e-36 * (1 + 2.0 ** -10)


def lru(x, r, i, lam, r_bias=None, i_bias=None, c=8.0, h0=None, reset=None, lengths=None, dout=None, dh_last=None):
    """{name: (value, bound before the last rounding)} of the outputs and of every gradient."""
    raw_r, raw_i, x, lam = d64(r), d64(i), d64(x), d64(lam)
    Bt, Dn, L = x.shape
    rb = torch.zeros(Dn).double() if r_bias is None else d64(r_bias)
    ib = torch.zeros(Dn).double() if i_bias is None else d64(i_bias)
    h = torch.zeros(Bt, Dn).double() if h0 is None else d64(h0)
    cut = torch.zeros(Bt, L).bool() if reset is None else reset.cpu().bool()
    n_live = torch.full((Bt,), L) if lengths is None else lengths.cpu().long().clamp(0, L)
    live = (torch.arange(L) < n_live[:, None])[:, None, :].expand_as(x)
    keep = (~cut)[:, None, :].expand_as(x)
    zero = lambda v, on: torch.where(on, v, torch.zeros_like(v))  # noqa: E731 (nothing of a masked step, NaN included)
    raw_r, raw_i, x = zero(raw_r, live), zero(raw_i, live), zero(x, live)
    u, v = raw_r + rb[:, None], raw_i + ib[:, None]
    gate = lambda raw, arg, bias: arg.abs() + raw.abs() / 2 + 1.5 * bias.abs()[:, None] + 17.0  # noqa: E731
    Kr, Kg = gate(raw_r, u, rb), gate(raw_i, v, ib)
    rr, omr, g, omg = sigmoid(u), sigmoid(-u), sigmoid(v), sigmoid(-v)
    sp = softplus(lam)
    y = c * sp[:, None] * rr
    a, n, s = torch.exp(-y), -torch.expm1(-y), -torch.expm1(-2 * y)
    m = torch.sqrt(s)
    Ky = Kr + 8.0
    Kn = Ky + 12.0
    Ka = y * (Ky + 2.0) + 6.0
    da = torch.minimum(a * Ka, n * Kn + 1.0)
    Km = Kn + 6.0
    mg, b = m * g, m * g * x
    Kb = Km + Kg + 3.0
    b_off = EPS * Kb * b.abs() + (2 * TINY) ** 0.5 * (g * x).abs()
    out, before, H_before, E_before, E_out, H_out = (torch.zeros(Bt, Dn, L).double() for _ in range(6))
    H, E = h.abs(), torch.zeros_like(h)  # the recurrence over absolute values; the error bound
    for t in range(L):
        on, k = live[..., t], keep[..., t]
        h1, H1, E1 = zero(h, k), zero(H, k), zero(E, k)
        before[..., t], H_before[..., t], E_before[..., t] = h1, H1, E1
        E_new = a[..., t] * E1 + EPS * (da[..., t] + 2 * a[..., t]) * H1 + b_off[..., t]
        h = torch.where(on, a[..., t] * h1 + b[..., t], h)
        H = torch.where(on, a[..., t] * H1 + b[..., t].abs(), H)
        E = torch.where(on, E_new, E)
        out[..., t], E_out[..., t], H_out[..., t] = zero(h, on), zero(E, on), zero(H, on)
    tree = 32.0 * EPS
    got = {"out": (out, E_out + tree * H_out), "h_last": (h, E + tree * H)}
    if dout is None:
        return got
    dout = zero(d64(dout), live)
    p = torch.zeros(Bt, Dn).double() if dh_last is None else d64(dh_last)
    P, F = p.abs(), torch.zeros_like(p)
    lm, LM, EL = (torch.zeros(Bt, Dn, L).double() for _ in range(3))
    for t in reversed(range(L)):
        on, k = live[..., t], keep[..., t]
        w, W = dout[..., t] + p, dout[..., t].abs() + P
        G = F + EPS * W
        lm[..., t], LM[..., t], EL[..., t] = zero(w, on), zero(W, on), zero(G, on)
        p = torch.where(on, zero(a[..., t] * w, k), p)
        P = torch.where(on, zero(a[..., t] * W, k), P)
        F = torch.where(on, zero(a[..., t] * G + EPS * (da[..., t] + a[..., t]) * W, k), F)
    EL = EL + tree * LM
    E_before = E_before + tree * H_before
    dx, di = zero(lm * mg, live), zero(lm * b * omg, live)
    e_dx = EL * mg + LM * (EPS * (Km + Kg + 3) * mg + (2 * TINY) ** 0.5 * g)
    e_di = omg * (EL * b.abs() + LM * (b_off + EPS * (Kg + 2) * b.abs()))
    # q = -lambda (y a h_before - y a^2 b / s): two terms and their errors, LM for |lambda|
    s1 = torch.where(s > 0, s, torch.ones_like(s))
    first, second = y * a * H_before, y * a * a * b.abs() / s1
    q = zero(-lm * (y * a * before - y * a * a * b / s1), live)
    e_q = EL * (first + second) + LM * (y * a * E_before + EPS * ((Ky + Ka + 4) * first + (Ky + 2 * Ka + Kb + 2 * Kn + 16) * second)
                                        + (TINY / 2) ** 0.5 * (g * x).abs() + TINY * H_before)
    dr = q * omr
    e_dr = omr * (e_q + EPS * (Kr + 2) * q.abs())
    # sums: a lane's share of the steps two at a time, pairs, lanes, warps, then the batch
    adds = EPS * (L / 64.0 + 48.0 + Bt)
    total = lambda v, e: (v.sum((0, 2)), (zero(e, live) + adds * v.abs()).sum((0, 2)))  # noqa: E731
    fac = torch.where(sp > 1e-30, sigmoid(lam) / sp.clamp(min=1e-300), torch.ones_like(sp))
    sq, eq = total(q, e_q)
    got.update(dx=(dx, zero(e_dx, live)), di=(di, zero(e_di, live)), dr=(dr, zero(e_dr, live)),
               dlam=(sq * fac, (eq + 16 * EPS * sq.abs()) * fac), dr_bias=total(dr, e_dr), di_bias=total(di, e_di), dh0=(p, F + tree * P))
    return got
