"""Measured cases of the gated linear recurrence (ssm_lru_fwd / _bwd / _step), of the normalisation and
rotation of queries and keys (ssm_qk_norm_rope_fwd / _bwd) and of the state-space-dual decode step
(ssm_ssd_step), with a plain form of each.

With ``own`` false, run() computes the operators from elementary torch operations in fp32; with
``own`` true it calls the library. exact() evaluates the definitions in float64, step by step.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
C_GATE = 8.0  # the recurrence's gate constant


# ---- the cases ---------------------------------------------------------------------------------


def _lru(name, direction, Bt, Dn, L, type="bf16", grad="f32", packed=False, padded=False):
    return {"name": name, "op": "lru", "dir": direction, "Bt": Bt, "Dn": Dn, "L": L, "type": type, "grad": grad,
            "packed": packed, "padded": padded}


def _qk(name, direction, Bt, L, Hq, Hk, D, rot, type="bf16", grad="f32", dout="bf16", norm=True,
        interleaved=False, time_last=False, far=0, scaling="none"):
    return {"name": name, "op": "qk", "dir": direction, "Bt": Bt, "L": L, "Hq": Hq, "Hk": Hk, "D": D, "rot": rot,
            "type": type, "grad": grad, "dout": dout, "norm": norm, "interleaved": interleaved,
            "time_last": time_last, "far": far, "scaling": scaling}


def _ssd(name, Bt, H, P, N, type="bf16"):
    return {"name": name, "op": "ssd_step", "Bt": Bt, "H": H, "P": P, "N": N, "type": type}


def listed():
    return [
        # one decode token for 64 sequences of a 4096-channel recurrent layer
        _lru("lru_step_64x4096", "step", 64, 4096, 1),
        # the forward of a small model's layer (the 130M-shaped block's sizes)
        _lru("lru_fwd_2x1536x2048", "fwd", 2, 1536, 2048),
        # prefill of one very long sequence (the long-context workload's sizes)
        _lru("lru_fwd_1x5120x65536", "fwd", 1, 5120, 65536),
        # a training step's forward and backward in bf16 throughout (the 1.4B-shaped block's sizes)
        _lru("lru_train_4x4096x4096", "train", 4, 4096, 4096, grad="bf16"),
        # fp32 training on short documents packed into rows of an odd length, the rows padded
        _lru("lru_train_ragged_f32", "train", 3, 1001, 2047, type="f32", packed=True, padded=True),
        # queries and keys of one decode token for 64 sequences, far into their contexts
        _qk("qk_decode_64", "fwd", 64, 1, 32, 8, 128, 128, far=200000, scaling="yarn"),
        # C and B in front of a state-space-dual layer (4 x 4096 steps, 128 states, one group)
        _qk("qk_fwd_ssd_4x4096", "fwd", 4, 4096, 1, 1, 128, 128),
        # grouped-head queries and keys in a training step, bf16 gradients
        _qk("qk_train_2x4096x40", "train", 2, 4096, 32, 8, 128, 128, grad="bf16"),
        # C and B in front of the selective scan, time innermost, with the scan's fp32 gradients
        _qk("qk_train_scan_4x16x4096", "train", 4, 4096, 1, 1, 16, 16, dout="f32", interleaved=True, time_last=True),
        # rotation alone of part of an odd head size, fp32, at odd lengths and far positions
        _qk("qk_rope_ragged_f32", "train", 3, 1001, 5, 1, 80, 48, type="f32", dout="f32", norm=False,
            interleaved=True, far=500000, scaling="linear"),
        # one decode token for 64 sequences of a state-space-dual layer (64 heads, 128 x 64 states)
        _ssd("ssd_step_64x64", 64, 64, 64, 128),
        # the same for a single sequence of a small layer
        _ssd("ssd_step_1x24", 1, 24, 64, 128),
    ]


def _span(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["lru", "lru", "qk", "qk", "qk", "ssd_step"])
    type = rng.choice(["bf16", "bf16", "f32"])
    if op == "lru":
        direction = rng.choice(["fwd", "train", "train", "step"])
        Bt, Dn = _span(rng, 1, 64 if direction == "step" else 8), _span(rng, 64, 5120)
        most = 1 << 25 if direction == "train" else 1 << 27
        L = 1 if direction == "step" else _span(rng, 1, max(1, min(65536, most // (Bt * Dn))))
        c = _lru("", direction, Bt, Dn, L, type, rng.choice(["f32", type]),
                 direction == "train" and rng.random() < 0.5, direction != "step" and rng.random() < 0.4)
    elif op == "qk":
        time_last = rng.random() < 0.35
        D = rng.choice([4, 8, 16, 24, 32, 33, 48, 64]) if time_last else rng.choice([16, 33, 64, 80, 96, 128, 192, 256])
        Hq, Hk = (rng.randint(1, 3), rng.randint(0, 2)) if time_last else (_span(rng, 1, 64), _span(rng, 1, 8))
        Bt = _span(rng, 1, 64)
        L = _span(rng, 1, max(1, min(16384, (1 << 25) // (Bt * (Hq + Hk) * D))))
        norm = rng.random() < 0.75
        rot = 2 * (D // 2) if rng.random() < 0.6 else 2 * rng.randint(0 if norm else 1, D // 2)
        c = _qk("", rng.choice(["fwd", "train"]), Bt, L, Hq, Hk, D, rot, type, rng.choice(["f32", type]),
                rng.choice(["f32", type]), norm, rng.random() < 0.5, time_last, rng.choice([0, 0, 100000, 1000000]),
                rng.choice(["none", "linear", "yarn"]))
    else:
        c = _ssd("", _span(rng, 1, 64), _span(rng, 4, 64), rng.choice([16, 32, 64, 96, 128]),
                 rng.choice([16, 33, 64, 96, 128]), type)
    del c["name"]
    return c


# ---- inputs ------------------------------------------------------------------------------------


class _Draws:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, *shape, std=1.0, dtype=torch.float32):
        v = torch.randn(shape, generator=self.g, device="cuda", dtype=torch.float32)
        return (v.mul_(std) if std != 1.0 else v).to(dtype)

    def uniform(self, *shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=self.g, device="cuda", dtype=torch.float32) * (hi - lo) + lo

    def integers(self, lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=self.g, device="cuda")


def _prepare_lru(c, d):
    t = TYPES[c["type"]]
    Bt, Dn, L = c["Bt"], c["Dn"], c["L"]
    shape = (Bt, Dn) if c["dir"] == "step" else (Bt, Dn, L)
    s = {"x": d.normal(*shape, dtype=t), "r": d.normal(*shape, dtype=t), "i": d.normal(*shape, dtype=t)}
    # a decay between 0.9 and 0.999 a step where the gate is fully open: softplus(lam) = -ln(decay) / c
    rate = -torch.log(d.uniform(Dn, lo=0.9, hi=0.999)) / C_GATE
    s["lam"] = torch.log(torch.expm1(rate))
    s["r_bias"], s["i_bias"] = d.normal(Dn, std=0.1), d.normal(Dn, std=0.1)
    h0 = d.normal(Bt, Dn)
    s["reset"] = s["lengths"] = None
    if c["dir"] == "step":
        s["h"] = h0
        return s
    s["h0"] = h0
    if c["packed"]:
        s["reset"] = d.uniform(Bt, L) < 1.0 / 300.0
    if c["padded"]:
        s["lengths"] = d.integers(0, L + 1, Bt).to(torch.int32)
    if c["dir"] == "train":
        s["dout"] = d.normal(*shape, dtype=t)
    return s


def _rope_table(rot, scaling):
    """(frequencies, factor on cosine and sine) of base 10000, as fp32 like a model's buffer."""
    j = torch.arange(0, rot, 2, dtype=torch.float64, device="cuda")
    f = 10000.0 ** (-j / max(rot, 1))
    if scaling == "linear":
        return (f / 4.0).float(), 1.0
    if scaling == "yarn":  # below 1 turn in 4096 tokens: a fourth of the angle; above 32: as it is
        turns = 4096.0 * f / (2.0 * math.pi)
        keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
        return (f * (keep + (1.0 - keep) / 4.0)).float(), 0.1 * math.log(4.0) + 1.0
    return f.float(), 1.0


def _prepare_qk(c, d):
    t, Bt, L, D = TYPES[c["type"]], c["Bt"], c["L"], c["D"]
    shape = lambda H: (Bt, H, D, L) if c["time_last"] else (Bt, L, H, D)  # noqa: E731
    s = {"q": d.normal(*shape(c["Hq"]), dtype=t), "k": d.normal(*shape(c["Hk"]), dtype=t) if c["Hk"] else None}
    s["q_weight"] = 1.0 + d.normal(D, std=0.1) if c["norm"] else None
    s["k_weight"] = 1.0 + d.normal(D, std=0.1) if c["norm"] and c["Hk"] else None
    s["inv_freq"], s["rot_scale"] = _rope_table(c["rot"], c["scaling"]) if c["rot"] else (None, 1.0)
    s["positions"] = d.integers(0, c["far"] + 1, Bt, 1) + torch.arange(L, device="cuda")
    if c["dir"] == "train":
        u = TYPES[c["dout"]]
        s["dq_out"] = d.normal(*shape(c["Hq"]), dtype=u)
        s["dk_out"] = d.normal(*shape(c["Hk"]), dtype=u) if c["Hk"] else None
    return s


def _prepare_ssd(c, d):
    t, Bt, H, P, N = TYPES[c["type"]], c["Bt"], c["H"], c["P"], c["N"]
    return {"x": d.normal(Bt, H, P, dtype=t), "dt": d.normal(Bt, H, dtype=t),
            "dt_bias": torch.log(torch.expm1(d.uniform(H, lo=0.001, hi=0.1))),
            "A_log": torch.log(d.uniform(H, lo=1.0, hi=16.0)), "B": d.normal(Bt, N, std=0.25, dtype=t),
            "C": d.normal(Bt, N, std=0.25, dtype=t), "D": d.normal(H), "h": d.normal(Bt, H, N, P)}


def prepare(case, seed):
    d = _Draws(seed)
    s = {"lru": _prepare_lru, "qk": _prepare_qk, "ssd_step": _prepare_ssd}[case["op"]](case, d)
    s["case"] = case
    return s


# ---- the plain forms ---------------------------------------------------------------------------


def _linear_scan(a, b):
    """h_t = a_t h_{t-1} + b_t along the last axis from h = 0, by halving: pairs of steps are one step of
    half as long a recurrence, whose results are the odd steps'."""
    if a.shape[-1] == 1:
        return b
    n = a.shape[-1] // 2 * 2
    a1, b1 = a[..., 1:n:2], b[..., 1:n:2]
    odd = _linear_scan(a1 * a[..., 0:n:2], torch.addcmul(b1, a1, b[..., 0:n:2]))
    h = b.clone()
    h[..., 1:n:2] = odd
    m = h[..., 2::2].shape[-1]
    h[..., 2::2] += a[..., 2::2] * odd[..., :m]
    return h


def _gates(s, x, r, i):
    """(x, decay gate, input gate, log decay, decay, sqrt(1 - decay^2)) in fp32."""
    col = (slice(None), None) if r.dim() == 3 else (slice(None),)
    rate = C_GATE * torch.nn.functional.softplus(s["lam"])
    open_r, g = torch.sigmoid(r.float() + s["r_bias"][col]), torch.sigmoid(i.float() + s["i_bias"][col])
    log_a = -rate[col] * open_r
    return x.float(), open_r, g, log_a, torch.exp(log_a), torch.sqrt(-torch.expm1(2.0 * log_a))


def _plain_lru(c, s):
    t = TYPES[c["type"]]
    x, open_r, g, log_a, a, m = _gates(s, s["x"], s["r"], s["i"])
    if c["dir"] == "step":
        h = a * s["h"] + m * g * x
        s["h"].copy_(h)
        return {"out": h.to(t), "h": s["h"]}
    L = c["L"]
    step = torch.arange(L, device=x.device)
    lengths = s["lengths"]
    live = None if lengths is None else (step < lengths[:, None])[:, None, :]
    carry = a if s["reset"] is None else a.masked_fill(s["reset"][:, None, :], 0.0)
    b = m * g * x
    b[..., 0] += carry[..., 0] * s["h0"]
    h = _linear_scan(carry, b)
    out = h if live is None else h.masked_fill(~live, 0.0)
    if c["dir"] == "fwd":
        if lengths is None:
            last = h[..., -1].clone()
        else:
            at = (lengths.long() - 1).clamp(min=0)[:, None, None].expand(-1, h.shape[1], 1)
            last = torch.where((lengths > 0)[:, None], h.gather(2, at)[..., 0], s["h0"])
        return {"out": out.to(t), "h_last": last}
    u = TYPES[c["grad"]]
    dout = s["dout"].float()
    if live is not None:
        dout = dout.masked_fill(~live, 0.0)
    after = torch.cat([carry[..., 1:], torch.zeros_like(carry[..., :1])], -1)
    lam = _linear_scan(after.flip(-1), dout.flip(-1)).flip(-1)
    before = torch.cat([s["h0"][..., None], h[..., :-1]], -1)
    dlog = lam * (carry * before - g * x * a * a / m) * log_a
    if live is not None:
        dlog = dlog.masked_fill(~live, 0.0)
    dr, dx, di = dlog * (1.0 - open_r), lam * m * g, lam * m * x * g * (1.0 - g)
    dlam = dlog.sum((0, 2)) * torch.sigmoid(s["lam"]) / torch.nn.functional.softplus(s["lam"])
    return {"out": out.to(t), "dx": dx.to(u), "dr": dr.to(u), "di": di.to(u), "dlam": dlam,
            "dr_bias": dr.sum((0, 2)), "di_bias": di.sum((0, 2)), "dh0": lam[..., 0] * carry[..., 0]}


def _turn(v, cos, sin, rot, interleaved):
    """The first rot elements of the last axis turned by the angles, pair by pair."""
    if rot == 0:
        return v
    if interleaved:
        p, q = v[..., 0:rot:2], v[..., 1:rot:2]
        w = torch.stack([p * cos - q * sin, q * cos + p * sin], -1).flatten(-2)
    else:
        p, q = v[..., :rot // 2], v[..., rot // 2:rot]
        w = torch.cat([p * cos - q * sin, q * cos + p * sin], -1)
    return torch.cat([w, v[..., rot:]], -1)


def _angles(c, s):
    if c["rot"] == 0:
        return None, None
    angle = (s["positions"].double()[..., None] * s["inv_freq"].double())[:, :, None, :]
    return (torch.cos(angle) * s["rot_scale"]).float(), (torch.sin(angle) * s["rot_scale"]).float()


def _inner(c, v):
    return v.permute(0, 3, 1, 2) if c["time_last"] else v


def _outer(c, v):
    return v.permute(0, 2, 3, 1).contiguous() if c["time_last"] else v.contiguous()


def _plain_heads(c, s, side, cos, sin):
    v, w = _inner(c, s[side]).float(), s[side + "_weight"]
    scale = torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6) if c["norm"] else None
    n = v * scale if c["norm"] else v
    got = {side + "_out": _outer(c, _turn(n * w if c["norm"] else n, cos, sin, c["rot"], c["interleaved"])).to(TYPES[c["type"]])}
    if c["dir"] == "train":
        back = _inner(c, s["d" + side + "_out"]).float()
        back = _turn(back, cos, None if sin is None else -sin, c["rot"], c["interleaved"])
        if c["norm"]:
            got["d%s_weight" % side] = (back * n).sum((0, 1, 2))
            back = back * w
            back = scale * (back - n * (back * n).mean(-1, keepdim=True))
        got["d" + side] = _outer(c, back).to(TYPES[c["grad"]])
    return got


def _plain_qk(c, s):
    cos, sin = _angles(c, s)
    got = _plain_heads(c, s, "q", cos, sin)
    if c["Hk"]:
        got.update(_plain_heads(c, s, "k", cos, sin))
    return got


def _plain_ssd(c, s):
    x = s["x"].float()
    delta = torch.nn.functional.softplus(s["dt"].float() + s["dt_bias"])
    A = -torch.exp(s["A_log"])
    a, beta = torch.exp(delta * A), torch.expm1(delta * A) / A
    h = a[..., None, None] * s["h"] + (beta[..., None] * s["B"].float()[:, None, :])[..., None] * x[:, :, None, :]
    y = (h * s["C"].float()[:, None, :, None]).sum(2) + s["D"][:, None] * x
    s["h"].copy_(h)
    return {"out": y.to(TYPES[c["type"]]), "h": s["h"]}


# ---- the library's calls -----------------------------------------------------------------------


def _own_lru(c, s):
    import selective_state_space_34_b200 as ssm
    kw = dict(r_bias=s["r_bias"], i_bias=s["i_bias"], c=C_GATE)
    if c["dir"] == "step":
        return {"out": ssm.ssm_lru_step(s["x"], s["r"], s["i"], s["lam"], s["h"], **kw), "h": s["h"]}
    kw.update(h0=s["h0"], reset=s["reset"], lengths=s["lengths"])
    if c["dir"] == "fwd":
        got = ssm.ssm_lru_fwd(s["x"], s["r"], s["i"], s["lam"], return_state=True, **kw)
        return {"out": got["out"], "h_last": got["h_last"]}
    got = ssm.ssm_lru_fwd(s["x"], s["r"], s["i"], s["lam"], save_states=True, **kw)
    grads = ssm.ssm_lru_bwd(s["dout"], s["x"], s["r"], s["i"], s["lam"], chunk_states=got["chunk_states"],
                            grad_dtype=TYPES[c["grad"]], **kw)
    return {"out": got["out"], **{n: grads[n] for n in ("dx", "dr", "di", "dlam", "dr_bias", "di_bias", "dh0")}}


def _own_qk(c, s):
    import selective_state_space_34_b200 as ssm
    kw = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], inv_freq=s["inv_freq"], positions=s["positions"],
              norm=c["norm"], eps=1e-6, interleaved=c["interleaved"], rot_scale=s["rot_scale"],
              layout="bhdl" if c["time_last"] else "blhd")
    q_out, k_out = ssm.ssm_qk_norm_rope_fwd(s["q"], s["k"], **kw)
    got = {"q_out": q_out}
    if c["Hk"]:
        got["k_out"] = k_out
    if c["dir"] == "train":
        got.update(ssm.ssm_qk_norm_rope_bwd(s["dq_out"], s["q"], s["dk_out"], s["k"], grad_dtype=TYPES[c["grad"]], **kw))
    return got


def _own_ssd(c, s):
    import selective_state_space_34_b200 as ssm
    out = ssm.ssm_ssd_step(s["x"], s["dt"], s["A_log"], s["B"], s["C"], s["h"], D=s["D"], dt_bias=s["dt_bias"])
    return {"out": out, "h": s["h"]}


def run(state):
    c = state["case"]
    if own:
        return {"lru": _own_lru, "qk": _own_qk, "ssd_step": _own_ssd}[c["op"]](c, state)
    return {"lru": _plain_lru, "qk": _plain_qk, "ssd_step": _plain_ssd}[c["op"]](c, state)


# ---- what a pass cannot do without -------------------------------------------------------------


def work(case):
    c = case
    e = 2 if c.get("type") == "bf16" else 4
    g = 2 if c.get("grad") == "bf16" else 4
    if c["op"] == "lru":
        rows = c["Bt"] * c["Dn"]
        n = rows * c["L"]
        if c["dir"] == "step":
            return {"bytes": 4 * e * n + 8 * n + 12 * c["Dn"], "flops": 20 * n}
        masks = (c["Bt"] * c["L"] if c["packed"] else 0) + (4 * c["Bt"] if c["padded"] else 0)
        if c["dir"] == "fwd":  # x, r, i in; out and the states at both ends
            return {"bytes": 4 * e * n + 8 * rows + 12 * c["Dn"] + masks, "flops": 20 * n}
        return {"bytes": 5 * e * n + 3 * g * n + 8 * rows + 24 * c["Dn"] + masks, "flops": 60 * n}
    if c["op"] == "qk":
        n = c["Bt"] * c["L"] * (c["Hq"] + c["Hk"]) * c["D"]
        o = 2 if c["dout"] == "bf16" else 4
        small = 8 * c["Bt"] * c["L"] + 2 * c["rot"] + (8 * c["D"] if c["norm"] else 0)
        if c["dir"] == "fwd":
            return {"bytes": 2 * e * n + small, "flops": 8 * n}
        return {"bytes": 2 * e * n + (o + g) * n + small, "flops": 22 * n}
    rows, n = c["Bt"] * c["H"], c["Bt"] * c["H"] * c["N"] * c["P"]
    return {"bytes": 8 * n + 2 * e * rows * c["P"] + e * rows + 2 * e * c["Bt"] * c["N"] + 12 * c["H"], "flops": 6 * n}


# ---- the definitions in 64 bits ----------------------------------------------------------------


def _exact_heads(c, s, side):
    D, rot = c["D"], c["rot"]
    first = lambda v: (v.permute(3, 0, 1, 2) if c["time_last"] else v.permute(1, 0, 2, 3)).double()  # noqa: E731
    last = lambda v: v.permute(1, 2, 3, 0) if c["time_last"] else v.permute(1, 0, 2, 3)  # noqa: E731
    v = first(s[side])  # (L, Bt, H, D)
    w = s[side + "_weight"].double() if c["norm"] else 1.0
    rms = torch.sqrt((v * v).sum(-1, keepdim=True) / D + 1e-6) if c["norm"] else 1.0
    unit = v / rms
    j = torch.arange(rot // 2, device=v.device)
    at = (2 * j, 2 * j + 1) if c["interleaved"] else (j, j + rot // 2)
    turn = torch.zeros(c["L"], c["Bt"], 1, rot // 2, dtype=torch.complex128, device=v.device)
    if rot:
        angle = s["positions"].t().double()[:, :, None, None] * s["inv_freq"].double()
        turn = torch.polar(torch.full_like(angle, s["rot_scale"]), angle)

    def turned(u, by):
        u = u.clone()
        z = torch.complex(u[..., at[0]], u[..., at[1]]) * by
        u[..., at[0]], u[..., at[1]] = z.real, z.imag
        return u

    got = {side + "_out": last(turned(unit * w, turn))}
    if c["dir"] == "train":
        b = turned(first(s["d" + side + "_out"]), turn.conj())
        if c["norm"]:
            got["d%s_weight" % side] = (b * unit).sum((0, 1, 2))
            e = b * w
            b = e / rms - v * ((e * v).sum(-1, keepdim=True) / (D * rms ** 3))
        got["d" + side] = last(b)
    return got


def _exact_ssd(c, s):
    x, h = s["x"].double(), s["h"].double()
    v = s["dt"].double() + s["dt_bias"].double()
    delta = torch.log1p(torch.exp(-v.abs())) + v.clamp(min=0)
    rate = torch.exp(s["A_log"].double())
    beta = (1.0 - torch.exp(-delta * rate)) / rate
    h = torch.exp(-delta * rate)[..., None, None] * h + torch.einsum("bh,bn,bhp->bhnp", beta, s["B"].double(), x)
    return {"out": torch.einsum("bn,bhnp->bhp", s["C"].double(), h) + s["D"].double()[:, None] * x, "h": h}


def exact(case, seed):
    def recurrence(c, s):
        lam, c_gate = s["lam"].double(), C_GATE
        sp = torch.log1p(torch.exp(-lam.abs())) + lam.clamp(min=0)
        first = lambda v: (v[None] if c["dir"] == "step" else v.permute(2, 0, 1)).double().contiguous()  # noqa: E731
        x, r, i = first(s["x"]), first(s["r"]), first(s["i"])
        T = x.shape[0]
        r = 1.0 / (1.0 + torch.exp(-(r + s["r_bias"].double())))
        g = 1.0 / (1.0 + torch.exp(-(i + s["i_bias"].double())))
        log_a = -c_gate * sp * r
        h = (s["h"] if c["dir"] == "step" else s["h0"]).double()
        Bt = h.shape[0]
        lengths = torch.full((Bt,), T, device=h.device) if s["lengths"] is None else s["lengths"]
        cut = torch.zeros(Bt, T, dtype=torch.bool, device=h.device) if s["reset"] is None else s["reset"]
        keep = (~cut).double()
        on = (torch.arange(T, device=h.device) < lengths[:, None]).double()
        m = torch.sqrt(-torch.expm1(2.0 * log_a))
        before, out = torch.empty_like(x), torch.empty_like(x)
        for t in range(T):
            before[t] = h * keep[:, t, None]
            new = torch.exp(log_a[t]) * before[t] + m[t] * g[t] * x[t]
            h = torch.where(on[:, t, None] > 0, new, h)
            out[t] = new * on[:, t, None]
        back = lambda v: v.permute(1, 2, 0)  # noqa: E731
        if c["dir"] == "step":
            return {"out": h, "h": h}
        if c["dir"] == "fwd":
            return {"out": back(out), "h_last": h}
        dout = first(s["dout"])
        got = {n: torch.empty_like(x) for n in ("dx", "dr", "di")}
        dlam = torch.zeros_like(lam)
        p = torch.zeros_like(h)  # the gradient that arrives at a step's state from behind it
        for t in reversed(range(T)):
            live = on[:, t, None]
            adj = (dout[t] + p) * live
            a = torch.exp(log_a[t])
            da = adj * before[t] - adj * g[t] * x[t] * a / m[t]  # through the decay and through sqrt(1 - a^2)
            dlog = da * a
            p = adj * a * keep[:, t, None] * live + p * (1.0 - live)
            got["dx"][t], got["di"][t] = adj * m[t] * g[t], adj * m[t] * x[t] * g[t] * (1.0 - g[t])
            got["dr"][t] = dlog * (-c_gate * sp) * r[t] * (1.0 - r[t])
            dlam += (dlog * (-c_gate) * r[t]).sum(0) / (1.0 + torch.exp(-lam))
        return {"out": back(out), **{n: back(v) for n, v in got.items()}, "dlam": dlam,
                "dr_bias": got["dr"].sum((0, 1)), "di_bias": got["di"].sum((0, 1)), "dh0": p}

    s = prepare(case, seed)
    if case["op"] == "lru":
        return recurrence(case, s)
    if case["op"] == "qk":
        return {**_exact_heads(case, s, "q"), **(_exact_heads(case, s, "k") if case["Hk"] else {})}
    return _exact_ssd(case, s)
