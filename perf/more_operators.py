"""The operators between the recurrence and a training step, as cases to measure.

Three operators, each in its directions:

  qk_norm   the norm of every query's and key's head with the position rotation
            in the same pass: prefill, single tokens, a training step
  glu       the gated feed-forward block's projections, activation and product:
            prefill, single tokens, a training step
  policy    the clipped policy loss with a KL term on logits: a rollout's
            log-probabilities, the loss, the loss with the logits' gradient

`run` computes them in elementary torch operations where `own` is false, and
calls the library's entry points where it is true.  `exact` is the definition
in 64 bits, through autograd where there are gradients.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-6
_IGNORED = -100          # the target of a row that takes no part
_CLIP = (0.2, 0.28)


# --------------------------------------------------------------------- cases
def listed():
    return [
        # prefill of 4 sequences x 4096 tokens: q and k of 16 heads of 128, every dimension rotated
        dict(name="qk_norm prefill 4x4096", op="qk", type="bf16", T=16384, Hq=16, Hk=16, d=128, rot=128,
             interleaved=False, l2=False, weight=True, far=False),
        # a ragged batch in fp32: shared keys, an odd head width, a part of it rotated in neighbouring pairs
        dict(name="qk_norm ragged fp32", op="qk", type="f32", T=3001, Hq=7, Hk=3, d=90, rot=40, interleaved=True,
             l2=False, weight=True, far=False),
        # decode: 64 sequences at far positions, 32 heads of 128, unit-length q and k as the recurrence takes them
        dict(name="qk_norm decode 64", op="qk", type="bf16", T=64, Hq=32, Hk=32, d=128, rot=64, interleaved=False,
             l2=True, weight=False, far=True),
        # trainer, 2 x 8192 tokens, 32 heads of 128: forward and gradients
        dict(name="qk_norm training 2x8192", op="qk_train", type="bf16", T=16384, Hq=32, Hk=32, d=128, rot=128,
             interleaved=False, l2=False, weight=True, far=False),
        # prefill of 4 sequences x 4096 tokens at width 2048 (16 heads of 128)
        dict(name="glu prefill 4x4096", op="glu", type="bf16", T=16384, D=2048, F=8192, act="silu"),
        # a short prompt with odd sizes
        dict(name="glu odd prompt", op="glu", type="bf16", T=333, D=1003, F=2777, act="gelu"),
        # decode: 64 sequences at width 4096 (32 heads of 128)
        dict(name="glu decode 64", op="glu", type="bf16", T=64, D=4096, F=8192, act="silu"),
        # decode of one sequence
        dict(name="glu decode 1", op="glu", type="bf16", T=1, D=2048, F=8192, act="silu"),
        # trainer, 2 x 4096 tokens at width 4096: forward and gradients
        dict(name="glu training 2x4096", op="glu_train", type="bf16", T=8192, D=4096, F=8192, act="silu"),
        # the sampled tokens' log-probabilities in one rollout step of 64 sequences
        dict(name="policy rollout 64", op="logprob", type="bf16", T=64, V=131072, tau=0.7),
        # a ragged micro-batch with fp32 logits and an odd vocabulary: the loss alone
        dict(name="policy loss ragged fp32", op="loss", type="f32", T=777, V=50021, tau=1.0, kl=0.05),
        # a trainer's micro-batch of 4096 tokens: the loss and the logits' gradient
        dict(name="policy training 4096", op="loss_train", type="bf16", T=4096, V=131072, tau=1.0, kl=0.05),
    ]


def _log_int(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, v))


def _width(rng, lo, hi):
    """A width of the range: a multiple of 64 half of the time, any number otherwise."""
    n = _log_int(rng, lo, hi)
    return max(64, n // 64 * 64) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["qk", "qk_train", "glu", "glu", "glu_train", "logprob", "loss", "loss_train"])
    if op.startswith("qk"):
        c = dict(op=op, type=rng.choice(["bf16", "bf16", "f32"]))
        c["d"] = rng.choice([16, 32, 64, 64, 128, 128, 256, 2 * rng.randint(8, 128)])
        c["Hk"] = _log_int(rng, 1, 32)
        c["Hq"] = c["Hk"] * rng.choice([1, 1, 2, 4, 8])
        size = (2 if c["type"] == "bf16" else 4) * (c["Hq"] + c["Hk"]) * c["d"]
        c["T"] = _log_int(rng, 1, min(65536, 16384 * 64 * 128 * 2 // size))
        c["rot"] = rng.choice([0, c["d"], c["d"], 2 * rng.randint(1, c["d"] // 2)])
        c.update(interleaved=rng.random() < 0.3, l2=rng.random() < 0.4, weight=rng.random() < 0.6,
                 far=rng.random() < 0.3)
        return c
    if op.startswith("glu"):
        c = dict(op=op, type="bf16", act=rng.choice(["silu", "silu", "gelu"]))
        c["D"], c["F"] = _width(rng, 64, 8192), _width(rng, 64, 16384)
        c["T"] = _log_int(rng, 1, max(1, min(32768, 8192 * 4096 * 8192 // (c["D"] * c["F"]))))
        return c
    c = dict(op=op, type=rng.choice(["bf16", "bf16", "f32"]))
    c["V"] = _width(rng, 100, 262144)
    c["T"] = _log_int(rng, 1, max(1, min(16384, 4096 * 131072 * 2 // (c["V"] * (2 if c["type"] == "bf16" else 4)))))
    c["tau"] = rng.choice([1.0, 1.0, 0.7])
    if op != "logprob":
        c["kl"] = rng.choice([0.0, 0.001, 0.05])
    return c


# -------------------------------------------------------------------- inputs
def _freqs(case):
    n = case["rot"] // 2
    return (1e4 ** (-torch.arange(n, dtype=torch.float64) / max(1, n))).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 1000003 + 29)
    dt = _TYPES[case["type"]]
    f32 = torch.float32

    def normal(*shape, scale=1.0, type=dt):
        return (torch.randn(*shape, generator=g, device=dev, dtype=f32) * scale).to(type)

    op, T, s = case["op"], case["T"], {"case": case}
    if op.startswith("qk"):
        Hq, Hk, d = case["Hq"], case["Hk"], case["d"]
        # slices of one projection's output, each head at a scale of its own
        scale = torch.exp(0.5 * torch.randn(Hq + Hk, 1, generator=g, device=dev))
        rows = (torch.randn(T, Hq + Hk, d, generator=g, device=dev) * scale).to(dt)
        s["q"], s["k"] = rows[:, :Hq], rows[:, Hq:]
        s["qw"] = 1 + normal(d, scale=0.1) if case["weight"] else None
        s["kw"] = 1 + normal(d, scale=0.1) if case["weight"] else None
        start = random.Random(seed).randint(100000, 1000000) if case["far"] else 0
        s["pos"] = (torch.arange(T, device=dev) % 8192 + start).to(torch.int32) if case["rot"] else None
        s["freq"] = _freqs(case).to(dev) if case["rot"] else None
        if op == "qk_train":
            s["dq"], s["dk"] = normal(T, Hq, d), normal(T, Hk, d)
    elif op.startswith("glu"):
        D, F = case["D"], case["F"]
        s["x"] = normal(T, D)
        s["wg"], s["wu"] = normal(F, D, scale=1 / math.sqrt(D)), normal(F, D, scale=1 / math.sqrt(D))
        if op == "glu_train":
            s["dh"] = normal(T, F)
    else:
        V = case["V"]
        z = normal(T, V, scale=2.5)
        y = torch.randint(0, V, (T,), generator=g, device=dev)
        rows = torch.arange(T, device=dev)
        # a sampled token has a high logit: a log-probability of mostly -5 to 0
        top = math.log(V) + 3.1
        z[rows, y] = (top + 8 * torch.rand(T, generator=g, device=dev) - 6).to(dt)
        s["z"], s["y"] = z, y
        if op != "logprob":
            lp = torch.cat([torch.log_softmax(p.float() / case["tau"], 1).gather(1, t[:, None])[:, 0]
                            for p, t in zip(z.split(256), y.split(256))])
            # ratios on both sides of the clip's borders, none within the rounding of a log-probability of one
            gap = 0.15 * torch.randn(T, generator=g, device=dev)
            for border in (math.log(1 - _CLIP[0]), math.log(1 + _CLIP[1])):
                gap = torch.where((gap - border).abs() < 1e-3, gap + 2e-3, gap)
            s["old"] = lp - gap
            s["ref"] = lp + 0.3 * torch.randn(T, generator=g, device=dev)
            s["adv"] = torch.randn(T, generator=g, device=dev)
            # prompt and padding rows
            y[torch.rand(T, generator=g, device=dev) < 0.1] = _IGNORED
            s["dloss"] = torch.full((T,), 1.0 / T, device=dev)
    return s


# ---------------------------------------------------------------- plain form
def _turn(s, dtype=torch.float32):
    """cos and sin [T, 1, rot / 2] of each token's angles, which are formed in 64 bits."""
    a = s["pos"].double()[:, None] * s["freq"].double()
    return torch.cos(a).to(dtype)[:, None], torch.sin(a).to(dtype)[:, None]


def _pairs(x, rot, interleaved):
    if interleaved:
        return x[..., 0:rot:2], x[..., 1:rot:2]
    return x[..., : rot // 2], x[..., rot // 2: rot]


def _rotate(s, x, sign=1.0):
    c = s["case"]
    rot = c["rot"]
    if rot == 0:
        return x
    cos, sin = _turn(s)
    a, b = _pairs(x, rot, c["interleaved"])
    ra, rb = a * cos - sign * b * sin, b * cos + sign * a * sin
    turned = torch.stack([ra, rb], -1).flatten(-2) if c["interleaved"] else torch.cat([ra, rb], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _qk_one(s, x, w):
    c, t = s["case"], x.dtype
    x = x.float()
    n = 1 if c["l2"] else c["d"]
    u = x / torch.sqrt((x * x).sum(-1, keepdim=True) / n + _EPS)
    if w is not None:
        u = u * w.float()
    return _rotate(s, u).to(t)


def _qk_one_grad(s, x, w, dy):
    c, t = s["case"], x.dtype
    x = x.float()
    n = 1 if c["l2"] else c["d"]
    r = 1 / torch.sqrt((x * x).sum(-1, keepdim=True) / n + _EPS)
    g = _rotate(s, dy.float(), -1.0)
    u = x * r
    dw = None
    if w is not None:
        dw = (g * u).sum((0, 1))
        g = g * w.float()
    return (r * (g - u * ((g * u).sum(-1, keepdim=True) / n))).to(t), dw


def _qk(s):
    return _qk_one(s, s["q"], s["qw"]), _qk_one(s, s["k"], s["kw"])


def _qk_train(s):
    dq, dqw = _qk_one_grad(s, s["q"], s["qw"], s["dq"])
    dk, dkw = _qk_one_grad(s, s["k"], s["kw"], s["dk"])
    return _qk(s) + (dq, dk, dqw, dkw)


def _act(v, act):
    """The activation and its derivative."""
    if act == "silu":
        e = 1 / (1 + torch.exp(-v))
        return v * e, e * (1 + v * (1 - e))
    # 0.5 v (1 + tanh t), t = c (v + 0.044715 v^3), through sigmoid(2 t)
    t = math.sqrt(8 / math.pi) * (v + 0.044715 * v * v * v)
    e = 1 / (1 + torch.exp(-t))
    return v * e, e + v * e * (1 - e) * math.sqrt(8 / math.pi) * (1 + 3 * 0.044715 * v * v)


def _glu(s):
    x = s["x"].float()
    a, _ = _act(x @ s["wg"].float().t(), s["case"]["act"])
    return (a * (x @ s["wu"].float().t())).to(s["x"].dtype)


def _glu_train(s):
    x, wg, wu, dh = s["x"].float(), s["wg"].float(), s["wu"].float(), s["dh"].float()
    g, u = x @ wg.t(), x @ wu.t()
    a, slope = _act(g, s["case"]["act"])
    dg, du = dh * u * slope, dh * a
    t = s["x"].dtype
    return (a * u).to(t), (dg @ wg + du @ wu).to(t), (dg.t() @ x).to(t), (du.t() @ x).to(t)


def _logprob(s):
    """Log-probabilities, softmax's logarithm's parts and which rows take part."""
    z = s["z"].float() / s["case"]["tau"]
    top = z.max(1, keepdim=True).values
    lse = top + torch.log(torch.exp(z - top).sum(1, keepdim=True))
    on = s["y"] >= 0
    lp = z.gather(1, s["y"].clamp(min=0)[:, None])[:, 0] - lse[:, 0]
    return z, lse, on, torch.where(on, lp, torch.zeros_like(lp))


def _loss_parts(s, lp):
    """The loss of each row and its derivative for the log-probability."""
    adv = s["adv"]
    ratio = torch.exp(lp - s["old"])
    lo, hi = 1 - _CLIP[0], 1 + _CLIP[1]
    free, held = -adv * ratio, -adv * torch.clamp(ratio, lo, hi)
    d = torch.where(free >= held, -adv * ratio, torch.zeros_like(lp))
    loss = torch.maximum(free, held)
    kl = s["case"]["kl"]
    if kl:
        gap = s["ref"] - lp
        loss = loss + kl * (torch.exp(gap) - gap - 1)
        d = d + kl * (1 - torch.exp(gap))
    return loss, d


def _policy(s):
    z, lse, on, lp = _logprob(s)
    if s["case"]["op"] == "logprob":
        return lp
    zero = torch.zeros_like(lp)
    loss, d = _loss_parts(s, lp)
    loss = torch.where(on, loss, zero)
    if s["case"]["op"] == "loss":
        return loss, lp
    d = torch.where(on, d * s["dloss"] / s["case"]["tau"], zero)
    grad = torch.exp(z - lse) * -d[:, None]
    grad[torch.arange(z.shape[0], device=z.device), s["y"].clamp(min=0)] += d
    return loss, lp, grad.to(s["z"].dtype)


_PLAIN = dict(qk=_qk, qk_train=_qk_train, glu=_glu, glu_train=_glu_train, logprob=_policy, loss=_policy,
              loss_train=_policy)


# ------------------------------------------------------------ the library's
def _own_run(s):
    from gated_deltanet_cpr_delta_b200 import gdn

    c = s["case"]
    op = c["op"]
    if op.startswith("qk"):
        kind = dict(q_weight=s["qw"], k_weight=s["kw"], positions=s["pos"], inv_freq=s["freq"],
                    interleaved=c["interleaved"], l2=c["l2"], eps=_EPS)
        y = gdn.gdn_qk_norm_forward(s["q"], s["k"], **kind)
        return y if op == "qk" else y + tuple(gdn.gdn_qk_norm_backward(s["q"], s["k"], s["dq"], s["dk"], **kind))
    if op.startswith("glu"):
        h, saved = gdn.gdn_glu_forward(s["x"], s["wg"], s["wu"], act=c["act"], save=op == "glu_train")
        if op == "glu":
            return h
        return (h,) + tuple(gdn.gdn_glu_backward(s["x"], s["wg"], s["wu"], s["dh"], saved, act=c["act"]))
    if op == "logprob":
        return gdn.gdn_policy_loss_forward(s["z"], s["y"], temperature=c["tau"])[1]
    kind = dict(old_logprob=s["old"], advantages=s["adv"], ref_logprob=s["ref"] if c["kl"] else None,
                kl_coef=c["kl"], clip_low=_CLIP[0], clip_high=_CLIP[1], temperature=c["tau"])
    if op == "loss":
        return gdn.gdn_policy_loss_forward(s["z"], s["y"], **kind)
    dz, loss, lp = gdn.gdn_policy_loss_backward(s["z"], s["y"], s["dloss"], **kind)
    return loss, lp, dz


def run(state):
    return _own_run(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------- work
def work(case):
    """Each input read once, each output written once; multiply-adds count two, exponentials one."""
    e = 2 if case["type"] == "bf16" else 4
    op, T = case["op"], case["T"]
    if op.startswith("qk"):
        n, d = T * (case["Hq"] + case["Hk"]) * case["d"], case["d"]
        extra = (4 * T + 2 * case["rot"] if case["rot"] else 0) + (2 * d * e if case["weight"] else 0)
        if op == "qk":
            return {"bytes": 2 * n * e + extra, "flops": 8 * n}
        return {"bytes": 4 * n * e + extra + (8 * d if case["weight"] else 0), "flops": 26 * n}
    if op.startswith("glu"):
        D, F = case["D"], case["F"]
        fwd = e * (T * D + 2 * F * D + T * F)
        if op == "glu":
            return {"bytes": fwd, "flops": 4 * T * D * F + 8 * T * F}
        return {"bytes": fwd + e * (T * F + T * D + 2 * F * D), "flops": 12 * T * D * F + 30 * T * F}
    n = T * case["V"]
    rows = T * (8 + 4 + (0 if op == "logprob" else 4 + 4 * (3 if case["kl"] else 2)))
    if op == "loss_train":
        return {"bytes": 2 * n * e + rows + 4 * T, "flops": 7 * n}
    return {"bytes": n * e + rows, "flops": 4 * n}


# --------------------------------------------------------------------- exact
def _exact_head(s, x, w):
    """One tensor's norm and rotation; the rotation as a product of complex numbers."""
    c = s["case"]
    y = x * torch.rsqrt((x.square().sum(-1, keepdim=True) if c["l2"] else x.square().mean(-1, keepdim=True)) + _EPS)
    y = y if w is None else y * w
    R = c["rot"]
    if R == 0:
        return y
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                       s["pos"].double()[:, None, None] * s["freq"].double())
    if c["interleaved"]:
        v = torch.view_as_real(torch.view_as_complex(y[..., :R].unflatten(-1, (R // 2, 2)).contiguous()) * turn)
        return torch.cat([v.flatten(-2), y[..., R:]], -1)
    v = torch.complex(y[..., : R // 2], y[..., R // 2: R]) * turn
    return torch.cat([v.real, v.imag, y[..., R:]], -1)


def _exact_policy(s, z, y, old, ref, adv):
    """Losses and log-probabilities of rows that all take part."""
    c = s["case"]
    lp = torch.log_softmax(z / c["tau"], 1)[torch.arange(z.shape[0], device=z.device), y]
    if c["op"] == "logprob":
        return None, lp
    r = (lp - old).exp()
    loss = -torch.minimum(r * adv, r.clamp(1 - _CLIP[0], 1 + _CLIP[1]) * adv)
    return loss + c["kl"] * ((ref - lp).exp() - (ref - lp) - 1), lp


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    p = {k: v.double() if torch.is_tensor(v) and k not in ("y", "pos", "freq", "z") else v for k, v in s.items()}
    if op.startswith("qk"):
        names = ["q", "k", "qw", "kw"]
        if op == "qk_train":
            for n in names:
                p[n] = p[n].clone().requires_grad_() if p[n] is not None else None
        yq, yk = _exact_head(s, p["q"], p["qw"]), _exact_head(s, p["k"], p["kw"])
        if op == "qk":
            return yq, yk
        loss = (yq * p["dq"]).sum() + (yk * p["dk"]).sum()
        have = [n for n in names if p[n] is not None]
        got = dict(zip(have, torch.autograd.grad(loss, [p[n] for n in have])))
        return (yq.detach(), yk.detach()) + tuple(got.get(n) for n in names)
    if op.startswith("glu"):
        if case["act"] == "silu":
            act = torch.nn.functional.silu
        else:
            act = lambda v: torch.nn.functional.gelu(v, approximate="tanh")  # noqa: E731
        leaves = [p["x"], p["wg"], p["wu"]]
        if op == "glu_train":
            for v in leaves:
                v.requires_grad_()
        h = act(p["x"] @ p["wg"].t()) * (p["x"] @ p["wu"].t())
        return h if op == "glu" else (h.detach(),) + torch.autograd.grad((h * p["dh"]).sum(), leaves)
    # some rows at a time: a row's 64-bit copies are many times its size
    T = case["T"]
    loss, lp = torch.zeros(2, T, dtype=torch.float64, device="cuda")
    grad = torch.zeros(T, case["V"], dtype=torch.float64, device="cuda") if op == "loss_train" else None
    for i in range(0, T, 512):
        rows = torch.arange(i, min(T, i + 512), device="cuda")
        rows = rows[s["y"][rows] >= 0]
        if rows.numel() == 0:
            continue
        z = s["z"][rows].double().requires_grad_(op == "loss_train")
        have = [p[n][rows] if n in p else None for n in ("old", "ref", "adv")]
        row_loss, row_lp = _exact_policy(s, z, s["y"][rows], *have)
        if grad is not None:
            grad[rows] = torch.autograd.grad((row_loss * p["dloss"][rows]).sum(), z)[0]
        lp[rows] = row_lp.detach()
        if row_loss is not None:
            loss[rows] = row_loss.detach()
    return lp if op == "logprob" else (loss, lp) if op == "loss" else (loss, lp, grad)
