"""The layer operators around the recurrent mixers, as cases to measure.

Three operators, each in its directions:

  conv        the short causal convolution of a packed batch (prefill), its
              gradients, and its single-token step on a cache
  ssm         the selective state space scan of a packed batch, a training step
              (forward and gradients), and its single-token step on a cache
  layer_norm  forward, and a training step with the weight's gradient

`run` computes them in elementary torch operations where `own` is false, and
calls the library's entry points where it is true.  `exact` is the definition
in 64 bits, written token by token or through autograd of a 64-bit forward.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-5


# --------------------------------------------------------------------- cases
def listed():
    return [
        # prefill of 4 sequences x 4096 tokens: the convolution over the joined q, k, v of 16 heads of 128
        dict(name="conv prefill 4x4096", op="conv", type="bf16", T=16384, seqs=4, ragged=False, D=6144, W=4,
             silu=True, bias=False, state=False),
        # an odd, ragged batch that continues from cached inputs, fp32, every option on
        dict(name="conv ragged fp32", op="conv", type="f32", T=3001, seqs=7, ragged=True, D=1003, W=3,
             silu=True, bias=True, state=True),
        # trainer gradients at 2 x 8192 tokens, the values of 16 heads of 128
        dict(name="conv gradients 2x8192", op="conv_grad", type="bf16", T=16384, seqs=2, ragged=False, D=2048, W=4,
             silu=True, bias=True, state=False),
        # decode: 64 sequences, the joined q, k, v of 32 heads of 128
        dict(name="conv step 64", op="conv_step", type="bf16", N=64, D=12288, W=4, silu=True, bias=True),
        # prefill of 4 x 4096 tokens, inner width of 16 heads of 128
        dict(name="ssm prefill 4x4096", op="ssm", type="bf16", T=16384, seqs=4, ragged=False, D=2048, S=16, G=1,
             z=True, state=False),
        # one short prompt, latency bound: 257 tokens, a wider state
        dict(name="ssm short prompt", op="ssm", type="bf16", T=257, seqs=1, ragged=False, D=1024, S=32, G=2,
             z=True, state=True),
        # a ragged fp32 batch with an odd width and no gate
        dict(name="ssm ragged fp32", op="ssm", type="f32", T=5003, seqs=9, ragged=True, D=777, S=16, G=1,
             z=False, state=True),
        # one training step, 2 x 4096 tokens
        dict(name="ssm training 2x4096", op="ssm_train", type="bf16", T=8192, seqs=2, ragged=False, D=2048, S=16,
             G=1, z=True, state=False),
        # decode: 64 sequences, inner width of 32 heads of 128
        dict(name="ssm step 64", op="ssm_step", type="bf16", N=64, D=4096, S=16, G=1, z=True),
        # the recurrence's output of 4 x 4096 tokens, normalised per head: 16 heads of 128
        dict(name="layer_norm heads", op="norm", type="bf16", R=262144, D=128, bias=False),
        # one decode step's 64 tokens at width 4096
        dict(name="layer_norm decode 64", op="norm", type="bf16", R=64, D=4096, bias=True),
        # training, 2 x 8192 tokens at width 4096
        dict(name="layer_norm training 2x8192", op="norm_train", type="bf16", R=16384, D=4096, bias=True),
    ]


def _log_int(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, v))


def _width(rng, lo, hi):
    """A width of the range: a multiple of 64 half of the time, any number otherwise."""
    d = _log_int(rng, lo, hi)
    return max(64, d // 64 * 64) if rng.random() < 0.5 else d


def draw(rng):
    op = rng.choice(["conv", "conv_grad", "conv_step", "ssm", "ssm_train", "ssm_step", "norm", "norm_train"])
    c = dict(op=op, type=rng.choice(["bf16", "bf16", "f32"]))
    size = 1 if c["type"] == "bf16" else 2
    yes = lambda: rng.random() < 0.5  # noqa: E731
    if op in ("conv", "conv_grad"):
        c["D"] = _width(rng, 64, 8192)
        c["T"] = _log_int(rng, 1, min(65536, (16384 * (6144 if op == "conv" else 2048)) // (size * c["D"])))
        c["seqs"] = _log_int(rng, 1, max(1, min(64, c["T"])))
        c.update(ragged=yes(), W=rng.choice([2, 3, 4]), silu=rng.random() < 0.8, bias=yes(), state=yes())
    elif op == "conv_step":
        c["D"] = _width(rng, 64, 16384)
        c.update(N=_log_int(rng, 1, 256), W=rng.choice([2, 3, 4]), silu=rng.random() < 0.8, bias=yes())
    elif op in ("ssm", "ssm_train"):
        c["S"] = rng.choice([16, 16, 32, 64])
        c["G"] = rng.choice([1, 1, 2, 4])
        c["D"] = max(1, _width(rng, 64, 4096) // c["G"]) * c["G"]
        most = (16384 if op == "ssm" else 8192) * 2048 * 16 // (size * c["D"] * c["S"])
        c["T"] = _log_int(rng, 1, min(32768, most))
        c["seqs"] = _log_int(rng, 1, max(1, min(32, c["T"])))
        c.update(ragged=yes(), z=yes(), state=yes())
    elif op == "ssm_step":
        c["S"] = rng.choice([16, 32, 64])
        c["G"] = rng.choice([1, 1, 2, 4])
        c["D"] = max(1, _width(rng, 64, 4096) // c["G"]) * c["G"]
        c.update(N=_log_int(rng, 1, 256), z=yes())
    else:
        c["D"] = _width(rng, 32, 16384)
        c["R"] = _log_int(rng, 1, max(1, min(262144, 16384 * 2048 // (size * c["D"]))))
        c["bias"] = yes()
    return c


# -------------------------------------------------------------------- inputs
def _lengths(case, seed):
    """Sequence lengths that add up to T; a ragged batch may hold empty sequences and single tokens."""
    T, n = case["T"], case["seqs"]
    if not case["ragged"]:
        return [T // n + (1 if i < T % n else 0) for i in range(n)]
    r = random.Random(seed * 7919 + T)
    cuts = sorted(r.randint(0, T) for _ in range(n - 1))
    cuts = [0] + cuts + [T]
    return [cuts[i + 1] - cuts[i] for i in range(n)]


def _offsets(lengths, device):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32).to(device)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 1000003 + 17)
    dt = _TYPES[case["type"]]
    f32 = torch.float32

    def normal(*shape, scale=1.0, type=dt):
        return (torch.randn(*shape, generator=g, device=dev, dtype=f32) * scale).to(type)

    op, s = case["op"], {"case": case}
    D = case["D"]
    if op.startswith("conv"):
        W = case["W"]
        s["weight"] = normal(D, W, scale=1.0 / math.sqrt(W))
        s["bias"] = normal(D, scale=0.1) if case["bias"] else None
        if op == "conv_step":
            s["x"], s["state"] = normal(case["N"], D), normal(case["N"], W - 1, D)
            return s
        s["cu"] = _offsets(_lengths(case, seed), dev)
        s["x"] = normal(case["T"], D)
        s["state_in"] = normal(case["seqs"], W - 1, D) if case["state"] else None
        if op == "conv_grad":
            s["dy"] = normal(case["T"], D)
            s["dstate_out"] = normal(case["seqs"], W - 1, D, type=f32) if case["state"] else None
    elif op.startswith("ssm"):
        S, G = case["S"], case["G"]
        R = case["N"] if op == "ssm_step" else case["T"]
        s["x"], s["dt"] = normal(R, D), normal(R, D, scale=0.3)
        s["B"], s["C"] = normal(R, G, S), normal(R, G, S)
        s["z"] = normal(R, D) if case["z"] else None
        # decay rates 1..S a head start apart, step widths from 0.001 to 0.1, as such layers are initialised
        rate = torch.arange(1, S + 1, device=dev, dtype=f32)
        s["A"] = -rate * torch.exp(0.1 * torch.randn(D, S, generator=g, device=dev, dtype=f32))
        width = torch.exp(torch.empty(D, device=dev).uniform_(math.log(1e-3), math.log(1e-1), generator=g))
        s["dt_bias"] = width + torch.log(-torch.expm1(-width))
        s["D"] = normal(D, type=f32)
        if op == "ssm_step":
            s["state"] = normal(R, D, S, type=f32)
            return s
        s["cu"] = _offsets(_lengths(case, seed), dev)
        s["state_in"] = normal(case["seqs"], D, S, type=f32) if case["state"] else None
        if op == "ssm_train":
            s["dy"] = normal(R, D)
            s["dstate_out"] = normal(case["seqs"], D, S, type=f32) if case["state"] else None
    else:
        s["x"] = normal(case["R"], D) + normal(case["R"], 1, scale=0.5)
        s["weight"] = 1 + normal(D, scale=0.1)
        s["bias"] = normal(D, scale=0.1) if case["bias"] else None
        if op == "norm_train":
            s["dy"] = normal(case["R"], D)
    return s


# ---------------------------------------------------------------- plain form
def _places(cu, T):
    """Each token's sequence and its position in it."""
    t = torch.arange(T, device=cu.device)
    seq = torch.searchsorted(cu, t.to(torch.int32), right=True) - 1
    return seq, t - cu[seq]


def _earlier(x, state, seq, pos, j, W):
    """x[t - j] within the sequence; before its start, the state (or zeros).  In 32 bits."""
    rows = torch.arange(x.shape[0], device=x.device)
    inside = (pos >= j)[:, None]
    v = torch.where(inside, x[(rows - j).clamp(min=0)].float(), torch.zeros((), device=x.device))
    if state is not None and j > 0:
        v = torch.where(inside, v, state[seq, (W - 1 + pos - j).clamp(0, W - 2)].float())
    return v


def _tail(x, state, cu, W):
    """The last W-1 inputs of each sequence, the state's where it is shorter."""
    L = (cu[1:] - cu[:-1]).long()[:, None]
    p = L - (W - 1) + torch.arange(W - 1, device=x.device)
    new = x[(cu[:-1].long()[:, None] + p).clamp(0, x.shape[0] - 1)]
    n = torch.arange(p.shape[0], device=x.device)[:, None]
    old = torch.zeros_like(new) if state is None else state[n, (W - 1 + p).clamp(0, W - 2)]
    return torch.where((p >= 0)[..., None], new, old)


def _act(v, silu):
    return v / (1 + torch.exp(-v)) if silu else v


def _act_grad(v, silu):
    if not silu:
        return torch.ones_like(v)
    s = 1 / (1 + torch.exp(-v))
    return s * (1 + v * (1 - s))


def _conv(s):
    c, x, w = s["case"], s["x"], s["weight"].float()
    W = c["W"]
    seq, pos = _places(s["cu"], c["T"])
    pre = sum(w[:, W - 1 - j] * _earlier(x, s["state_in"], seq, pos, j, W) for j in range(W))
    if s["bias"] is not None:
        pre = pre + s["bias"].float()
    return pre, seq, pos


def _conv_forward(s):
    pre, _, _ = _conv(s)
    return _act(pre, s["case"]["silu"]).to(s["x"].dtype), _tail(s["x"], s["state_in"], s["cu"], s["case"]["W"])


def _conv_grad(s):
    c, x, w, cu = s["case"], s["x"], s["weight"].float(), s["cu"].long()
    T, W = c["T"], c["W"]
    pre, seq, pos = _conv(s)
    g = s["dy"].float() * _act_grad(pre, c["silu"])
    rows = torch.arange(T, device=x.device)
    L = cu[1:] - cu[:-1]
    zero = torch.zeros((), device=x.device)
    dx, dw = 0, []
    dstate = torch.zeros(c["seqs"], W - 1, c["D"], device=x.device)
    i = torch.arange(W - 1, device=x.device)
    for j in range(W):
        later = (pos + j < L[seq])[:, None]
        dx = dx + w[:, W - 1 - j] * torch.where(later, g[(rows + j).clamp(max=T - 1)], zero)
        dw.append((g * _earlier(x, s["state_in"], seq, pos, j, W)).sum(0))
        at = (i - (W - 1) + j)[None, :]                       # the position that reads state row i at distance j
        ok = (at >= 0) & (at < L[:, None])
        dstate = dstate + w[:, W - 1 - j] * torch.where(ok[..., None], g[(cu[:-1, None] + at).clamp(0, T - 1)], zero)
    if s["dstate_out"] is not None:
        do = s["dstate_out"]
        k = pos - L[seq] + (W - 1)                            # the state row that this token ends up in
        dx = dx + torch.where((k >= 0)[:, None], do[seq, k.clamp(0, W - 2)], zero)
        k = i[None, :] - L[:, None]                           # where the old row i ends up
        n = torch.arange(c["seqs"], device=x.device)[:, None]
        dstate = dstate + torch.where((k >= 0)[..., None], do[n, k.clamp(0, W - 2)], zero)
    db = g.sum(0) if s["bias"] is not None else None
    return dx.to(x.dtype), torch.stack(dw[::-1], 1), db, dstate


def _conv_step(s):
    c, w = s["case"], s["weight"].float()
    window = torch.cat([s["state"], s["x"][:, None]], 1)
    pre = (window.float() * w.t()).sum(1)
    if s["bias"] is not None:
        pre = pre + s["bias"].float()
    return _act(pre, c["silu"]).to(s["x"].dtype), window[:, 1:].contiguous()


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along the first axis (a_0 is not read), in log2(T) doublings."""
    d = 1
    while d < a.shape[0]:
        b = torch.cat([b[:d], b[d:] + a[d:] * b[:-d]])
        a = torch.cat([a[:d], a[d:] * a[:-d]])
        d *= 2
    return b


def _step_width(s):
    v = s["dt"].float() + s["dt_bias"]
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs())), v


def _per_channel(v, D):
    """[.., G, S] of groups of channels -> [.., D, S]."""
    return v.float().repeat_interleave(D // v.shape[-2], dim=-2)


def _gate(z):
    return z.float() / (1 + torch.exp(-z.float()))


def _ssm_parts(s):
    """Step widths, decays (zero at each sequence's first token, whose state enters b), inputs and states."""
    c, cu = s["case"], s["cu"].long()
    delta, v = _step_width(s)
    decay = torch.exp(delta[:, :, None] * s["A"])
    b = (delta * s["x"].float())[:, :, None] * _per_channel(s["B"], c["D"])
    L = cu[1:] - cu[:-1]
    first = cu[:-1].clamp(max=c["T"] - 1)
    a = decay.clone()
    if s["state_in"] is not None:
        b.index_add_(0, first, decay[first] * s["state_in"] * (L > 0)[:, None, None])
    a[_places(s["cu"], c["T"])[1] == 0] = 0
    return delta, v, decay, a, _scan(a, b)


def _last_states(s, h):
    cu = s["cu"].long()
    old = torch.zeros_like(h[:1]) if s["state_in"] is None else s["state_in"]
    return torch.where((cu[1:] > cu[:-1])[:, None, None], h[(cu[1:] - 1).clamp(min=0)], old)


def _ssm_out(s, h):
    raw = (h * _per_channel(s["C"], s["case"]["D"])).sum(-1) + s["D"] * s["x"].float()
    return raw, (raw * _gate(s["z"]) if s["z"] is not None else raw).to(s["x"].dtype)


def _ssm_forward(s):
    _, _, _, _, h = _ssm_parts(s)
    return _ssm_out(s, h)[1], _last_states(s, h)


def _ssm_train(s):
    c, x, cu = s["case"], s["x"].float(), s["cu"].long()
    T, D, S, G = c["T"], c["D"], c["S"], c["G"]
    delta, v, decay, a, h = _ssm_parts(s)
    raw, y = _ssm_out(s, h)
    dy, dz = s["dy"].float(), None
    if s["z"] is not None:
        dz = (dy * raw * _act_grad(s["z"].float(), True)).to(s["x"].dtype)
        dy = dy * _gate(s["z"])
    L = cu[1:] - cu[:-1]
    Bc, Cc = _per_channel(s["B"], D), _per_channel(s["C"], D)
    q = Cc * dy[:, :, None]
    if s["dstate_out"] is not None:
        q.index_add_(0, (cu[1:] - 1).clamp(min=0), s["dstate_out"] * (L > 0)[:, None, None])
    after = torch.cat([a[1:], torch.zeros_like(a[:1])])       # the decay from a token to the next of its sequence
    g = _scan(after.flip(0), q.flip(0)).flip(0)               # dL/dh_t
    dC = (h * dy[:, :, None]).reshape(T, G, D // G, S).sum(2)
    dB = (g * (delta * x)[:, :, None]).reshape(T, G, D // G, S).sum(2)
    gB = (g * Bc).sum(-1)
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    first = cu[:-1].clamp(max=T - 1)
    before[_places(s["cu"], T)[1] == 0] = 0
    if s["state_in"] is not None:
        before.index_add_(0, first, s["state_in"] * (L > 0)[:, None, None])
    e = g * before * decay                                    # dL/d(delta A)
    dA = (e * delta[:, :, None]).sum(0)
    ddelta = (e * s["A"]).sum(-1) + gB * x
    dv = ddelta / (1 + torch.exp(-v))
    dx = delta * gB + s["D"] * dy
    dstate = decay[first] * g[first] * (L > 0)[:, None, None]
    if s["dstate_out"] is not None:
        dstate = dstate + s["dstate_out"] * (L == 0)[:, None, None]
    t = s["x"].dtype
    return (y, _last_states(s, h), dx.to(t), dv.to(t), dA, dB.to(t), dC.to(t), (dy * x).sum(0), dz, dv.sum(0), dstate)


def _ssm_step(s):
    c = s["case"]
    delta, _ = _step_width(s)
    x = s["x"].float()
    h = torch.exp(delta[:, :, None] * s["A"]) * s["state"] + (delta * x)[:, :, None] * _per_channel(s["B"], c["D"])
    return _ssm_out(s, h)[1], h


def _norm_parts(s):
    x = s["x"].float()
    mean = x.mean(1)
    rstd = 1 / torch.sqrt(((x - mean[:, None]) ** 2).mean(1) + _EPS)
    return x, mean, rstd


def _norm_forward(s):
    x, mean, rstd = _norm_parts(s)
    y = (x - mean[:, None]) * rstd[:, None] * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["x"].dtype), mean, rstd


def _norm_train(s):
    x, mean, rstd = _norm_parts(s)
    y = _norm_forward(s)[0]
    dy, n = s["dy"].float(), (x - mean[:, None]) * rstd[:, None]
    g = dy * s["weight"].float()
    dx = rstd[:, None] * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True))
    return y, dx.to(s["x"].dtype), (dy * n).sum(0), dy.sum(0)


_PLAIN = dict(conv=_conv_forward, conv_grad=_conv_grad, conv_step=_conv_step, ssm=_ssm_forward, ssm_train=_ssm_train,
              ssm_step=_ssm_step, norm=_norm_forward, norm_train=_norm_train)


# ------------------------------------------------------------ the library's
def _own_run(s):
    from gated_deltanet_cpr_delta_b200 import gdn

    c = s["case"]
    op = c["op"]
    if op == "conv":
        return gdn.gdn_conv_forward(s["x"], s["weight"], s["cu"], bias=s["bias"], state_in=s["state_in"],
                                    silu=c["silu"])
    if op == "conv_grad":
        return gdn.gdn_conv_backward(s["x"], s["weight"], s["dy"], s["cu"], bias=s["bias"], state_in=s["state_in"],
                                     silu=c["silu"], dstate_out=s["dstate_out"])
    if op == "conv_step":
        state = torch.empty_like(s["state"])
        y = gdn.gdn_conv_step(s["x"], s["weight"], s["state"], bias=s["bias"], silu=c["silu"], state_out=state)
        return y, state
    if op in ("ssm", "ssm_train"):
        y, last, states = gdn.gdn_ssm_forward(s["x"], s["dt"], s["A"], s["B"], s["C"], s["cu"], D=s["D"], z=s["z"],
                                              dt_bias=s["dt_bias"], state_in=s["state_in"],
                                              save_states=op == "ssm_train")
        if op == "ssm":
            return y, last
        grads = gdn.gdn_ssm_backward(s["x"], s["dt"], s["A"], s["B"], s["C"], s["dy"], states, s["cu"], D=s["D"],
                                     z=s["z"], dt_bias=s["dt_bias"], dstate_out=s["dstate_out"])
        return (y, last) + tuple(grads)
    if op == "ssm_step":
        state = torch.empty_like(s["state"])
        y = gdn.gdn_ssm_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["state"], D=s["D"], z=s["z"],
                             dt_bias=s["dt_bias"], state_out=state)
        return y, state
    y, mean, rstd = gdn.gdn_layer_norm_forward(s["x"], s["weight"], bias=s["bias"], eps=_EPS)
    if op == "norm":
        return y, mean, rstd
    return (y,) + tuple(gdn.gdn_layer_norm_backward(s["x"], s["weight"], s["dy"], mean, rstd))


def run(state):
    return _own_run(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------- work
def work(case):
    """Each input read once, each output written once; multiply-adds count two, exponentials one."""
    e = 2 if case["type"] == "bf16" else 4
    op, D = case["op"], case["D"]
    if op.startswith("conv"):
        W = case["W"]
        weight = D * W * e + (D * e if case["bias"] else 0)
        if op == "conv_step":
            n = case["N"] * D
            return {"bytes": n * e * (2 + 2 * (W - 1)) + weight, "flops": n * (2 * W + 4)}
        n, tail = case["T"] * D, case["seqs"] * (W - 1) * D
        if op == "conv":
            return {"bytes": n * e * 2 + tail * e * (2 if case["state"] else 1) + weight, "flops": n * (2 * W + 4)}
        return {"bytes": n * e * 3 + tail * (4 + (4 + e if case["state"] else 0)) + weight + D * 4 * (W + 1),
                "flops": n * (6 * W + 10)}
    if op.startswith("ssm"):
        S, G = case["S"], case["G"]
        z = 1 if case["z"] else 0
        R = case["N"] if op == "ssm_step" else case["T"]
        n, per = R * D, D * S * 4 + 8 * D
        if op == "ssm_step":
            return {"bytes": n * e * (3 + z) + 2 * R * G * S * e + per + 2 * n * S * 4, "flops": n * (7 * S + 12)}
        states = case["seqs"] * D * S * 4
        if op == "ssm":
            return {"bytes": n * e * (3 + z) + 2 * R * G * S * e + per + states * (2 if case["state"] else 1),
                    "flops": n * (7 * S + 12)}
        return {"bytes": n * e * (6 + 2 * z) + 4 * R * G * S * e + 2 * per + states * (4 if case["state"] else 2),
                "flops": n * (21 * S + 30)}
    n, rows = case["R"] * D, case["R"]
    b = D * e * (2 if case["bias"] else 1)
    if op == "norm":
        return {"bytes": n * e * 2 + rows * 8 + b, "flops": n * 7}
    return {"bytes": n * e * 4 + b + 8 * D, "flops": n * 20}


# --------------------------------------------------------------------- exact
def _spans(s):
    cu = s["cu"].tolist()
    return [(n, cu[n], cu[n + 1]) for n in range(len(cu) - 1)]


def _exact_conv(s, x, w, b, st):
    """Per sequence: a padded convolution in 64 bits.  Returns outputs and final states."""
    c = s["case"]
    W = c["W"]
    ys, tails = [], []
    for n, lo, hi in _spans(s):
        head = st[n] if st is not None else x.new_zeros(W - 1, c["D"])
        full = torch.cat([head, x[lo:hi]])
        if hi > lo:
            pre = torch.einsum("tdw,dw->td", full.unfold(0, W, 1), w)
            pre = pre + b if b is not None else pre
            ys.append(torch.nn.functional.silu(pre) if c["silu"] else pre)
        tails.append(full[full.shape[0] - (W - 1):])
    return torch.cat(ys), torch.stack(tails)


def _exact_scan(s, p):
    """Token by token in 64 bits.  p: the inputs as 64-bit tensors."""
    c = s["case"]
    D, S, G = c["D"], c["S"], c["G"]
    delta = torch.nn.functional.softplus(p["dt"] + p["dt_bias"], threshold=1e9)
    u = delta * p["x"]
    ys, last = [], []
    for n, lo, hi in _spans(s):
        h = p["state_in"][n] if p["state_in"] is not None else p["x"].new_zeros(D, S)
        for t in range(lo, hi):
            Bt = p["B"][t][:, None].expand(G, D // G, S).reshape(D, S)
            Ct = p["C"][t][:, None].expand(G, D // G, S).reshape(D, S)
            h = torch.exp(delta[t][:, None] * p["A"]) * h + u[t][:, None] * Bt
            ys.append(torch.einsum("ds,ds->d", h, Ct))
        last.append(h)
    y = torch.stack(ys) + p["D"] * p["x"]
    if p["z"] is not None:
        y = y * torch.nn.functional.silu(p["z"])
    return y, torch.stack(last)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    grad = op in ("conv_grad", "ssm_train", "norm_train")
    # token by token with a graph for the gradients: about 0.3 ms a token
    if op == "ssm_train" and case["T"] > 9000 or op == "ssm" and case["T"] > 40000:
        return None
    p = {k: v.double().requires_grad_(grad) if torch.is_tensor(v) and k != "cu" else v for k, v in s.items()}

    def gradients(loss, names):
        have = [k for k in names if p[k] is not None]
        got = dict(zip(have, torch.autograd.grad(loss, [p[k] for k in have], allow_unused=True)))
        return [None if p[k] is None else torch.zeros_like(p[k]) if got[k] is None else got[k] for k in names]

    if op == "conv":
        return _exact_conv(s, p["x"], p["weight"], p["bias"], p["state_in"])
    if op == "conv_grad":
        if p["state_in"] is None:
            p["state_in"] = torch.zeros(case["seqs"], case["W"] - 1, case["D"], dtype=torch.float64, device="cuda",
                                        requires_grad=True)
        y, tail = _exact_conv(s, p["x"], p["weight"], p["bias"], p["state_in"])
        loss = (y * p["dy"]).sum() + ((tail * p["dstate_out"]).sum() if p["dstate_out"] is not None else 0)
        return gradients(loss, ("x", "weight", "bias", "state_in"))
    if op == "conv_step":
        full = torch.cat([p["state"], p["x"][:, None]], 1)
        pre = torch.einsum("nwd,dw->nd", full, p["weight"])
        pre = pre + p["bias"] if p["bias"] is not None else pre
        return torch.nn.functional.silu(pre) if case["silu"] else pre, full[:, 1:]
    if op == "ssm":
        return _exact_scan(s, p)
    if op == "ssm_train":
        if p["state_in"] is None:
            p["state_in"] = torch.zeros(case["seqs"], case["D"], case["S"], dtype=torch.float64, device="cuda",
                                        requires_grad=True)
        y, last = _exact_scan(s, p)
        loss = (y * p["dy"]).sum() + ((last * p["dstate_out"]).sum() if p["dstate_out"] is not None else 0)
        names = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "state_in")
        return [y.detach(), last.detach()] + gradients(loss, names)
    if op == "ssm_step":
        N, D, S = p["state"].shape
        spread = lambda v: v[:, :, None].expand(N, case["G"], D // case["G"], S).reshape(N, D, S)  # noqa: E731
        delta = torch.nn.functional.softplus(p["dt"] + p["dt_bias"], threshold=1e9)
        h = torch.exp(delta[..., None] * p["A"]) * p["state"] + (delta * p["x"])[..., None] * spread(p["B"])
        y = torch.einsum("nds,nds->nd", h, spread(p["C"])) + p["D"] * p["x"]
        return y * torch.nn.functional.silu(p["z"]) if p["z"] is not None else y, h
    y = torch.nn.functional.layer_norm(p["x"], (case["D"],), p["weight"], p["bias"], _EPS)
    if op == "norm":
        var, mean = torch.var_mean(p["x"], dim=1, correction=0)
        return y, mean, torch.rsqrt(var + _EPS)
    shift = p["bias"] if p["bias"] is not None else torch.zeros(case["D"], dtype=torch.float64, device="cuda",
                                                                requires_grad=True)
    if p["bias"] is None:
        y = y + shift
    dx, dw, db = torch.autograd.grad((y * p["dy"]).sum(), [p["x"], p["weight"], shift])
    return y.detach(), dx, dw, db
