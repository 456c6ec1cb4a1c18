"""The norm of queries and keys, the gated block and the policy loss as a program uses them: a step of a small
model from its tokens' embeddings to the loss and back, the same model token by token, several streams, and
tensors beyond 2^31 elements."""
import numpy as np
import pytest
import torch

from gated_deltanet_cpr_delta_b200 import gdn
from oracle import block_ops as ops
from test_gpu_layer_ops import U

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
E, H, D, F, V, C = 128, 2, 32, 192, 500, 16   # width, heads, head width, inner width, vocabulary, chunk
LENGTHS = [40, 17, 1, 30]


def model(seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s, scale=1.0: (torch.randn(*s, generator=g, device="cuda") * scale).to(BF)  # noqa: E731
    p = dict(qkv=r(3 * H * D, E, scale=E ** -0.5), conv=r(3 * H * D, 4, scale=0.5), qw=1 + r(D, scale=0.1), kw=1 + r(D, scale=0.1),
             norm=1 + r(E, scale=0.1), o=r(E, H * D, scale=(H * D) ** -0.5), wg=r(F, E, scale=E ** -0.5), wu=r(F, E, scale=E ** -0.5),
             down=r(E, F, scale=F ** -0.5), head=r(V, E, scale=2 * E ** -0.5))
    T = sum(LENGTHS)
    cu_h = np.concatenate([[0], np.cumsum(LENGTHS)]).tolist()
    b = dict(x=r(T, E), alpha=torch.rand(T, H, generator=g, device="cuda") * 0.4 + 0.6, beta=torch.rand(T, H, generator=g, device="cuda"),
             pos=torch.cat([torch.arange(n) for n in LENGTHS]).to(torch.int32).cuda(), cu=torch.tensor(cu_h, dtype=torch.int32).cuda(),
             freq=100.0 ** (-torch.arange(D // 4, device="cuda", dtype=F32) / (D // 4)),
             y=torch.randint(0, V, (T,), generator=g, device="cuda"), adv=torch.randn(T, generator=g, device="cuda"))
    b["y"][5:9] = -100
    return p, b, cu_h


def step(p, b, cu_h):
    """The library's forward and backward; the plain products in between are the program's own."""
    T = b["x"].shape[0]
    rot = dict(q_weight=p["qw"], k_weight=p["kw"], positions=b["pos"], inv_freq=b["freq"], l2=True)
    qkv = b["x"] @ p["qkv"].t()
    c, _ = gdn.gdn_conv_forward(qkv, p["conv"], b["cu"])
    q, k, v = (c[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)) for i in range(3))
    qn, kn = gdn.gdn_qk_norm_forward(q, k, **rot)
    vc = v.contiguous()
    o, states = gdn.gdn_cpr_forward(qn, kn, vc, b["alpha"], b["beta"], b["cu"], C, cu_seqlens_host=cu_h)
    x1 = b["x"] + o.flatten(1) @ p["o"].t()
    n, mean, rstd = gdn.gdn_layer_norm_forward(x1, p["norm"])
    h, saved = gdn.gdn_glu_forward(n, p["wg"], p["wu"], save=True)
    x2 = x1 + h @ p["down"].t()
    logits = x2 @ p["head"].t()
    lp = gdn.gdn_policy_loss_forward(logits, b["y"])[1]
    pol = dict(old_logprob=lp - 0.05, advantages=b["adv"], ref_logprob=lp + 0.2, kl_coef=0.1)
    w = torch.full((T,), 1.0, device="cuda")
    dz, loss, lp2 = gdn.gdn_policy_loss_backward(logits, b["y"], w, **pol)
    assert torch.equal(lp, lp2)
    g = dict(head=dz.t() @ x2)
    dx2 = dz @ p["head"]
    g["down"] = dx2.t() @ h
    dn, g["wg"], g["wu"] = gdn.gdn_glu_backward(n, p["wg"], p["wu"], dx2 @ p["down"], saved)
    dx1, g["norm"], _ = gdn.gdn_layer_norm_backward(x1, p["norm"], dn, mean, rstd)
    dx1 = dx1 + dx2
    g["o"] = dx1.t() @ o.flatten(1)
    dq, dk, dv, da, db, _ = gdn.gdn_cpr_backward(qn, kn, vc, b["alpha"], b["beta"], (dx1 @ p["o"]).unflatten(1, (H, D)), states,
                                                 b["cu"], C, cu_seqlens_host=cu_h)
    dq, dk, g["qw"], g["kw"] = gdn.gdn_qk_norm_backward(q, k, dq.to(BF), dk.to(BF), **rot)
    dc = torch.cat([dq.flatten(1), dk.flatten(1), dv.to(BF).flatten(1)], 1)
    dqkv, g["conv"], _, _ = gdn.gdn_conv_backward(qkv, p["conv"], dc, b["cu"])
    g["qkv"] = dqkv.t() @ b["x"]
    g["alpha"], g["beta"] = da, db
    return loss, lp, logits, g


def reference(p, b, cu_h):
    """The same in 64 bits, through autograd."""
    p = {k: v.double().requires_grad_() for k, v in p.items()}
    al, be = b["alpha"].double().requires_grad_(), b["beta"].double().requires_grad_()
    x, silu = b["x"].double(), torch.nn.functional.silu

    def head(u, w):
        u = u / torch.sqrt((u * u).sum(-1, keepdim=True) + 1e-6) * w
        a = b["pos"].double()[:, None] * b["freq"].double()
        c, s, R = torch.cos(a)[:, None], torch.sin(a)[:, None], D // 4
        return torch.cat([u[..., :R] * c - u[..., R:2 * R] * s, u[..., R:2 * R] * c + u[..., :R] * s, u[..., 2 * R:]], -1)

    def ln(u, w):
        return torch.nn.functional.layer_norm(u, u.shape[-1:], w, None, 1e-5)

    qkv = x @ p["qkv"].t()
    rows, outs = [], []
    for lo, hi in zip(cu_h[:-1], cu_h[1:]):
        full = torch.cat([qkv.new_zeros(3, qkv.shape[1]), qkv[lo:hi]])
        rows.append(silu(torch.einsum("tdw,dw->td", full.unfold(0, 4, 1), p["conv"])))
    c = torch.cat(rows)
    q, k, v = (c[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)) for i in range(3))
    q, k = head(q, p["qw"]), head(k, p["kw"])
    for lo, hi in zip(cu_h[:-1], cu_h[1:]):
        S = qkv.new_zeros(H, D, D)
        for t in range(lo, hi):
            S = al[t][:, None, None] * (S - be[t][:, None, None] * torch.einsum("hij,hj,hk->hik", S, k[t], k[t])) \
                + be[t][:, None, None] * torch.einsum("hi,hj->hij", v[t], k[t])
            outs.append(torch.einsum("hij,hj->hi", S, q[t]))
    x1 = x + torch.stack(outs).flatten(1) @ p["o"].t()
    n = ln(x1, p["norm"])
    x2 = x1 + (silu(n @ p["wg"].t()) * (n @ p["wu"].t())) @ p["down"].t()
    logits = x2 @ p["head"].t()
    on = b["y"] >= 0
    lp = torch.log_softmax(logits, 1).gather(1, b["y"].clamp(min=0)[:, None])[:, 0]
    old, ref, adv = lp.detach() - 0.05, lp.detach() + 0.2, b["adv"].double()
    r = (lp - old).exp()
    loss = -torch.minimum(r * adv, r.clamp(0.8, 1.2) * adv) + 0.1 * ((ref - lp).exp() - (ref - lp) - 1)
    (loss * on).sum().backward()
    g = {k: v.grad for k, v in p.items()}
    g["alpha"], g["beta"] = al.grad, be.grad
    return loss.detach() * on, lp.detach() * on, logits.detach(), g


def test_a_training_step():
    """Every tensor between two operators is rounded to bf16, 2^-8 of its values at most: 12 roundings on the way to
    the logits and 14 on the way back, each of which moves a gradient by at most 2^-8 of its norm (the norms and the loss take
    out scales, the residuals add), some of them twice (a product's two factors): 40 2^-8 in the 2-norm."""
    p, b, cu_h = model()
    loss, lp, logits, g = step(p, b, cu_h)
    wloss, wlp, wlogits, wg = reference(p, b, cu_h)
    near = lambda a, w: float((a.double() - w).norm() / w.norm())  # noqa: E731
    assert near(logits, wlogits) <= 12 * 2 ** -8
    size = float(wlogits.norm(dim=1).max()) / V ** 0.5
    assert (lp - wlp).abs().max() <= 12 * 2 ** -8 * 8 * max(1.0, size)
    for k, w in wg.items():
        assert near(g[k], w) <= 40 * 2 ** -8, (k, near(g[k], w))
    again = step(p, b, cu_h)
    assert torch.equal(loss, again[0]) and all(torch.equal(g[k], again[3][k]) for k in g)
    assert (loss[5:9] == 0).all() and (lp[5:9] == 0).all()


def test_token_by_token():
    """Prefill of all tokens but three, then three steps on the caches: the log-probabilities of the whole forward,
    within the roundings of test_a_training_step (the products of single tokens are summed in another order)."""
    p, b, _ = model()
    n, more = 40, 3
    one = {k: v[:n] if v.shape[:1] == b["x"].shape[:1] else v for k, v in b.items()}
    one["cu"], one["y"] = torch.tensor([0, n], dtype=torch.int32).cuda(), torch.randint(0, V, (n,), device="cuda")
    _, lp, logits, _ = step(p, one, [0, n])
    m = n - more
    rot = lambda s: dict(q_weight=p["qw"], k_weight=p["kw"], positions=b["pos"][s], inv_freq=b["freq"], l2=True)  # noqa: E731
    cut = lambda c: (c[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)) for i in range(3))  # noqa: E731

    def rest(x, o, y):
        x1 = x + o.flatten(1) @ p["o"].t()
        h, _ = gdn.gdn_glu_forward(gdn.gdn_layer_norm_forward(x1, p["norm"])[0], p["wg"], p["wu"])
        z = (x1 + h @ p["down"].t()) @ p["head"].t()
        return z, gdn.gdn_policy_loss_forward(z, y)[1]

    c, tail = gdn.gdn_conv_forward(b["x"][:m] @ p["qkv"].t(), p["conv"])
    q, k, v = cut(c)
    q, k = gdn.gdn_qk_norm_forward(q, k, **rot(slice(0, m)))
    cache = gdn.new_cache(1, H, D, D, C, BF)
    o, _ = gdn.gdn_cpr_forward(q, k, v.contiguous(), b["alpha"][:m], b["beta"][:m], torch.tensor([0, m], dtype=torch.int32).cuda(), C,
                               cu_seqlens_host=[0, m], cache_out=cache)
    got = [rest(b["x"][:m], o, one["y"][:m])]
    for t in range(m, n):
        s = slice(t, t + 1)
        c = gdn.gdn_conv_step(b["x"][s] @ p["qkv"].t(), p["conv"], tail)
        q, k, v = cut(c)
        q, k = gdn.gdn_qk_norm_forward(q, k, **rot(s))
        o = gdn.gdn_decode_step(q, k, v.contiguous(), b["alpha"][s], b["beta"][s], cache, C)
        got.append(rest(b["x"][s], o, one["y"][s]))
    z, l = (torch.cat([g[i] for g in got]) for i in range(2))
    assert float((z.double() - logits.double()).norm() / logits.double().norm()) <= 12 * 2 ** -8
    # the log-probabilities of the same logits have the same bits in one row and in many
    for t in range(m, n):
        assert torch.equal(gdn.gdn_policy_loss_forward(logits[t:t + 1], one["y"][t:t + 1])[1][0], lp[t])
    assert (l - lp).abs().max() <= 12 * 2 ** -8 * 8 * max(1.0, float(logits.double().norm(dim=1).max()) / V ** 0.5)


def calls():
    """Each operator's passes on inputs of its own: functions without arguments that return their outputs."""
    g = torch.Generator(device="cuda").manual_seed(7)
    r = lambda *s, t=BF: torch.randn(*s, generator=g, device="cuda").to(t)  # noqa: E731
    q, k, dq, dk, w = r(300, 4, 64), r(300, 2, 64), r(300, 4, 64), r(300, 2, 64), r(64)
    rot = dict(q_weight=w, k_weight=w, positions=torch.arange(300, dtype=torch.int32, device="cuda"), inv_freq=torch.rand(32, device="cuda", generator=g))
    x, wg, wu, dh = r(700, 200), r(300, 200), r(300, 200), r(700, 300)
    z, y, old, adv = r(60, 40001), torch.randint(0, 40001, (60,), device="cuda", generator=g), r(60, t=F32) - 10, r(60, t=F32)

    def glu(n):
        h, saved = gdn.gdn_glu_forward(x[:n], wg, wu, save=True)
        return (h,) + tuple(gdn.gdn_glu_backward(x[:n], wg, wu, dh[:n], saved))

    return [lambda: gdn.gdn_qk_norm_forward(q, k, **rot) + tuple(gdn.gdn_qk_norm_backward(q, k, dq, dk, **rot)),
            lambda: glu(700), lambda: glu(20),
            lambda: gdn.gdn_policy_loss_backward(z, y, adv, old_logprob=old, advantages=adv)]


def test_two_streams_at_once():
    fs = calls()
    want = [f() for f in fs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(3)], []
    for i in range(12):
        with torch.cuda.stream(streams[i % 3]):
            got.append((i % 4, fs[i % 4]()))
    torch.cuda.synchronize()
    for i, outs in got:
        assert all(torch.equal(a, b) for a, b in zip(outs, want[i])), i


def test_two_captured_graphs_replayed_in_turn():
    fs = calls()
    want = [f() for f in fs]
    graphs, outs = [], []
    for f in fs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(f())
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_policy_beyond_2_31_elements():
    T, V_ = 17000, 131072
    z = torch.zeros(T, V_, dtype=BF, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = [0, 16383, 16384, T - 1]
    some = (torch.randn(len(rows), V_, generator=g, device="cuda") * 2).to(BF)
    z[rows] = some
    y = torch.full((T,), -100, dtype=torch.int64, device="cuda")
    y[rows] = torch.tensor([3, 5, 131071, 70000], device="cuda")
    old, adv, w = (torch.randn(T, generator=g, device="cuda") for _ in range(3))
    dz, loss, lp = gdn.gdn_policy_loss_backward(z, y, w, old_logprob=old - 12, advantages=adv)
    want = gdn.gdn_policy_loss_backward(some, y[rows], w[rows], old_logprob=old[rows] - 12, advantages=adv[rows])
    assert torch.equal(dz[rows], want[0]) and torch.equal(loss[rows], want[1]) and torch.equal(lp[rows], want[2])
    assert not dz[1:16383:97].any() and not dz[16385:T - 1:97].any()


def test_qk_norm_beyond_2_31_elements():
    T, H_, d = 70000, 128, 256
    q = torch.ones(T, H_, d, dtype=BF, device="cuda")
    k = torch.ones(T, 1, d, dtype=BF, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = [0, 65535, 65536, T - 1]
    some = torch.randn(len(rows), H_, d, generator=g, device="cuda").to(BF)
    q[rows] = some
    pos, freq = torch.arange(T, dtype=torch.int32, device="cuda"), torch.rand(64, generator=g, device="cuda")
    w = torch.rand(d, generator=g, device="cuda").to(BF)
    a = dict(q_weight=w, k_weight=w, inv_freq=freq)
    want = gdn.gdn_qk_norm_forward(some, k[rows], positions=pos[rows], **a)
    got = gdn.gdn_qk_norm_forward(q, k, positions=pos, **a)
    assert torch.equal(got[0][rows], want[0]) and torch.equal(got[1][rows], want[1])
    dq = got[0]
    want = gdn.gdn_qk_norm_backward(some, k[rows], dq[rows], got[1][rows], positions=pos[rows], **a)
    got = gdn.gdn_qk_norm_backward(q, k, dq, got[1], positions=pos, **a)
    assert torch.equal(got[0][rows], want[0]) and torch.equal(got[1][rows], want[1])


def test_glu_beyond_2_31_elements():
    T, D_, F_ = 270000, 64, 8192
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, D_, generator=g, device="cuda").to(BF)
    wg, wu = (torch.randn(F_, D_, generator=g, device="cuda").to(BF) / 8 for _ in range(2))
    h, saved = gdn.gdn_glu_forward(x, wg, wu, save=True)
    rows = slice(T - 300, T)
    want, _ = gdn.gdn_glu_forward(x[rows], wg, wu)
    assert torch.equal(h[rows], want) and torch.equal(h[262100:262200], gdn.gdn_glu_forward(x[262000:262300], wg, wu)[0][100:200])
    dh = torch.zeros_like(h)
    dh[rows] = h[rows]
    small = gdn.gdn_glu_forward(x[rows], wg, wu, save=True)[1]
    want = gdn.gdn_glu_backward(x[rows], wg, wu, dh[rows], small)
    got = gdn.gdn_glu_backward(x, wg, wu, dh, saved)
    # 300 rows share the sum over 16384 between blocks: either side is off by (16384 / 4 + 8) units of the magnitudes' sum,
    # and by half a step, 2^-8
    G, u, silu = x[rows].double() @ wg.double().t(), x[rows].double() @ wu.double().t(), torch.nn.functional.silu
    M = (1.13 * dh[rows].double() * u).abs() @ wg.double().abs() + (dh[rows].double() * silu(G)).abs() @ wu.double().abs()
    assert ((got[0][rows].double() - want[0].double()).abs() <= 2 ** -7 * want[0].double().abs() + 2 * 4104 * U * M).all()
    assert not got[0][:T - 300].any()
    # sums over 270000 rows, all but 300 of them zero: one more bf16 rounding, the sums' order differs
    for a, b in zip(got[1:], want[1:]):
        assert ((a.double() - b.double()).abs() <= 2 ** -7 * b.double().abs() + 1e-3 * float(b.abs().max())).all()


def test_qk_norm_gradients_against_differences():
    """fp32, along a random direction v with step e = 2^-5: the difference is off by e^2 / 6 of the third derivative (of the
    order of the function itself, as the rows are of size 1: at most 16 |L|) and by the outputs' rounding,
    24 units on each of the terms, over e."""
    g = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q, k, dq, dk, w = r(5, 2, 16) + 1, r(5, 1, 16) - 1, r(5, 2, 16), r(5, 1, 16), r(16)
    a = dict(positions=torch.arange(5, dtype=torch.int32, device="cuda") * 3, inv_freq=torch.rand(8, generator=g, device="cuda"))
    out = lambda q, k, w: [v.double() for v in gdn.gdn_qk_norm_forward(q, k, q_weight=w, k_weight=w, **a)]  # noqa: E731
    loss = lambda q, k, w: sum(float((o * d.double()).sum()) for o, d in zip(out(q, k, w), (dq, dk)))  # noqa: E731
    size = sum(float((o * d.double()).abs().sum()) for o, d in zip(out(q, k, w), (dq, dk)))
    gq, gk, gw, gw2 = gdn.gdn_qk_norm_backward(q, k, dq, dk, q_weight=w, k_weight=w, **a)
    e = 2.0 ** -5
    for i, (x, grad) in enumerate(((q, gq), (k, gk), (w, gw + gw2))):
        v = r(*x.shape)
        v /= v.norm()
        args = [q, k, w]
        args[i] = x + e * v
        up = loss(*args)
        args[i] = x - e * v
        diff = (up - loss(*args)) / (2 * e)
        assert abs(diff - float((grad * v).double().sum())) <= e * e / 6 * 16 * size + 24 * U * 2 * size / e


def test_glu_gradients_against_differences():
    """Along a direction of bf16 values, step 2^-4 of inputs of size 1: truncation e^2 / 6 of a third derivative of at
    most 4 of the sum of magnitudes; h's rounding of half a step, 2^-8 of each term at most; the gradients' own roundings, 2^-7."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x, wg, wu, dh = (torch.randn(*s, generator=g, device="cuda").to(BF) for s in ((8, 32), (48, 32), (48, 32), (8, 48)))
    wg, wu = wg / 8, wu / 8
    run = lambda x: float((gdn.gdn_glu_forward(x, wg, wu)[0].double() * dh.double()).sum())  # noqa: E731
    h, saved = gdn.gdn_glu_forward(x, wg, wu, save=True)
    dx = gdn.gdn_glu_backward(x, wg, wu, dh, saved)[0].double()
    v = dx.sign() * 0.5  # the steepest of the directions with entries of 1 / 2
    e = 0.125
    up, down = (x.double() + e * v).to(BF), (x.double() - e * v).to(BF)  # rounded: the step that is taken is up - down
    size = float((h.double() * dh.double()).abs().sum())
    want = float((dx * (up.double() - down.double())).sum())
    assert abs(run(up) - run(down) - want) <= 2 * 2 ** -8 * size * 1.5 + 2 ** -7 * abs(want) + e ** 3 / 3 * 4 * size


def test_a_graph_of_copies_branches_and_calls():
    """Calls behind copies, fills, other kernels and a join of two streams in one captured graph."""
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *n, t=torch.bfloat16: torch.randn(*n, generator=g, device="cuda").to(t)  # noqa: E731
    T, H, d, D, F, V = 300, 4, 64, 256, 512, 40000
    fresh = dict(q=r(T, H, d), k=r(T, H, d), x=r(T, D), xs=r(5, D), z=r(6, V), w=r(d), dh=r(T, F))
    wg, wu, w = r(F, D), r(F, D), r(d)
    y = torch.arange(6, device="cuda") * 7
    adv = r(6, t=torch.float32)
    kept = {n: torch.zeros_like(v) for n, v in fresh.items()}

    def calls(v, side=None):
        main = torch.cuda.current_stream()
        q, k = gdn.gdn_qk_norm_forward(v["q"], v["k"], q_weight=v["w"])
        grads = gdn.gdn_qk_norm_backward(v["q"], v["k"], q, k, q_weight=v["w"])
        h, saved = gdn.gdn_glu_forward(v["x"], wg, wu, save=True)
        few, _ = gdn.gdn_glu_forward(v["xs"], wg, wu)
        if side is not None:
            side.wait_stream(main)
            with torch.cuda.stream(side):
                _, lp = gdn.gdn_policy_loss_forward(v["z"], y)
            main.wait_stream(side)
        else:
            _, lp = gdn.gdn_policy_loss_forward(v["z"], y)
        dx, dwg, dwu = gdn.gdn_glu_backward(v["x"], wg, wu, v["dh"], saved)
        dz, loss, _ = gdn.gdn_policy_loss_backward(v["z"], y, adv, old_logprob=lp, advantages=adv)
        return [q, k, *grads[:3], h, few, lp, dx, dwg, dwu, dz, loss]

    want = calls(fresh)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for n, v in kept.items():
            v.copy_(fresh[n])
        got = calls(kept, side)
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), i
