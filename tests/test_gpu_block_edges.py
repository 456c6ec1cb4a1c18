"""The norm of queries and keys, the gated block and the policy loss where a call's form, sizes or values are at an edge."""
import itertools
import threading

import numpy as np
import pytest
import torch

from gated_deltanet_cpr_delta_b200 import gdn
from oracle import block_ops as ops
from test_gpu_glu import case as glu_case, check as glu_check
from test_gpu_layer_ops import HALF, TYPES, U

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def rand(seed, *shape, t=BF, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(t)


@pytest.mark.parametrize("T", [7, 300])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_gated_block_gradients_partly_given(T, dtype):
    """Buffers that the caller leaves out are made in the type of those that are given; the values are the same."""
    D, F = 200, 72
    x, wg, wu, dh = rand(1, T, D), rand(2, F, D, scale=0.1), rand(3, F, D, scale=0.1), rand(4, T, F)
    _, saved = gdn.gdn_glu_forward(x, wg, wu, save=True)
    full = lambda: (torch.empty(T, D, dtype=BF, device="cuda"),) + tuple(torch.empty(F, D, dtype=dtype, device="cuda") for _ in range(2))  # noqa: E731
    want = gdn.gdn_glu_backward(x, wg, wu, dh, saved, grads=full())
    for given in itertools.product([0, 1], repeat=3):
        if not given[1] and not given[2] and dtype is F32:
            continue
        got = gdn.gdn_glu_backward(x, wg, wu, dh, saved, grads=tuple(b if on else None for b, on in zip(full(), given)))
        for a, b in zip(got, want):
            assert a.dtype is b.dtype and torch.equal(a, b), given


def entry(monkeypatch, f):
    """f(), and the library's last entry that it called with its arguments, as a function of the stream."""
    ready, call = [], gdn._call

    def record(dev, what, fn, *args):
        ready.append((fn, args))
        call(dev, what, fn, *args)

    with monkeypatch.context() as m:
        m.setattr(gdn, "_call", record)
        keep = f()
    fn, args = ready[-1]
    return keep, lambda stream: fn(*args, stream.cuda_stream)


def test_a_thread_whose_first_call_this_is(monkeypatch):
    """Each entry, as the first that a thread calls of CUDA."""
    x, w, dh, q = rand(1, 300, 64), rand(2, 200, 64), rand(3, 300, 200), rand(4, 20, 2, 64)
    z, y, adv = rand(5, 9, 1000), torch.arange(9, device="cuda"), rand(6, 9, t=F32)
    _, saved = gdn.gdn_glu_forward(x, w, w, save=True)
    calls = [lambda: gdn.gdn_glu_forward(x, w, w), lambda: gdn.gdn_glu_forward(x[:5], w, w),
             lambda: gdn.gdn_glu_backward(x, w, w, dh, saved), lambda: gdn.gdn_qk_norm_forward(q, q),
             lambda: gdn.gdn_qk_norm_backward(q, q, q, q), lambda: gdn.gdn_policy_loss_forward(z, y),
             lambda: gdn.gdn_policy_loss_backward(z, y, adv, old_logprob=adv, advantages=adv)]
    stream = torch.cuda.Stream()
    for f in calls:
        workspaces, scratch = [], gdn._scratch
        with monkeypatch.context() as m:  # kept for the second call
            m.setattr(gdn, "_scratch", lambda *a: workspaces.append(scratch(*a)) or workspaces[-1])
            outs, again = entry(monkeypatch, f)
        outs = [t for t in outs if t is not None]
        want = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        got = []
        t = threading.Thread(target=lambda: got.append(again(stream)))
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert got == [gdn.GDN_OK]
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_threads_with_calls_of_different_sizes(monkeypatch):
    """Threads call the same kernels with different amounts of shared memory, each on its own stream: every call launches, and
    the results are those of one thread.  The library's entries are called with arguments that are ready, so that the calls
    meet."""
    def norm(seed, d, rot):
        x, dy = rand(seed, 12, 4, d, t=F32), rand(seed + 1, 12, 4, d, t=F32)
        kw = dict(positions=torch.arange(12, dtype=torch.int32, device="cuda"), inv_freq=torch.ones(rot // 2, device="cuda")) if rot else {}
        out = torch.empty_like(x), torch.empty_like(x), None, None
        return out[:2], lambda: gdn.gdn_qk_norm_backward(x, x, dy, dy, grads=out, **kw)

    def block(seed, D, F):
        x, w, h = rand(seed, 4, D), rand(seed + 1, F, D, scale=D ** -0.5), torch.empty(4, F, dtype=BF, device="cuda")
        return (h,), lambda: gdn.gdn_glu_forward(x, w, w, h=h)

    def layer_norm(seed, D):
        x, w, y = rand(seed, 8, D, t=F32), rand(seed + 1, D, t=F32), torch.empty(8, D, device="cuda")
        return (y,), lambda: gdn.gdn_layer_norm_forward(x, w, y=y)

    pairs = [(norm(1, 128, 0), norm(7, 128, 128)), (block(3, 1024, 640), block(9, 256, 4096)), (layer_norm(5, 6000), layer_norm(11, 8192))]
    streams = [torch.cuda.Stream() for _ in range(4)]
    for pair in pairs:
        want, entries = [], []
        for out, f in pair:
            entries.append(entry(monkeypatch, f))
            want.append([t.clone() for t in out])
            for t in out:
                t.zero_()
        torch.cuda.synchronize()
        bad, start = [], threading.Barrier(4)

        def work(i):
            again = entries[i % 2][1]
            torch.zeros(1, device="cuda")
            start.wait()
            for _ in range(4000):
                st = again(streams[i])
                if st != gdn.GDN_OK:
                    bad.append((i, st))

        threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        assert not bad, (len(bad), bad[:4])
        for (out, _), w in zip(pair, want):
            assert all(torch.equal(a, b) for a, b in zip(out, w))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("V", [40, 3001, 60000, 140001])
@pytest.mark.parametrize("tau", [1.0, 0.5, 4.0])
def test_finite_logits_at_the_ends_of_the_range(dtype, V, tau):
    """Rows that a mask of the type's lowest value fills, wholly or in part, and values beyond fp32's range times log2(e) / tau: a
    finite logit counts as what it is.  Tolerances: as in the policy loss's tests, e_lp = 2^-24 (101 + 21 (V / 4096) + 4 range +
    2 |lp|) with the range of the logits whose probability is not 0 (at most 20 / tau here); log-probabilities beyond fp32's range are
    infinite.  Below 2^30 a row's maximum times log2(e) / tau is rounded by up to 32, which adds four roundings of 32."""
    t, inf = TYPES[dtype], float("inf")
    low, top = torch.finfo(t).min, torch.finfo(t).max
    near = float(torch.tensor(low, dtype=t).view({BF: torch.int16, F32: torch.int32}[t]).sub(1).view(t))  # the next value
    R = 15
    z = rand(V, R, V, t=t, scale=2.0).clamp_(-10, 10)
    y = torch.tensor([3, 5, 7, 9, 11, 13, 15, 17, 19, 20, 21, 22, 23, 24, 25], device="cuda") + (V - 30) // 2
    y[14] = V - 1
    z[0] = low                                  # all masked
    z[1], z[1, 1::2] = -inf, low                # all masked, one half by each kind
    z[1, y[1]] = low
    z[2, y[2]] = low                            # the target alone masked
    z[3, 2], z[3, y[3]] = top, 1.0              # one beyond all
    z[4, y[4]] = top                            # which is the target
    z[5], z[5, : V // 2] = low, near            # two values beyond the range
    z[6] = top
    z[7], z[7, y[7]] = low, 2.0                 # all but the target masked
    z[8], z[8, y[8]:] = low, -1e38              # masked, and beyond the range for small temperatures only
    z[9, V // 3:] = low
    z[10], z[11], z[12] = -1e9, -1e10, 1e30     # other values that masks take, and rows far off as a whole
    z[13] -= 3e4
    z[14, : V // 2] = -1e10
    n64 = lambda v: v.double().cpu().numpy()  # noqa: E731
    z64, y_, tau64 = n64(z), y.cpu().numpy(), float(np.float32(tau))
    with np.errstate(over="ignore"):
        lp = ops.policy(z64, y_, tau=tau64)[1]
        assert np.isfinite(lp).all()
    old = torch.from_numpy(np.clip(lp, -1e30, None).astype(np.float32)).cuda() - 0.05
    adv, w = rand(V + 1, R, t=F32), rand(V + 2, R, t=F32)
    dz, loss, got = gdn.gdn_policy_loss_backward(z, y, w, old_logprob=old, advantages=adv, temperature=tau)
    loss2, got2 = gdn.gdn_policy_loss_forward(z, y, old_logprob=old, advantages=adv, temperature=tau)
    place = z.clone()
    third = gdn.gdn_policy_loss_backward(place, y, w, old_logprob=old, advantages=adv, temperature=tau, dlogits=place)
    assert torch.equal(got, got2) and torch.equal(loss, loss2) and all(torch.equal(a, b) for a, b in zip(third, (dz, loss, got)))
    o = dict(old=n64(old), adv=n64(adv), lo=float(np.float32(0.2)), hi=float(np.float32(0.2)), tau=tau64)
    wl, _, wd, p = ops.policy(z64, y_, **o)
    wz = ops.policy_backward(z64, y_, n64(w), **o)
    e = U * (101 + 21 * (V // 4096) + 4 * 32 + 4 * 20 / tau + 2 * np.abs(lp))
    got, loss, dz = n64(got), n64(loss), n64(dz)
    far = lp < -torch.finfo(F32).max * (1 + 2.0 ** -25)  # rounds to -inf
    assert (got[far] == -inf).all() and (np.abs(got - lp) <= e)[~far].all(), (got, lp)
    e = np.where(lp < -1e30, 0, e)  # their ratio is 0, and stays it
    ratio = np.exp(lp - o["old"])
    e1 = np.abs(o["adv"]) * ratio * (e + 8 * U) + 4 * U * np.abs(wl)
    assert (np.abs(loss - wl) <= e1).all(), (loss, wl)
    hot = np.zeros_like(p)
    hot[np.arange(R), y_] = 1
    tol = e1[:, None] * (hot + p) + np.abs(wd)[:, None] * (p * (e + 8 * U)[:, None] + 4 * U * hot)
    bad = ~(np.abs(dz - wz) <= tol * np.abs(n64(w))[:, None] / tau64 + HALF[t] * np.abs(wz) * 1.01 + 1e-37)
    assert not bad.any(), (np.argwhere(bad)[:4], dz[bad][:4], wz[bad][:4])


@pytest.mark.parametrize("scale", [1e-4, 1e-3, 1e-2, 0.3, 0.6, 3.0])
def test_the_kl_term_of_policies_that_are_close(scale):
    """e^g - g - 1 for given gaps g: its own rounding is 3 units of 2^-24 of its value up to 1/2, beyond it e^g - 1 is off by 2 units, up
    to 4.4 times the difference's size; with the product and the sum's rounding at most 16 units of the value, however small the gap is.
    The slope 1 - e^g: 2 units, products 4; a probability by e_lp + 8 units."""
    R, V, kl = 64, 50, 0.3
    z, y = rand(1, R, V, t=F32), torch.arange(R, device="cuda") % V
    _, lp = gdn.gdn_policy_loss_forward(z, y)
    ref = lp + rand(2, R, t=F32).clamp_(-3, 3) * scale
    w, zero = rand(3, R, t=F32), torch.zeros(R, device="cuda")
    dz, loss, _ = gdn.gdn_policy_loss_backward(z, y, w, old_logprob=lp, advantages=zero, ref_logprob=ref, kl_coef=kl)
    n64 = lambda v: v.double().cpu().numpy()  # noqa: E731
    g = n64(ref - lp)
    series = sum(g ** n / float(np.prod(np.arange(1.0, n + 1))) for n in range(2, 40))
    want = float(np.float32(kl)) * np.where(np.abs(g) < 2, series, np.expm1(g) - g)
    loss = n64(loss)
    assert (loss >= 0).all() and (np.abs(loss - want) <= 16 * U * want).all(), np.max(np.abs(loss - want) / want) / U
    z64, y_ = n64(z), y.cpu().numpy()
    wp, p = ops.policy(z64, y_)[1], ops.policy(z64, y_)[3]
    d = -float(np.float32(kl)) * np.expm1(g)
    hot = np.eye(V)[y_]
    wz = (n64(w) * d)[:, None] * (hot - p)
    e = U * (101 + 4 * np.ptp(z64, 1) + 2 * np.abs(wp))
    assert (np.abs(n64(dz) - wz) <= np.abs(n64(w) * d)[:, None] * (p * (e[:, None] + 8 * U) + 8 * U * hot) + U * np.abs(wz) + 1e-37).all()


def test_without_a_kl_weight_the_reference_takes_no_part():
    """However far the reference is."""
    R, V = 20, 300
    z, y = rand(1, R, V), torch.arange(R, device="cuda")
    _, lp = gdn.gdn_policy_loss_forward(z, y)
    adv, w = rand(2, R, t=F32), rand(3, R, t=F32)
    for ref in (lp + 200, lp - 200, torch.full_like(lp, float("inf"))):
        args = dict(old_logprob=lp - 0.1, advantages=adv)
        want = gdn.gdn_policy_loss_backward(z, y, w, **args)
        got = gdn.gdn_policy_loss_backward(z, y, w, ref_logprob=ref, kl_coef=0.0, **args)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T,Hq,Hk,d,rot,inter,shift", [
    (1, 1, 1, 16, 0, False, 0), (70, 4, 4, 128, 128, False, 0), (33, 7, 3, 90, 40, True, 0), (65, 1, 2, 64, 32, True, 4), (300, 3, 3, 8, 8, False, 0),
    (40, 4, 2, 64, 64, False, 1), (9, 2, 2, 256, 256, False, 2), (2000, 16, 4, 128, 64, False, 0), (17, 5, 1, 34, 22, False, 0)])
@pytest.mark.parametrize("weight", [False, True])
def test_the_norms_gradients_from_those_of_the_recurrence(T, Hq, Hk, d, rot, inter, shift, weight):
    """Gradients of the outputs in fp32 beside bf16 inputs: values that bf16 holds give the bits of a call in bf16, others the definition's
    values (tolerances as in the norm's tests: dx half a step and 64 units, dw 24 and one for each row, with its fp32 result's own)."""
    q, k, qw = rand(1, T, Hq, d), rand(2, T, Hk, d, scale=3.0), rand(3, d) if weight else None
    pos, freq = torch.arange(T, dtype=torch.int32, device="cuda") * 7, 1e2 ** (-torch.arange(rot // 2, device="cuda", dtype=F32) / max(1, rot // 2))
    args = dict(q_weight=qw, k_weight=qw, interleaved=inter, l2=True)
    if rot:
        args.update(positions=pos, inv_freq=freq)
    wide = torch.full((T, (Hq + Hk) * d + 2 * shift), float("nan"), device="cuda")  # both in one tensor's rows
    dq, dk = (wide[:, a:a + H * d].unflatten(1, (H, d)) for a, H in ((shift, Hq), (shift + Hq * d, Hk)))
    dq.copy_(rand(4, T, Hq, d)), dk.copy_(rand(5, T, Hk, d))
    got = gdn.gdn_qk_norm_backward(q, k, dq, dk, **args)
    want = gdn.gdn_qk_norm_backward(q, k, dq.to(BF), dk.to(BF), **args)
    assert got[0].dtype is BF and got[1].dtype is BF
    for a, b in zip(got, want):
        assert (a is None and b is None) or torch.equal(a, b)
    dq.copy_(rand(6, T, Hq, d, t=F32)), dk.copy_(rand(7, T, Hk, d, t=F32))
    got = gdn.gdn_qk_norm_backward(q, k, dq, dk, **args)
    n64 = lambda v: v.double().cpu().numpy()  # noqa: E731
    kw = dict(inter=inter, l2=True, pos=pos.cpu().numpy() if rot else None, freq=n64(freq) if rot else None)
    for i, (x, dy) in enumerate(((q, dq), (k, dk))):
        w = n64(qw) if weight else None
        dx, dw = ops.head_norm_backward(n64(x), n64(dy), w, **kw)
        Mx, Mw = ops.head_norm_backward(n64(x), n64(dy), w, bound=True, **kw)
        assert (np.abs(n64(got[i]) - dx) <= HALF[BF] * np.abs(dx) * 1.01 + 64 * U * Mx).all()
        assert not weight or (np.abs(n64(got[2 + i]) - dw) <= U * np.abs(dw) + (24 + x.shape[0] * x.shape[1]) * U * Mw).all()


def test_the_norms_gradients_of_mixed_types_are_refused():
    x, g = rand(1, 5, 2, 16), rand(2, 5, 2, 16, t=F32)
    for a, b in ((x, g), (g, x)):
        with pytest.raises(ValueError, match="dk_out"):
            gdn.gdn_qk_norm_backward(x, x, a, b)
    with pytest.raises(ValueError, match="dq_out"):
        gdn.gdn_qk_norm_backward(g, g, x, x)


def test_the_recurrences_gradients_go_to_the_norm_as_they_are():
    """Norm, recurrence and back: dq and dk of gdn_cpr_backward are the norm's gradients without a cast; dx as the definition has it
    for them (tolerance as above)."""
    T, H, D, C = 70, 2, 32, 16
    qk, v = rand(1, T, 2 * H, D), rand(2, T, H, D)
    q, k = qk[:, :H], qk[:, H:]
    pos, freq = torch.arange(T, dtype=torch.int32, device="cuda"), 1e2 ** (-torch.arange(D // 2, device="cuda", dtype=F32) / (D // 2))
    g = torch.Generator(device="cuda").manual_seed(3)
    alpha, beta = torch.rand(T, H, generator=g, device="cuda") * 0.4 + 0.6, torch.rand(T, H, generator=g, device="cuda")
    cu_h = [0, 30, 70]
    cu = torch.tensor(cu_h, dtype=torch.int32, device="cuda")
    args = dict(positions=pos, inv_freq=freq, l2=True)
    qn, kn = gdn.gdn_qk_norm_forward(q, k, **args)
    o, states = gdn.gdn_cpr_forward(qn, kn, v, alpha, beta, cu, C, cu_seqlens_host=cu_h)
    dqn, dkn, *_ = gdn.gdn_cpr_backward(qn, kn, v, alpha, beta, rand(4, T, H, D), states, cu, C, cu_seqlens_host=cu_h)
    assert dqn.dtype is F32
    got = gdn.gdn_qk_norm_backward(q, k, dqn, dkn, **args)
    n64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    kw = dict(l2=True, pos=n64(pos).astype(np.int64), freq=n64(freq))
    for x, dy, dx in ((q, dqn, got[0]), (k, dkn, got[1])):
        want, M = (ops.head_norm_backward(n64(x), n64(dy), bound=b, **kw)[0] for b in (False, True))
        assert dx.dtype is BF and (np.abs(n64(dx) - want) <= HALF[BF] * np.abs(want) * 1.01 + 64 * U * M).all()


@pytest.mark.parametrize("T", [1, 16, 33, 128, 129, 200, 256])
@pytest.mark.parametrize("D,F", [(72, 4097), (200, 9473), (64, 11008), (136, 20480), (8, 28672), (72, 40001)])
def test_wide_gated_blocks_of_few_tokens(T, D, F):
    """Inner widths for which an SM holds one, two and three blocks at a time, and more than run at once."""
    glu_check(glu_case(T, D, F), "gelu" if T & 1 else "silu", backward=F < 10000)


@pytest.mark.parametrize("T", [64, 640])
def test_what_the_gated_blocks_backward_reads_is_not_drawn_towards_zero(T):
    """The forward saves g cut off to 24 bits, by up to 2^-15, and the backward multiplies it with 1 + 2^-16 ln 2: off by at most 2^-15 -
    2^-16 ln 2 = 1.31 2^-16, and 2^-24 of either rounding.  dw_up = (act(g) dh)^T x with one token for each column of x: each element is
    one product, within two bf16 terms (2^-16) of act of that.  (Here g = w + 2^-8 w' in [1, 2) has few bits: w' in [2^-k, 2^-k+1) is
    a multiple of 2^-8-k, and the cut takes 2^-15 (1 - 2^-k) / 2, 2^-15 / 3 on average; so what is read is 2^-16 ln 2 / 3 of the
    value too large, and was twice that too small.)"""
    F = 20480 // 64 if T == 640 else 320
    D = 64
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.zeros(T, D, device="cuda")
    rows = torch.arange(T, device="cuda")
    x[rows, rows % (D // 2)], x[rows, D // 2 + rows % (D // 2)] = 1.0, 2.0 ** -8
    x = x.to(BF)
    wg = torch.rand(F, D, generator=g, device="cuda")
    wg[:, : D // 2] += 1.0
    wg = wg.to(BF)
    wu = torch.zeros(F, D, dtype=BF, device="cuda")
    dh = torch.zeros(T, F, dtype=BF, device="cuda")
    keep = rows < D // 2
    dh[keep] = 1.0
    _, saved = gdn.gdn_glu_forward(x, wg, wu, save=True)
    words = saved.view(torch.int16).view(3, T, F).to(torch.int32) & 0xffff
    G = (x.double() @ wg.double().t())[keep]
    cut = ((words[0] << 16) | ((words[2] & 0xff) << 8)).view(F32)[keep]
    read = (cut * (1 + 89 * 2.0 ** -23)).double()
    ln2 = float(np.log(2))
    assert ((read - G).abs() <= 1.35 * 2.0 ** -16 * G).all()
    assert abs(float(((read - G) / G).mean()) - 2.0 ** -16 * ln2 / 3) <= 2.0 ** -20
    assert abs(float(((cut.double() - G) / G).mean()) + 2.0 ** -16 * ln2 * 2 / 3) <= 2.0 ** -20
    f32 = torch.empty(F, D, device="cuda")
    grads = gdn.gdn_glu_backward(x, wg, wu, dh, saved, grads=(None, f32, torch.empty_like(f32)))
    got = grads[2][:, : D // 2].t().double()  # [token, unit]
    want = torch.nn.functional.silu(read)
    step = 2.0 ** -8 if T > 128 else 2.0 ** -16
    assert ((got - want).abs() <= (step + 16 * U) * want).all()
    # 10240 roundings of at most `step`, as often up as down: within 6 standard errors, and the arithmetic's own 16 units
    assert abs(float(((got - want) / want).mean())) <= 6 * step / 3 ** 0.5 / got.numel() ** 0.5 + 16 * U
    # what stands for 0 or for an infinity is read as it is
    _, zeros = gdn.gdn_glu_forward(torch.zeros_like(x), wg, torch.ones_like(wu), save=True)
    for out in gdn.gdn_glu_backward(torch.zeros_like(x), wg, torch.ones_like(wu), torch.full_like(dh, 1e4), zeros):
        assert not out.any()
    planes = saved.view(torch.int16).view(3, T, F)
    planes[1, 0, 0], planes[2, 0, 0] = 0x7f80, planes[2, 0, 0] & 0xff  # u = inf
    dx = gdn.gdn_glu_backward(x, wg, wu, dh, saved)[0]
    assert (dx[0] == float("inf")).all() and torch.isfinite(dx[1:]).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,Hq,Hk,d,shift", [(30000, 2, 2, 16, 0), (16384, 16, 4, 128, 0), (5000, 3, 1, 90, 0), (5000, 4, 2, 64, 1), (9, 145, 3, 256, 0), (1, 1, 1, 2, 0),
                                            (700, 32, 32, 64, 0)])
def test_the_norms_weight_gradients_count_every_row(dtype, T, Hq, Hk, d, shift):
    """Rows of unit length with one element that is not 0, and gradients of 1 to 3: every product and every partial sum is a whole
    number below 2^24, so the sums over tokens and heads are exact in any order, and a row that is missed or counted twice shows."""
    t = TYPES[dtype]

    def part(H, seed):
        row = torch.arange(T * H, device="cuda")
        at, value = (row * 7 + seed + row // d) % d, 1.0 + (row + seed) % 3
        wide = torch.full((T, H * d + 2 * shift), float("nan"), dtype=t, device="cuda")
        x = wide[:, shift:shift + H * d].unflatten(1, (H, d))
        x.copy_(torch.zeros(T * H, d, device="cuda").scatter_(1, at[:, None], 1.0).view(T, H, d))
        g = torch.full((T, H, d), 2.0, dtype=t, device="cuda")
        g.view(T * H, d).scatter_(1, at[:, None], value.to(t)[:, None])
        return x, g, torch.zeros(d, device="cuda", dtype=torch.float64).index_add_(0, at, value.double())

    (q, dq, wq), (k, dk, wk) = part(Hq, 1), part(Hk, 2)
    w = torch.ones(d, dtype=t, device="cuda")
    args = dict(q_weight=w, k_weight=w, l2=True, eps=0.0)
    for gq, gk in ((dq, dk), (dq.float(), dk.float())):
        got = gdn.gdn_qk_norm_backward(q, k, gq, gk, **args)
        assert torch.equal(got[2].double(), wq) and torch.equal(got[3].double(), wk)


@pytest.mark.parametrize("D,F", [(200, 300), (512, 1024), (264, 5000)])
def test_a_rows_bits_in_the_gated_block(D, F):
    """The same in every call of the same sizes, wherever the row is and whatever stands beside it; in batches of other sizes the
    sums' order may differ, within e = (D / 4 + 8) 2^-24 of the magnitudes' sum on either side and half a step of the result."""
    x, wg, wu = rand(1, 600, D), rand(2, F, D, scale=D ** -0.5), rand(3, F, D, scale=D ** -0.5)
    X, G, V = x.double(), x.double() @ wg.double().t(), x.double() @ wu.double().t()
    eg, eu = ((D / 4 + 8) * U * (X.abs() @ w.double().abs().t()) for w in (wg, wu))
    act = torch.nn.functional.silu(G)
    tol = 2 * (1.13 * V.abs() * eg + (act.abs() + 1.13 * eg) * eu + 16 * U * (act * V).abs()) + 2 * HALF[BF] * (act * V).abs() * 1.02
    full = gdn.gdn_glu_forward(x, wg, wu)[0]
    for T in (1, 16, 17, 128, 129, 256, 257, 600):
        h = gdn.gdn_glu_forward(x[:T], wg, wu)[0]
        assert ((h.double() - full[:T].double()).abs() <= tol[:T]).all()
        turned = x[:T].roll(T // 2, 0).contiguous()
        assert torch.equal(gdn.gdn_glu_forward(turned, wg, wu)[0], h.roll(T // 2, 0)), T


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("V", [1, 4, 13, 1003, 20001])
def test_the_logits_gradient_has_the_same_bits_at_every_address(dtype, V):
    """Targets at the rows' ends among them, which come element by element where a row starts or ends inside 16 bytes."""
    t, R = TYPES[dtype], 60
    z, w, adv = rand(1, R, V, t=t, scale=3.0), rand(2, R, t=F32), rand(3, R, t=F32)
    y = torch.tensor([0, 1, 2, V - 1, V - 2, V - 3, V // 2, 5, 7, V - 8] * (R // 10), device="cuda").clamp(0, V - 1)
    kw = dict(old_logprob=gdn.gdn_policy_loss_forward(z, y)[1] + 0.1, advantages=adv)
    want = gdn.gdn_policy_loss_backward(z, y, w, **kw)
    for at in range(9):
        place = torch.full((R * V + 24,), 7.0, dtype=t, device="cuda")
        view = place[at:at + R * V].view(R, V)
        view.copy_(z)
        apart = torch.full((R * V + 24,), 7.0, dtype=t, device="cuda")
        for got in (gdn.gdn_policy_loss_backward(view, y, w, dlogits=apart[3:3 + R * V].view(R, V), **kw),
                    gdn.gdn_policy_loss_backward(view, y, w, dlogits=view, **kw)):
            assert all(torch.equal(a, b) for a, b in zip(got, want)), at
        for b, o in ((place, at), (apart, 3)):
            assert (b[:o] == 7).all() and (b[o + R * V:] == 7).all()
