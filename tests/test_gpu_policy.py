"""The clipped policy loss against its 64-bit definition.

Tolerances.  With range = (max z - min z) / tau of a row's finite logits: an exponent (z - max) / tau is off by
2 units of 2^-24 of its size (log2(e) / tau rounded once, one multiply-add), 2^x by 2.5 units; a sum
of positive terms passes a rescaling (4 units) and 17 additions per tile of 4096 or more elements in a thread, and
10 joins (4 units each) in the block: 21 (V / 4096 + 1) + 40; log2 of it, at most 20, 2 units.  So lp is off by at most
    e_lp = 2^-24 (80 + 21 (V / 4096 + 1) + 4 range + 2 |lp|),
and what follows by the chain rule: ratio by ratio (e_lp + 8 units), e^(ref - lp) alike, a probability by
p (e_lp + 4 units).
"""
import numpy as np
import pytest
import torch

from gated_deltanet_cpr_delta_b200 import gdn
from oracle import block_ops as ops
from test_gpu_layer_ops import HALF, TYPES, U

pytestmark = pytest.mark.gpu
F32 = torch.float32


def case(t, R, V, tau=1.0, kl=0.1, seed=0, scale=2.5):
    rng = np.random.default_rng([seed, R, V])
    z = torch.from_numpy((rng.standard_normal((R, V)) * scale).astype(np.float32)).to(t)
    y = rng.integers(0, V, R)
    z[np.arange(R), y] += float(np.log(V))
    z64 = z.double().numpy()
    lp = ops.policy(z64, y, tau=tau)[1]
    gap = rng.standard_normal(R) * 0.2
    for b in (np.log(0.8), np.log(1.3)):  # off the borders, where the gradient jumps
        gap = np.where(np.abs(gap - b) < 1e-3, b + 2e-3, gap)
    f = lambda v: torch.from_numpy(v.astype(np.float32)).cuda()  # noqa: E731
    c = dict(z=z.cuda(), y=torch.from_numpy(y).cuda(), old=f(lp - gap), adv=f(rng.standard_normal(R)),
             ref=f(lp + rng.standard_normal(R) * 0.4) if kl else None, w=f(rng.standard_normal(R)))
    return c, z64, dict(clip_low=0.2, clip_high=0.3, kl_coef=kl, temperature=tau)


def n64(v):
    return None if v is None else v.double().cpu().numpy()


def near(name, got, want, tol):
    got = n64(got)
    bad = ~((np.abs(got - want) <= tol) | ((got == want)) | (np.isnan(got) & np.isnan(want)))
    assert not bad.any(), (name, int(bad.sum()), np.argwhere(bad)[:3], np.abs(got - want)[bad][:3], tol[bad][:3])


def check(c, z64, kw, z=None):
    z = c["z"] if z is None else z
    args = dict(old_logprob=c["old"], advantages=c["adv"], ref_logprob=c["ref"], **kw)
    loss, lp = gdn.gdn_policy_loss_forward(z, c["y"], **args)
    dz, loss2, lp2 = gdn.gdn_policy_loss_backward(z, c["y"], c["w"], **args)
    none, lp3 = gdn.gdn_policy_loss_forward(z, c["y"], temperature=kw["temperature"])
    assert none is None and torch.equal(lp, lp2) and torch.equal(lp, lp3) and torch.equal(loss, loss2)
    y, tau, kl = c["y"].cpu().numpy(), kw["temperature"], kw["kl_coef"]
    o = dict(old=n64(c["old"]), adv=n64(c["adv"]), ref=n64(c["ref"]), lo=kw["clip_low"], hi=kw["clip_high"], kl=kl, tau=tau)
    o["lo"], o["hi"] = float(np.float32(o["lo"])), float(np.float32(o["hi"]))
    tau = o["tau"] = float(np.float32(tau))
    kl = o["kl"] = float(np.float32(kl))
    wl, wp, wd, p = ops.policy(z64, y, **o)
    fin = np.where(np.isfinite(z64), z64, np.nan)
    e = U * (101 + 21 * (z64.shape[1] // 4096) + 4 * (np.nanmax(fin, 1) - np.nanmin(fin, 1)) / tau + 2 * np.abs(wp))
    near("lp", lp, wp, e)
    ratio, gap = np.exp(wp - o["old"]), (o["ref"] - wp) if o["ref"] is not None else np.zeros(len(y))
    e1 = np.abs(o["adv"]) * ratio * (e + 8 * U) + kl * np.exp(gap) * (e + 8 * U)
    near("loss", loss, wl, e1 + kl * (e + 4 * U * (np.abs(gap) + 1)) + 4 * U * np.abs(wl))
    want = ops.policy_backward(z64, y, n64(c["w"]), **o)
    hot = np.zeros_like(p)
    on = (y >= 0) & (y < z64.shape[1])
    hot[np.arange(len(y))[on], y[on]] = 1
    e1 = (e1 + 4 * U * np.abs(wd))[:, None] * (hot + p) + np.abs(wd)[:, None] * (p * (e + 8 * U)[:, None] + 4 * U * hot)
    near("dz", dz, want, e1 * np.abs(n64(c["w"]))[:, None] / tau + HALF[z.dtype] * np.abs(want) * 1.01 + 1e-37)
    return loss, lp, dz


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("R,V,tau,kl", [
    (1, 1, 1.0, 0.1), (5, 2, 1.0, 0.0), (3, 7, 0.5, 0.1), (2, 8, 1.0, 0.1), (70, 100, 1.0, 0.05), (9, 1000, 2.0, 0.1), (9, 4097, 1.0, 0.1), (9, 4099, 1.0, 0.1), (9, 8193, 1.0, 0.1), (9, 8199, 1.0, 0.0), (9, 2047, 1.0, 0.1),
    (3, 16384, 1.0, 0.0), (3, 16391, 0.7, 0.1), (5, 32768, 1.0, 0.1), (2, 50021, 1.0, 0.1), (2, 65537, 1.0, 0.1), (3, 131072, 0.7, 0.05)])
def test_sizes(dtype, R, V, tau, kl):
    check(*case(TYPES[dtype], R, V, tau, kl))


@pytest.mark.parametrize("dtype,V", [("bf16", 524288), ("f32", 262144), ("f32", 262143), ("bf16", 700001), ("f32", 24577)])
def test_the_largest_rows(dtype, V):
    check(*case(TYPES[dtype], 3, V))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("V", [77, 1024, 20001])
def test_rows_that_take_no_part_and_bad_targets(dtype, V):
    c, z64, kw = case(TYPES[dtype], 900, V)
    c["y"][::3], c["y"][4], c["y"][899] = -100, V - 1, -1
    c["z"][::3] = float("nan")  # not read
    z64 = n64(c["z"])
    with np.errstate(invalid="ignore"):
        z64[::3] = 0
    loss, lp, dz = check(c, z64, kw)
    for v in (loss, lp, dz):
        assert (v[::3] == 0).all()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_policy_loss_forward(c["z"], c["y"], status=status)
    assert status.item() == gdn.GDN_OK
    c["y"][5] = V
    _, lp2 = gdn.gdn_policy_loss_forward(c["z"], c["y"], status=status)
    assert status.item() == gdn.GDN_ERR_DEVICE_INPUT and lp2[5] == 0
    keep = torch.arange(900, device="cuda") != 5
    a, b = gdn.gdn_policy_loss_forward(c["z"], c["y"], temperature=kw["temperature"])[1], lp
    assert torch.equal(a[keep], b[keep])
    c["y"].fill_(-100)
    loss, lp, dz = check(c, np.zeros_like(z64), kw)
    assert not loss.any() and not lp.any() and not dz.any()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("V,shift", [(1000, 0), (1000, 1), (1003, 0), (40000, 3), (40001, 0)])
def test_the_same_bits_in_every_place(dtype, V, shift):
    """A row's results do not depend on its place, its stride, its alignment or the rows beside it."""
    t = TYPES[dtype]
    c, z64, kw = case(t, 12, V)
    loss, lp, dz = check(c, z64, kw)
    wide = torch.full((12, V + shift + 5), float("nan"), dtype=t, device="cuda")
    view = wide[:, shift:shift + V]
    view.copy_(c["z"])
    for a, b in zip(check(c, z64, kw, view), (loss, lp, dz)):
        assert torch.equal(a, b)
    for i in (0, 7, 11):
        one = {k: None if v is None else v[i:i + 1].clone() for k, v in c.items()}
        for a, b in zip(check(one, z64[i:i + 1], kw), (loss, lp, dz)):
            assert torch.equal(a[0], b[i])


@pytest.mark.parametrize("dtype,V,shift", [("bf16", 65536, 0), ("bf16", 65537, 0), ("bf16", 131072, 3), ("bf16", 150001, 1), ("bf16", 262144, 0),
                                           ("f32", 32768, 0), ("f32", 40003, 2), ("f32", 131071, 0), ("f32", 140000, 0)])
def test_few_rows_share_the_blocks(dtype, V, shift):
    """Rows cut over 8, 4, 2 and 1 blocks: the same bits, and the definition's values.  (The up to 8 joins of the
    parts, 4 units each, stand for less than half of what the tolerance counts per tile and does not come up: 8 tiles and more,
    each of 11 units in place of 21.)"""
    t, R = TYPES[dtype], 280
    c, z64, kw = case(t, 9, V)
    c["y"][3] = -1
    c["z"][4, V // 3:] = -float("inf")  # parts of nothing but masked logits
    c["y"][4], c["y"][5], c["y"][6] = 5, 0, V - 1
    z64 = n64(c["z"])
    o = ops.policy(z64, c["y"].cpu().numpy(), tau=kw["temperature"])[1]
    c["old"], c["ref"] = (torch.from_numpy(np.where(np.isfinite(o), o, 0) + d).float().cuda() for d in (0.05, -0.1))
    wide = torch.full((R, V + shift), float("nan"), dtype=t, device="cuda")
    view = wide[:, shift:shift + V]
    view[:9].copy_(c["z"])
    results = check(c, z64, kw, view[:9])
    big = {k: v[:1].repeat((R,) + (1,) * (v.dim() - 1)) if v.dim() == 1 else view for k, v in c.items()}
    for k in ("y", "old", "adv", "ref", "w"):
        big[k][:9] = c[k]
    view[9:].copy_(c["z"][:1].expand(R - 9, V))
    for n in (1, 2, 9, 33, 64, 70, 129, R):
        part = {k: v[:n] for k, v in big.items()}
        args = dict(advantages=part["adv"], old_logprob=part["old"], ref_logprob=part["ref"], **kw)
        loss, lp = gdn.gdn_policy_loss_forward(part["z"], part["y"], **args)
        dz, loss2, lp2 = gdn.gdn_policy_loss_backward(part["z"], part["y"], part["w"], **args)
        assert torch.equal(loss, loss2) and torch.equal(lp, lp2)
        k = min(n, 9)
        for got, want in zip((loss, lp, dz), results):
            assert torch.equal(got[:k], want[:k]), n
            assert n <= 9 or torch.equal(got[9:], want[:1].expand(got[9:].shape)), n
        if shift == 0:
            place = part["z"].clone()
            gdn.gdn_policy_loss_backward(place, part["y"], part["w"], dlogits=place, **args)
            assert torch.equal(place, dz), n


@pytest.mark.parametrize("dtype", list(TYPES))
def test_masked_logits_and_rows_that_are_not_finite(dtype):
    t, V, inf = TYPES[dtype], 5000, float("inf")
    c, z64, kw = case(t, 8, V, kl=0.1)
    low = torch.finfo(t).min
    keep = c["z"][torch.arange(8), c["y"]].clone()
    c["z"][0, ::2], c["z"][1, 1:] = -inf, -inf   # half the vocabulary; all but two tokens
    c["z"][2, ::2] = low                         # the type's lowest value
    c["z"][torch.arange(8), c["y"]] = keep
    c["y"][1] = 0
    c["z"][3] = -inf
    c["z"][4, 17] = inf
    c["z"][5, 17] = float("nan")
    args = dict(old_logprob=c["old"], advantages=c["adv"], ref_logprob=c["ref"], **kw)
    dz, loss, lp = gdn.gdn_policy_loss_backward(c["z"], c["y"], c["w"], **args)
    for r in (3, 4, 5):
        assert torch.isnan(lp[r]) and torch.isnan(loss[r])
    assert dz[0, 0 if c["y"][0] else 2] == 0
    rows = [0, 1, 6, 7]
    some = {k: v[rows] for k, v in c.items()}
    check(some, n64(some["z"]), kw)
    # a logit of the type's lowest value has probability 0 as well, and its row's results are those of -inf
    b = c["z"][2:3].clone()
    b[b == low] = -inf
    a = gdn.gdn_policy_loss_forward(c["z"][2:3], c["y"][2:3])[1]
    assert torch.equal(a, gdn.gdn_policy_loss_forward(b, c["y"][2:3])[1])
    # the target itself masked: lp = -inf, ratio 0, no KL
    c["z"][6, c["y"][6]] = -inf
    loss, lp = gdn.gdn_policy_loss_forward(c["z"][6:7], c["y"][6:7], old_logprob=c["old"][6:7], advantages=c["adv"][6:7].abs())
    assert lp[0] == -inf and loss[0] == 0


def test_advantages_of_zero_and_extreme_ratios():
    c, z64, kw = case(F32, 6, 300, kl=0.0)
    c["old"][:] = torch.tensor([-1e4, -1e4, -1e4, 1e4, 1e4, 1e4])
    c["adv"][:] = torch.tensor([0.0, 1.0, -1.0, 0.0, 1.0, -1.0])
    dz, loss, _ = gdn.gdn_policy_loss_backward(c["z"], c["y"], c["w"], old_logprob=c["old"], advantages=c["adv"], **kw)
    hi, lo = float(np.float32(1) + np.float32(0.3)), float(np.float32(1) - np.float32(0.2))
    assert loss.tolist() == [0.0, -hi, float("inf"), 0.0, 0.0, lo]
    assert not dz[0].any() and not dz[1].any() and not dz[3].any() and not dz[4].any() and not dz[5].any()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("V", [1000, 33333])
def test_the_gradient_in_the_logits_place(dtype, V):
    c, z64, kw = case(TYPES[dtype], 50, V)
    c["y"][7] = -100
    args = dict(old_logprob=c["old"], advantages=c["adv"], ref_logprob=c["ref"], **kw)
    want = gdn.gdn_policy_loss_backward(c["z"], c["y"], c["w"], **args)
    z = c["z"].clone()
    got = gdn.gdn_policy_loss_backward(z, c["y"], c["w"], dlogits=z, **args)
    assert got[0].data_ptr() == z.data_ptr()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("R,V", [(40, 9000), (5, 131072)])
def test_a_graph_replays_other_values(R, V):
    c, z64, kw = case(torch.bfloat16, R, V)
    args = dict(old_logprob=c["old"], advantages=c["adv"], ref_logprob=c["ref"], **kw)
    out = dict(dlogits=torch.empty_like(c["z"]), loss=torch.empty(R, device="cuda"), logprob=torch.empty(R, device="cuda"))
    gdn.gdn_policy_loss_backward(c["z"], c["y"], c["w"], **args, **out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_policy_loss_backward(c["z"], c["y"], c["w"], **args, **out)
    d, _, _ = case(torch.bfloat16, R, V, seed=9)
    d["y"][3] = -100
    for k in c:
        c[k].copy_(d[k])
    graph.replay()
    want = gdn.gdn_policy_loss_backward(d["z"], d["y"], d["w"], old_logprob=d["old"], advantages=d["adv"], ref_logprob=d["ref"], **kw)
    for a, b in zip((out["dlogits"], out["loss"], out["logprob"]), want):
        assert torch.equal(a, b)


def test_gradient_against_differences():
    """fp32 differences over a step of 0.25: the loss's third derivative adds 0.25^2 / 6 of its scale."""
    c, z64, kw = case(F32, 1, 50, kl=0.2, scale=1.0)
    args = dict(old_logprob=c["old"], advantages=c["adv"], ref_logprob=c["ref"], **kw)
    c["old"].copy_(gdn.gdn_policy_loss_forward(c["z"], c["y"])[1])  # ratio 1, far from the borders
    dz = gdn.gdn_policy_loss_backward(c["z"], c["y"], torch.ones(1, device="cuda"), **args)[0][0]
    scale = float(c["adv"].abs()) * 1.3 + 0.2 * 4
    h = 0.02
    for v in (int(c["y"]), (int(c["y"]) + 1) % 50, 7):
        z = [c["z"].clone(), c["z"].clone()]
        z[0][0, v] += h
        z[1][0, v] -= h
        up, down = (float(gdn.gdn_policy_loss_forward(a, c["y"], **args)[0]) for a in z)
        # rounding: two losses of size at most 4, each off by 400 units; truncation h^2 / 6 times a third derivative of at most 8 scales
        assert abs((up - down) / (2 * h) - float(dz[v])) <= 400 * U * 4 / h + h * h / 6 * 8 * scale
