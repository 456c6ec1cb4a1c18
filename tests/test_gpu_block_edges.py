"""The norm of queries and keys, the gated block and the policy loss where a call's form, sizes or values are at an edge."""
import itertools
import threading

import pytest
import torch

from gated_deltanet_cpr_delta_b200 import gdn

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
