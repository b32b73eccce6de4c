"""GPU checks of the q/k norm at the edges of what its header and binding allow."""
import numpy as np
import pytest
import torch

from oracle import qk_norm

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def gdn():
    from rl_train_numerics_b200 import _abi
    return _abi


def f64(t):
    return t.detach().double().cpu().numpy()


def draw(T, Hq, Hk, d, seed, dt=BF, gdt=F32):
    r = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=r)  # noqa: E731
    return (rand(T, Hq, d).to(dt).cuda(), rand(T, Hk, d).to(dt).cuda(),
            rand(T, Hq, d).to(gdt).cuda(), rand(T, Hk, d).to(gdt).cuda(),
            (1 + 0.3 * rand(d)).cuda(), (1 + 0.3 * rand(d)).cuda())


@pytest.mark.parametrize("have", [(), ("dq",), ("dk", "dwk"), ("dwq",)])
def test_gradient_buffers_that_are_not_given_are_made(gdn, have):
    q, k, doq, dok, wq, wk = draw(9, 4, 2, 64, 3)
    kw = dict(norm="rms", wq=wq, wk=wk)
    want = gdn.qk_norm_backward(q, k, doq, dok, **kw)
    buf = {s: torch.empty_like(want[s]) for s in have}
    got = gdn.qk_norm_backward(q, k, doq, dok, grads=buf, **kw)
    assert set(got) == set(want) and all(got[s] is buf[s] for s in have)
    assert all(torch.equal(got[s], want[s]) for s in want)


@pytest.mark.parametrize("norm", ["l2", "rms"])
@pytest.mark.parametrize("T,Hq,Hk,d,dt,gdt", [(20000, 1, 1, 128, BF, F32), (9001, 4, 1, 64, F32, BF),
                                              (5003, 2, 3, 256, BF, BF), (700, 33, 1, 128, F32, F32)])
def test_weights_of_many_tokens_without_a_rotation(gdn, T, Hq, Hk, d, dt, gdt, norm):
    """Sums of a weight's gradient whose blocks make several passes, with one weight and
    with both."""
    q, k, doq, dok, wq, wk = draw(T, Hq, Hk, d, 4, dt, gdt)
    kw = dict(norm=norm, wq=wq, wk=wk)
    grads = gdn.qk_norm_backward(q, k, doq, dok, **kw)
    again = gdn.qk_norm_backward(q, k, doq, dok, **kw)
    assert all(torch.equal(grads[s], again[s]) for s in grads)
    for s, x, dy, w in (("q", q, doq, wq), ("k", k, dok, wk)):
        args = (f64(x), f64(dy), f64(w))
        dx, dw = qk_norm.backward(*args, norm=norm)
        bx, bw = qk_norm.backward_bound(*args, norm=norm)
        if dt == BF:    # one rounding to bf16: half a step, 2^-8 of the value
            bx = bx + 2.0 ** -8 * (np.abs(dx) + bx)
        assert (np.abs(f64(grads["d" + s]) - dx) <= bx).all()
        assert (np.abs(f64(grads["dw" + s]) - dw) <= bw).all()
    one = gdn.qk_norm_backward(q, k, doq, dok, norm=norm, wk=wk)
    assert one["dwq"] is None and torch.equal(one["dwk"], grads["dwk"])
    assert torch.equal(one["dk"], grads["dk"])


@pytest.mark.parametrize("T,Hq,Hk,d", [(1, 4, 1, 128), (300, 5, 3, 64), (2000, 16, 4, 128),
                                       (500, 8, 2, 256)])
@pytest.mark.parametrize("out", [F32, BF])
def test_fp32_heads_without_a_rotation(gdn, T, Hq, Hk, d, out):
    q, k, _, _, wq, wk = draw(T, Hq, Hk, d, 5, F32)
    oq, ok = gdn.qk_norm_forward(q, k, norm="rms", wq=wq, wk=wk, out_dtype=out)
    for y, x, w in ((oq, q, wq), (ok, k, wk)):
        want = qk_norm.forward(f64(x), f64(w), norm="rms")
        bound = qk_norm.forward_bound(f64(x), f64(w), norm="rms")
        if out == BF:
            bound = bound + 2.0 ** -8 * (np.abs(want) + bound)
        assert y.dtype == out and (np.abs(f64(y) - want) <= bound).all()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_offsets_beyond_32_bits(gdn, d):
    """Tokens 2^20 elements apart: from token 2048 on an element's offset passes 2^31."""
    T, Hq, Hk = 2100, 2, 1
    wide = torch.empty((T, 1 << 20), dtype=BF, device="cuda")
    q, k, doq, dok, wq, wk = draw(T, Hq, Hk, d, 6, gdt=BF)
    views, at = [], 0
    for t in (q, k, doq, dok, q, k, q, k):
        views.append(wide[:, at:at + t.shape[1] * d].unflatten(1, (t.shape[1], d)))
        at += t.shape[1] * d
        views[-1].copy_(t)
    kw = dict(norm="rms", wq=wq, wk=wk, positions=torch.arange(T, dtype=torch.int32).cuda(),
              inv_freq=torch.rand(d // 4).cuda())
    oq, ok = gdn.qk_norm_forward(q, k, **kw)
    a, b = gdn.qk_norm_forward(views[0], views[1], oq=views[4], ok=views[5], **kw)
    assert torch.equal(a, oq) and torch.equal(b, ok)
    want = gdn.qk_norm_backward(q, k, doq, dok, **kw)
    got = gdn.qk_norm_backward(*views[:4], grads={"dq": views[6], "dk": views[7]}, **kw)
    assert all(torch.equal(got[s], want[s]) for s in want)
