"""GPU checks of the q/k norm with rotation (gdn_qk_norm_forward, _backward)
against the fp64 oracle within its fp32 bounds (oracle/qk_norm.py)."""
import itertools

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
    return None if t is None else t.detach().double().cpu().numpy()


def draw(T, Hq, Hk, d, seed, dt=BF, gdt=F32, weights=True, rot=0, far=0, fused=False):
    r = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=r)  # noqa: E731
    y = (rand(T, (Hq + Hk) * d) * rand(T, 1).exp()).to(dt).cuda()
    q, k = y[:, :Hq * d].unflatten(1, (Hq, d)), y[:, Hq * d:].unflatten(1, (Hk, d))
    if not fused:
        q, k = q.contiguous(), k.contiguous()
    kw = {}
    if weights:
        kw.update(wq=(1 + 0.3 * rand(d)).cuda(), wk=(1 + 0.3 * rand(d)).cuda())
    if rot:
        kw["positions"] = (far + torch.randint(0, 4096, (T,), generator=r)).to(torch.int32).cuda()
        kw["inv_freq"] = (10000.0 ** (-torch.arange(rot // 2) / (rot // 2))).float().cuda()
    return q, k, rand(T, Hq, d).to(gdt).cuda(), rand(T, Hk, d).to(gdt).cuda(), kw


def sides(q, k, dq, dk, kw):
    rot = (f64(kw.get("positions")), f64(kw.get("inv_freq")))
    return [(f64(q), f64(dq), (f64(kw.get("wq")), *rot)), (f64(k), f64(dk), (f64(kw.get("wk")), *rot))]


def close(got, want, bound, dt=F32):
    if dt == BF:    # one rounding to bf16: half a step, 2^-8 of the value
        bound = bound + 2.0 ** -8 * (np.abs(want) + bound)
    err = np.abs(f64(got) - want)
    assert (err <= bound).all(), float((err / bound).max())


def check(gdn, q, k, doq, dok, kw, opts):
    oq, ok = gdn.qk_norm_forward(q, k, out_dtype=F32, **opts, **kw)
    bq, bk = gdn.qk_norm_forward(q, k, out_dtype=BF, **opts, **kw)
    assert torch.equal(bq, oq.to(BF)) and torch.equal(bk, ok.to(BF))
    grads = gdn.qk_norm_backward(q, k, doq, dok, **opts, **kw)
    for (x, dy, rest), y, s in zip(sides(q, k, doq, dok, kw), (oq, ok), "qk"):
        if x.shape[1] == 0:
            continue
        close(y, qk_norm.forward(x, *rest, **opts), qk_norm.forward_bound(x, *rest, **opts))
        dx, dw = qk_norm.backward(x, dy, *rest, **opts)
        bx, bw = qk_norm.backward_bound(x, dy, *rest, **opts)
        assert grads["d" + s].dtype == q.dtype
        close(grads["d" + s], dx, bx, q.dtype)
        if rest[0] is None:
            assert grads["dw" + s] is None
        else:
            close(grads["dw" + s], dw, bw)


@pytest.mark.parametrize("d,norm,dt", list(itertools.product([64, 128, 256], ["l2", "rms"], [BF, F32])))
def test_norms_and_rotations(gdn, d, norm, dt):
    for i, (rot, inter) in enumerate([(0, False), (16, False), (d // 2, True), (d, False),
                                      (d - 16, True), (d - 16, False), (d, True)]):
        q, k, dq, dk, kw = draw(21, 5, 3, d, 100 + d + i, dt, BF if i % 2 else F32,
                                weights=i % 3 != 0, rot=rot, far=[0, 8192, 1000000][i % 3],
                                fused=i % 2 == 0)
        check(gdn, q, k, dq, dk, kw, dict(norm=norm, eps=1e-6, interleaved=inter))


@pytest.mark.parametrize("T,Hq,Hk", [(1, 1, 1), (1, 16, 16), (2, 32, 1), (7, 1, 9), (700, 3, 1),
                                     (1500, 4, 4), (65, 40, 8)])
def test_sizes(gdn, T, Hq, Hk):
    q, k, dq, dk, kw = draw(T, Hq, Hk, 128, 7 + T, rot=64)
    check(gdn, q, k, dq, dk, kw, dict(norm="rms"))


def test_one_side_and_no_tokens(gdn):
    q, k, dq, dk, kw = draw(9, 4, 2, 64, 71)
    kw.pop("wk")
    oq, ok = gdn.qk_norm_forward(q, k, norm="rms", **kw)
    a, none = gdn.qk_norm_forward(q, None, norm="rms", **kw)
    assert none is None and torch.equal(a, oq)
    none, b = gdn.qk_norm_forward(None, k, norm="rms")
    assert none is None and torch.equal(b, ok)
    both = gdn.qk_norm_backward(q, k, dq, dk, norm="rms", **kw)
    one = gdn.qk_norm_backward(None, k, None, dk, norm="rms")
    assert one["dq"] is None and torch.equal(one["dk"], both["dk"]) and both["dwk"] is None
    one = gdn.qk_norm_backward(q, None, dq, None, norm="rms", want_dw=False, **kw)
    assert torch.equal(one["dq"], both["dq"]) and one["dwq"] is None
    z, zk, dz, dzk, kw = draw(0, 4, 2, 64, 72, rot=32)
    oq, ok = gdn.qk_norm_forward(z, zk, **kw)
    assert oq.shape == (0, 4, 64) and ok.shape == (0, 2, 64)
    grads = gdn.qk_norm_backward(z, zk, dz, dzk, **kw)
    assert not grads["dwq"].any() and not grads["dwk"].any()


def test_bits_are_a_heads_own(gdn):
    q, k, dq, dk, kw = draw(300, 6, 2, 128, 73, rot=128)
    oq, ok = gdn.qk_norm_forward(q, k, **kw)
    grads = gdn.qk_norm_backward(q, k, dq, dk, **kw)
    again = gdn.qk_norm_backward(q, k, dq, dk, **kw)
    assert all(torch.equal(grads[s], again[s]) for s in grads)
    kw1 = dict(kw, positions=kw["positions"][250:251])
    # one token alone, other heads around it, keys in the queries' place
    o1, k1 = gdn.qk_norm_forward(q[250:251], k[250:251], **kw1)
    assert torch.equal(o1[0], oq[250]) and torch.equal(k1[0], ok[250])
    o2, _ = gdn.qk_norm_forward(q[250:251, 3:4], None, **kw1)
    assert torch.equal(o2[0, 0], oq[250, 3])
    _, o3 = gdn.qk_norm_forward(None, q[250:251], **dict(kw1, wk=kw["wq"]))
    assert torch.equal(o3[0], oq[250])
    g1 = gdn.qk_norm_backward(q[250:251], k[250:251], dq[250:251], dk[250:251], **kw1)
    assert torch.equal(g1["dq"][0], grads["dq"][250])


def test_strides_and_in_place(gdn):
    q, k, dq, dk, kw = draw(50, 4, 2, 64, 74, rot=64, fused=True)
    oq, ok = gdn.qk_norm_forward(q, k, **kw)
    out = torch.full((50, 6 * 64 + 16), 5.0, dtype=BF, device="cuda")
    vq, vk = out[:, :256].unflatten(1, (4, 64)), out[:, 256:384].unflatten(1, (2, 64))
    gdn.qk_norm_forward(q, k, oq=vq, ok=vk, **kw)
    assert torch.equal(vq, oq) and torch.equal(vk, ok) and (out[:, 384:] == 5).all()
    grads = gdn.qk_norm_backward(q, k, dq, dk, **kw)
    gdn.qk_norm_backward(q, k, dq, dk, grads=dict(dq=vq, dk=vk, dwq=grads["dwq"].clone(),
                                                  dwk=grads["dwk"].clone()), **kw)
    assert torch.equal(vq, grads["dq"]) and (out[:, 384:] == 5).all()
    gdn.qk_norm_forward(q, k, oq=q, ok=k, **kw)     # in place, in the fused projection
    assert torch.equal(q, oq) and torch.equal(k, ok)


def test_extreme_values(gdn):
    """A head of zeros gives zeros; tiny and huge heads stay finite; a NaN stays in
    its head; positions of any sign and size turn a head without changing its length."""
    q, k, dq, dk, kw = draw(6, 2, 1, 128, 75, dt=F32, weights=False, rot=128)
    q[0, 0] = 0
    q[1, 0] *= 1e-18
    q[2, 0] *= 1e15
    q[3, 0, 5] = float("nan")
    kw["positions"].copy_(torch.tensor([0, -5, 2 ** 31 - 1, 3, -2 ** 24, 7], dtype=torch.int32))
    oq, _ = gdn.qk_norm_forward(q, k, **kw)
    grads = gdn.qk_norm_backward(q, k, dq, dk, **kw)
    assert not oq[0, 0].any() and torch.isfinite(grads["dq"][:3]).all()
    fine = torch.isfinite(oq).all(-1)
    assert fine.sum() == 11 and not fine[3, 0]
    assert torch.isfinite(grads["dq"]).all(-1).sum() == 11
    keep = [4, 5]
    x, p = f64(q[keep]), f64(kw["positions"])[keep]
    close(oq[keep], qk_norm.forward(x, None, p, f64(kw["inv_freq"])),
          qk_norm.forward_bound(x, None, p, f64(kw["inv_freq"])))
    close(oq[:1], qk_norm.forward(f64(q[:1])), qk_norm.forward_bound(f64(q[:1])))  # no turn
    length = (oq[2, 0].double() ** 2).sum()
    assert abs(float(length) - 1) < 1e-5


def test_streams_and_graphs(gdn):
    q, k, dq, dk, kw = draw(200, 4, 4, 128, 76, rot=64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = gdn.qk_norm_backward(q, k, dq, dk, stream=side, **kw)
    torch.cuda.current_stream().wait_stream(side)
    b = gdn.qk_norm_backward(q, k, dq, dk, **kw)
    assert all(torch.equal(a[s], b[s]) for s in a)
    graphs, outs = [], []
    for _ in range(2):      # two graphs, each with its own scratch
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            oq, ok = gdn.qk_norm_forward(q, k, **kw)
            outs.append((oq, ok, gdn.qk_norm_backward(q, k, dq, dk, **kw)))
    q.copy_(torch.randn_like(q.float()).to(BF))
    for gph in graphs:
        gph.replay()
    oq, ok = gdn.qk_norm_forward(q, k, **kw)
    b = gdn.qk_norm_backward(q, k, dq, dk, **kw)
    for cq, ck, c in outs:
        assert torch.equal(cq, oq) and torch.equal(ck, ok)
        assert all(torch.equal(c[s], b[s]) for s in b)


def test_binding_refuses(gdn):
    q, k, dq, dk, kw = draw(4, 2, 2, 64, 77, rot=32)
    with pytest.raises(ValueError, match="contiguous"):
        gdn.qk_norm_forward(q.transpose(1, 2).contiguous().transpose(1, 2), k)
    with pytest.raises(ValueError, match="together"):
        gdn.qk_norm_forward(q, k, positions=kw["positions"])
    with pytest.raises(ValueError, match="int32"):
        gdn.qk_norm_forward(q, k, positions=kw["positions"].long(), inv_freq=kw["inv_freq"])
    with pytest.raises(ValueError, match="shape"):
        gdn.qk_norm_forward(q, k[:3])
    with pytest.raises(ValueError, match="norm"):
        gdn.qk_norm_forward(q, k, norm="l1")
    with pytest.raises(ValueError, match="go with"):
        gdn.qk_norm_backward(q, k, dq, None)
    with pytest.raises(ValueError, match="float32|wq"):
        gdn.qk_norm_forward(q, k, wq=kw["wq"].to(BF))
    with pytest.raises(gdn.GdnError, match="UNSUPPORTED"):
        gdn.qk_norm_forward(q[..., :32].contiguous(), None)
    with pytest.raises(gdn.GdnError, match="UNSUPPORTED"):
        gdn.qk_norm_forward(q, k, positions=kw["positions"], inv_freq=kw["inv_freq"][:5])


@pytest.mark.parametrize("interleaved", [False, True])
def test_idle_groups_add_nothing_to_the_weights(gdn, interleaved):
    """Lane groups without a token must not read what an earlier kernel left in
    shared memory: here a run over NaNs, which fills it on every multiprocessor."""
    nan = torch.full((2048, 2048), float("nan"), device="cuda")
    cu = torch.tensor([0, 1000, 2048], dtype=torch.int32, device="cuda")
    q, k, dq, dk, kw = draw(37, 5, 1, 128, 78, rot=64)
    for rot in (16, 64):
        kw["inv_freq"] = kw["inv_freq"][:rot // 2].contiguous()
        gdn.glr_forward(nan, nan, cu)
        grads = gdn.qk_norm_backward(q, k, dq, dk, norm="rms", interleaved=interleaved, **kw)
        for (x, dy, rest), s in zip(sides(q, k, dq, dk, kw), "qk"):
            opts = dict(norm="rms", interleaved=interleaved)
            close(grads["dw" + s], qk_norm.backward(x, dy, *rest, **opts)[1],
                  qk_norm.backward_bound(x, dy, *rest, **opts)[1])


@pytest.mark.parametrize("norm", ["l2", "rms"])
def test_smallest_eps(gdn, norm):
    """A head of zeros with an eps whose r^2 is out of fp32's range: dx = r e."""
    eps = float(np.float32(1e-42))
    q, k, doq, dok, kw = draw(5, 3, 2, 64, 30)
    q[1], k[:, 0] = 0, 0
    grads = gdn.qk_norm_backward(q, k, doq, dok, norm=norm, eps=eps, **kw)
    assert all(torch.isfinite(g).all() for g in grads.values())
    check(gdn, q, k, doq, dok, kw, {"norm": norm, "eps": eps})
