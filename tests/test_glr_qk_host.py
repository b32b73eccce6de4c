"""CPU checks of the q/k norm and the gated linear recurrence: the fp64 oracles
against finite differences and independent forms, and every host-side refusal of
the library's entry points and of the binding.

Calls of the library below are ones it must refuse, or valid empty ones; none
reaches a launch, so the fake pointers are never dereferenced.
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle import glr, qk_norm
from rl_train_numerics_b200 import build_lib

build_lib.build()
from rl_train_numerics_b200 import _abi as gdn  # noqa: E402

FAKE, ODD = 0x10000, 0x10001
BAD, UNS, WS, OK = (gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED, gdn.GDN_ERR_WORKSPACE,
                    gdn.GDN_OK)


# ---------------------------------------------------------------------------
# Oracles
# ---------------------------------------------------------------------------

def draw_glr(T, N, D, seed):
    r = np.random.default_rng(seed)
    return (r.standard_normal((T, D)), -np.log1p(np.exp(r.standard_normal((T, D)))),
            r.standard_normal((N, D)), r.standard_normal((T, D)), r.standard_normal((N, D)))


@pytest.mark.parametrize("complement", [False, True])
def test_glr_oracle_gradients_are_differences(complement):
    """Central differences: the loss is smooth with derivatives of order one, so
    a step of 1e-4 leaves errors of about 1e-8 (truncation) + 1e-12 (rounding)."""
    lens = [3, 0, 1, 5]
    x, g, h0, dh, ds = draw_glr(9, 4, 2, 1)

    def loss(x, g, h0):
        h, s = glr.forward(x, g, lens, h0, complement)
        return (h * dh).sum() + (s * ds).sum()

    got = glr.backward(x, g, lens, dh, h0, ds, complement)
    args = [x, g, h0]
    for i, grad in enumerate(got):
        for at in np.ndindex(args[i].shape):
            up, dn = [a.copy() for a in args], [a.copy() for a in args]
            up[i][at] += 1e-4
            dn[i][at] -= 1e-4
            assert abs((loss(*up) - loss(*dn)) / 2e-4 - grad[at]) < 1e-6, (i, at)


def test_glr_oracle_closed_forms():
    x, g, h0, _, _ = draw_glr(6, 1, 3, 2)
    h, s = glr.forward(x, 0 * g, [6], h0)
    assert np.allclose(h, h0 + np.cumsum(x, 0), rtol=1e-14) and np.array_equal(s[0], h[-1])
    h, _ = glr.forward(x, g, [6], h0, complement=True)
    a = np.exp(g)
    want = [np.prod(a[:t + 1], 0) * h0[0] + sum(np.prod(a[i + 1:t + 1], 0) * (1 - a[i]) * x[i]
                                                for i in range(t + 1)) for t in range(6)]
    assert np.allclose(h, want, rtol=1e-13)
    h, _ = glr.forward(x, 0 * g - np.inf, [6], h0)
    assert np.array_equal(h, x)


@pytest.mark.parametrize("mistake", ["late decay", "no h0", "shifted h"])
def test_glr_oracle_catches(mistake):
    x, g, h0, dh, ds = draw_glr(5, 1, 2, 3)
    dx, dg, dh0 = glr.backward(x, g, [5], dh, h0, ds)
    if mistake == "late decay":     # h = a (h + b)
        bad, s = np.zeros_like(x), h0[0]
        for t in range(5):
            s = np.exp(g[t]) * (s + x[t])
            bad[t] = s
        bound, _ = glr.forward_bound(x, g, [5], h0)
        assert (np.abs(bad - glr.forward(x, g, [5], h0)[0]) > 100 * bound).any()
        return
    bound = glr.backward_bound(x, g, [5], dh, h0, ds)[1]
    if mistake == "no h0":
        bad = glr.backward(x, g, [5], dh, None, ds)[1]
    else:                           # dg from h_t in place of h_{t-1}
        h, _ = glr.forward(x, g, [5], h0)
        before = np.concatenate([h0, h[:-1]])
        bad = dg / before * h
    assert (np.abs(bad - dg) > 100 * bound).any()


@pytest.mark.parametrize("complement", [False, True])
def test_glr_chunk_schedule_in_fp32_is_within_the_bound(complement):
    """The kernels' schedule (chunks of 16, A and B from 1 and 0, h = A H + B) run
    in numpy fp32 stays within the oracle's bound."""
    lens = [1, 15, 16, 17, 40, 0, 200]
    T, D = sum(lens), 8
    x, g, h0, _, _ = draw_glr(T, len(lens), D, 4)
    x, g, h0 = x.astype(np.float32), g.astype(np.float32), h0.astype(np.float32)
    a = np.exp(g)
    b = -np.expm1(g) * x if complement else x
    h, t = np.zeros_like(x), 0
    for n, L in enumerate(lens):
        H = h0[n]
        for i in range(L):
            if i % 16 == 0:
                A, B = np.ones(D, np.float32), np.zeros(D, np.float32)
            A, B = a[t] * A, a[t] * B + b[t]
            h[t] = A * H + B
            if i % 16 == 15:
                H = h[t]
            t += 1
    ref, _ = glr.forward(x, g, lens, h0, complement)
    bound, _ = glr.forward_bound(x, g, lens, h0, complement)
    assert (np.abs(h - ref) <= bound).all()


@pytest.mark.parametrize("norm", ["l2", "rms"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_qk_oracle_gradients_are_differences(norm, interleaved):
    r = np.random.default_rng(5)
    T, H, d, F = 2, 2, 8, 3
    x, dy, w = r.standard_normal((T, H, d)), r.standard_normal((T, H, d)), 1 + r.random(d)
    pos, inv = np.array([3, -7]), 10.0 ** -np.arange(F)
    kw = dict(norm=norm, eps=1e-3, interleaved=interleaved)

    def loss(x, w):
        return (qk_norm.forward(x, w, pos, inv, **kw) * dy).sum()

    dx, dw = qk_norm.backward(x, dy, w, pos, inv, **kw)
    for args, grad, i in (((x, w), dx, 0), ((x, w), dw, 1)):
        for at in np.ndindex(args[i].shape):
            up, dn = [a.copy() for a in args], [a.copy() for a in args]
            up[i][at] += 1e-4
            dn[i][at] -= 1e-4
            assert abs((loss(*up) - loss(*dn)) / 2e-4 - grad[at]) < 1e-6


def test_qk_oracle_norms_and_turns():
    r = np.random.default_rng(6)
    x = r.standard_normal((4, 3, 16))
    y = qk_norm.forward(x, None, np.arange(4), np.array([0.5, 0.1]), eps=1e-30)
    assert np.allclose((y * y).sum(-1), 1, atol=1e-12)      # a turn keeps the length
    assert np.array_equal(y[0], qk_norm.forward(x, eps=1e-30)[0])   # position 0
    assert np.array_equal(y[..., 4:], qk_norm.forward(x, eps=1e-30)[..., 4:])
    z = qk_norm.forward(x, norm="rms", eps=1e-30)
    assert np.allclose((z * z).mean(-1), 1, atol=1e-12)
    # scores depend on the difference of positions only
    q, inv = r.standard_normal((1, 1, 16)), np.array([1.0, 0.3, 0.01])
    at = lambda v, p: qk_norm.rotate(v, np.array([p]), inv, False)  # noqa: E731
    k = r.standard_normal((1, 1, 16))
    assert np.allclose((at(q, 9) * at(k, 4)).sum(), (at(q, 105) * at(k, 100)).sum(), atol=1e-12)


# ---------------------------------------------------------------------------
# Refusals of the library
# ---------------------------------------------------------------------------

def qk_fwd(**over):
    a = dict(q=FAKE, ldq=512, k=FAKE, ldk=256, dt=0, T=8, Hq=4, Hk=2, d=128, norm=0, eps=1e-6,
             wq=FAKE, wk=None, pos=FAKE, inv=FAKE, rot=64, inter=0, oq=FAKE, ldoq=512, ok=FAKE,
             ldok=256, odt=0)
    a.update(over)
    return gdn.lib.gdn_qk_norm_forward(*a.values(), None)


@pytest.mark.parametrize("over,expect", [
    (dict(T=-1), BAD), (dict(Hq=-1), BAD), (dict(Hq=0, Hk=0), BAD), (dict(d=0), BAD),
    (dict(d=96), UNS), (dict(d=512), UNS), (dict(T=1 << 31), UNS), (dict(Hk=65536), UNS),
    (dict(dt=2), BAD), (dict(odt=-1), BAD), (dict(norm=2), BAD), (dict(eps=0.0), BAD),
    (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD),
    (dict(rot=-16), BAD), (dict(rot=144), BAD), (dict(rot=40), UNS), (dict(inter=2), BAD),
    (dict(pos=None), BAD), (dict(inv=None), BAD), (dict(pos=ODD), BAD), (dict(inv=ODD), BAD),
    (dict(q=None), BAD), (dict(k=None), BAD), (dict(oq=None), BAD), (dict(ok=None), BAD),
    (dict(q=FAKE + 8), BAD), (dict(ok=FAKE + 8), BAD), (dict(wq=FAKE + 4), BAD),
    (dict(ldq=504), BAD), (dict(ldq=516), BAD), (dict(ldok=255), BAD), (dict(ldq=0), BAD),
    (dict(ldq=1 << 41), UNS),
])
def test_qk_forward_refuses(over, expect):
    assert qk_fwd(**over) == expect


def test_qk_forward_without_tokens():
    assert qk_fwd(T=0, q=None, k=None, oq=None, ok=None, pos=None, inv=None) == OK


def qk_bwd(**over):
    a = dict(q=FAKE, ldq=512, k=FAKE, ldk=256, dt=0, T=8, Hq=4, Hk=2, d=128, norm=1, eps=1e-6,
             wq=FAKE, wk=FAKE, pos=None, inv=None, rot=0, inter=0, doq=FAKE, lddoq=512, dok=FAKE,
             lddok=256, gdt=1, dq=FAKE, lddq=512, dk=FAKE, lddk=256, dwq=FAKE, dwk=None, ws=FAKE,
             wsb=1 << 30)
    a.update(over)
    return gdn.lib.gdn_qk_norm_backward(*a.values(), None)


@pytest.mark.parametrize("over,expect", [
    (dict(T=-1), BAD), (dict(d=72), UNS), (dict(gdt=5), BAD), (dict(rot=16), BAD),
    (dict(doq=None), BAD), (dict(dok=FAKE + 8), BAD), (dict(lddok=128), BAD),
    (dict(lddok=258), BAD), (dict(dq=None), BAD), (dict(lddk=252), BAD), (dict(wq=None), BAD),
    (dict(dwk=FAKE + 4), BAD), (dict(ws=None), WS), (dict(wsb=16), WS), (dict(ws=FAKE + 8), BAD),
])
def test_qk_backward_refuses(over, expect):
    assert qk_bwd(**over) == expect


def test_qk_workspace_query():
    w = gdn.qk_norm_backward_workspace_bytes
    assert w(1, 4, 2, 128) == 2 * 128 * 4
    assert w(100000, 4, 2, 128) <= 592 * 2 * 128 * 4
    assert w(0, 4, 2, 128) == 0
    assert w(8, 4, 2, 100) == 0 and w(-1, 4, 2, 128) == 0 and w(8, 0, 0, 128) == 0
    assert qk_bwd(T=0, dwq=None, ws=None, q=None) == OK


def glr_fwd(**over):
    a = dict(x=FAKE, ldx=100, dt=0, g=FAKE, ldg=100, gdt=1, cu=FAKE, N=2, T=9, D=100, mode=0,
             h0=None, h=FAKE, ldh=100, odt=0, sf=None, st=None, slot=None, carry=None, err=None)
    a.update(over)
    if a["st"] is not None:
        a["st"] = ctypes.byref(a["st"])
    return gdn.lib.gdn_glr_forward(*a.values(), None)


def glr_state(**over):
    f = dict(h=FAKE, a=FAKE, b=FAKE, pos=FAKE, error=FAKE, n_slots=2)
    f.update(over)
    return gdn.GlrStateStruct(*f.values())


BAD_BATCH = [
    (dict(N=-1), BAD), (dict(T=-1), BAD), (dict(T=1 << 31), UNS), (dict(N=0), BAD),
    (dict(D=0), BAD), (dict(D=-4), BAD), (dict(D=(1 << 24) + 1, ldx=1 << 25, ldg=1 << 25,
                                               ldh=1 << 25), UNS),
    (dict(N=1 << 30, D=128, ldx=128, ldg=128, ldh=128), UNS), (dict(dt=3), BAD),
    (dict(gdt=-1), BAD), (dict(mode=2), BAD), (dict(cu=None), BAD), (dict(cu=ODD), BAD),
    (dict(x=None), BAD), (dict(g=None), BAD), (dict(x=ODD), BAD), (dict(g=FAKE + 2), BAD),
    (dict(ldx=99), BAD), (dict(ldg=0), BAD), (dict(ldx=1 << 41), UNS), (dict(err=ODD), BAD),
]


@pytest.mark.parametrize("over,expect", BAD_BATCH + [
    (dict(odt=2), BAD), (dict(h=None), BAD), (dict(h=ODD), BAD), (dict(ldh=64), BAD),
    (dict(h0=ODD), BAD), (dict(sf=FAKE + 2), BAD), (dict(carry=ODD), BAD),
    (dict(slot=FAKE), BAD), (dict(st=glr_state(n_slots=1)), BAD),
    (dict(st=glr_state(n_slots=0)), BAD), (dict(st=glr_state(h=None)), BAD),
    (dict(st=glr_state(pos=None)), BAD), (dict(st=glr_state(a=FAKE + 4)), BAD),
    (dict(st=glr_state(error=None)), BAD), (dict(st=glr_state(), slot=ODD), BAD),
])
def test_glr_forward_refuses(over, expect):
    assert glr_fwd(**over) == expect


def glr_bwd(**over):
    a = dict(x=FAKE, ldx=100, dt=0, g=FAKE, ldg=100, gdt=1, cu=FAKE, N=2, T=9, D=100, mode=0,
             carry=FAKE, dh=FAKE, lddh=100, ddt=0, ds=None, dx=FAKE, lddx=100, dg=FAKE, lddg=100,
             dh0=None, err=None)
    a.update({k: v for k, v in over.items() if k != "ldh"})
    return gdn.lib.gdn_glr_backward(*a.values(), None)


@pytest.mark.parametrize("over,expect", BAD_BATCH + [
    (dict(carry=None), BAD), (dict(carry=FAKE + 2), BAD), (dict(dh=None), BAD),
    (dict(ddt=9), BAD), (dict(lddh=64), BAD), (dict(dx=None), BAD), (dict(dx=ODD), BAD),
    (dict(lddx=99), BAD), (dict(dg=None), BAD), (dict(lddg=99), BAD), (dict(ds=FAKE + 2), BAD),
    (dict(dh0=ODD), BAD),
])
def test_glr_backward_refuses(over, expect):
    assert glr_bwd(**over) == expect


def glr_step(state=None, **over):
    a = dict(x=FAKE, ldx=100, dt=0, g=FAKE, ldg=100, gdt=1, slot=None, B=2, D=100, mode=0,
             st=state or glr_state(), h=FAKE, ldh=100, odt=0)
    a.update(over)
    return gdn.lib.gdn_glr_decode_step(*a.values(), None)


@pytest.mark.parametrize("over,expect", [
    (dict(B=-1), BAD), (dict(B=3), BAD), (dict(D=0), BAD), (dict(mode=-1), BAD),
    (dict(x=None), BAD), (dict(h=None), BAD), (dict(ldg=4), BAD), (dict(slot=ODD), BAD),
    (dict(state=glr_state(b=None)), BAD), (dict(state=glr_state(b=FAKE + 4)), BAD),
    (dict(state=glr_state(n_slots=-1)), BAD), (dict(odt=4), BAD), (dict(dt=4), BAD),
])
def test_glr_step_refuses(over, expect):
    assert glr_step(**over) == expect


def test_glr_empty_calls():
    none = dict(x=None, g=None, cu=None, N=0, T=0)
    assert glr_fwd(**none, h=None) == OK
    assert glr_bwd(**none, carry=None, dh=None, dx=None, dg=None) == OK
    assert glr_step(B=0, x=None, g=None, h=None) == OK


def test_glr_carry_rows():
    rows = gdn.glr_carry_rows
    assert rows(0, 0) == 0 and rows(3, 0) == 3 and rows(1, 128) == 2 and rows(5, 1000) == 12
    assert rows(-1, 5) == 0 and rows(1, -5) == 0 and rows(1, 1 << 31) == 0
    # the row of tile j of sequence n is cu[n] / 128 + n + j: inside, and no two the same
    rng = np.random.default_rng(7)
    for _ in range(50):
        lens = rng.integers(0, 400, rng.integers(1, 9))
        cu = np.concatenate([[0], np.cumsum(lens)])
        at = [cu[n] // 128 + n + j for n, L in enumerate(lens) for j in range(-(-L // 128))]
        assert len(set(at)) == len(at) and all(0 <= i < rows(len(lens), int(cu[-1])) for i in at)


# ---------------------------------------------------------------------------
# Refusals of the binding
# ---------------------------------------------------------------------------

def test_binding_refuses_cpu_tensors():
    x, g = torch.zeros((4, 8)), torch.zeros((4, 8))
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.glr_forward(x, g, cu)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.glr_backward(x, g, cu, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.glr_decode_step(gdn.GlrDecodeState(4, 8, device="cpu"), x, g)
    q = torch.zeros((4, 2, 64))
    with pytest.raises(ValueError, match="CUDA"):
        gdn.qk_norm_forward(q, q)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.qk_norm_backward(q, q, q, q)
    with pytest.raises(ValueError, match="tokens, heads"):
        gdn.qk_norm_forward(None, None)
