"""The q/k norm, the Gated DeltaNet layer and the gated linear recurrence run
together, as a stack does: projections -> norm -> layer -> recurrence.

Prefill, a prefix continued by decode steps, and another batch composition have
the same bits at the end of the stack; the gradients that travel back through
the three are each within the bounds of their own oracle on what they received.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle import glr, qk_norm
from rl_train_numerics_b200 import workloads as W

pytestmark = pytest.mark.gpu
H, D = 2, 128
LENS = [70, 0, 130, 5]
NORM = dict(norm="l2", eps=1e-6)


@pytest.fixture(scope="module")
def gdn():
    from rl_train_numerics_b200 import _abi
    return _abi


def f64(t):
    return t.detach().double().cpu().numpy()


@pytest.fixture(scope="module")
def inputs():
    r = torch.Generator().manual_seed(61)
    T = sum(LENS)
    rand = lambda *s: torch.randn(s, generator=r)  # noqa: E731
    proj = rand(T, 3 * H * D).to(torch.bfloat16).cuda()   # q, k, v of one projection
    q, k, v = (proj[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)) for i in range(3))
    gates = dict(beta=torch.sigmoid(rand(T, H)).cuda(),
                 g=-torch.nn.functional.softplus(rand(T, H)).cuda(),
                 g2=-torch.nn.functional.softplus(rand(T, H * D)).cuda())
    return q, k, v.contiguous(), gates, rand(T, H * D).to(torch.bfloat16).cuda()


def rows(inputs, idx):
    q, k, v, gt, _ = inputs
    return q[idx], k[idx], v[idx], {s: t[idx] for s, t in gt.items()}


def stack(gdn, q, k, v, gt, lens, **kw):
    cu = W.cu_seqlens_of(lens, "cuda")
    qn, kn = gdn.qk_norm_forward(q, k, **NORM)
    o, srun, sbnd, ws = gdn.forward(qn, kn, v, gt["beta"], gt["g"], cu, **kw.get("layer", {}))
    assert gdn.check_error(ws) == 0
    h, _, carry, err = gdn.glr_forward(o.flatten(1), gt["g2"], cu, complement=True,
                                       **kw.get("glr", {}))
    assert gdn.check_error(err) == 0
    return qn, kn, o, srun, sbnd, h, carry, cu


def test_decode_and_other_batches_are_bitwise_the_prefill(gdn, inputs):
    q, k, v, gt, _ = inputs
    h = stack(gdn, q, k, v, gt, LENS)[5]
    edges = W.cu_seqlens_of(LENS).tolist()
    order = [3, 2, 0]
    idx = torch.cat([torch.arange(edges[n], edges[n + 1]) for n in order]).cuda()
    assert torch.equal(stack(gdn, *rows(inputs, idx), [LENS[n] for n in order])[5], h[idx])
    # prefixes of 30 and 60 tokens of the two long sequences, then decode
    seqs, prefix, steps = [0, 2], [30, 60], 40
    idx = torch.cat([torch.arange(edges[n], edges[n] + p) for n, p in zip(seqs, prefix)]).cuda()
    layer, vec = gdn.DecodeState(2, H, D, D), gdn.GlrDecodeState(2, H * D)
    scale = torch.empty((2, H), device="cuda")
    qn, kn, _, srun, sbnd, hp, _, cu = stack(gdn, *rows(inputs, idx), prefix,
                                             layer=dict(s_run_scale=scale), glr=dict(state=vec))
    assert torch.equal(hp, h[idx])
    gdn.decode_state_from_prefill(layer, kn, v[idx], gt["beta"][idx], gt["g"][idx], cu, srun,
                                  sbnd, s_run_scale=scale)
    for j in range(steps):
        t = torch.tensor([edges[n] + p + j for n, p in zip(seqs, prefix)]).cuda()
        qt, kt, vt, gtt = rows(inputs, t)
        qn, kn = gdn.qk_norm_forward(qt, kt, **NORM)
        o = gdn.decode_step(layer, qn, kn, vt, gtt["beta"], gtt["g"])
        out = gdn.glr_decode_step(vec, o.flatten(1), gtt["g2"], complement=True)
        assert torch.equal(out, h[t]), j
    assert gdn.check_error(layer.error) == 0 and gdn.check_error(vec.error) == 0


def test_gradients_travel_back(gdn, inputs):
    q, k, v, gt, dh = inputs
    qn, kn, o, _, _, h, carry, cu = stack(gdn, q, k, v, gt, LENS, glr=dict(want_carry=True))
    g1, err = gdn.glr_backward(o.flatten(1), gt["g2"], cu, carry, dh, complement=True)
    assert gdn.check_error(err) == 0
    g2, ws = gdn.backward(qn, kn, v, gt["beta"], gt["g"], cu, g1["dx"].unflatten(1, (H, D)))
    assert gdn.check_error(ws) == 0
    g3 = gdn.qk_norm_backward(q, k, g2["dq"], g2["dk"], **NORM)
    args = (f64(o.flatten(1)), f64(gt["g2"]), LENS, f64(dh))
    want = glr.backward(*args, complement=True)
    bound = glr.backward_bound(*args, complement=True)
    half = 2.0 ** -8    # of a bf16 step
    assert (np.abs(f64(g1["dx"]) - want[0]) <= bound[0] + half * (np.abs(want[0]) + bound[0])).all()
    assert (np.abs(f64(g1["dg"]) - want[1]) <= bound[1]).all()
    ref = oracle.backward(f64(qn), f64(kn), f64(v), f64(gt["beta"]), f64(gt["g"]),
                          cu.cpu().numpy(), f64(g1["dx"].unflatten(1, (H, D))))
    for s in ("dq", "dk"):      # the layer's own bound for bf16 inputs
        rms = np.sqrt(np.mean(ref[s] ** 2))
        assert np.abs(f64(g2[s]) - ref[s]).max() <= 1e-4 * rms
    for x, s in ((q, "dq"), (k, "dk")):
        dx, _ = qk_norm.backward(f64(x), f64(g2[s]), **NORM)
        b, _ = qk_norm.backward_bound(f64(x), f64(g2[s]), **NORM)
        assert (np.abs(f64(g3[s]) - dx) <= b + half * (np.abs(dx) + b)).all()
