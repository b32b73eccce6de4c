"""GPU checks of the gated linear recurrence (gdn_glr_forward, _backward,
_decode_step) against the fp64 oracle within its fp32 bounds (oracle/glr.py),
and of its bit promises: decode, batch composition, widths and strides.
"""
import itertools

import numpy as np
import pytest
import torch

from oracle import glr
from rl_train_numerics_b200 import workloads as W

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
RAGGED = [1, 15, 16, 0, 17, 127, 128, 129, 0, 300, 2, 1100]


@pytest.fixture(scope="module")
def gdn():
    from rl_train_numerics_b200 import _abi
    return _abi


def draw(lens, D, seed, dt=BF, gt=F32, gates="softplus"):
    """x, g, d_h [T, D], h0, ds [N, D] and cu_seqlens, on the GPU."""
    r = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    z = torch.randn((T, D), generator=r)
    g = -torch.nn.functional.softplus(z)
    if gates == "stress":   # decays from none to a reset, a few of them growing
        u = torch.rand((T, D), generator=r)
        g = -torch.nn.functional.softplus(2.5 * z)
        g = torch.where(u < 0.03, torch.full_like(g, -1e4), g)
        g = torch.where((u > 0.1) & (u < 0.2), torch.full_like(g, -1e-7), g)
        g = torch.where((u > 0.2) & (u < 0.22), torch.full_like(g, 0.3), g)
        g = torch.where((u > 0.25) & (u < 0.26), torch.full_like(g, float("-inf")), g)
    rand = lambda *s: torch.randn(s, generator=r)  # noqa: E731
    return (rand(T, D).to(dt).cuda(), g.to(gt).cuda(), rand(T, D).to(dt).cuda(),
            rand(N, D).cuda(), rand(N, D).cuda(), W.cu_seqlens_of(lens, "cuda"))


def f64(t):
    return t.detach().double().cpu().numpy()


def close(got, want, bound, what=""):
    err = np.abs(f64(got) - want)
    assert (err <= bound).all(), (what, float((err / bound).max()))


def ok(gdn, error):
    assert gdn.check_error(error) == 0


def check_all(gdn, lens, D, seed, dt, gt, complement, gates="softplus"):
    x, g, dh, h0, ds, cu = draw(lens, D, seed, dt, gt, gates)
    ref_in = (f64(x), f64(g), lens)
    h, fin, carry, err = gdn.glr_forward(x, g, cu, h0=h0, complement=complement, out_dtype=F32,
                                         want_carry=True)
    ok(gdn, err)
    want, want_fin = glr.forward(*ref_in, f64(h0), complement)
    bh, bf = glr.forward_bound(*ref_in, f64(h0), complement)
    close(h, want, bh, "h")
    close(fin, want_fin, bf, "s_final")
    h16, _, _, _ = gdn.glr_forward(x, g, cu, h0=h0, complement=complement, out_dtype=BF)
    assert torch.equal(h16, h.to(BF))
    for d_h in {dt: dh, F32: dh.float()}.values():
        grads, err = gdn.glr_backward(x, g, cu, carry, d_h, ds_final=ds, complement=complement)
        ok(gdn, err)
        wx, wg, w0 = glr.backward(*ref_in, f64(dh), f64(h0), f64(ds), complement)
        bx, bg, b0 = glr.backward_bound(*ref_in, f64(dh), f64(h0), f64(ds), complement)
        if dt == BF:    # one rounding to bf16: half a step, 2^-8 of the value
            bx = bx + 2.0 ** -8 * (np.abs(wx) + bx)
        if gt == BF:
            bg = bg + 2.0 ** -8 * (np.abs(wg) + bg)
        assert grads["dx"].dtype == dt and grads["dg"].dtype == gt
        close(grads["dx"], wx, bx, "dx")
        close(grads["dg"], wg, bg, "dg")
        close(grads["dh0"], w0, b0, "dh0")


@pytest.mark.parametrize("dt,gt,complement", list(itertools.product([BF, F32], [BF, F32],
                                                                    [False, True])))
@pytest.mark.parametrize("D", [64, 1, 37, 130])
def test_ragged(gdn, D, dt, gt, complement):
    check_all(gdn, RAGGED, D, 11 + D, dt, gt, complement)


@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("lens", [[1], [16], [5000], [40] * 33])
def test_lengths_with_stress_gates(gdn, lens, complement):
    check_all(gdn, lens, 96, 23, BF, F32, complement, gates="stress")


def test_defaults(gdn):
    """No h0, no ds_final, no state, no carry: zeros, and nothing else changes."""
    lens = [70, 3, 0, 140]
    x, g, dh, h0, ds, cu = draw(lens, 48, 31)
    h, fin, carry, _ = gdn.glr_forward(x, g, cu, want_carry=True)
    hz, finz, carryz, _ = gdn.glr_forward(x, g, cu, h0=torch.zeros_like(h0), want_carry=True)
    assert torch.equal(h, hz) and torch.equal(fin, finz) and not fin[2].any()
    h1, none, no_carry, err = gdn.glr_forward(x, g, cu, want_state=False)
    assert none is None and no_carry is None and torch.equal(h1, h)
    ok(gdn, err)
    a, _ = gdn.glr_backward(x, g, cu, carry, dh)
    b, _ = gdn.glr_backward(x, g, cu, carryz, dh, ds_final=torch.zeros_like(ds))
    assert all(torch.equal(a[k], b[k]) for k in a)
    c, _ = gdn.glr_backward(x, g, cu, carry, dh, want_dh0=False)
    assert c["dh0"] is None and torch.equal(c["dx"], a["dx"])


def test_plain_is_linear_in_x_and_h0(gdn):
    """The loss <h, d_h> + <s_final, ds> is linear in (x, h0) when g is fixed, so a
    difference over any step is the gradient's product with it, up to rounding."""
    lens = [50, 200]
    x, g, dh, h0, ds, cu = draw(lens, 64, 33, dt=F32)
    x2, _, _, h02, _, _ = draw(lens, 64, 34, dt=F32)
    h, fin, carry, _ = gdn.glr_forward(x, g, cu, h0=h0, want_carry=True)
    h2, fin2, _, _ = gdn.glr_forward(x2, g, cu, h0=h02)
    grads, _ = gdn.glr_backward(x, g, cu, carry, dh, ds_final=ds)
    loss = lambda a, b: (a.double() * dh).sum() + (b.double() * ds).sum()  # noqa: E731
    step = (grads["dx"].double() * (x2.double() - x)).sum() + \
        (grads["dh0"].double() * (h02.double() - h0)).sum()
    args = (f64(x), f64(g), lens)
    slack = 0.0
    for xs, hs in ((x, h0), (x2, h02)):
        bh, bf = glr.forward_bound(f64(xs), f64(g), lens, f64(hs))
        slack += (bh * np.abs(f64(dh))).sum() + (bf * np.abs(f64(ds))).sum()
    bx, _, b0 = glr.backward_bound(*args, f64(dh), f64(h0), f64(ds))
    slack += (bx * np.abs(f64(x2) - f64(x))).sum() + (b0 * np.abs(f64(h02) - f64(h0))).sum()
    assert abs(float(loss(h2, fin2) - loss(h, fin) - step)) <= slack


@pytest.mark.parametrize("complement", [False, True])
def test_dg_is_a_difference(gdn, complement):
    """One gate at a time moved by +-1/8 in g (fp32): the central difference of
    the loss has a truncation error of at most step^2 / 6 times its third
    derivative; moving one g scales that token's carried part by e^step, whose
    odd part is sinh(step) / step = 1 + step^2 / 6 exactly."""
    x, g, dh, h0, ds, cu = draw([40], 32, 35, dt=F32)
    _, _, carry, _ = gdn.glr_forward(x, g, cu, h0=h0, complement=complement, want_carry=True)
    grads, _ = gdn.glr_backward(x, g, cu, carry, dh, ds_final=ds, complement=complement)
    step, sinh = 0.125, float(np.sinh(0.125)) / 0.125
    for t in (0, 15, 16, 39):
        val = []
        slack = 0.0
        for s in (step, -step):
            g2 = g.clone()
            g2[t] += s
            moved = (g2[t] - g[t]).double()
            h, fin, _, _ = gdn.glr_forward(x, g2, cu, h0=h0, complement=complement)
            val.append((h.double() * dh).sum(0) + (fin.double() * ds).sum(0))
            bh, bf = glr.forward_bound(f64(x), f64(g2), [40], f64(h0), complement)
            slack = slack + (bh * np.abs(f64(dh))).sum(0) + (bf * np.abs(f64(ds))).sum(0)
            # g + step is rounded to fp32: at most 2^-24 |g2| off, in a relative step
            slack = slack + np.abs(f64(grads["dg"][t])) * 2 * (f64(moved) - s).__abs__()
        diff = (val[0] - val[1]).cpu().numpy()
        bg = glr.backward_bound(f64(x), f64(g), [40], f64(dh), f64(h0), f64(ds), complement)[1][t]
        want = f64(grads["dg"][t]) * 2 * step * sinh
        assert (np.abs(diff - want) <= slack + bg * 2 * step * sinh).all(), t


@pytest.mark.parametrize("D,dt,gt,complement", [(64, BF, F32, False), (37, F32, BF, True),
                                                (2050, BF, F32, True)])
def test_prefix_and_decode_are_bitwise_the_forward(gdn, D, dt, gt, complement):
    prefix = [0, 1, 15, 16, 17, 40, 130]
    steps = 35
    full = [p + steps for p in prefix]
    x, g, _, h0, _, cu = draw(full, D, 41, dt, gt, gates="stress")
    kw = dict(complement=complement, out_dtype=F32)
    h_all, fin, _, _ = gdn.glr_forward(x, g, cu, h0=h0, **kw)
    at = [int(c) for c in cu[:-1]]
    idx = torch.cat([torch.arange(a, a + p) for a, p in zip(at, prefix)]).cuda()
    slots = torch.tensor([8, 0, 3, 5, 1, 7, 2], dtype=torch.int32, device="cuda")
    state = gdn.GlrDecodeState(9, D)
    h_pre, _, _, err = gdn.glr_forward(x[idx], g[idx], W.cu_seqlens_of(prefix, "cuda"), h0=h0,
                                       state=state, slot_idx=slots, **kw)
    ok(gdn, err)
    ok(gdn, state.error)
    assert torch.equal(h_pre, h_all[idx])
    assert state.pos.tolist() == [1, 1, 2, 15, 0, 0, 0, 8, 0]
    untouched = [4, 6]
    assert not state.h[untouched].any() and (state.a[untouched] == 1).all()
    base = torch.tensor(at, device="cuda") + torch.tensor(prefix, device="cuda")
    for j in range(steps):
        t = base + j
        o = gdn.glr_decode_step(state, x[t], g[t], slot_idx=slots, **kw)
        assert torch.equal(o, h_all[t]), j
    ok(gdn, state.error)
    # the decode state is the one a forward over everything leaves
    whole = gdn.GlrDecodeState(9, D)
    gdn.glr_forward(x, g, cu, h0=h0, state=whole, slot_idx=slots, **kw)
    assert all(torch.equal(a, b) for a, b in zip(state.tensors(), whole.tensors()))
    value = torch.where((whole.pos > 0)[:, None], whole.a * whole.h + whole.b, whole.h)
    assert torch.allclose(value[slots.long()], fin, rtol=1e-6, atol=1e-6)


def test_forward_in_two_parts_is_bitwise_one(gdn):
    x, g, _, h0, _, cu = draw([400], 100, 43)
    h, fin, _, _ = gdn.glr_forward(x, g, cu, h0=h0)
    for cut in (16, 128, 208):
        a, mid, _, _ = gdn.glr_forward(x[:cut], g[:cut], W.cu_seqlens_of([cut], "cuda"), h0=h0)
        b, end, _, _ = gdn.glr_forward(x[cut:], g[cut:], W.cu_seqlens_of([400 - cut], "cuda"),
                                       h0=mid)
        assert torch.equal(torch.cat([a, b]), h) and torch.equal(end, fin), cut


def test_bits_do_not_depend_on_batch_width_or_stride(gdn):
    lens = [5, 700, 64, 1, 129, 0, 2000, 33]
    D = 96
    x, g, dh, h0, ds, cu = draw(lens, D, 44)

    def both(x, g, dh, h0, ds, cu):
        h, fin, carry, _ = gdn.glr_forward(x, g, cu, h0=h0, want_carry=True)
        grads, _ = gdn.glr_backward(x, g, cu, carry, dh, ds_final=ds)
        return h, fin, grads

    h, fin, gr = both(x, g, dh, h0, ds, cu)
    h2, fin2, gr2 = both(x, g, dh, h0, ds, cu)
    assert torch.equal(h, h2) and all(torch.equal(gr[k], gr2[k]) for k in gr)
    edges = cu.tolist()
    for n in (0, 1, 6):     # a sequence alone: other launch shapes
        sl = slice(edges[n], edges[n + 1])
        h1, fin1, gr1 = both(x[sl], g[sl], dh[sl], h0[n:n + 1], ds[n:n + 1],
                             W.cu_seqlens_of([lens[n]], "cuda"))
        assert torch.equal(h1, h[sl]) and torch.equal(fin1[0], fin[n])
        assert torch.equal(gr1["dx"], gr["dx"][sl]) and torch.equal(gr1["dg"], gr["dg"][sl])
        assert torch.equal(gr1["dh0"][0], gr["dh0"][n])
    # an odd slice of the channels, at odd element offsets and strides
    cols = slice(3, 90)
    wide = torch.zeros((sum(lens), 2 * D + 7), dtype=BF, device="cuda")
    wide[:, 5:5 + 87] = x[:, cols]
    h3, _, gr3 = both(wide[:, 5:5 + 87], g[:, cols], dh[:, cols], h0[:, cols].contiguous(),
                      ds[:, cols].contiguous(), cu)
    assert torch.equal(h3, h[:, cols]) and torch.equal(gr3["dg"], gr["dg"][:, cols])
    # outputs written into strided memory touch nothing else
    out = torch.full((sum(lens), D + 9), 7.0, dtype=BF, device="cuda")
    gdn.glr_forward(x, g, cu, h0=h0, h=out[:, 4:4 + D])
    assert torch.equal(out[:, 4:4 + D], h)
    assert (out[:, :4] == 7).all() and (out[:, 4 + D:] == 7).all()


def test_long_and_wide(gdn):
    """One sequence long enough for every split of the work; sampled channels."""
    x, g, dh, h0, ds, cu = draw([9000], 256, 45)
    h, fin, carry, err = gdn.glr_forward(x, g, cu, h0=h0, out_dtype=F32, want_carry=True)
    ok(gdn, err)
    grads, _ = gdn.glr_backward(x, g, cu, carry, dh, ds_final=ds)
    ch = [0, 1, 63, 64, 255]
    args = (f64(x[:, ch]), f64(g[:, ch]), [9000])
    close(h[:, ch], glr.forward(*args, f64(h0[:, ch]))[0],
          glr.forward_bound(*args, f64(h0[:, ch]))[0])
    want = glr.backward(*args, f64(dh[:, ch]), f64(h0[:, ch]), f64(ds[:, ch]))
    bound = glr.backward_bound(*args, f64(dh[:, ch]), f64(h0[:, ch]), f64(ds[:, ch]))
    close(grads["dg"][:, ch], want[1], bound[1])


def test_bad_sequences_and_slots_set_error_words(gdn):
    x, g, dh, h0, ds, _ = draw([30, 20], 64, 46)
    good = W.cu_seqlens_of([30, 20], "cuda")
    for bad in ([0, 60, 50], [1, 30, 50], [0, 30, 49], [0, -3, 50]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        h = torch.full_like(x, 3.0)
        _, _, carry, err = gdn.glr_forward(x, g, cu, h0=h0, h=h, want_carry=True)
        torch.cuda.synchronize()
        assert int(err.item()) & gdn.GDN_DEVERR_CU_SEQLENS
        assert (h[30:] == 3).all()
        _, err = gdn.glr_backward(x, g, cu, carry, dh)
        assert gdn.check_error(err) & gdn.GDN_DEVERR_CU_SEQLENS
        _, _, _, err = gdn.glr_forward(x, g, good, error=err)   # the next call clears it
        ok(gdn, err)
    state = gdn.GlrDecodeState(2, 64)
    for slots in ([0, 2], [-1, 1], [1, 1]):
        before = state.clone()
        gdn.glr_forward(x, g, good, h0=h0, state=state,
                        slot_idx=torch.tensor(slots, dtype=torch.int32, device="cuda"))
        assert gdn.check_error(state.error) & gdn.GDN_DEVERR_POS
        bad = [i for i in (0, 1) if i not in slots]
        assert all(torch.equal(a[bad], b[bad]) for a, b in zip(state.tensors(), before.tensors()))


def test_decode_refuses_bad_rows(gdn):
    D = 70
    x, g, _, _, _, _ = draw([4], D, 47)
    state = gdn.GlrDecodeState(6, D)
    state.h.normal_()
    state.pos[4] = 16
    state.pos[5] = -1
    before = state.clone()
    h = torch.full((4, D), 9.0, dtype=BF, device="cuda")
    idx = torch.tensor([2, 6, 2, 4], dtype=torch.int32, device="cuda")  # 6: none; 2: twice
    gdn.glr_decode_step(state, x, g, slot_idx=idx, h=h)
    assert gdn.check_error(state.error) & gdn.GDN_DEVERR_POS
    assert (h[1:] == 9).all() and not (h[0] == 9).all()
    rest = [0, 1, 3, 4, 5]
    assert all(torch.equal(a[rest], b[rest]) for a, b in zip(state.tensors(), before.tensors()))
    assert int(state.pos[2]) == 1
    # the first of the two rows is the one that ran
    one = before.clone()
    want = gdn.glr_decode_step(one, x[:1], g[:1], slot_idx=idx[:1])
    assert torch.equal(want[0], h[0]) and torch.equal(one.h, state.h)
    gdn.glr_decode_step(state, x[:1], g[:1], h=h[:1],
                        slot_idx=torch.tensor([5], dtype=torch.int32, device="cuda"))
    assert gdn.check_error(state.error) & gdn.GDN_DEVERR_POS


def test_stale_values_of_a_fresh_chunk_do_not_matter(gdn):
    x, g, _, _, _, _ = draw([3], 40, 48)
    state = gdn.GlrDecodeState(3, 40)
    state.h.normal_()
    other = state.clone()
    other.a.fill_(float("nan"))
    other.b.fill_(float("inf"))
    assert torch.equal(gdn.glr_decode_step(state, x, g), gdn.glr_decode_step(other, x, g))
    assert all(torch.equal(a, b) for a, b in zip(state.tensors(), other.tensors()))


def test_empty_batches(gdn):
    z = torch.zeros((0, 64), dtype=BF, device="cuda")
    zg = torch.zeros((0, 64), device="cuda")
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    err = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    h, fin, carry, _ = gdn.glr_forward(z, zg, cu, want_carry=True, error=err)
    assert h.shape == (0, 64) and fin.shape == (0, 64) and carry.shape == (0, 64)
    ok(gdn, err)
    gdn.glr_backward(z, zg, cu, carry, z, error=err)
    ok(gdn, err)
    # sequences without tokens: the states pass through
    h0 = torch.randn((3, 64), device="cuda")
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    state = gdn.GlrDecodeState(3, 64)
    _, fin, carry, _ = gdn.glr_forward(z, zg, cu, h0=h0, state=state, want_carry=True)
    assert torch.equal(fin, h0) and torch.equal(state.h, h0)
    grads, _ = gdn.glr_backward(z, zg, cu, carry, z, ds_final=h0)
    assert torch.equal(grads["dh0"], h0)
    assert gdn.glr_decode_step(state, z, zg).shape == (0, 64)


def test_streams_and_graphs(gdn):
    x, g, dh, h0, ds, cu = draw([300, 40], 128, 49)
    want_h, want_fin, carry, _ = gdn.glr_forward(x, g, cu, h0=h0, want_carry=True)
    want, _ = gdn.glr_backward(x, g, cu, carry, dh, ds_final=ds)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    h, fin, c2, err = gdn.glr_forward(x, g, cu, h0=h0, want_carry=True, stream=side)
    got, _ = gdn.glr_backward(x, g, cu, c2, dh, ds_final=ds, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(h, want_h) and all(torch.equal(got[k], want[k]) for k in want)
    ok(gdn, err)
    # a captured step replayed on changing inputs; eager calls in between
    state = gdn.GlrDecodeState(4, 128)
    eager = state.clone()
    xs, gs = x[:4].clone(), g[:4].clone()
    out = torch.empty((4, 128), dtype=BF, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.glr_decode_step(state, xs, gs, h=out)
    for i in range(20):
        xs.copy_(x[i:i + 4])
        gs.copy_(g[i:i + 4])
        graph.replay()
        assert torch.equal(out, gdn.glr_decode_step(eager, x[i:i + 4], g[i:i + 4])), i
    assert all(torch.equal(a, b) for a, b in zip(state.tensors(), eager.tensors()))
    # forward and backward captured together
    graph = torch.cuda.CUDAGraph()
    buf = {k: torch.empty_like(v) for k, v in want.items()}
    with torch.cuda.graph(graph):
        h, fin, c3, e3 = gdn.glr_forward(x, g, cu, h0=h0, want_carry=True)
        gdn.glr_backward(x, g, cu, c3, dh, ds_final=ds, grads=buf)
    x.copy_(torch.randn_like(x.float()).to(BF))
    graph.replay()
    want_h, _, carry, _ = gdn.glr_forward(x, g, cu, h0=h0, want_carry=True)
    want, _ = gdn.glr_backward(x, g, cu, carry, dh, ds_final=ds)
    assert torch.equal(h, want_h) and all(torch.equal(buf[k], want[k]) for k in want)


def test_binding_refuses(gdn):
    x, g, dh, h0, ds, cu = draw([8], 16, 50)
    with pytest.raises(ValueError, match="shape"):
        gdn.glr_forward(x, g[:4], cu)
    with pytest.raises(ValueError, match="contiguous"):
        gdn.glr_forward(x.t().contiguous().t(), g, cu)
    with pytest.raises(ValueError, match="int32"):
        gdn.glr_forward(x, g, cu.long())
    with pytest.raises(ValueError, match="unsupported dtype"):
        gdn.glr_forward(x.half(), g, cu)
    with pytest.raises(ValueError, match="h0"):
        gdn.glr_forward(x, g, cu, h0=h0.to(BF))
    with pytest.raises(ValueError, match="carry"):
        gdn.glr_backward(x, g, cu, None, dh)
    with pytest.raises(gdn.GdnError):   # rows that repeat (stride 0) cannot be written
        gdn.glr_forward(x, g, cu, h=torch.empty((1, 16), dtype=BF, device="cuda").expand(8, 16))
    with pytest.raises(ValueError, match="state"):
        gdn.glr_decode_step(gdn.GlrDecodeState(8, 15), x, g)


SHAPES = {  # (lengths, channels): the launch shapes that sizes choose between
    "short": ([3, 0, 17, 64, 1, 130, 40, 16] * 8, 512),        # many short sequences
    "short, one long": ([2] * 60 + [900], 513),
    "tiles": ([300, 5, 700, 129] * 4, 512),                    # a block for each slab
    "clusters of 8": ([5000], 64),
    "clusters of 4": ([3000, 1, 2000], 512),
    "two for uneven": ([1500, 10, 300, 0, 700], 2048),
    "last step partly empty": ([129], 32),
    "rows off 16 bytes": ([700, 300], 1027),
}


@pytest.mark.parametrize("name", list(SHAPES))
@pytest.mark.parametrize("complement", [False, True])
def test_every_launch_shape_has_the_same_bits(gdn, name, complement):
    """Each sequence of the batch alone, and its first 32 and last odd channels
    alone, go through other kernels, clusters and stages: the bits are the same."""
    lens, D = SHAPES[name]
    x, g, dh, h0, ds, cu = draw(lens, D, 61)
    edges = cu.tolist()

    def both(rows, cols, n):
        c = W.cu_seqlens_of([lens[i] for i in n], "cuda")
        take = lambda t: t[rows][:, cols].contiguous()  # noqa: E731
        per = lambda t: t[n][:, cols].contiguous()      # noqa: E731
        a = (take(x), take(g), c)
        h, fin, carry, err = gdn.glr_forward(*a, h0=per(h0), complement=complement,
                                             want_carry=True)
        ok(gdn, err)
        grads, err = gdn.glr_backward(*a, carry, take(dh), ds_final=per(ds),
                                      complement=complement)
        ok(gdn, err)
        return (h, grads["dx"], grads["dg"]), (fin, grads["dh0"])

    everything = list(range(len(lens)))
    tok, seq = both(slice(None), slice(None), everything)
    for n in sorted({0, len(lens) // 2, len(lens) - 1}):
        rows = slice(edges[n], edges[n + 1])
        for cols in (slice(None), slice(0, 32), slice(D - 7, D)):
            t1, s1 = both(rows, cols, [n])
            assert all(torch.equal(a, b[rows][:, cols]) for a, b in zip(t1, tok)), (n, cols)
            assert all(torch.equal(a[0], b[n][cols]) for a, b in zip(s1, seq)), (n, cols)
    # and the oracle, on a few channels
    ch = [0, D // 2, D - 1]
    args = (f64(x[:, ch]), f64(g[:, ch]), lens)
    want, _ = glr.forward(*args, f64(h0[:, ch]), complement)
    bound, _ = glr.forward_bound(*args, f64(h0[:, ch]), complement)
    close(tok[0][:, ch], want, bound + 2.0 ** -8 * (np.abs(want) + bound))
    wx, wg, w0 = glr.backward(*args, f64(dh[:, ch]), f64(h0[:, ch]), f64(ds[:, ch]), complement)
    bx, bg, b0 = glr.backward_bound(*args, f64(dh[:, ch]), f64(h0[:, ch]), f64(ds[:, ch]),
                                    complement)
    close(tok[2][:, ch], wg, bg, "dg")
    close(seq[1][:, ch], w0, b0, "dh0")


def test_decode_states_from_short_sequences(gdn):
    """The short kernel's final states: slots, positions and a twice-named slot."""
    lens, D = [3, 0, 17, 64, 1, 33, 40, 16] * 8, 512
    x, g, _, h0, _, cu = draw(lens, D, 62)
    idx = torch.randperm(64, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    idx[9] = idx[4]
    state = gdn.GlrDecodeState(64, D)
    _, fin, _, err = gdn.glr_forward(x, g, cu, h0=h0, state=state, slot_idx=idx.cuda())
    ok(gdn, err)
    assert gdn.check_error(state.error) & gdn.GDN_DEVERR_POS
    value = torch.where((state.pos > 0)[:, None], state.a * state.h + state.b, state.h)
    keep = [n for n in range(64) if n != 9]
    slots = idx[keep].long()
    assert state.pos[slots].tolist() == [lens[n] % 16 for n in keep]
    assert torch.allclose(value[slots], fin[keep], rtol=1e-6, atol=1e-6)
    one = gdn.GlrDecodeState(64, D)     # a sequence alone takes the tile kernel
    edges = cu.tolist()
    rows = slice(edges[2], edges[3])
    gdn.glr_forward(x[rows], g[rows], W.cu_seqlens_of([lens[2]], "cuda"), h0=h0[2:3], state=one)
    assert all(torch.equal(a[0], b[int(idx[2])]) for a, b in zip(one.tensors(), state.tensors()))


def test_two_threads_with_different_shapes(gdn):
    """Calls of one kernel with different launch shapes, at once from two host threads."""
    import threading
    jobs = []
    for lens, D in (([5000], 64), ([700] * 40, 512), ([129, 300], 2048)):
        x, g, dh, h0, ds, cu = draw(lens, D, 70)

        def job(x=x, g=g, dh=dh, h0=h0, ds=ds, cu=cu):
            h, fin, carry, err = gdn.glr_forward(x, g, cu, h0=h0, want_carry=True)
            grads, err2 = gdn.glr_backward(x, g, cu, carry, dh, ds_final=ds)
            return h, fin, grads["dx"], grads["dg"], grads["dh0"], err, err2
        jobs.append((job, [t.clone() for t in job()]))
    torch.cuda.synchronize()
    failed = []

    def loop(job, want, stream):
        try:
            with torch.cuda.stream(stream):
                for _ in range(200):
                    got = job()
                stream.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want)):
                failed.append("other bits")
        except Exception as e:  # a refused launch
            failed.append(e)
    threads = [threading.Thread(target=loop, args=(*j, torch.cuda.Stream())) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


@pytest.mark.parametrize("lens,D", [([2], 64), ([2], 37), ([130, 2], 64), ([2] * 64, 256)])
def test_identity_steps_keep_the_sign_of_a_zero(gdn, lens, D):
    """A sum that underflowed to -0 at a sequence's last token is -0 in its final
    and decode state too.  x = (-2^-149, 0), a = exp(-1.4) < 1/2: B = -2^-149, then
    fma(a, -2^-149, 0) rounds to -0, and h = fma(A, -0, -0) = -0."""
    T, N = sum(lens), len(lens)
    x = torch.zeros((T, D), device="cuda")
    cu = W.cu_seqlens_of(lens, "cuda")
    x[(cu[1:] - 2).long()] = -2.0 ** -149
    g = torch.full((T, D), -1.4, device="cuda")
    h0 = torch.full((N, D), -0.0, device="cuda")
    state, steps = gdn.GlrDecodeState(N, D), gdn.GlrDecodeState(N, D)
    h, fin, _, err = gdn.glr_forward(x, g, cu, h0=h0, state=state)
    ok(gdn, err)
    bits = lambda t: t.view(torch.int32)  # noqa: E731
    last = (cu[1:] - 1).long()
    assert torch.equal(bits(fin), bits(h[last]))
    if max(lens) == 2:
        assert (bits(fin) == -2 ** 31).all()
        steps.h.copy_(h0)
        for t in range(2):
            hd = gdn.glr_decode_step(steps, x[last - 1 + t], g[last - 1 + t])
            assert torch.equal(bits(hd), bits(h[last - 1 + t]))
        for a, b in zip(steps.tensors(), state.tensors()):
            assert torch.equal(bits(a), bits(b))


@pytest.mark.parametrize("lens", [[300, 5, 300, 0, 129, 700, 17, 300] * 4, [40, 900, 0, 900, 900]])
def test_batches_whose_longest_start_first(gdn, lens):
    """More blocks than places: sequences of equal and no length, their decode
    states, and a batch with a bad sequence, whose others are not touched by it."""
    D, N = 2048, len(lens)
    x, g, dh, h0, ds, cu = draw(lens, D, 71)
    slots = torch.arange(N, dtype=torch.int32, device="cuda").flip(0).contiguous()
    state = gdn.GlrDecodeState(N, D)
    h, fin, carry, err = gdn.glr_forward(x, g, cu, h0=h0, state=state, slot_idx=slots,
                                         want_carry=True)
    ok(gdn, err)
    grads, err = gdn.glr_backward(x, g, cu, carry, dh, ds_final=ds)
    ok(gdn, err)
    edges = cu.tolist()
    for n in sorted({*range(6), N - 2, N - 1} & set(range(N))):
        rows = slice(edges[n], edges[n + 1])
        one = gdn.GlrDecodeState(1, D)
        c = W.cu_seqlens_of([lens[n]], "cuda")
        h1, f1, c1, _ = gdn.glr_forward(x[rows], g[rows], c, h0=h0[n:n + 1], state=one,
                                        want_carry=True)
        g1, _ = gdn.glr_backward(x[rows], g[rows], c, c1, dh[rows], ds_final=ds[n:n + 1])
        assert torch.equal(h1, h[rows]) and torch.equal(f1[0], fin[n])
        assert torch.equal(g1["dx"], grads["dx"][rows])
        assert torch.equal(g1["dg"], grads["dg"][rows])
        assert torch.equal(g1["dh0"][0], grads["dh0"][n])
        for a, b in zip(one.tensors(), state.tensors()):
            assert torch.equal(a[0], b[slots[n]])
    # sequence 1 ends before it starts: it and the next, which then overlaps 0, are not looked at
    bad = cu.clone()
    bad[2] = 0
    out = torch.full_like(h, 7.0)
    _, f2, _, err = gdn.glr_forward(x, g, bad, h0=h0, h=out)
    assert err.item() == gdn.GDN_DEVERR_CU_SEQLENS
    for n in range(3, N):
        rows = slice(edges[n], edges[n + 1])
        assert torch.equal(out[rows], h[rows]) and torch.equal(f2[n], fin[n])
