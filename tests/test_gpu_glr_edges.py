"""GPU checks of the gated linear recurrence at the edges of what its header
allows: the gates themselves, slow gates, batches of very unequal sequences,
gates that grow, invalid cu_seqlens and what lies behind a sequence's end.
"""
import numpy as np
import pytest
import torch

from oracle import glr
from rl_train_numerics_b200 import workloads as W

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def gdn():
    from rl_train_numerics_b200 import _abi
    return _abi


def f64(t):
    return t.detach().double().cpu().numpy()


def draw(lens, D, seed, dt=BF, gt=F32):
    """x, g, d_h [T, D], h0, ds [N, D] and cu_seqlens, on the GPU."""
    r = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    rand = lambda *s: torch.randn(s, generator=r)  # noqa: E731
    g = -torch.nn.functional.softplus(rand(T, D))
    return (rand(T, D).to(dt).cuda(), g.to(gt).cuda(), rand(T, D).to(dt).cuda(),
            rand(N, D).cuda(), rand(N, D).cuda(), W.cu_seqlens_of(lens, "cuda"))


def close(got, want, bound, what=""):
    err = np.abs(f64(got) - want)
    assert (err <= bound).all(), (what, float((err / bound).max()))


def ok(gdn, error):
    assert gdn.check_error(error) == 0


@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("lens,D", [([1], 4096), ([1], 4095), ([1] * 4, 4096), (None, 4096),
                                    (None, 4095)])
def test_a_gate_is_as_exact_as_stated(gdn, lens, D, complement):
    """One token with x = 0 from h0 = 1 returns its decay: A = a, B = 0, h = fma(a, 1, 0).
    Tiles, rows no tensor map describes, short sequences and the decode step (None)."""
    r = np.random.default_rng(5)
    size = 10.0 ** r.uniform(-7, 2, (4, D))
    size[:, ::3] = r.uniform(0, 0.6, size[:, ::3].shape)    # slow gates, and the forms' borders
    g = torch.from_numpy(-size).float()
    g[:, 1::7] = -g[:, 1::7].clamp(min=-0.45)               # some of them growing
    g = g[:len(lens) if lens else 4].cuda().contiguous()
    N = g.shape[0]
    x = torch.zeros_like(g)
    one = torch.ones((N, D), device="cuda")
    if lens:
        a, fin, _, err = gdn.glr_forward(x, g, W.cu_seqlens_of(lens, "cuda"), h0=one,
                                         complement=complement)
        ok(gdn, err)
        assert torch.equal(a, fin)
    else:
        state = gdn.GlrDecodeState(N, D)
        state.h.copy_(one)
        a = gdn.glr_decode_step(state, x, g, complement=complement)
        ok(gdn, state.error)
    want = np.exp(f64(g))
    bound = want * glr.decay_bound(f64(g), complement) * 1.01
    bound = np.where(want < 2.0 ** -125, want, bound)       # a below 2^-126 counts as 0
    close(a, want, bound)
    if not complement:      # half a step towards 0, where a state lives long
        slow = (f64(g) < 0) & (f64(g) > -0.125)
        err = np.abs(f64(a) - want) / want
        assert slow.sum() > 100 and err[slow].max() <= 0.8 * 2.0 ** -24


@pytest.mark.parametrize("complement", [False, True])
def test_slow_gates_over_a_long_sequence(gdn, complement):
    """States that live for 10^2 to 10^5 tokens: the sums take a gate's error up as often."""
    T, D = 30000, 8
    r = torch.Generator().manual_seed(9)
    x = (1 + 0.5 * torch.randn((T, D), generator=r)).cuda()
    rate = torch.tensor([1e-2, 1e-3, 3e-4, 1e-4, 7e-5, 3e-5, 1.1e-5, 0.06])
    g = (-rate).expand(T, D).contiguous().cuda()
    dh = torch.randn((T, D), generator=r).cuda()
    cu = W.cu_seqlens_of([T], "cuda")
    h, fin, carry, err = gdn.glr_forward(x, g, cu, complement=complement, want_carry=True)
    ok(gdn, err)
    args = (f64(x), f64(g), [T])
    close(h, glr.forward(*args, None, complement)[0],
          glr.forward_bound(*args, None, complement)[0], "h")
    grads, err = gdn.glr_backward(x, g, cu, carry, dh, complement=complement)
    ok(gdn, err)
    want = glr.backward(*args, f64(dh), complement=complement)
    bound = glr.backward_bound(*args, f64(dh), complement=complement)
    for got, w, b in zip((grads["dx"], grads["dg"], grads["dh0"]), want, bound):
        close(got, w, b)


@pytest.mark.parametrize("have", [(), ("dx",), ("dg",), ("dh0",), ("dx", "dg")])
def test_gradient_buffers_that_are_not_given_are_made(gdn, have):
    x, g, dh, h0, ds, cu = draw([20, 5], 64, 12)
    _, _, carry, _ = gdn.glr_forward(x, g, cu, h0=h0, want_carry=True)
    want, _ = gdn.glr_backward(x, g, cu, carry, dh, ds_final=ds)
    buf = {k: torch.empty_like(want[k]) for k in have}
    mine = dict(buf)
    got, _ = gdn.glr_backward(x, g, cu, carry, dh, ds_final=ds, grads=buf)
    assert got is buf and set(got) == {"dx", "dg", "dh0"}
    assert all(got[k] is mine[k] for k in have)
    assert all(torch.equal(got[k], want[k]) for k in want)
    got, _ = gdn.glr_backward(x, g, cu, carry, dh, grads={"dh0": None}, want_dh0=False)
    assert got["dh0"] is None and got["dg"] is not None


UNEQUAL = {  # mostly short sequences, some far longer: both kinds of kernels in one call
    "one": ([1] * 40 + [3600] + [2] * 59, 512),
    "borders": ([512, 3] * 2 + [513, 1024, 0, 1025, 511] + [1] * 80, 512),
    "first and last": ([1500] + [0] * 60 + [7] * 9 + [2100], 1024),
    "rows off 16 bytes": ([5] * 30 + [2000, 0, 1300] + [9] * 70, 257),
    "many": (([0, 1, 3, 2] * 300 + [3000]) * 3 + [600, 1030] + [4] * 200, 64),
}


@pytest.mark.parametrize("name", list(UNEQUAL))
@pytest.mark.parametrize("complement", [False, True])
def test_unequal_sequences(gdn, name, complement):
    """Bits of sequences alone, final and decode states, and the oracle."""
    lens, D = UNEQUAL[name]
    N = len(lens)
    x, g, dh, h0, ds, cu = draw(lens, D, 81)
    slots = torch.arange(N, dtype=torch.int32, device="cuda").flip(0).contiguous()
    state = gdn.GlrDecodeState(N, D)
    kw = dict(complement=complement)
    fill = torch.full((sum(lens), D), float("nan"), dtype=BF, device="cuda")
    h, fin, carry, err = gdn.glr_forward(x, g, cu, h0=h0, state=state, slot_idx=slots, h=fill,
                                         want_carry=True, **kw)
    ok(gdn, err)
    ok(gdn, state.error)
    assert state.pos.flip(0).tolist() == [n % 16 for n in lens]
    grads, err = gdn.glr_backward(x, g, cu, carry, dh, ds_final=ds, **kw)
    ok(gdn, err)
    edges = cu.tolist()
    order = sorted(range(N), key=lambda n: -lens[n])
    for n in order[:6] + order[-2:] + [order[N // 2]]:
        rows = slice(edges[n], edges[n + 1])
        one = gdn.GlrDecodeState(1, D)
        c = W.cu_seqlens_of([lens[n]], "cuda")
        h1, f1, c1, _ = gdn.glr_forward(x[rows], g[rows], c, h0=h0[n:n + 1], state=one,
                                        want_carry=True, **kw)
        g1, _ = gdn.glr_backward(x[rows], g[rows], c, c1, dh[rows], ds_final=ds[n:n + 1], **kw)
        assert torch.equal(h1, h[rows]) and torch.equal(f1[0], fin[n]), n
        assert torch.equal(g1["dx"], grads["dx"][rows]) and torch.equal(g1["dg"],
                                                                        grads["dg"][rows]), n
        assert torch.equal(g1["dh0"][0], grads["dh0"][n]), n
        assert all(torch.equal(a[0], b[N - 1 - n]) for a, b in zip(one.tensors(),
                                                                   state.tensors())), n
    ch = [0, D - 1]
    args = (f64(x[:, ch]), f64(g[:, ch]), lens)
    init = f64(h0[:, ch])
    want, wfin = glr.forward(*args, init, complement)
    bound, bfin = glr.forward_bound(*args, init, complement)
    close(h[:, ch], want, bound + 2.0 ** -8 * (np.abs(want) + bound), "h")
    close(fin[:, ch], wfin, bfin, "s_final")
    want = glr.backward(*args, f64(dh[:, ch]), init, f64(ds[:, ch]), complement)
    bound = glr.backward_bound(*args, f64(dh[:, ch]), init, f64(ds[:, ch]), complement)
    close(grads["dx"][:, ch], want[0], bound[0] + 2.0 ** -8 * (np.abs(want[0]) + bound[0]), "dx")
    close(grads["dg"][:, ch], want[1], bound[1], "dg")
    close(grads["dh0"][:, ch], want[2], bound[2], "dh0")


def test_unequal_sequences_captured_and_on_a_side_stream(gdn):
    lens, D = UNEQUAL["first and last"]
    x, g, dh, h0, ds, cu = draw(lens, D, 82)

    def both():
        h, fin, carry, _ = gdn.glr_forward(x, g, cu, h0=h0, want_carry=True)
        grads, err = gdn.glr_backward(x, g, cu, carry, dh, ds_final=ds)
        return h, fin, grads["dx"], grads["dg"], grads["dh0"], err, h.float() + 1

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(20):
            got = both()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    x.neg_()
    dh.mul_(2)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, both()))


def test_a_long_sequence_among_short_ones_is_not_walked_by_one_thread(gdn):
    """Within four times the same sequence alone (1.5 measured; a walk by one thread for
    each channel takes 8 times as long forward and 17 backward)."""
    D, L = 4096, 3968
    x, g, dh, h0, ds, cu = draw([1] * 40 + [L] + [1] * 23, D, 83)

    def best(x, g, dh, h0, ds, cu):
        _, _, carry, err = gdn.glr_forward(x, g, cu, h0=h0, want_carry=True)
        grads, _ = gdn.glr_backward(x, g, cu, carry, dh, ds_final=ds)
        kw = dict(h=dh.clone(), s_final=ds.clone(), error=err)
        calls = (lambda: gdn.glr_forward(x, g, cu, h0=h0, carry=carry, **kw),
                 lambda: gdn.glr_backward(x, g, cu, carry, dh, ds_final=ds, grads=grads,
                                          error=err))
        out = []
        for call in calls:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                for _ in range(5):
                    call()
            times = []
            for _ in range(7):
                a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
                a.record()
                graph.replay()
                b.record()
                b.synchronize()
                times.append(a.elapsed_time(b))
            out.append(min(times))
        return out

    among = best(x, g, dh, h0, ds, cu)
    rows = slice(40, 40 + L)
    alone = best(x[rows], g[rows], dh[rows], h0[:1], ds[:1], W.cu_seqlens_of([L], "cuda"))
    assert among[0] < 4 * alone[0] and among[1] < 4 * alone[1], (among, alone)


@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("lens,D", [([40], 64), ([40], 33), ([40] * 64, 256)])
def test_gates_that_grow_up_to_the_stated_sum(gdn, lens, D, complement):
    """A chunk whose gates sum to 88 (A = 1.65e38), one that takes it back, then a
    reset: exact within the bounds, states of zero stay zero, and the decode steps
    follow."""
    N, L = len(lens), lens[0]
    g = torch.zeros((L, D))
    g[:16], g[16:32], g[32:] = 5.5, -5.5, -0.5
    g[36] = float("-inf")
    g = g.repeat(N, 1).cuda()
    x = torch.zeros_like(g)
    h0 = torch.linspace(-1e-3, 1e-3, N * D).reshape(N, D).cuda()
    h0[:, 5] = 0
    x[:, 7:] = h0.repeat_interleave(L, 0)[:, 7:]
    cu = W.cu_seqlens_of(lens, "cuda")
    h, fin, carry, err = gdn.glr_forward(x, g, cu, h0=h0, complement=complement, want_carry=True)
    ok(gdn, err)
    args = (f64(x), f64(g), lens, f64(h0), complement)
    assert not h[:, 5].any() and not fin[:, 5].any()
    close(h, glr.forward(*args)[0], glr.forward_bound(*args)[0])
    dh = torch.zeros_like(x)
    dh[::7] = 1
    grads, err = gdn.glr_backward(x, g, cu, carry, dh, complement=complement)
    ok(gdn, err)
    args = (*args[:3], f64(dh), f64(h0), None, complement)
    for got, w, b in zip(grads.values(), glr.backward(*args), glr.backward_bound(*args)):
        close(got, w, b)
    state = gdn.GlrDecodeState(N, D)
    state.h.copy_(h0)
    first = cu[:-1].long()
    for t in range(L):
        step = gdn.glr_decode_step(state, x[first + t], g[first + t], complement=complement)
        assert torch.equal(step, h[first + t]), t


@pytest.mark.parametrize("lens,D", [([40, 0, 60], 96), ([40, 0, 60], 97),     # tiles
                                    ([9, 5] * 60, 512), ([9, 5] * 60, 257),   # short
                                    ([3] * 50 + [1500] + [2] * 50, 512)])     # both
@pytest.mark.parametrize("how", ["overlap", "falls", "starts late", "ends early", "ends late",
                                 "negative", "far out", "all alike"])
def test_invalid_cu_seqlens_are_reported_and_stay_inside(gdn, lens, D, how):
    """The error word is set, nothing around the outputs is written, and the next call
    clears the word and is right."""
    x, g, dh, h0, ds, cu = draw(lens, D, 84)
    T, N = x.shape[0], len(lens)
    bad = cu.tolist()
    m = max(2, N // 2)
    if how == "overlap":    # (at an edge behind a sequence that has tokens: not valid)
        assert bad[m - 1] > 0
        bad[m] = 0
    elif how == "falls":
        bad[m] = bad[m + 1] + 1
    elif how == "starts late":
        bad[0] = 1
    elif how == "ends early":
        bad[N] = T - 1
    elif how == "ends late":
        bad[N] = T + 1
    elif how == "negative":
        bad[1] = -5
    elif how == "far out":
        bad[m] = 2 ** 31 - 1
    else:
        bad = [T // 2] * (N + 1)
    bad = torch.tensor(bad, dtype=torch.int32, device="cuda")

    def guarded(shape, dtype):
        whole = torch.full((shape[0] + 4, shape[1]), 7.0, dtype=dtype, device="cuda")
        return whole, whole[2:-2]
    rows = gdn.glr_carry_rows(N, T)
    bufs = [guarded(s, d) for s, d in (((T, D), BF), ((N, D), F32), ((rows, D), F32),
                                       ((T, D), BF), ((T, D), F32), ((N, D), F32))]
    h, fin, carry, dx, dg, dh0 = (b[1] for b in bufs)
    state = gdn.GlrDecodeState(N, D)
    carry.zero_()   # (the rows of sequences that are left out are read by the backward)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.glr_forward(x, g, bad, h0=h0, h=h, s_final=fin, carry=carry, state=state, error=err)
    assert gdn.check_error(err) == gdn.GDN_DEVERR_CU_SEQLENS
    err.zero_()
    gdn.glr_backward(x, g, bad, carry, dh, ds_final=ds, error=err,
                     grads={"dx": dx, "dg": dg, "dh0": dh0})
    assert gdn.check_error(err) == gdn.GDN_DEVERR_CU_SEQLENS
    for whole, _ in bufs:
        assert (whole[:2] == 7).all() and (whole[-2:] == 7).all()
    assert state.pos.min() >= 0 and state.pos.max() < 16
    want = gdn.glr_forward(x, g, cu, h0=h0)[0]
    gdn.glr_forward(x, g, cu, h0=h0, h=h, s_final=fin, carry=carry, error=err)
    ok(gdn, err)
    assert torch.equal(h, want)


@pytest.mark.parametrize("D", [64, 63])
@pytest.mark.parametrize("L", [5000, 129])
def test_a_sequence_alone_has_the_bits_of_any_cluster_size(gdn, L, D):
    """Alone, a sequence of 64 channels is taken by clusters of 8 blocks forward and 4
    backward (2 of them for its 129 tokens); among 300 others of 130 tokens by one
    block, among 49 by two, among 19 of 300 by four or eight.  All outputs, and the
    oracle for all of them."""
    x, g, dh, h0, ds, cu = draw([L], D, 85)

    def both(x, g, dh, h0, ds, cu):
        h, fin, carry, err = gdn.glr_forward(x, g, cu, h0=h0, want_carry=True, out_dtype=F32)
        ok(gdn, err)
        grads, err = gdn.glr_backward(x, g, cu, carry, dh, ds_final=ds)
        ok(gdn, err)
        return h, fin, grads["dx"], grads["dg"], grads["dh0"]

    alone = both(x, g, dh, h0, ds, cu)
    for length, n in ((130, 300), (130, 49), (300, 19)):
        for at in (0, n // 2, n):
            lens = [length] * at + [L] + [length] * (n - at)
            others = draw(lens, D, 86)[:5]
            start = length * at
            for mine, t in zip((x, g, dh), others):
                t[start:start + L] = mine
            others[3][at], others[4][at] = h0[0], ds[0]
            got = both(*others, W.cu_seqlens_of(lens, "cuda"))
            rows = slice(start, start + L)
            want = (got[0][rows], got[1][at:at + 1], got[2][rows], got[3][rows],
                    got[4][at:at + 1])
            assert all(torch.equal(a, b) for a, b in zip(alone, want)), (length, n, at)
    args = (f64(x), f64(g), [L])
    for got, w, b in zip(alone[:2], glr.forward(*args, f64(h0)),
                         glr.forward_bound(*args, f64(h0))):
        close(got, w, b)
    want = glr.backward(*args, f64(dh), f64(h0), f64(ds))
    bound = list(glr.backward_bound(*args, f64(dh), f64(h0), f64(ds)))
    bound[0] = bound[0] + 2.0 ** -8 * (np.abs(want[0]) + bound[0])
    for got, w, b in zip(alone[2:], want, bound):
        close(got, w, b)


@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("lens,D", [([130, 20, 300], 64), ([130, 20, 300], 61), ([5000, 3], 64),
                                    ([5, 20, 17] * 40, 512),
                                    ([3, 2] * 40 + [1300] + [2] * 40, 512)])
def test_what_lies_behind_a_sequence_does_not_matter(gdn, lens, D, complement):
    """NaN and infinities in every second sequence, which a tile's copies bring in with
    the first's last tokens, in the rows behind the batch and in the columns beside it."""
    x, g, dh, h0, ds, cu = draw(lens, D, 87)
    edges = cu.tolist()
    T = edges[-1]
    kw = dict(complement=complement)

    def both(x, g, dh):
        h, fin, carry, err = gdn.glr_forward(x, g, cu, h0=h0, want_carry=True, **kw)
        ok(gdn, err)
        grads, err = gdn.glr_backward(x, g, cu, carry, dh, ds_final=ds, **kw)
        ok(gdn, err)
        return (h, grads["dx"], grads["dg"]), (fin, grads["dh0"])

    want_tok, want_seq = both(x, g, dh)
    wide = []
    for t, junk in ((x, float("nan")), (g, float("nan")), (dh, float("inf"))):
        w = torch.full((T + 140, D + 64), junk, dtype=t.dtype, device="cuda")
        w[:T, 16:16 + D] = t
        for n in range(1, len(lens), 2):
            w[edges[n]:edges[n + 1]] = junk
        wide.append(w[:T, 16:16 + D])
    tok, seq = both(*wide)
    for n in range(0, len(lens), 2):
        rows = slice(edges[n], edges[n + 1])
        assert all(torch.equal(a[rows], b[rows]) for a, b in zip(tok, want_tok)), n
        assert all(torch.equal(a[n], b[n]) for a, b in zip(seq, want_seq)), n


@pytest.mark.parametrize("D", [64, 63])
def test_offsets_beyond_32_bits(gdn, D):
    """Rows 2^20 elements apart: from row 2048 on an element's offset passes 2^31, in the
    inputs and in the outputs."""
    T, lens = 2100, [900, 1200]
    wide = torch.empty((T, 1 << 20), dtype=BF, device="cuda")
    x, g, dh, h0, ds, cu = draw(lens, D, 88, gt=BF)
    cols = [wide[:, 64 * i:64 * i + D] for i in range(6)]
    for c, t in zip(cols, (x, g, dh)):
        c.copy_(t)
    for c in cols[3:]:
        c.fill_(7)
    h, fin, carry, err = gdn.glr_forward(x, g, cu, h0=h0, want_carry=True)
    grads, _ = gdn.glr_backward(x, g, cu, carry, dh, ds_final=ds)
    got, fin2, carry2, err = gdn.glr_forward(cols[0], cols[1], cu, h0=h0, h=cols[3],
                                             want_carry=True)
    ok(gdn, err)
    out, err = gdn.glr_backward(cols[0], cols[1], cu, carry2, cols[2], ds_final=ds,
                                grads={"dx": cols[4], "dg": cols[5]})
    ok(gdn, err)
    assert torch.equal(got, h) and torch.equal(fin2, fin)
    assert all(torch.equal(out[k], grads[k]) for k in grads)


def test_decode_slots_beyond_32_bits(gdn):
    """A slot of 2^20 channels whose elements lie behind 2^31 others."""
    D, n = 1 << 20, 2060
    state = gdn.GlrDecodeState(n, D)
    small = gdn.GlrDecodeState(2, D)
    x, g, _, h0, _, _ = draw([2], D, 89)
    slots = torch.tensor([n - 1, 0], dtype=torch.int32, device="cuda")
    state.h[slots.long()] = h0.expand(2, D)
    small.h.copy_(h0.expand(2, D))
    for _ in range(2):
        a = gdn.glr_decode_step(state, x, g, slot_idx=slots)
        assert torch.equal(a, gdn.glr_decode_step(small, x, g))
    ok(gdn, state.error)
    assert all(torch.equal(big[slots.long()], s) for big, s in zip(state.tensors(),
                                                                   small.tensors()))


@pytest.mark.parametrize("D", [1, 2, 6, 30, 34])
def test_narrow_rows_of_a_wide_buffer(gdn, D):
    """Rows that start on 16 bytes, with fewer channels than a slab or a few more."""
    lens = [300, 1, 140]
    x, g, dh, h0, ds, cu = draw(lens, D, 90)
    T = x.shape[0]
    wide = [torch.full((T, 64), float("nan"), dtype=t.dtype, device="cuda") for t in (x, g, dh)]
    for w, t in zip(wide, (x, g, dh)):
        w[:, 8:8 + D] = t
    a = [w[:, 8:8 + D] for w in wide]
    h, fin, carry, err = gdn.glr_forward(a[0], a[1], cu, h0=h0, want_carry=True, out_dtype=F32)
    ok(gdn, err)
    grads, err = gdn.glr_backward(a[0], a[1], cu, carry, a[2], ds_final=ds)
    ok(gdn, err)
    args = (f64(x), f64(g), lens)
    for got, w, b in zip((h, fin), glr.forward(*args, f64(h0)),
                         glr.forward_bound(*args, f64(h0))):
        close(got, w, b)
    want = glr.backward(*args, f64(dh), f64(h0), f64(ds))
    bound = list(glr.backward_bound(*args, f64(dh), f64(h0), f64(ds)))
    bound[0] = bound[0] + 2.0 ** -8 * (np.abs(want[0]) + bound[0])
    for got, w, b in zip((grads["dx"], grads["dg"], grads["dh0"]), want, bound):
        close(got, w, b)


def test_some_of_a_longer_list_of_sequences(gdn):
    """n_seqs sequences at the front of a longer cu_seqlens."""
    x, g, dh, h0, ds, cu = draw([50, 7, 300, 20], 64, 91)
    T = 57
    h, fin, carry, err = gdn.glr_forward(x, g, cu, h0=h0, want_carry=True)
    part, fin2, carry2, err = gdn.glr_forward(x[:T], g[:T], cu, n_seqs=2, h0=h0[:2],
                                              want_carry=True)
    ok(gdn, err)
    assert torch.equal(part, h[:T]) and torch.equal(fin2, fin[:2])
    grads, err = gdn.glr_backward(x, g, cu, carry, dh, ds_final=ds)
    some, err = gdn.glr_backward(x[:T], g[:T], cu, carry2, dh[:T], n_seqs=2, ds_final=ds[:2])
    ok(gdn, err)
    assert torch.equal(some["dg"], grads["dg"][:T]) and torch.equal(some["dh0"], grads["dh0"][:2])
    with pytest.raises(ValueError, match="entries"):
        gdn.glr_forward(x, g, cu, n_seqs=5)
