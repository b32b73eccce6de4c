"""Cases that measure the library's q/k norm and its gated linear recurrence.

The two operators around the Gated DeltaNet layer that work on a layer's raw
projections:

* q/k norm: the norm of every head's query and key (l2 over the head, or root
  mean square with a weight), with the position rotation in the same pass.
* gated linear recurrence (glr): h_t = exp(g_t) h_{t-1} + b_t for each channel
  of packed sequences, b = x or (1 - exp(g)) x.

``run`` computes them in plain torch operations (``own`` false) or calls the
library (``own`` true); ``exact`` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

CHUNK = 16  # tokens after which a decode state is folded into its entry state


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _glr(op, tokens, seqs, width, split=0, dtype="bf16", g_dtype="f32", gates="softplus",
         complement=False, fused=True):
    """split 0: sequences of (nearly) equal length; otherwise the seed of random
    cuts, among them empty sequences.  fused: x and g are column blocks of one
    wider projection (of one type) or of their own wider buffers."""
    return dict(op=op, tokens=tokens, seqs=seqs, width=width, split=split, dtype=dtype,
                g_dtype=g_dtype, gates=gates, complement=complement, fused=fused)


def _qk(op, tokens, hq, hk, d, norm="l2", rot=0, interleaved=False, dtype="bf16", dy="f32",
        far=0, fused=True):
    """rot: rotated channels of a head; far: first position of the tokens (decode
    rows draw theirs up to it); fused: q and k are column blocks of one projection."""
    return dict(op=op, tokens=tokens, hq=hq, hk=hk, d=d, norm=norm, rot=rot,
                interleaved=interleaved, dtype=dtype, dy=dy, far=far, fused=fused)


def listed():
    def named(name, case):
        return dict(name=name, **case)
    return [
        # One sequence's next token in a latency-bound rollout: the smallest calls.
        named("glr_decode_1", _glr("glr_decode", 1, 1, 2048)),
        named("qk_decode_1", _qk("qk_forward", 1, 16, 16, 128)),
        # The rollout decode shape: 256 slots, far positions of a rotated head.
        named("glr_decode_256", _glr("glr_decode", 256, 256, 4096)),
        named("qk_decode_256", _qk("qk_forward", 256, 32, 8, 128, norm="rms", rot=64,
                                   far=131072)),
        # Rollout prefill of 5 x 2048 tokens, 16 heads of 128: what the layer's forward reads.
        named("qk_prefill", _qk("qk_forward", 10240, 16, 16, 128)),
        named("glr_prefill", _glr("glr_forward", 10240, 5, 2048)),
        # One long prompt alone: few channels beside its length.
        named("glr_long", _glr("glr_forward", 65536, 1, 2048, g_dtype="bf16", gates="long")),
        # Trainer step over 10240 tokens: forward and backward; the fp32 gradient of the
        # layer's q and k, or a bf16 one through rotation and weights.
        named("qk_train", _qk("qk_train", 10240, 16, 16, 128)),
        named("qk_train_rot", _qk("qk_train", 16384, 32, 8, 128, norm="rms", rot=128, dy="bf16")),
        named("glr_train", _glr("glr_train", 10240, 5, 2048, split=3)),
        # 64 ragged sequences with no-decay and reset gates, wide layer: the largest.
        named("glr_train_ragged", _glr("glr_train", 57344, 64, 4096, split=4, gates="stress",
                                       complement=True)),
        # Odd widths and fp32 data, as a small research model or a parity check has them.
        named("glr_train_odd", _glr("glr_train", 4099, 7, 1001, split=5, dtype="f32",
                                    fused=False)),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["glr_decode", "glr_forward", "glr_train", "qk_forward", "qk_train"])
    if op.startswith("glr"):
        width = _log(rng, 64, 4096)
        if rng.random() < 0.6:
            width = max(64, width // 64 * 64)
        tokens = _log(rng, 1, 512) if op == "glr_decode" else _log(rng, 1, 65536)
        tokens = min(tokens, 57344 * 4096 // width)
        seqs = tokens if op == "glr_decode" else _log(rng, 1, 64)
        return _glr(op, tokens, seqs, width, split=rng.choice([0, rng.randrange(1, 10 ** 6)]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]),
                    g_dtype=rng.choice(["f32", "f32", "bf16"]),
                    gates=rng.choice(["softplus", "stress", "long"]),
                    complement=rng.random() < 0.4, fused=rng.random() < 0.6)
    d = rng.choice([64, 128, 128, 256])
    hk = rng.choice([1, 2, 3, 4, 8, 16])
    hq = min(32, hk * rng.choice([1, 1, 2, 4, 5, 8]))
    tokens = min(_log(rng, 1, 32768), 16384 * 40 * 128 // ((hq + hk) * d))
    rot = rng.choice([0, d // 4, d // 2, d, rng.randrange(1, d // 16 + 1) * 16])
    return _qk(op, tokens, hq, hk, d, norm=rng.choice(["l2", "rms"]), rot=rot,
               interleaved=rng.random() < 0.3, dtype=rng.choice(["bf16", "bf16", "f32"]),
               dy=rng.choice(["f32", "bf16"]), far=rng.choice([0, 0, 8192, 131072, 1000000]),
               fused=rng.random() < 0.6)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}


def _lengths(case):
    T, N = case["tokens"], case["seqs"]
    if case["split"]:
        r = random.Random(case["split"])
        cuts = sorted(r.randint(0, T) for _ in range(N - 1))
    else:
        cuts = [T * (i + 1) // N for i in range(N - 1)]
    edges = [0] + cuts + [T]
    return [b - a for a, b in zip(edges, edges[1:])]


def _edges(lengths):
    edges = [0]
    for n in lengths:
        edges.append(edges[-1] + n)
    return edges


def _block(x, fused):
    """x [T, n], or the same values as a column block of a wider buffer."""
    if not fused:
        return x
    wide = torch.empty((x.shape[0], x.shape[1] + 64), dtype=x.dtype, device=x.device)
    wide[:, :x.shape[1]] = x
    return wide[:, :x.shape[1]]


def _gates(case, shape, gen, dev):
    z = torch.randn(shape, generator=gen, device=dev)
    if case["gates"] == "softplus":  # the layer's own gates
        return -torch.nn.functional.softplus(z)
    if case["gates"] == "long":      # decays of 0.9 to 0.9999 a token
        return -torch.exp(-4.5 + 1.5 * z.clamp(-3, 1.5))
    g = (-torch.nn.functional.softplus(2.5 * z)).clamp(min=-8.0)
    u = torch.rand(shape, generator=gen, device=dev)
    g = torch.where(u < 0.01, torch.full_like(g, -8.0), g)
    g = torch.where((u >= 0.01) & (u < 0.02), torch.full_like(g, -1e-7), g)
    return torch.where((u >= 0.02) & (u < 0.021), torch.full_like(g, -1e4), g)  # resets


def _prepare_glr(case, seed, dev):
    gen = torch.Generator(device=dev).manual_seed(seed)
    T, D = case["tokens"], case["width"]
    rand = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
    st = dict(case=case)
    st["x"] = _block(rand(T, D).to(_DT[case["dtype"]]), case["fused"])
    st["g"] = _block(_gates(case, (T, D), gen, dev).to(_DT[case["g_dtype"]]), case["fused"])
    if case["op"] == "glr_decode":
        pos = torch.randint(0, CHUNK, (T,), generator=gen, device=dev, dtype=torch.int32)
        started = (pos > 0)[:, None]
        st["pos"] = pos
        st["h_in"] = rand(T, D) * 0.7
        st["a_in"] = torch.where(started, torch.rand((T, D), generator=gen, device=dev),
                                 torch.ones((), device=dev))
        st["b_in"] = torch.where(started, rand(T, D) * 0.5, torch.zeros((), device=dev))
        if own:
            from rl_train_numerics_b200 import gdn
            s = gdn.GlrDecodeState(T, D, device=dev)
            s.h, s.a, s.b, s.pos = st["h_in"], st["a_in"], st["b_in"], st["pos"]
            st["state"] = s
        return st
    lengths = _lengths(case)
    st["edges"] = _edges(lengths)
    st["cu"] = torch.tensor(st["edges"], dtype=torch.int32, device=dev)
    st["h0"] = rand(len(lengths), D) * 0.5
    if case["op"] == "glr_train":
        st["dh"] = rand(T, D).to(_DT[case["dtype"]])
        st["ds"] = rand(len(lengths), D)
    return st


def _prepare_qk(case, seed, dev):
    gen = torch.Generator(device=dev).manual_seed(seed)
    T, hq, hk, d = case["tokens"], case["hq"], case["hk"], case["d"]
    rand = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
    dt = _DT[case["dtype"]]
    st = dict(case=case)
    # projections: channels of unequal size, tokens of unequal size
    size = (0.5 * rand(1, (hq + hk) * d)).exp() * (0.5 * rand(T, 1)).exp()
    y = (rand(T, (hq + hk) * d) * size).to(dt)
    if case["fused"]:
        st["q"], st["k"] = y[:, :hq * d], y[:, hq * d:]
    else:
        st["q"], st["k"] = y[:, :hq * d].contiguous(), y[:, hq * d:].contiguous()
    st["q"] = st["q"].unflatten(1, (hq, d))
    st["k"] = st["k"].unflatten(1, (hk, d))
    st["wq"] = st["wk"] = None
    if case["norm"] == "rms":
        st["wq"] = 1 + 0.2 * rand(d)
        st["wk"] = 1 + 0.2 * rand(d)
    st["positions"] = st["inv_freq"] = None
    if case["rot"]:
        if T <= 512 and case["far"]:  # decode rows: each at its own position
            pos = torch.randint(0, case["far"], (T,), generator=gen, device=dev)
        else:
            pos = case["far"] + torch.arange(T, device=dev) % 8192
        st["positions"] = pos.to(torch.int32)
        F = case["rot"] // 2
        st["inv_freq"] = (10000.0 ** (-torch.arange(F, device=dev, dtype=torch.float64) / F)
                          ).float()
    if case["op"] == "qk_train":
        st["dq"] = rand(T, hq, d).to(_DT[case["dy"]])
        st["dk"] = rand(T, hk, d).to(_DT[case["dy"]])
    return st


def prepare(case, seed):
    dev = torch.device("cuda")
    make = _prepare_glr if case["op"].startswith("glr") else _prepare_qk
    return make(case, seed, dev)


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t down the rows from h = 0, by doubling: after the
    pass of stride s every row holds the composition of its last 2s steps."""
    T, s = a.shape[0], 1
    while s < T:
        b = torch.cat([b[:s], b[s:] + a[s:] * b[:-s]])
        if 2 * s < T:
            a = torch.cat([a[:s], a[s:] * a[:-s]])
        s *= 2
    return b


def _gate_plain(x, g, complement):
    x, g = x.float(), g.float()
    a = torch.exp(g)
    return x, a, (-torch.expm1(g) if complement else None)


def _glr_forward_plain(st):
    case = st["case"]
    x, a, c = _gate_plain(st["x"], st["g"], case["complement"])
    b = x if c is None else c * x
    cu = st["cu"].long()
    first = cu[:-1][cu[1:] > cu[:-1]]
    h0 = st["h0"][cu[1:] > cu[:-1]]
    ar = a.clone()
    ar[first] = 0.0                      # nothing crosses a sequence's first token
    b = b.clone()
    b[first] += a[first] * h0
    h = _scan(ar, b)
    fin = st["h0"].clone()
    fin[cu[1:] > cu[:-1]] = h[cu[1:][cu[1:] > cu[:-1]] - 1]
    return x, a, c, h, fin, ar


def _glr_train_plain(st):
    case = st["case"]
    x, a, c, h, fin, ar = _glr_forward_plain(st)
    cu = st["cu"].long()
    some = cu[1:] > cu[:-1]
    first, last = cu[:-1][some], cu[1:][some] - 1
    dh = st["dh"].float().clone()
    dh[last] += st["ds"][some]
    # lam_t = dh_t + a_{t+1} lam_{t+1}: the same scan, rows reversed
    nxt = torch.cat([ar[1:], torch.zeros_like(ar[:1])])
    lam = _scan(nxt.flip(0), dh.flip(0)).flip(0)
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    before[first] = st["h0"][some]
    mu = a * lam
    dh0 = st["ds"].clone()
    dh0[some] = mu[first]
    if c is None:
        dx, dg = lam, mu * before
    else:
        dx, dg = lam * c, mu * (before - x)
    dt = _DT[case["dtype"]]
    return dict(h=h.to(dt), s_final=fin, dx=dx.to(dt), dg=dg.to(_DT[case["g_dtype"]]), dh0=dh0)


def _glr_decode_plain(st):
    case = st["case"]
    x, a, c = _gate_plain(st["x"], st["g"], case["complement"])
    b = x if c is None else c * x
    H, A, B, pos = st["h_in"], st["a_in"], st["b_in"], st["pos"]
    A2, B2 = a * A, a * B + b
    h = A2 * H + B2
    full = (pos == CHUNK - 1)[:, None]
    H.copy_(torch.where(full, h, H))
    A.copy_(torch.where(full, torch.ones((), device=h.device), A2))
    B.copy_(torch.where(full, torch.zeros((), device=h.device), B2))
    pos.copy_((pos + 1) % CHUNK)
    return dict(h=h.to(_DT[case["dtype"]]), state_h=H, state_a=A, state_b=B, pos=pos)


def _angles(st):
    ang = st["positions"].double()[:, None] * st["inv_freq"].double()
    return torch.cos(ang).float()[:, None, :], torch.sin(ang).float()[:, None, :]


def _rotate(n, cos, sin, interleaved):
    F = cos.shape[-1]
    y = n.clone()
    if interleaved:
        u, v = n[..., 0:2 * F:2], n[..., 1:2 * F:2]
        y[..., 0:2 * F:2] = u * cos - v * sin
        y[..., 1:2 * F:2] = v * cos + u * sin
    else:
        u, v = n[..., :F], n[..., F:2 * F]
        y[..., :F] = u * cos - v * sin
        y[..., F:2 * F] = v * cos + u * sin
    return y


EPS = 1e-6


def _qk_plain(st):
    case = st["case"]
    train = case["op"] == "qk_train"
    out = {}
    rot = _angles(st) if case["rot"] else None
    for s in ("q", "k"):
        x = st[s].float()
        w = st["w" + s]
        m = (lambda v: v.mean(-1, keepdim=True)) if case["norm"] == "rms" else \
            (lambda v: v.sum(-1, keepdim=True))
        r = torch.rsqrt(m(x * x) + EPS)
        n = x * r if w is None else x * r * w
        y = n if rot is None else _rotate(n, rot[0], rot[1], case["interleaved"])
        out["o" + s] = y.to(_DT[case["dtype"]])
        if not train:
            continue
        dn = st["d" + s].float()
        if rot is not None:
            dn = _rotate(dn, rot[0], -rot[1], case["interleaved"])
        e = dn if w is None else dn * w
        out["d" + s] = (r * (e - x * (r * r * m(x * e)))).to(_DT[case["dtype"]])
        if w is not None:
            out["dw" + s] = (dn * x * r).sum((0, 1))
    return out


# ---------------------------------------------------------------------------
# The library's operators
# ---------------------------------------------------------------------------

def _run_own(st):
    from rl_train_numerics_b200 import gdn
    case = st["case"]
    op = case["op"]
    if op == "glr_decode":
        s = st["state"]
        h = gdn.glr_decode_step(s, st["x"], st["g"], complement=case["complement"])
        return dict(h=h, state_h=s.h, state_a=s.a, state_b=s.b, pos=s.pos)
    if op.startswith("glr"):
        train = op == "glr_train"
        h, fin, carry, _ = gdn.glr_forward(st["x"], st["g"], st["cu"], h0=st["h0"],
                                           complement=case["complement"], want_carry=train)
        if not train:
            return dict(h=h, s_final=fin)
        grads, _ = gdn.glr_backward(st["x"], st["g"], st["cu"], carry, st["dh"],
                                    ds_final=st["ds"], complement=case["complement"])
        return dict(h=h, s_final=fin, dx=grads["dx"], dg=grads["dg"], dh0=grads["dh0"])
    kw = dict(norm=case["norm"], eps=EPS, wq=st["wq"], wk=st["wk"], positions=st["positions"],
              inv_freq=st["inv_freq"], interleaved=case["interleaved"])
    oq, ok = gdn.qk_norm_forward(st["q"], st["k"], **kw)
    if op == "qk_forward":
        return dict(oq=oq, ok=ok)
    grads = gdn.qk_norm_backward(st["q"], st["k"], st["dq"], st["dk"], **kw)
    out = {}
    for s, y in (("q", oq), ("k", ok)):
        out["o" + s], out["d" + s] = y, grads["d" + s]
        if case["norm"] == "rms":
            out["dw" + s] = grads["dw" + s]
    return out


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "glr_decode":
        return _glr_decode_plain(state)
    if op == "glr_forward":
        _, _, _, h, fin, _ = _glr_forward_plain(state)
        return dict(h=h.to(_DT[state["case"]["dtype"]]), s_final=fin)
    if op == "glr_train":
        return _glr_train_plain(state)
    return _qk_plain(state)


# ---------------------------------------------------------------------------
# Work
# ---------------------------------------------------------------------------

def work(case):
    T = case["tokens"]
    if case["op"].startswith("glr"):
        D = case["width"]
        n, sx, sg = T * D, _SIZE[case["dtype"]], _SIZE[case["g_dtype"]]
        if case["op"] == "glr_decode":
            return dict(bytes=n * (sx + sg + 12 + sx + 8), flops=7 * n)
        rows = case["seqs"] * D * 4
        if case["op"] == "glr_forward":
            return dict(bytes=n * (2 * sx + sg) + 2 * rows, flops=4 * n)
        # the forward, then the backward, which reads x, g, dh and writes dx, dg
        return dict(bytes=n * (2 * sx + sg) + n * (3 * sx + 2 * sg) + 4 * rows, flops=12 * n)
    n, sx = T * (case["hq"] + case["hk"]) * case["d"], _SIZE[case["dtype"]]
    fwd = n * 2 * sx + T * 4 * (1 if case["rot"] else 0)
    if case["op"] == "qk_forward":
        return dict(bytes=fwd, flops=8 * n)
    return dict(bytes=fwd + n * (2 * sx + _SIZE[case["dy"]]), flops=24 * n)


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def _exact_glr(case, st):
    x, g = st["x"].double(), st["g"].double()
    a = torch.exp(g)
    gain = -torch.expm1(g) if case["complement"] else torch.ones_like(g)
    if case["op"] == "glr_decode":
        # a row's state is A H + B; a row that fills its chunk starts a new one
        A, B = a * st["a_in"].double(), a * st["b_in"].double() + gain * x
        h = A * st["h_in"].double() + B
        fills = [int(p) == CHUNK - 1 for p in st["pos"].cpu()]
        H = st["h_in"].double().clone()
        for i, f in enumerate(fills):
            if f:
                H[i], A[i], B[i] = h[i], 1.0, 0.0
        pos = torch.tensor([0 if f else int(p) + 1 for f, p in zip(fills, st["pos"].cpu())],
                           dtype=torch.int32, device=x.device)
        return dict(h=h, state_h=H, state_a=A, state_b=B, pos=pos)
    # token by token, every sequence that is long enough at once (longest first)
    edges = st["edges"]
    N = len(edges) - 1
    lens = [edges[i + 1] - edges[i] for i in range(N)]
    order = sorted(range(N), key=lambda i: -lens[i])
    start = torch.tensor([edges[i] for i in order], device=x.device)
    perm = torch.tensor(order, device=x.device)
    longest = lens[order[0]]
    alive = [N] * longest
    count = N
    for t in range(longest):
        while count and lens[order[count - 1]] <= t:
            count -= 1
        alive[t] = count
    prev = torch.empty_like(x)           # the state before each token
    h = torch.empty_like(x)
    s = st["h0"].double()[perm].clone()
    for t in range(longest):
        m = alive[t]
        rows = start[:m] + t
        prev[rows] = s[:m]
        s[:m] = a[rows] * s[:m] + gain[rows] * x[rows]
        h[rows] = s[:m]
    fin = torch.empty_like(s)
    fin[perm] = s
    out = dict(h=h, s_final=fin)
    if case["op"] == "glr_forward":
        return out
    dh = st["dh"].double()
    u = st["ds"].double()[perm].clone()
    dx, dg = torch.empty_like(x), torch.empty_like(x)
    for t in reversed(range(longest)):
        m = alive[t]
        rows = start[:m] + t
        u[:m] += dh[rows]
        dx[rows] = u[:m] * gain[rows]
        carried = prev[rows] - x[rows] if case["complement"] else prev[rows]
        u[:m] *= a[rows]
        dg[rows] = u[:m] * carried
    dh0 = torch.empty_like(u)
    dh0[perm] = u
    out.update(dx=dx, dg=dg, dh0=dh0)
    return out


def _exact_qk(case, st):
    out = {}
    d, R = case["d"], case["rot"]
    turn = None
    if R:
        # each rotated pair as one complex number
        F = R // 2
        phase = torch.outer(st["positions"].double(), st["inv_freq"].double())
        turn = torch.polar(torch.ones_like(phase), phase)[:, None, :]
        ch = torch.arange(R, device=phase.device)
        re, im = (ch[0::2], ch[1::2]) if case["interleaved"] else (ch[:F], ch[F:])

    def spin(v, by):
        z = torch.complex(v[..., re], v[..., im]) * by
        v = v.clone()
        v[..., re], v[..., im] = z.real, z.imag
        return v

    for s in ("q", "k"):
        x = st[s].double()
        div = d if case["norm"] == "rms" else 1
        length = torch.sqrt((x ** 2).sum(-1, keepdim=True) / div + EPS)
        unit = x / length
        w = torch.ones(d, dtype=torch.float64, device=x.device) if st["w" + s] is None \
            else st["w" + s].double()
        y = unit * w
        out["o" + s] = spin(y, turn) if R else y
        if case["op"] != "qk_train":
            continue
        back = st["d" + s].double()
        if R:
            back = spin(back, turn.conj())
        along = (unit * back * w).sum(-1, keepdim=True) / div
        out["d" + s] = (back * w - unit * along) / length
        if st["w" + s] is not None:
            out["dw" + s] = torch.einsum("thd,thd->d", back, unit)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_glr(case, st) if case["op"].startswith("glr") else _exact_qk(case, st)
