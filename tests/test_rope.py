"""Rotary positions with several axes, alone and behind the per-head RMSNorm
(rmsnorm_rope_fwd / rmsnorm_rope_bwd), against a plain evaluation in 64 bits.

Tolerances, with u = 2^-24 (half a step of fp32):
  * A sine or cosine is off by at most pi 2^-25 (the angle, a fraction of half a
    turn below 1, rounded to fp32) plus 2^-23 (two units in the last place of
    sincospif): below 2^-22.  A rotated value is two products and a sum: with its
    roundings (2 u each of |u| + |v|) the error is below TURN = 2^-21 times |u| + |v|,
    the magnitudes of its pair.
  * A normed value x rstd gamma: the sum of squares of positive terms is off by at
    most depth u relative, depth <= 32 (terms per lane, then shuffles; the scalar
    form: D / threads, shuffles, 8 warps), half of it in rstd, and six roundings
    more: below NORM = 2^-19 relative.
  * dx = r (gamma g - x c): each of the two terms within TURN + NORM of its
    magnitude, where |g| is bounded by the pair's magnitude G = |dyu| + |dyv| and c by
    C = r^2 / D sum gamma G |x|, whose sum carries another depth u.
  * dgamma = sum over n rows of g x r: every term within TURN + NORM of G |x| r, and a
    sum of n terms in any order within (n - 1) u of the sum of the magnitudes.
  * bf16 outputs add half a step of the rounded value, 2^-8 relative.
"""
import numpy as np
import pytest
import torch

import row_wise_normalization_02_gb300 as rn

gpu = pytest.mark.gpu
TD = {"bf16": torch.bfloat16, "f32": torch.float32}
TURN, NORM, U = 2.0 ** -21, 2.0 ** -19, 2.0 ** -24
FAKE = 1 << 40


def half_step(dt):
    return torch.finfo(TD[dt]).eps / 2


# ---------------------------------------------------------------- 64-bit reference

def axis_of(i, sections, order):
    if order == "interleaved":
        a = i % len(sections)
        return a if i < sections[a] * len(sections) else 0
    return int(np.searchsorted(np.cumsum(sections), i, side="right"))


def angles(positions, inv_freq, sections, order):
    """[T, R / 2] cosines and sines, the products in extended precision."""
    p = positions.astype(np.longdouble)
    f = inv_freq.astype(np.longdouble)
    th = np.stack([p[axis_of(i, sections, order)] * f[i] for i in range(len(f))], -1)
    return np.cos(th).astype(np.float64), np.sin(th).astype(np.float64)


def split(x, R, pairs):
    return ((x[..., :R // 2], x[..., R // 2:R]) if pairs == "halves" else
            (x[..., 0:R:2], x[..., 1:R:2]))


def turn(x, cos, sin, R, pairs):
    y = x.copy()
    u, v = split(x, R, pairs)
    yu, yv = split(y, R, pairs)
    yu[...] = u * cos[:, None] - v * sin[:, None]
    yv[...] = u * sin[:, None] + v * cos[:, None]
    return y


def magnitude(x, R, pairs):
    """|u| + |v| of each element's pair, |x| of the columns that do not turn."""
    m = np.abs(x)
    u, v = split(m, R, pairs)
    s = u + v
    u[...], v[...] = s, s
    return m


def ref_fwd(x, gamma, eps, cos, sin, R, pairs):
    z, slack = x, TURN
    if gamma is not None:
        z = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * gamma
        slack += NORM
    return turn(z, cos, sin, R, pairs), slack * magnitude(z, R, pairs)


def ref_bwd(dy, x, gamma, eps, cos, sin, R, pairs):
    g, G = turn(dy, cos, -sin, R, pairs), magnitude(dy, R, pairs)
    if gamma is None:
        return g, TURN * G, None, None
    D = x.shape[-1]
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    c = r * r / D * (gamma * g * x).sum(-1, keepdims=True)
    C = r * r / D * (np.abs(gamma) * G * np.abs(x)).sum(-1, keepdims=True)
    dx = r * (gamma * g - x * c)
    tol = (TURN + NORM) * r * (np.abs(gamma) * G + 2 * np.abs(x) * C)
    term = g * x * r
    n = term.shape[0] * term.shape[1]
    return dx, tol, term.sum((0, 1)), (TURN + NORM + n * U) * (G * np.abs(x) * r).sum((0, 1))


# ---------------------------------------------------------------- a case on the device

class Case:
    def __init__(self, T, hq, hk, D, R, sections, pairs="halves", order="blocks", xd="bf16",
                 wd=None, norm=True, layout="packed", offset=0, seed=0, far=0, in_place=False):
        self.__dict__.update(locals())
        self.wd = wd or xd
        r = np.random.RandomState(seed)
        dev = torch.device("cuda")
        self.eps = float(np.float32(1e-6))
        rows = hq + hk + (3 if layout == "packed" else 0)

        def block(heads):
            t = torch.from_numpy(r.standard_normal((T, heads, D)).astype(np.float32)).to(TD[xd])
            flat = torch.full((t.numel() + 64,), 7.0, dtype=TD[xd], device=dev)
            v = flat[16 + offset:16 + offset + t.numel()].view(T, heads, D)
            v.copy_(t)
            return v

        def two(heads_q, heads_k):
            if layout == "packed":       # [q | k | v] rows
                b = block(rows)
                return b[:, :heads_q], b[:, heads_q:heads_q + heads_k], b
            if layout == "turns":        # q and k heads in turn (hq == hk)
                b = block(2 * heads_q).view(T, heads_q, 2, D)
                return b[:, :, 0], b[:, :, 1], b
            if layout == "heads":        # [H, T, D]
                return (block(heads_q).view(heads_q, T, D).transpose(0, 1),
                        block(heads_k).view(heads_k, T, D).transpose(0, 1), None)
            if layout == "heads, in turn":   # [H, T, q and k, D] (hq == hk)
                b = block(2 * heads_q).view(heads_q, T, 2, D).transpose(0, 1)
                return b[:, :, 0], b[:, :, 1], b
            return block(heads_q), block(heads_k), None

        self.q, self.k, self.base = two(hq, hk)
        self.dyq, self.dyk, self.dbase = two(hq, hk)
        w = [torch.from_numpy(1 + 0.3 * r.standard_normal(D)).to(TD[self.wd]).to(dev)
             for _ in range(2)]
        self.gq, self.gk = w if norm else (None, None)
        A = len(sections)
        self.positions = (far + torch.from_numpy(r.randint(-50, 5000, (A, T)))).to(dev)
        self.inv_freq = torch.from_numpy(
            (10000.0 ** (-np.arange(0, R, 2) / R)).astype(np.float32)).to(dev)
        self.rope = rn.Rope(self.positions, self.inv_freq, sections, R, pairs, order)
        self.cos, self.sin = angles(self.positions.cpu().numpy(), self.inv_freq.cpu().numpy(),
                                    sections, order)

    def host(self, t):
        return None if t is None else t.detach().double().cpu().numpy()

    def run_fwd(self, stream=None):
        qo, ko = (self.q, self.k) if self.in_place else (torch.empty_like(self.q),
                                                         torch.empty_like(self.k))
        has_k = self.hk > 0
        rn.rmsnorm_rope_fwd(rn.Heads.of(self.q), rn.Heads.of(self.k) if has_k else None, self.gq,
                            self.gk if has_k else None, rn.Heads.of(qo),
                            rn.Heads.of(ko) if has_k else None, self.rope, self.T, self.D,
                            self.eps, self.xd, self.wd, stream)
        return qo, ko

    def run_bwd(self, stream=None, want=(True, True)):
        has_k = self.hk > 0
        dq, dk = (self.dyq, self.dyk) if self.in_place else (torch.empty_like(self.dyq),
                                                             torch.empty_like(self.dyk))
        n = rn.rmsnorm_rope_bwd_workspace_size(self.T, self.hq, self.hk, self.D, self.xd, self.wd)
        ws = torch.full((n + 64,), 0xA5, dtype=torch.uint8, device="cuda")
        gq, gk = (torch.full((self.D,), float("nan"), device="cuda")
                  if self.norm and want[i] and (i == 0 or has_k) else None for i in range(2))
        rn.rmsnorm_rope_bwd(rn.Heads.of(self.dyq), rn.Heads.of(self.dyk) if has_k else None,
                            rn.Heads.of(self.q) if self.norm else None,
                            rn.Heads.of(self.k) if self.norm and has_k else None, self.gq,
                            self.gk if has_k else None, rn.Heads.of(dq),
                            rn.Heads.of(dk) if has_k else None, gq, gk, ws, n, self.rope, self.T,
                            self.D, self.eps, self.xd, self.wd, stream)
        torch.cuda.synchronize()
        assert bool((ws[n:] == 0xA5).all()), "write behind the workspace"
        return dq, dk, gq, gk


def check(got, ref, tol, dt=None, what=""):
    got = got.detach().double().cpu().numpy()
    tol = tol + (half_step(dt) * np.abs(ref) if dt == "bf16" else 0)
    bad = ~(np.abs(got - ref) <= tol + 1e-30)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], ref[bad][:4], tol[bad][:4])


def check_case(c):
    x = [c.host(c.q), c.host(c.k)]
    dy = [c.host(c.dyq), c.host(c.dyk)]
    g = [c.host(c.gq), c.host(c.gk)]
    base = None if c.base is None else c.base.clone()
    out = c.run_fwd()
    torch.cuda.synchronize()
    for i in range(2 if c.hk else 1):
        y, tol = ref_fwd(x[i], g[i], c.eps, c.cos, c.sin, c.R, c.pairs)
        check(out[i], y, tol, c.xd, f"fwd {i}")
    if base is not None and c.in_place and c.layout == "packed":
        assert torch.equal(base[:, c.hq + c.hk:], c.base[:, c.hq + c.hk:]), "v was touched"
    if c.in_place:
        c.q.copy_(torch.from_numpy(x[0]))
        c.k.copy_(torch.from_numpy(x[1]))
    got = c.run_bwd()
    for i in range(2 if c.hk else 1):
        dx, tol, dg, dgtol = ref_bwd(dy[i], x[i], g[i], c.eps, c.cos, c.sin, c.R, c.pairs)
        check(got[i], dx, tol, c.xd, f"dx {i}")
        if c.norm:
            check(got[2 + i], dg, dgtol, None, f"dgamma {i}")


S3 = lambda R: [R // 2 - 2 * (R // 6), R // 6, R // 6]   # noqa: E731


@gpu
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("pairs", ["halves", "adjacent"])
@pytest.mark.parametrize("xd,wd", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("T,hq,hk,D,R", [
    (1, 1, 0, 64, 64), (1, 32, 8, 128, 128), (7, 5, 1, 128, 64), (67, 12, 4, 80, 80),
    (33, 3, 3, 96, 32), (130, 4, 2, 256, 256), (9, 2, 1, 192, 64), (5, 3, 1, 512, 512),
    (19, 6, 2, 36, 36), (21, 4, 1, 20, 10), (3, 2, 2, 2, 2), (4, 1, 1, 1000, 990)])
def test_sizes(T, hq, hk, D, R, xd, wd, pairs, norm):
    check_case(Case(T, hq, hk, D, R, S3(R), pairs, "blocks", xd, wd, norm))


@gpu
@pytest.mark.parametrize("order,sections", [
    ("blocks", [32]), ("interleaved", [32]), ("blocks", [0, 32]), ("blocks", [8, 8, 8, 8]),
    ("blocks", [16, 0, 16]), ("interleaved", [12, 10, 10]), ("interleaved", [31, 1, 0]),
    ("interleaved", [32, 0, 0, 0]), ("interleaved", [8, 8, 8, 8])])
@pytest.mark.parametrize("pairs", ["halves", "adjacent"])
def test_axes(order, sections, pairs):
    check_case(Case(50, 8, 2, 80, 64, sections, pairs, order, norm=False))
    check_case(Case(50, 8, 2, 80, 64, sections, pairs, order, "f32", layout="apart"))


@gpu
@pytest.mark.parametrize("far", [1 << 20, (1 << 31) - 6000, -(1 << 31) + 60])
def test_far_and_negative_positions(far):
    check_case(Case(40, 4, 2, 128, 128, [24, 20, 20], xd="f32", far=far))


@gpu
@pytest.mark.parametrize("layout", ["packed", "apart", "turns", "heads", "heads, in turn"])
@pytest.mark.parametrize("offset", [0, 1, 8])
@pytest.mark.parametrize("in_place", [False, True])
def test_layouts(layout, offset, in_place):
    for xd, norm in (("bf16", True), ("f32", False)):
        check_case(Case(45, 4, 4, 64, 64, [12, 10, 10], layout=layout, offset=offset, xd=xd,
                        norm=norm, in_place=in_place))


@gpu
@pytest.mark.parametrize("xd,norm", [("bf16", True), ("f32", True), ("bf16", False)])
@pytest.mark.parametrize("pairs", ["halves", "adjacent"])
@pytest.mark.parametrize("D,R,offset", [
    (80, 40, 0), (36, 36, 0), (36, 18, 0), (250, 250, 0), (250, 2, 0), (128, 128, 1), (256, 256, 1),
    (256, 128, 2), (258, 258, 0), (512, 256, 4), (512, 512, 2), (130, 66, 3), (1024, 1024, 4),
    (1030, 1030, 0)])
def test_vectors_below_sixteen_bytes(D, R, offset, pairs, xd, norm):
    check_case(Case(23, 5, 3, D, R, S3(R), pairs, "interleaved", xd, None, norm, "apart", offset))


@gpu
def test_many_tokens_and_heads():
    check_case(Case(5000, 6, 2, 64, 64, [12, 10, 10], order="interleaved"))
    check_case(Case(2, 300, 7, 128, 128, [24, 20, 20]))
    check_case(Case(700, 2, 1, 36, 36, [6, 6, 6]))
    # several tokens an item, rows of 5, 6 and 10 lanes
    check_case(Case(9000, 1, 1, 80, 80, [20, 10, 10]))
    check_case(Case(8200, 2, 1, 96, 96, [16, 16, 16], norm=False))
    check_case(Case(8200, 2, 1, 96, 96, [16, 16, 16], "adjacent"))
    check_case(Case(8200, 1, 1, 80, 64, [16, 8, 8], "adjacent", xd="f32"))


@gpu
def test_gradient_against_differences():
    # central differences of the 64-bit forward through the kernel's backward: the loss sum(dy * y)
    c = Case(3, 2, 1, 32, 32, [6, 5, 5], xd="f32", layout="apart")
    dq, _, gq, _ = c.run_bwd()
    x, dy, w = c.host(c.q), c.host(c.dyq), c.host(c.gq)
    f = lambda x, w: (dy * ref_fwd(x, w, c.eps, c.cos, c.sin, c.R, c.pairs)[0]).sum()  # noqa: E731
    h = 1e-5
    for idx in [(0, 0, 0), (1, 1, 17), (2, 0, 31)]:
        e = np.zeros_like(x)
        e[idx] = h
        num = (f(x + e, w) - f(x - e, w)) / (2 * h)
        # truncation h^2 f''' / 6 and cancellation 2^-52 |f| / h stay below 1e-8 here
        assert abs(num - float(dq[idx])) <= 1e-5 * (1 + abs(num))
    for j in (0, 9, 31):
        e = np.zeros_like(w)
        e[j] = h
        num = (f(x, w + e) - f(x, w - e)) / (2 * h)
        assert abs(num - float(gq[j])) <= 1e-5 * (1 + abs(num))


@gpu
def test_repeats_give_the_same_bits_and_skipped_gradients_stay_out():
    c = Case(900, 8, 2, 128, 128, [24, 20, 20])
    a, b = c.run_bwd(), c.run_bwd()
    for u, v in zip(a, b):
        assert torch.equal(u, v)
    for want in ((True, False), (False, True), (False, False)):
        d = c.run_bwd(want=want)
        assert torch.equal(d[0], a[0]) and torch.equal(d[1], a[1])
        for i in range(2):
            assert torch.equal(d[2 + i], a[2 + i]) if want[i] else d[2 + i] is None


@gpu
def test_no_rows():
    c = Case(0, 4, 2, 64, 64, [32])
    c.run_fwd()
    _, _, gq, gk = c.run_bwd()
    assert not gq.any() and not gk.any()
    c = Case(3, 0, 2, 64, 64, [32])
    check_case(c)


@gpu
@pytest.mark.parametrize("norm", [False, True])
def test_tokens_further_apart_than_32_bits(norm):
    c = Case(3, 4, 2, 64, 64, [12, 10, 10], layout="apart", norm=norm)
    stride = (1 << 31) + 8
    far = torch.empty(2 * stride + (4 << 20), dtype=torch.bfloat16, device="cuda")
    for name in ("q", "k", "dyq", "dyk"):
        t = getattr(c, name)
        at = {"q": 0, "k": 1 << 20, "dyq": 2 << 20, "dyk": 3 << 20}[name]
        v = far.as_strided(t.shape, (stride, 64, 1), at)
        v.copy_(t)
        setattr(c, name, v)
    check_case(c)
    c.in_place = True
    check_case(c)


@gpu
def test_a_view_of_no_heads_has_a_zero_gradient():
    for D in (64, 2050):      # the vectors' kernel and the scalar one
        c = Case(5, 3, 2, D, D, [D // 2], layout="apart")
        none = rn.Heads(None, 0, 0, 0)
        gq, gk = torch.full((2, D), float("nan"), device="cuda")
        n = rn.rmsnorm_rope_bwd_workspace_size(5, 3, 0, D, "bf16", "bf16")
        ws, dq = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(c.dyq)
        rn.rmsnorm_rope_bwd(rn.Heads.of(c.dyq), none, rn.Heads.of(c.q), none, c.gq, c.gk,
                            rn.Heads.of(dq), none, gq, gk, ws, n, c.rope, 5, D, c.eps, "bf16",
                            "bf16")
        dx, tol, dg, dgtol = ref_bwd(c.host(c.dyq), c.host(c.q), c.host(c.gq), c.eps, c.cos, c.sin,
                                     D, "halves")
        check(dq, dx, tol, "bf16")
        check(gq, dg, dgtol)
        assert not gk.any()


@gpu
def test_special_values_stay_in_their_row():
    c = Case(6, 4, 1, 64, 64, [32], xd="f32")
    clean = [t.clone() for t in c.run_fwd()]
    c.q[2, 1, 5] = float("nan")
    c.q[4, 0, 6] = float("inf")
    c.q[5, 3] = 0
    q, k = c.run_fwd()
    assert bool(q[2, 1].isnan().all()) and not bool(q[4, 0].isfinite().all())
    assert not q[5, 3].any() and torch.equal(k, clean[1])
    keep = torch.ones(6, 4, dtype=torch.bool)
    keep[2, 1] = keep[4, 0] = keep[5, 3] = False
    assert torch.equal(q[keep], clean[0][keep])


@gpu
def test_replayed_graph_and_two_streams():
    c = Case(300, 8, 2, 128, 128, [24, 20, 20])
    want = [t.clone() for t in c.run_fwd()] + [t.clone() for t in c.run_bwd()]
    outs = [torch.empty_like(t) for t in want]
    n = rn.rmsnorm_rope_bwd_workspace_size(c.T, c.hq, c.hk, c.D, c.xd, c.wd)
    s = torch.cuda.Stream()
    H = rn.Heads.of

    def step(o, ws, st):
        rn.rmsnorm_rope_fwd(H(c.q), H(c.k), c.gq, c.gk, H(o[0]), H(o[1]), c.rope, c.T, c.D, c.eps,
                            c.xd, c.wd, st)
        rn.rmsnorm_rope_bwd(H(c.dyq), H(c.dyk), H(c.q), H(c.k), c.gq, c.gk, H(o[2]), H(o[3]), o[4],
                            o[5], ws, n, c.rope, c.T, c.D, c.eps, c.xd, c.wd, st)

    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    step(outs, ws, s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step(outs, ws, torch.cuda.current_stream())
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    # a workspace each: two streams at once
    sets = [([torch.zeros_like(t) for t in want], torch.empty(n, dtype=torch.uint8, device="cuda"),
             torch.cuda.Stream()) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for o, w, st in sets:
            step(o, w, st)
    torch.cuda.synchronize()
    for o, _, _ in sets:
        assert all(torch.equal(a, b) for a, b in zip(o, want))


# ---------------------------------------------------------------- refusals (no GPU)

@pytest.fixture(scope="module")
def lib():
    from row_wise_normalization_02_gb300 import _build
    _build.build()
    return rn.load_library()


def args(**kw):
    a = dict(q=rn.Heads(FAKE, 640, 64, 8), k=rn.Heads(FAKE + 1024, 640, 64, 2),
             gq=FAKE + (1 << 32), gk=FAKE + (1 << 32) + 4096,
             qo=rn.Heads(FAKE + (2 << 32), 512, 64, 8),
             ko=rn.Heads(FAKE + (3 << 32), 128, 64, 2), T=4, D=64, eps=1e-6, xd=1, wd=1,
             sections=[12, 10, 10], R=64, positions=FAKE + (4 << 32), pst=4,
             inv_freq=FAKE + (5 << 32), pairs=0, order=0, axes=None)
    a.update(kw)
    r = rn.Rope(a["positions"], a["inv_freq"], a["sections"], a["R"], positions_stride=a["pst"])
    r.pairs, r.order = a["pairs"], a["order"]
    if a["axes"] is not None:
        r.axes = a["axes"]
    a["rope"] = r if kw.get("rope", 1) is not None else None
    return a


H = rn.Heads
REFUSED = [
    (dict(q=None), 1), (dict(qo=None), 1), (dict(ko=None), 1), (dict(k=None), 1),
    (dict(gq=None), 1),
    (dict(gk=None), 1), (dict(rope=None), 1), (dict(T=-1), 1), (dict(T=1 << 30), 1), (dict(D=0), 1),
    (dict(D=8193), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(R=63), 1),
    (dict(R=0, sections=[0, 0, 0]), 1), (dict(R=66, sections=[13, 10, 10]), 1),
    (dict(sections=[12, 10, 9]), 1), (dict(sections=[12, 10, 11]), 1),
    (dict(sections=[-2, 24, 10]), 1),
    (dict(sections=[2, 20, 10], order=1), 1), (dict(axes=0), 1), (dict(axes=5), 1),
    (dict(pairs=2), 1), (dict(pairs=-1), 1), (dict(order=2), 1), (dict(pst=3), 1),
    (dict(positions=None), 1), (dict(inv_freq=None), 1), (dict(positions=FAKE + (4 << 32) + 4), 3),
    (dict(inv_freq=FAKE + (5 << 32) + 2), 3), (dict(q=H(FAKE + 1, 640, 64, 8)), 3),
    (dict(gq=FAKE + (1 << 32) + 1), 3), (dict(q=H(None, 640, 64, 8)), 1),
    (dict(q=H(FAKE, 640, 32, 8)), 1), (dict(q=H(FAKE, 500, 64, 8)), 1),
    (dict(q=H(FAKE, -640, 64, 8)), 1),
    (dict(q=H(FAKE, 64, 255, 8)), 1), (dict(q=H(FAKE, 63, 256, 8)), 1),   # heads first
    (dict(q=H(FAKE, 256, 1 << 58, 8)), 1), (dict(pst=1 << 57), 1),
    (dict(q=H(FAKE, 640, 64, -8)), 1), (dict(q=H(FAKE, 640, 64, 7)), 1),
    (dict(q=H(FAKE, 1 << 62, 64, 8)), 1), (dict(q=H(FAKE, 640, 1 << 62, 8)), 1),
    (dict(q=H(FAKE, 1 << 23, 64, 1 << 17), qo=H(FAKE + (2 << 32), 1 << 23, 64, 1 << 17)), 1),
    (dict(qo=H(FAKE + 64, 640, 64, 8)), 1),            # over q, not in place
    (dict(qo=H(FAKE, 512, 64, 8)), 1),                 # over q with other strides
    (dict(ko=H(FAKE, 640, 64, 2)), 1),                 # k_out over q
    (dict(ko=H(FAKE + (2 << 32) + 896, 512, 64, 2)), 1),  # k_out over q_out's last head
    (dict(qo=H(FAKE + (1 << 32), 512, 64, 8)), 1),     # over gamma
    (dict(qo=H(FAKE + (4 << 32), 512, 64, 8)), 1),     # over positions
    (dict(xd=0, wd=1), 2), (dict(xd=7), 2), (dict(wd=5), 2),
]


@pytest.mark.parametrize("kw,status", REFUSED)
def test_forward_refusals(lib, kw, status):
    a = args(**kw)
    with pytest.raises(rn.RMSNormError) as e:
        rn.rmsnorm_rope_fwd(a["q"], a["k"], a["gq"], a["gk"], a["qo"], a["ko"], a["rope"], a["T"],
                            a["D"], a["eps"], a["xd"], a["wd"])
    assert e.value.status == status


@pytest.mark.parametrize("kw,status", [
    (dict(dq=None), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(ws=None), 4),
    (dict(ws=FAKE + (9 << 32) + 8), 4), (dict(dgq=FAKE + (7 << 32) + 2), 3),
    (dict(k=H(FAKE, 640, 64, 0), dk=H(FAKE, 640, 64, 0), dxk=H(FAKE, 640, 64, 0),
          dgk=FAKE + (7 << 32) + 5), 3),                # of no heads
    (dict(k=H(FAKE, 640, 64, 0), dk=H(FAKE, 640, 64, 0), dxk=H(FAKE, 640, 64, 0),
          dgk=FAKE + (7 << 32)), 1),
    (dict(dgk=FAKE + (7 << 32)), 1),                    # both gradients in one place
    (dict(dq=H(FAKE + (8 << 32), 512, 64, 7)), 1),
    (dict(dxq=H(FAKE, 640, 64, 8)), 1),                 # dq over q
    (dict(gq=None, gk=None), 1),                        # weight gradients without weights
    (dict(xd=0, wd=1), 2),
])
def test_backward_refusals(lib, kw, status):
    a = args(**{k: v for k, v in kw.items() if k in ("q", "k", "gq", "gk", "xd", "wd")})
    b = dict(dq=H(FAKE + (8 << 32), 512, 64, 8), dk=H(FAKE + (8 << 32) + (1 << 20), 128, 64, 2),
             dxq=H(FAKE + (2 << 32), 512, 64, 8), dxk=H(FAKE + (3 << 32), 128, 64, 2),
             dgq=FAKE + (7 << 32), dgk=FAKE + (7 << 32) + 4096, ws=FAKE + (9 << 32))
    b.update({k: v for k, v in kw.items() if k in b})
    with pytest.raises(rn.RMSNormError) as e:
        rn.rmsnorm_rope_bwd(b["dq"], b["dk"], a["q"], a["k"], a["gq"], a["gk"], b["dxq"], b["dxk"],
                            b["dgq"], b["dgk"], b["ws"], 1 << 30, a["rope"], a["T"], a["D"],
                            a["eps"], a["xd"], a["wd"])
    assert e.value.status == status


def test_workspace_refusals(lib):
    for bad in ((-1, 8, 2, 64), (4, -1, 2, 64), (4, 8, 2, 0), (4, 8, 2, 9000), (4, 1 << 17, 0, 64)):
        with pytest.raises(rn.RMSNormError) as e:
            rn.rmsnorm_rope_bwd_workspace_size(*bad, "bf16", "bf16")
        assert e.value.status == 1
    assert rn.rmsnorm_rope_bwd_workspace_size(0, 8, 2, 64, "bf16", "bf16") == 0


def test_no_tokens_touch_nothing(lib):
    a = args(T=0, q=H(None, 0, 64, 8), k=None, gk=None, qo=H(None, 0, 64, 8), ko=None,
             positions=None, inv_freq=None, pst=0)
    rn.rmsnorm_rope_fwd(a["q"], None, a["gq"], None, a["qo"], None, a["rope"], 0, 64, 1e-6, 1, 1)


def test_binding_checks_its_descriptors():
    p, f = torch.zeros(3, 5, dtype=torch.int64), torch.ones(32)
    rn.Rope(p, f, [12, 10, 10], 64)
    for bad, err in ((lambda: rn.Rope(p, f, [16, 16], 64), ValueError),
                     (lambda: rn.Rope(p.int(), f, [12, 10, 10], 64), TypeError),
                     (lambda: rn.Rope(p, f.double(), [12, 10, 10], 64), TypeError),
                     (lambda: rn.Rope(p, f[:31], [12, 10, 10], 64), ValueError),
                     (lambda: rn.Rope(p, f, [6, 6, 6, 7, 7], 64), ValueError),
                     (lambda: rn.Rope(p[0], f, [16, 16], 64), ValueError),
                     (lambda: rn.Rope(p, f, [12, 10, 10], 64, "thirds"), KeyError),
                     (lambda: rn.Heads.of(torch.zeros(4, 8)), ValueError),
                     (lambda: rn.Heads.of(torch.zeros(4, 64, 8).transpose(1, 2)), ValueError)):
        with pytest.raises(err):
            bad()
