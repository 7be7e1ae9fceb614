"""Token log-probabilities, the clipped policy loss and the preference loss, with
the gradient of the logits, against a plain evaluation in 64 bits.

Tolerances, with u = 2^-24 (half a step of fp32) and a_j = (x_j - max) log2(e) /
temperature, the exponents of a row's terms:
  * s = sum 2^a_j: a term is off by 2^-22 (ex2.approx) and by the rounding of its
    exponent, 2^-24 |a_j| for the fma and 2^-25 |a_j| for the constant, both times ln 2;
    under the weights of the terms, |a_j| averages to at most log2(V) + 1 (the entropy
    of the softmax bounds it).  A sum of positive terms in fp32 adds its depth in
    roundings: a thread's share over its four accumulators, V / 4 / 64 at the fewest
    threads and V / 4 / 256 for long rows, and 40 for the batches' rescaling, the
    shuffles, the warps and the cluster.
  * logp, and rel_lse = -logp: that, absolutely (d log s = ds / s), and one rounding u of
    the result.
  * p_j = exp(z_j - z_t - rel): the error of rel and the roundings of z_j - z_t, of its
    product with the two parts of the scale and of rel, u (4 |z_j - z_t| + 4 |rel|) +
    2^-21, relative (where rel > 64 the sum is taken again, and the exponents are those
    from the maximum: smaller).  dlogits = g ([j = t] - p): that times p |g|, and three
    roundings of the result.
  * the policy's ratio carries the error of logp; loss terms and slopes a few roundings
    more (POINT = 2^-20) of the magnitudes of their parts.
  * margins: the errors of their rows' logp added up, times beta, and a rounding.
  * bf16 gradients add half a step, 2^-8 relative.
"""
import math

import numpy as np
import pytest
import torch

import row_wise_normalization_02_gb300 as rn

gpu = pytest.mark.gpu
TD = {"bf16": torch.bfloat16, "f32": torch.float32}
U, POINT = 2.0 ** -24, 2.0 ** -20
FAKE = 1 << 40
IGNORE = -100


def half_step(dt):
    return torch.finfo(TD[dt]).eps / 2


def logp_tol(V):
    depth = V / 4 / (256 if V >= 8192 else 64) + 40
    return 2.0 ** -22 + 1.5 * U * (math.log2(V) + 1) + depth * U


def rows(M, V, dt, ld=None, offset=0, seed=0, scale=2.0, lift=6.0):
    """[M, V] logits on the device, row stride ld, `offset` elements past a 16-byte
    boundary, canaries around them; targets with a fifth left out."""
    ld = ld or V
    r = np.random.RandomState(seed)
    x = scale * r.standard_normal((M, V)).astype(np.float32)
    t = r.randint(0, V, M)
    x[np.arange(M), t] += lift * r.rand(M).astype(np.float32)
    flat = torch.full((16 + offset + M * ld + 64,), 3.0, dtype=TD[dt], device="cuda")
    v = flat[16 + offset:16 + offset + M * ld].view(M, ld)[:, :V]
    v.copy_(torch.from_numpy(x))
    t[r.rand(M) < 0.2] = IGNORE
    return v, torch.from_numpy(t).cuda(), flat


class Ref:
    """The row's 64-bit values."""

    def __init__(self, x, t, inv_t):
        self.z = x.double() * inv_t
        self.live = t >= 0
        self.t = t.clamp(min=0)
        m = self.z.amax(1, keepdim=True)
        log_s = (self.z - m).exp().sum(1).log()
        self.p = (self.z - m - log_s[:, None]).exp()
        # the difference first: 64 bits too lose log s beside a mask's lowest value
        self.zt = self.z.gather(1, self.t[:, None])
        self.logp = (self.z.gather(1, self.t[:, None]) - m)[:, 0] - log_s
        self.logp[~self.live] = 0
        self.rel = -self.logp
        self.inv_t = inv_t

    def grad(self, dlogp):
        """Gradient for dlogp, and its tolerance for an error `rel` of g."""
        g = torch.where(self.live, dlogp, 0.0)[:, None] * self.inv_t
        p = torch.where(self.live[:, None], self.p, 0.0)
        one = torch.zeros_like(p).scatter_(1, self.t[:, None], 1.0)
        V = p.shape[1]
        size = torch.where(self.z.isinf(), 0.0, (self.z - self.zt).abs())    # p is 0 there
        err = p * (logp_tol(V) + U * (4 * size + 4 * self.rel.abs()[:, None]) + 2.0 ** -21)
        return g * (one - p), g.abs() * (err + 3 * U * (one + p))


def close(got, ref, tol, what=""):
    got = got.double()
    assert got.shape == ref.shape
    bad = ~((got - ref).abs() <= tol + 1e-30)
    assert not bool(bad.any()), (what, int(bad.sum()), got[bad][:4], ref[bad][:4])


def check_grad(got, r, dlogp, dt, what="", gtol=None):
    d, tol = r.grad(dlogp)
    if gtol is not None:     # dlogp itself carries an error
        tol = tol + gtol[:, None] * r.inv_t * (d.abs() / dlogp.abs().clamp(min=1e-30)[:, None])
    if dt == "bf16":
        tol = tol + half_step(dt) * d.abs()
    close(got, d, tol, what)


def fwd(x, t, inv_t=1.0, dt="bf16", stream=None):
    M, V = x.shape
    logp, lse = torch.full((2, M), float("nan"), device="cuda")
    rn.rmsnorm_token_logprob_fwd(x, x.stride(0), t, inv_t, logp, lse, M, V, dt, stream)
    return logp, lse


def bwd(x, t, lse, dlogp, scale=None, inv_t=1.0, dt="bf16", out=None, stream=None):
    M, V = x.shape
    if out is None:
        out = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda")
    rn.rmsnorm_token_logprob_bwd(x, x.stride(0), t, inv_t, lse, dlogp, scale, out, out.stride(0),
                                 M, V, dt, stream)
    return out


def check_logprob(x, t, dt, inv_t=1.0, out=None):
    M, V = x.shape
    r = Ref(x, t, inv_t)
    logp, lse = fwd(x, t, inv_t, dt)
    close(logp, r.logp, logp_tol(V) + U * r.logp.abs(), "logp")
    assert torch.equal(lse, -logp)
    dlogp = torch.randn(M, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    scale = torch.tensor(1.5, device="cuda")
    d = bwd(x, t, lse, dlogp, scale, inv_t, dt, out)
    check_grad(d, r, dlogp.double() * 1.5, dt, "dlogits")
    return d


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("M,V", [(1, 1), (3, 2), (5, 7), (9, 8), (4, 33), (300, 1000), (700, 1025),
                                 (17, 5003), (400, 4096), (64, 32768), (1, 131072), (5, 50257),
                                 (40, 65536), (160, 20000)])
def test_sizes(M, V, dt):
    x, t, _ = rows(M, V, dt, seed=M + V)
    check_logprob(x, t, dt)


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V,pad,offset", [(1000, 24, 0), (1001, 0, 0), (1001, 7, 3), (5000, 1, 1),
                                          (3, 1, 2), (50257, 47, 0)])
@pytest.mark.parametrize("inv_t", [1.0, 1 / 0.7, 0.25])
def test_strides_offsets_and_temperature(V, pad, offset, dt, inv_t):
    x, t, flat = rows(30, V, dt, V + pad, offset, seed=V)
    before = flat.clone()
    check_logprob(x, t, dt, inv_t)
    # a gradient whose rows start elsewhere modulo 16 bytes
    other = torch.full((30 * (V + 5) + 64,), 9.0, dtype=TD[dt], device="cuda")
    out = other[1:1 + 30 * (V + 5)].view(30, V + 5)[:, :V]
    check_logprob(x, t, dt, inv_t, out)
    assert torch.equal(flat, before)
    assert bool((other[1:1 + 30 * (V + 5)].view(30, V + 5)[:, V:] == 9).all()) and other[0] == 9
    # in place
    want = check_logprob(x, t, dt, inv_t).clone()
    _, lse = fwd(x, t, inv_t, dt)
    dlogp = torch.randn(30, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    bwd(x, t, lse, dlogp, torch.tensor(1.5, device="cuda"), inv_t, dt, out=x)
    assert torch.equal(x, want)
    gap = flat[16 + offset:16 + offset + 30 * (V + pad)].view(30, V + pad)[:, V:]
    assert bool((gap == 3).all()) and bool((flat[:16 + offset] == 3).all())


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_large_magnitudes_and_order(dt):
    # rows whose maximum comes last, comes first, and far apart values
    for scale in (30.0, 1000.0, 1e6):
        x, t, _ = rows(8, 30000, dt, scale=scale)
        x[0], _ = x[0].sort()
        x[1], _ = x[1].sort(descending=True)
        r = Ref(x, t, 1.0)
        logp, lse = fwd(x, t, 1.0, dt)
        # logp is the difference of values far larger than the softmax's spread
        close(logp, r.logp, logp_tol(30000) + U * r.logp.abs(), "logp")
        assert torch.equal(lse, -logp)
        # a rel_lse too large for its fp32 digits: the backward takes the sum again, and a term
        # is off by its exponent's rounding, 2 u |z - max|; smaller ones are within the usual bound
        dlogp = torch.linspace(-1, 1, 8, device="cuda")
        far = r.rel > 64
        p = torch.where(r.live[:, None], r.p, 0.0)
        one = torch.zeros_like(p).scatter_(1, r.t[:, None], 1.0)
        want = torch.where(r.live, dlogp.double(), 0.0)[:, None] * (one - p)
        size = torch.where(far[:, None], 4 * (r.z - r.z.amax(1, keepdim=True)).abs(),
                           4 * (r.z - r.zt).abs() + 4 * r.rel.abs()[:, None])
        tol = dlogp.abs()[:, None] * (p * (logp_tol(30000) + U * size + 2.0 ** -21) +
                                      3 * U * (one + p)) + half_step(dt) * want.abs() * (dt == "bf16")
        close(bwd(x, t, lse, dlogp, dt=dt), want, tol, "dlogits")
        bwd(x, t, lse, dlogp, dt=dt, out=x)
        close(x, want, tol, "dlogits in place")


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_masked_vocabulary_and_special_rows(dt):
    x, t, _ = rows(12, 2000, dt, seed=5)
    t[:] = torch.arange(12, device="cuda")
    t[11] = IGNORE
    x[0, 500:] = float("-inf")          # a masked vocabulary
    x[1] = float("-inf")                # nothing left
    x[2] = float("-inf")
    x[2, 2] = -5.0                      # one token left: certain
    x[3, 3] = float("-inf")             # the target is masked
    x[4, 900] = float("nan")
    x[5, 900] = float("inf")
    x[6] = torch.finfo(TD[dt]).min      # masks of the lowest value
    x[11, :] = float("nan")             # left out: not read
    t[7] = 2000                         # past the row
    t[8] = 1 << 40
    logp, lse = fwd(x, t, 1.0, dt)
    dlogp = torch.ones(12, device="cuda")
    d = bwd(x, t, lse, dlogp, dt=dt)
    r = Ref(x[[0, 2, 6, 9, 10]].clone(), t[[0, 2, 6, 9, 10]], 1.0)
    close(logp[[0, 2, 6, 9, 10]], r.logp, logp_tol(2000) + U * r.logp.abs())
    check_grad(d[[0, 2, 6, 9, 10]], r, dlogp[:5].double(), dt)
    # one value everywhere: a uniform row whatever the value
    even = torch.full((2000,), -1 / 2000, device="cuda", dtype=torch.float64)
    even[6] += 1
    close(d[6], even, even.abs() * (2.0 ** -18 + (half_step(dt) if dt == "bf16" else 0)))
    assert not d[0, 500:].any()
    assert logp[2] == 0 and not d[2].any()
    assert logp[3] == float("-inf") and bool(d[3].isfinite().all())
    for bad in (1, 4, 5, 7, 8):
        assert bool(logp[bad].isnan()) and bool(d[bad].isnan().any()), bad
    assert bool(d[7].isnan().all())
    assert logp[11] == 0 and lse[11] == 0 and not d[11].any()
    assert torch.equal(bwd(x, t, lse, dlogp, dt=dt, out=x).isnan(), d.isnan())    # in place


# ---------------------------------------------------------------- policy loss

def policy_inputs(r, seed=0, kl=True):
    M = r.logp.numel()
    g = torch.Generator("cuda").manual_seed(seed)
    n = lambda: torch.randn(M, device="cuda", generator=g)  # noqa: E731
    ratio = (0.3 * n()).double().exp()
    for border in (0.8, 1.3):    # no 32-bit logp decides a ratio this near a border
        ratio = torch.where((ratio - border).abs() < 2e-3, ratio + 5e-3, ratio)
    old = (r.logp - ratio.log()).float()
    ref = (r.logp + 0.4 * n()).float() if kl else None
    return old, ref, n(), torch.rand(M, device="cuda", generator=g) / M


def policy_ref(r, old, ref, A, w, kl):
    A, w = A.double(), w.double() if w is not None else torch.ones_like(A).double()
    w = torch.where(r.live, w, 0.0)
    ratio = (r.logp - old.double()).exp()
    s = torch.minimum(ratio * A, ratio.clamp(0.8, 1.3) * A)
    clipped = torch.where(A >= 0, ratio > 1.3, ratio < 0.8)
    term, slope = -s, torch.where(clipped, 0.0, -A * ratio)
    size = (A * ratio).abs()
    if ref is not None:
        d = ref.double() - r.logp
        term = term + kl * (torch.expm1(d) - d)
        slope = slope - kl * torch.expm1(d)
        size = size + kl * (d.exp() + d.abs() + 1)
    tol = w * size * (logp_tol(r.z.shape[1]) + POINT)
    return w * term, w * slope, tol


def policy(x, t, old, ref, A, w, kl, dt, inv_t=1.0, out=None, want=True, stream=None):
    M, V = x.shape
    loss = torch.full((), float("nan"), device="cuda")
    token, logp, lse, dlogp = torch.full((4, M), float("nan"), device="cuda")
    if out is None and want:
        out = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda")
    rn.rmsnorm_policy_loss_fwd(x, x.stride(0), t, inv_t, old, ref, A, w, 0.2, 0.3, kl, loss, token,
                               logp, lse, dlogp, out if want else None,
                               out.stride(0) if want else 0, M, V, dt, stream)
    return loss, token, logp, lse, dlogp, out


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kl", [None, 0.0, 0.1])
@pytest.mark.parametrize("M,V,pad,inv_t", [(1, 5, 0, 1.0), (2, 300, 0, 1.0), (33, 1001, 0, 1 / 0.7),
                                           (400, 4096, 0, 1.0), (7, 50257, 47, 1.0),
                                           (3, 131072, 0, 1.0), (500, 20000, 8, 0.5)])
def test_policy_loss(M, V, pad, inv_t, kl, dt):
    x, t, _ = rows(M, V, dt, V + pad, seed=M)
    r = Ref(x, t, inv_t)
    old, ref, A, w = policy_inputs(r, M, kl is not None)
    for weights in (w, None):
        term, slope, tol = policy_ref(r, old, ref, A, weights, kl or 0.0)
        # with the gradient in the same pass, and without it (another kernel)
        for want in (True, False):
            loss, token, logp, lse, dlogp, d = policy(x, t, old, ref, A, weights, kl or 0.0, dt,
                                                      inv_t, want=want)
            close(logp, r.logp, logp_tol(V) + U * r.logp.abs(), "logp")
            assert torch.equal(lse, -logp)
            close(token, term, tol, "token loss")
            close(loss, term.sum(), tol.sum() + U * term.sum().abs(), "loss")
            close(dlogp, slope, tol, "dlogp")
            if want:
                check_grad(d, r, slope, dt, "dlogits", tol)
                one_pass = d
        check_grad(bwd(x, t, lse, dlogp, None, inv_t, dt), r, slope, dt, "backward", tol)
    # in place, and rows that start elsewhere modulo 16 bytes
    other = torch.empty(M * (V + 3) + 16, dtype=TD[dt], device="cuda")[1:1 + M * (V + 3)]
    other = other.view(M, V + 3)[:, :V]
    policy(x, t, old, ref, A, None, kl or 0.0, dt, inv_t, out=other)
    check_grad(other, r, slope, dt, "dlogits elsewhere", tol)
    x2 = x.clone() if pad == 0 else x
    policy(x2, t, old, ref, A, None, kl or 0.0, dt, inv_t, out=x2)
    assert torch.equal(x2, one_pass)


@gpu
def test_policy_loss_where_nothing_is_left():
    x, t, _ = rows(6, 700, "bf16")
    r = Ref(x, t, 1.0)
    old, ref, A, w = policy_inputs(r)
    t[:] = IGNORE
    x[:] = float("nan")
    loss, token, logp, lse, dlogp, d = policy(x, t, old, ref, A, w, 0.1, "bf16")
    for v in (loss, token, logp, lse, dlogp, d):
        assert not v.any()
    loss = policy(x[:0], t[:0], old[:0], ref[:0], A[:0], w[:0], 0.1, "bf16")[0]
    assert loss == 0
    # a weight of zero is worth nothing, whatever else the row holds
    x, t, _ = rows(6, 700, "bf16")
    t[:] = torch.arange(6, device="cuda")
    old[2], A[2], w[2] = float("nan"), float("inf"), 0.0
    loss, token, _, _, dlogp, d = policy(x, t, old, ref, A, w, 0.1, "bf16")
    assert bool(loss.isfinite()) and token[2] == 0 and dlogp[2] == 0 and not d[2].any()
    # a NaN shows
    old[3] = float("nan")
    loss, _, _, _, _, d = policy(x, t, old, ref, A, w, 0.1, "bf16")
    assert bool(loss.isnan()) and bool(d[3].isnan().any()) and bool(d[4].isfinite().all())


@gpu
def test_policy_gradient_against_differences():
    x, t, _ = rows(5, 40, "f32", seed=3)
    t[:] = torch.tensor([3, 39, 0, 17, IGNORE], device="cuda")
    r = Ref(x, t, 1 / 0.8)
    old, ref, A, w = policy_inputs(r, 2)
    d = policy(x, t, old, ref, A, w, 0.2, "f32", 1 / 0.8)[-1]
    h = 1e-6

    def f(x):
        return float(policy_ref(Ref(x, t, 1 / 0.8), old, ref, A, w, 0.2)[0].sum())

    for i, j in [(0, 3), (1, 5), (2, 0), (3, 30), (4, 2)]:
        e = torch.zeros(5, 40, device="cuda", dtype=torch.float64)
        e[i, j] = h
        num = (f(x.double() + e) - f(x.double() - e)) / (2 * h)
        # cancellation 2^-52 |f| / h and truncation stay below 1e-9
        assert abs(num - float(d[i, j])) <= 1e-8 + 1e-5 * abs(num)


@gpu
def test_rows_further_apart_than_32_bits():
    # 8.6 GB apart, of which only the rows are touched
    M, V, ld = 3, 1003, (1 << 31) + 5
    x, t, _ = rows(M, V, "bf16")
    t[1] = 1002
    r = Ref(x, t, 1.0)
    old, ref, A, w = policy_inputs(r)
    far = torch.empty((M - 1) * ld + V, dtype=torch.bfloat16, device="cuda")
    far = far.as_strided((M, V), (ld, 1))
    far.copy_(x)
    logp, lse = fwd(far, t)
    close(logp, r.logp, logp_tol(V) + U * r.logp.abs())
    near = torch.empty(M, V + 1, dtype=torch.bfloat16, device="cuda")[:, :V]
    _, _, _, lse, dlogp, _ = policy(far, t, old, ref, A, w, 0.1, "bf16", out=near)
    want = near.clone()
    policy(far, t, old, ref, A, w, 0.1, "bf16", out=far)      # in place
    _, slope, tol = policy_ref(r, old, ref, A, w, 0.1)
    for got in (want, far):
        check_grad(got, r, slope, "bf16", "dlogits", tol)
    far.copy_(x)
    check_grad(bwd(far, t, lse, dlogp, out=far), r, slope, "bf16", "in place", tol)


@gpu
def test_a_wait_that_runs_out_is_reported(debug_env):
    """A negative limit makes every wait of a cluster for its peers give up at once.  The
    kernel has to end all the same, and the next call to be right."""
    x, t, _ = rows(5, 65536, "bf16")
    r = Ref(x, t, 1.0)
    old, ref, A, w = policy_inputs(r)
    want = policy(x, t, old, ref, A, w, 0.1, "bf16")
    rn.rmsnorm_check_device()
    debug_env.set("RMSNORM_WAIT_LIMIT_CYCLES", "-1")
    policy(x, t, old, ref, A, w, 0.1, "bf16")
    with pytest.raises(rn.RMSNormError) as e:
        rn.rmsnorm_check_device()
    assert e.value.status == 6                   # RMSNORM_ERR_TIMEOUT
    debug_env.delete("RMSNORM_WAIT_LIMIT_CYCLES")
    got = policy(x, t, old, ref, A, w, 0.1, "bf16")
    rn.rmsnorm_check_device()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@gpu
def test_another_familys_forced_variant_is_none_of_theirs(debug_env):
    x, t, _ = rows(40, 3000, "bf16")
    r = Ref(x, t, 1.0)
    old, ref, A, w = policy_inputs(r)
    want = (*fwd(x, t, 1.0, "bf16"), *policy(x, t, old, ref, A, w, 0.1, "bf16"))
    debug_env.set("RMSNORM_FORCE_VARIANT", "cta:t=512:cl=3")
    got = (*fwd(x, t, 1.0, "bf16"), *policy(x, t, old, ref, A, w, 0.1, "bf16"))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# ---------------------------------------------------------------- preference loss

def preference(x, t, ref, cu, beta, ls, dt, inv_t=1.0, stream=None):
    M, V = x.shape
    pairs = (cu.numel() - 1) // 2
    loss = torch.full((), float("nan"), device="cuda")
    margins = torch.full((pairs,), float("nan"), device="cuda")
    logp, lse, dlogp = torch.full((3, M), float("nan"), device="cuda")
    rn.rmsnorm_preference_loss_fwd(x, x.stride(0), t, inv_t, ref, cu, pairs, beta, ls, loss,
                                   margins, logp, lse, dlogp, M, V, dt, stream)
    return loss, margins, logp, lse, dlogp


def preference_ref(r, ref, cu, beta, ls):
    cu = cu.tolist()
    B = (len(cu) - 1) // 2
    gap = r.logp - (ref.double() if ref is not None else 0.0)
    gap = torch.where(r.live, gap, 0.0)
    M, V = r.z.shape
    S = torch.stack([gap[cu[s]:cu[s + 1]].sum() for s in range(2 * B)])
    # an error per row: logp's, and the rounding of the difference
    e = torch.where(r.live, logp_tol(V) + U * gap.abs(), 0.0)
    E = torch.stack([e[cu[s]:cu[s + 1]].sum() for s in range(2 * B)])
    h = beta * (S[:B] - S[B:])
    htol = abs(beta) * (E[:B] + E[B:]) + 2 * U * h.abs()
    sp = torch.nn.functional.softplus
    loss = ((1 - ls) * sp(-h) + ls * sp(h)).mean()
    slope = (ls * torch.sigmoid(h) - (1 - ls) * torch.sigmoid(-h)) * beta / B
    stol = abs(beta) / B * (htol / 4 + POINT)
    d, dtol = torch.zeros(M, device="cuda", dtype=torch.float64), torch.zeros(
        M, device="cuda", dtype=torch.float64)
    for s in range(2 * B):
        a, b = cu[s], cu[s + 1]
        d[a:b] = slope[s % B] if s < B else -slope[s % B]
        dtol[a:b] = stol[s % B]
    d[~r.live] = 0
    return loss, h, d, htol.mean() + POINT * loss, htol, dtol


@gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("with_ref", [True, False])
@pytest.mark.parametrize("cu,M,V", [
    ([0, 1, 2], 2, 30), ([0, 0, 5], 5, 100), ([0, 5, 5], 5, 100), ([0, 0, 0], 3, 100),
    ([2, 30, 41, 41, 80], 90, 1001), ([0, 300, 301, 500, 777, 900, 1200], 1203, 500),
    ([3, 10, 20], 30, 60000), (list(range(0, 82, 1)) + [90, 100, 300], 310, 70),
    ([0, 20000, 20001, 39000, 40000], 40000, 50)])
def test_preference_loss(cu, M, V, with_ref, dt):
    x, t, _ = rows(M, V, dt, seed=V)
    r = Ref(x, t, 1.0)
    ref = (r.logp + 0.3 * torch.randn(M, device="cuda")).float() if with_ref else None
    c = torch.tensor(cu, device="cuda")
    for beta, ls in ((0.1, 0.0), (0.5, 0.2)):
        loss, margins, logp, lse, dlogp = preference(x, t, ref, c, beta, ls, dt)
        L, h, d, ltol, htol, dtol = preference_ref(r, ref, c, beta, ls)
        close(margins, h, htol, "margins")
        close(loss, L, ltol, "loss")
        close(logp, r.logp, logp_tol(V) + U * r.logp.abs(), "logp")
        close(dlogp, d, dtol, "dlogp")
        check_grad(bwd(x, t, lse, dlogp, dt=dt), r, d, dt, "dlogits", dtol)


@gpu
def test_preference_edges():
    x, t, _ = rows(40, 300, "f32")
    r = Ref(x, t, 1.0)
    # offsets behind and before the batch are cut to it
    a = preference(x, t, None, torch.tensor([-5, 20, 99], device="cuda"), 0.3, 0.1, "f32")
    b = preference(x, t, None, torch.tensor([0, 20, 40], device="cuda"), 0.3, 0.1, "f32")
    for u, v in zip(a, b):
        assert torch.equal(u, v)
    # no rows at all: every sequence is empty
    loss, margins, *_ = preference(x[:0], t[:0], None, torch.zeros(5, dtype=torch.long,
                                                                   device="cuda"), 0.3, 0.1, "f32")
    assert abs(float(loss) - math.log(2)) < 1e-6 and not margins.any()
    # margins far out: the loss stays finite
    big = torch.full((40,), -1e4, device="cuda")
    cu = torch.tensor([0, 20, 20], device="cuda")
    loss, margins, _, _, dlogp = preference(x, t, big, cu, 1.0, 0.0, "f32")
    assert float(loss) == 0.0 and float(margins) > 1e4 and not dlogp.any()
    loss, margins, _, _, dlogp = preference(x, t, -big, cu, 1.0, 0.0, "f32")
    assert abs(float(loss) + float(margins)) <= 1e-6 * abs(float(loss))
    assert float(dlogp.min()) == -1.0
    # a NaN shows in its pair and in the loss, not in the others
    x[3, 5] = float("nan")
    t[3] = 1
    loss, margins, *_ = preference(x, t, None, torch.tensor([0, 10, 20, 30, 40], device="cuda"),
                                   0.3, 0.1, "f32")
    assert bool(loss.isnan()) and margins.isnan().tolist() == [True, False]
    del r


# ---------------------------------------------------------------- repeats, graphs, streams

@gpu
@pytest.mark.parametrize("M,V", [(3, 65536), (500, 3001)])
def test_repeats_graphs_and_streams(M, V):
    x, t, _ = rows(M, V, "bf16", V + 7)
    r = Ref(x, t, 1.0)
    old, ref, A, w = policy_inputs(r)
    cu = torch.tensor([0, M // 2, M], device="cuda")

    def step(st):
        p = policy(x, t, old, ref, A, w, 0.1, "bf16", stream=st)
        q = preference(x, t, ref, cu, 0.1, 0.1, "bf16", stream=st)
        return [*p, *q, bwd(x, t, q[3], q[4], stream=st)]

    cur = torch.cuda.current_stream()
    want = [v.clone() for v in step(cur)]
    for a, b in zip(want, step(cur)):
        assert torch.equal(a, b)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        outs = step(torch.cuda.current_stream())
    for _ in range(2):
        for o in outs:
            o.fill_(5)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, outs):
            assert torch.equal(a, b)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for st in streams:
        with torch.cuda.stream(st):
            got.append(step(st))
    torch.cuda.synchronize()
    for o in got:
        for a, b in zip(want, o):
            assert torch.equal(a, b)


# ---------------------------------------------------------------- refusals (no GPU)

@pytest.fixture(scope="module")
def lib():
    from row_wise_normalization_02_gb300 import _build
    _build.build()
    return rn.load_library()


G = 1 << 32
BASE = dict(x=FAKE, ld=1000, t=FAKE + G, inv_t=1.0, logp=FAKE + 2 * G, lse=FAKE + 3 * G, M=4,
            V=1000, dt=1)
SHARED = [
    (dict(M=-1), 1), (dict(M=1 << 28), 1), (dict(V=0), 1), (dict(V=(1 << 30) + 1), 1),
    (dict(ld=999), 1), (dict(ld=1 << 62), 1), (dict(ld=-1000), 1), (dict(inv_t=0.0), 1),
    (dict(inv_t=-1.0), 1), (dict(inv_t=float("nan")), 1), (dict(inv_t=float("inf")), 1),
    (dict(inv_t=1e300), 1), (dict(inv_t=1e-300), 1), (dict(dt=2), 2), (dict(x=None), 1),
    (dict(t=None), 1), (dict(lse=None), 1), (dict(x=FAKE + 1), 3), (dict(t=FAKE + G + 4), 3),
    (dict(lse=FAKE + 3 * G + 2), 3),
]


def refused(status, call):
    with pytest.raises(rn.RMSNormError) as e:
        call()
    assert e.value.status == status


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(logp=None), 1), (dict(logp=FAKE), 1), (dict(logp=FAKE + 3 * G + 8), 1),
    (dict(lse=FAKE + G + 8), 1)])
def test_logprob_refusals(lib, kw, status):
    a = {**BASE, **kw}
    refused(status, lambda: rn.rmsnorm_token_logprob_fwd(
        a["x"], a["ld"], a["t"], a["inv_t"], a["logp"], a["lse"], a["M"], a["V"], a["dt"]))


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(dlogp=None), 1), (dict(out=None), 1), (dict(out=FAKE + 16), 1), (dict(ldo=999), 1),
    (dict(out=FAKE, ldo=1008), 1), (dict(out=FAKE + 1), 3), (dict(scale=FAKE + 6 * G + 1), 3),
    (dict(scale=FAKE + 5 * G + 16), 1), (dict(out=FAKE + 4 * G - 64), 1)])
def test_logits_gradient_refusals(lib, kw, status):
    a = {**BASE, "dlogp": FAKE + 4 * G, "out": FAKE + 5 * G, "ldo": 1000, "scale": None, **kw}
    refused(status, lambda: rn.rmsnorm_token_logprob_bwd(
        a["x"], a["ld"], a["t"], a["inv_t"], a["lse"], a["dlogp"], a["scale"], a["out"], a["ldo"],
        a["M"], a["V"], a["dt"]))


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(old=None), 1), (dict(A=None), 1), (dict(loss=None), 1), (dict(token=None), 1),
    (dict(dlogp=None), 1), (dict(lo=-0.1), 1), (dict(lo=1.5), 1), (dict(hi=-0.1), 1),
    (dict(hi=float("inf")), 1), (dict(lo=float("nan")), 1), (dict(kl=-1.0), 1),
    (dict(kl=float("nan")), 1), (dict(w=FAKE + 9 * G + 2), 3), (dict(loss=FAKE + 3 * G), 1),
    (dict(out=FAKE + 16), 1), (dict(ldo=10), 1), (dict(token=FAKE + 4 * G), 1)])
def test_policy_refusals(lib, kw, status):
    a = {**BASE, "old": FAKE + 4 * G, "ref": FAKE + 5 * G, "A": FAKE + 6 * G, "w": FAKE + 9 * G,
         "lo": 0.2, "hi": 0.2, "kl": 0.1, "loss": FAKE + 7 * G, "token": FAKE + 8 * G,
         "dlogp": FAKE + 10 * G, "out": FAKE + 11 * G, "ldo": 1000, **kw}
    refused(status, lambda: rn.rmsnorm_policy_loss_fwd(
        a["x"], a["ld"], a["t"], a["inv_t"], a["old"], a["ref"], a["A"], a["w"], a["lo"], a["hi"],
        a["kl"], a["loss"], a["token"], a["logp"], a["lse"], a["dlogp"], a["out"], a["ldo"],
        a["M"], a["V"], a["dt"]))


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(cu=None), 1), (dict(pairs=0), 1), (dict(pairs=1 << 24), 1), (dict(pairs=-2), 1),
    (dict(beta=float("inf")), 1), (dict(ls=-0.1), 1), (dict(ls=1.1), 1), (dict(ls=float("nan")), 1),
    (dict(loss=None), 1), (dict(margins=None), 1), (dict(dlogp=None), 1),
    (dict(cu=FAKE + 6 * G + 4), 3), (dict(margins=FAKE + 6 * G), 1)])
def test_preference_refusals(lib, kw, status):
    a = {**BASE, "ref": FAKE + 5 * G, "cu": FAKE + 6 * G, "pairs": 2, "beta": 0.1, "ls": 0.0,
         "loss": FAKE + 7 * G, "margins": FAKE + 8 * G, "dlogp": FAKE + 10 * G, **kw}
    refused(status, lambda: rn.rmsnorm_preference_loss_fwd(
        a["x"], a["ld"], a["t"], a["inv_t"], a["ref"], a["cu"], a["pairs"], a["beta"], a["ls"],
        a["loss"], a["margins"], a["logp"], a["lse"], a["dlogp"], a["M"], a["V"], a["dt"]))


def test_no_rows_touch_nothing(lib):
    rn.rmsnorm_token_logprob_fwd(None, 0, None, 1.0, None, None, 0, 1000, "bf16")
    rn.rmsnorm_token_logprob_bwd(None, 0, None, 1.0, None, None, None, None, 0, 0, 1000, "bf16")
