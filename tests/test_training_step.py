"""The rotary and token-loss autograd functions: against a plain PyTorch graph in
64 bits, alone and together as a post-training step runs them -- RMSNorm, a fused
projection, the per-head norm with rotary positions over its q and k slices,
attention, the final fused-add RMSNorm, logits, and the policy or the preference
loss, backward to every weight.

Tolerance of the step: in fp32, activations of magnitude about one pass through some
ten operations of at most 512-term sums; with independent roundings of 2^-24 a
relative error of 2^-24 * sqrt(10 * 512) = 4e-6 of a gradient's norm is expected;
5e-5 allows an order for terms that cancel.  A mistake in a kernel or in a
marshalled argument is wrong by orders more.  The single functions are held to
1e-5 of the norm.
"""
import pytest
import torch

import row_wise_normalization_02_gb300 as rn
from row_wise_normalization_02_gb300 import autograd as ag

gpu = pytest.mark.gpu


def near(got, ref, tol=1e-5):
    assert got.shape == ref.shape
    got, ref = got.detach(), ref.detach()
    err = float((got.double() - ref.double()).norm())
    assert err <= tol * float(ref.double().norm()) + 1e-12, (err, float(ref.norm()))


def plain_rms(x, w, eps=1e-6):
    return x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w


def plain_rope(x, positions, inv_freq, sections, pairs, order):
    R, A = 2 * sum(sections), len(sections)
    if order == "blocks":
        axis = [a for a in range(A) for _ in range(sections[a])]
    else:
        axis = [i % A if i < sections[i % A] * A else 0 for i in range(R // 2)]
    th = (positions.reshape(A, -1)[axis].double() * inv_freq.double()[:, None]).t()
    c, s = (f(th).reshape(*x.shape[:-2], 1, R // 2) for f in (torch.cos, torch.sin))
    if pairs == "halves":
        u, v = x[..., :R // 2], x[..., R // 2:R]
        return torch.cat([u * c - v * s, u * s + v * c, x[..., R:]], -1)
    u, v = x[..., 0:R:2], x[..., 1:R:2]
    return torch.cat([torch.stack([u * c - v * s, u * s + v * c], -1).flatten(-2), x[..., R:]], -1)


def gen(seed=0):
    return torch.Generator("cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


@gpu
@pytest.mark.parametrize("pairs,order", [("halves", "interleaved"), ("adjacent", "blocks")])
@pytest.mark.parametrize("layout", ["packed", "heads first", "broadcast", "alone"])
@pytest.mark.parametrize("norm", [False, True])
def test_rope_functions(pairs, order, layout, norm):
    B, S, Hq, Hk, D, sections = 2, 37, 6, 2, 96, [12, 10, 10]
    g = gen(1)
    pos = torch.randint(0, 5000, (3, B, S), device="cuda", generator=g)
    inv = (10000.0 ** (-torch.arange(32, device="cuda") / 32)).float()
    wq, wk = ((1 + 0.2 * randn(g, D)).requires_grad_() for _ in range(2))
    if layout == "packed":
        leaf = randn(g, B, S, (Hq + 2 * Hk) * D).requires_grad_()
        cut = lambda t: (t.view(B, S, -1, D)[:, :, :Hq],  # noqa: E731
                         t.view(B, S, -1, D)[:, :, Hq:Hq + Hk])
    elif layout == "heads first":
        leaf = randn(g, B, Hq + Hk, S, D).requires_grad_()
        cut = lambda t: (t[:, :Hq].transpose(1, 2), t[:, Hq:].transpose(1, 2))  # noqa: E731
    elif layout == "broadcast":      # one key head expanded over two
        leaf = randn(g, B, S, Hq + 1, D).requires_grad_()
        cut = lambda t: (t[:, :, :Hq], t[:, :, Hq:].expand(B, S, Hk, D))  # noqa: E731
    else:
        leaf = randn(g, B, S, Hq, D).requires_grad_()
        cut = lambda t: (t, None)  # noqa: E731
    q, k = cut(leaf)
    if norm:
        yq, yk = ag.rms_norm_rope(q, k, wq, wk if k is not None else None, pos, inv, sections,
                                  pairs, order)
    else:
        yq, yk = ag.rope(q, k, pos, inv, sections, pairs, order)
    leaf64 = leaf.detach().double().requires_grad_()
    w64 = [w.detach().double().requires_grad_() for w in (wq, wk)]
    ys, grads = [yq] + [yk] * (k is not None), []
    refs = []
    for x, w in zip(cut(leaf64), w64):
        if x is not None:
            x = plain_rms(x, w) if norm else x
            refs.append(plain_rope(x, pos, inv, sections, pairs, order))
    for y, r in zip(ys, refs):
        near(y, r)
        grads.append(randn(g, *y.shape))
    torch.autograd.backward(ys, grads)
    torch.autograd.backward(refs, [d.double() for d in grads])
    near(leaf.grad, leaf64.grad)
    if norm:
        near(wq.grad, w64[0].grad)
        if k is not None:
            near(wk.grad, w64[1].grad)


@gpu
def test_rope_bf16_and_one_axis_without_its_dimension():
    g = gen(2)
    x = randn(g, 50, 4, 64).bfloat16().requires_grad_()
    pos = torch.arange(50, device="cuda")
    inv = (10000.0 ** (-torch.arange(32, device="cuda") / 32)).float()
    w = torch.ones(64, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    y, none = ag.rms_norm_rope(x, None, w, None, pos, inv, [32])
    assert none is None
    y.sum().backward()         # an expanded gradient
    x64, w64 = (t.detach().double().requires_grad_() for t in (x, w))
    r = plain_rope(plain_rms(x64, w64), pos, inv, [32], "halves", "blocks")
    r.sum().backward()
    # one rounding to bf16: 2^-8 of each value
    near(y, r, 2 ** -8)
    near(x.grad, x64.grad, 2 ** -8)
    near(w.grad, w64.grad, 2 ** -8)
    assert w.grad.dtype == torch.bfloat16


def losses64(z, t, kind, extra):
    """The loss of 64-bit scaled logits as a plain graph."""
    live = t >= 0
    logp = torch.log_softmax(z, -1).gather(-1, t.clamp(min=0)[..., None])[..., 0]
    logp = torch.where(live, logp, torch.zeros_like(logp))
    if kind == "policy":
        old, adv, ref, kl, w = extra
        r = (logp - old.double()).exp()
        s = torch.minimum(r * adv, r.clamp(0.8, 1.2) * adv)
        d = ref.double() - logp
        each = kl * (d.exp() - d - 1) - s
        w = live.double() / live.sum() if w is None else w.double()
        return (torch.where(live, each, torch.zeros_like(each)) * w).sum(), logp
    cu, ref, beta = extra
    gap = torch.where(live, logp - ref.double(), torch.zeros_like(logp)).reshape(-1)
    B = (len(cu) - 1) // 2
    S = [gap[cu[i]:cu[i + 1]].sum() for i in range(2 * B)]
    h = beta * torch.stack([S[b] - S[B + b] for b in range(B)])
    return torch.nn.functional.softplus(-h).mean(), h


@gpu
@pytest.mark.parametrize("padded", [0, 7, 47])
@pytest.mark.parametrize("kind", ["logprob", "policy", "preference"])
def test_loss_functions(kind, padded):
    B, S, V, T = 4, 25, 1009, 0.8
    g = gen(3)
    leaf = randn(g, B, S, V + padded).requires_grad_()
    t = torch.randint(0, V, (B, S), device="cuda", generator=g)
    t[torch.rand(B, S, device="cuda", generator=g) < 0.3] = -100
    leaf64 = leaf.detach().double().requires_grad_()
    z = leaf64[..., :V] / T
    old = (torch.log_softmax(z, -1).gather(-1, t.clamp(min=0)[..., None])[..., 0].detach()
           + 0.05 * randn(g, B, S)).float()
    ref, adv = old + 0.1 * randn(g, B, S), randn(g, B, S)
    up = 3.0
    if kind == "logprob":
        logp = ag.token_logprobs(leaf[..., :V], t, T)
        want = losses64(z, t, "policy", (old, adv, ref, 0.1, None))[1]
        near(logp, want)
        d = randn(g, B, S)
        logp.backward(d)
        want.backward(d.double())
    else:
        if kind == "policy":
            loss, more = ag.policy_loss(leaf[..., :V], t, old, adv, ref, clip_low=0.2,
                                        clip_high=0.2, kl_coef=0.1, temperature=T)
            want, wm = losses64(z, t, "policy", (old, adv, ref, 0.1, None))
        else:
            cu = [0, 25, 40, 75, 98]
            loss, more = ag.preference_loss(leaf[..., :V], t, torch.tensor(cu, device="cuda"), ref,
                                            0.2, temperature=T)
            want, wm = losses64(z, t, "preference", (cu, ref, 0.2))
        near(loss, want.detach())
        near(more, wm.detach(), 1e-4)
        assert not more.requires_grad
        (loss * up).backward()
        (want * up).backward()
    near(leaf.grad, leaf64.grad)
    if padded:
        assert not leaf.grad[..., V:].any()


@gpu
def test_loss_gradient_twice_and_transposed_logits():
    g = gen(4)
    base = randn(g, 300, 40).requires_grad_()
    logits = base.t()                               # rows that are not contiguous: copied
    t = torch.randint(0, 300, (40,), device="cuda", generator=g)
    old, adv = randn(g, 40) - 6, randn(g, 40)
    loss, _ = ag.policy_loss(logits, t, old, adv, weights=torch.rand(40, device="cuda"))
    a, = torch.autograd.grad(loss, base, retain_graph=True)
    b, = torch.autograd.grad(loss, base)
    assert torch.equal(a, b)
    with torch.no_grad():                           # nothing is kept without a gradient
        assert ag.token_logprobs(logits, t).grad_fn is None


def weights(g, dt, D=128, H=4, Hk=2, dh=32, V=503):
    w = {"emb": randn(g, V, D), "n1": 1 + 0.1 * randn(g, D), "n2": 1 + 0.1 * randn(g, D),
         "qkv": randn(g, (H + 2 * Hk) * dh, D) / D ** 0.5, "o": randn(g, D, H * dh) / D ** 0.5,
         "qn": 1 + 0.1 * randn(g, dh), "kn": 1 + 0.1 * randn(g, dh), "head": randn(g, V, D) / 6}
    return {k: v.to(dt).requires_grad_() for k, v in w.items()}


def model(w, tokens, pos, inv, sections, ours, H=4, Hk=2, dh=32):
    B, S = tokens.shape
    x = w["emb"][tokens]
    n = ag.rms_norm(x, w["n1"]) if ours else plain_rms(x, w["n1"])
    qkv = (n @ w["qkv"].t()).view(B, S, H + 2 * Hk, dh)
    q, k, v = qkv[:, :, :H], qkv[:, :, H:H + Hk], qkv[:, :, H + Hk:]
    if ours:
        q, k = ag.rms_norm_rope(q, k, w["qn"], w["kn"], pos, inv, sections, "halves",
                                "interleaved")
    else:
        q = plain_rope(plain_rms(q, w["qn"]), pos, inv, sections, "halves", "interleaved")
        k = plain_rope(plain_rms(k, w["kn"]), pos, inv, sections, "halves", "interleaved")
    k, v = (a.repeat_interleave(H // Hk, 2).transpose(1, 2) for a in (k, v))
    a = q.transpose(1, 2) @ k.transpose(2, 3) / dh ** 0.5
    a = a + torch.full((S, S), float("-inf"), device="cuda", dtype=a.dtype).triu(1)
    o = (a.softmax(-1) @ v).transpose(1, 2).reshape(B, S, H * dh) @ w["o"].t()
    y = ag.fused_add_rms_norm(o, x, w["n2"])[0] if ours else plain_rms(x + o, w["n2"])
    return y @ w["head"].t()


@gpu
@pytest.mark.parametrize("kind", ["policy", "preference"])
def test_a_step_of_all_of_them(kind):
    g = gen(5)
    B, S = 4, 24
    w = weights(g, torch.float32)
    w64 = {k: v.detach().double().requires_grad_() for k, v in w.items()}
    tokens = torch.randint(0, 503, (B, S), device="cuda", generator=g)
    t = tokens.roll(-1, 1).clone()
    t[:, -1] = -100
    t[0, :9] = -100
    pos = torch.randint(0, 300, (3, B, S), device="cuda", generator=g).sort(-1)[0]
    inv = (10000.0 ** (-torch.arange(16, device="cuda") / 16)).float()
    sections = [6, 5, 5]
    with torch.no_grad():
        old = ag.token_logprobs(model(w, tokens, pos, inv, sections, True), t)
    old, ref, adv = old + 0.03 * randn(g, B, S), old + 0.1 * randn(g, B, S), randn(g, B, S)
    logits = model(w, tokens, pos, inv, sections, True)
    z = model(w64, tokens, pos, inv, sections, False)
    near(logits, z.detach(), 5e-5)
    if kind == "policy":
        loss, _ = ag.policy_loss(logits, t, old, adv, ref, kl_coef=0.05)
        want, _ = losses64(z, t, kind, (old, adv, ref, 0.05, None))
    else:
        cu = [0, S, 2 * S, 3 * S, 4 * S]
        loss, _ = ag.preference_loss(logits, t, torch.tensor(cu, device="cuda"), ref, 0.1)
        want, _ = losses64(z, t, kind, (cu, ref, 0.1))
    loss.backward()
    want.backward()
    near(loss.detach(), want.detach(), 5e-5)
    for k in w:
        near(w[k].grad, w64[k].grad, 5e-5)


@gpu
def test_a_captured_step_replays_on_new_inputs():
    g = gen(7)
    B, S = 2, 16
    w = weights(g, torch.float32)
    inv, sections = (10000.0 ** (-torch.arange(16, device="cuda") / 16)).float(), [6, 5, 5]

    def inputs():
        tokens = torch.randint(0, 503, (B, S), device="cuda", generator=g)
        return [tokens, tokens.roll(-1, 1), torch.randint(0, 300, (3, B, S), device="cuda",
                                                          generator=g),
                -6 + 0.1 * randn(g, B, S), randn(g, B, S)]

    def step(tokens, t, pos, old, adv):
        loss, _ = ag.policy_loss(model(w, tokens, pos, inv, sections, True), t, old, adv, old,
                                 kl_coef=0.05)
        return (loss, *torch.autograd.grad(loss, list(w.values())))

    held = inputs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*held)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*held)
    for _ in range(2):
        new = inputs()
        for a, b in zip(held, new):
            a.copy_(b)
        graph.replay()
        for a, b in zip(out, step(*new)):
            near(a.detach(), b.detach().double(), 5e-5)


@gpu
def test_one_pass_gradient_matches_the_autograd_step():
    # the C ABI's one-pass policy gradient is the autograd functions' gradient
    g = gen(6)
    M, V = 200, 3001
    x = randn(g, M, V).requires_grad_()
    t = torch.randint(-1, V, (M,), device="cuda", generator=g)
    old, adv, w = randn(g, M) - 8, randn(g, M), torch.rand(M, device="cuda", generator=g)
    loss, logp = ag.policy_loss(x, t, old, adv, weights=w)
    loss.backward()
    out, l1 = torch.empty_like(x), torch.empty((), device="cuda")
    tk, lp, ls, dl = torch.empty(4, M, device="cuda")
    rn.rmsnorm_policy_loss_fwd(x, V, t, 1.0, old, None, adv, w, 0.2, 0.2, 0.0, l1, tk, lp, ls, dl,
                               out, V, M, V, "f32", torch.cuda.current_stream())
    # (another kernel, its sums split another way)
    near(l1, loss)
    near(lp, logp)
    near(out, x.grad)


def test_arguments_are_checked_before_any_call():
    x, t = torch.randn(3, 8), torch.zeros(3, dtype=torch.int64)
    q, pos, inv = torch.randn(5, 2, 8), torch.zeros(1, 5, dtype=torch.int64), torch.ones(4)
    for call in (lambda: ag.token_logprobs(x, t), lambda: ag.policy_loss(x, t, x[:, 0], x[:, 0]),
                 lambda: ag.preference_loss(x, t, torch.zeros(3, dtype=torch.int64)),
                 lambda: ag.rope(q, None, pos, inv, [4]),
                 lambda: ag.rms_norm_rope(q, None, torch.ones(8), None, pos, inv, [4])):
        with pytest.raises(ValueError):
            call()


@gpu
def test_positions_as_they_come():
    # one row of positions for every axis, and positions held token by token
    g = torch.Generator("cuda").manual_seed(3)
    q = torch.randn(2, 9, 3, 32, device="cuda", generator=g)
    inv = 100.0 ** (-torch.arange(16, device="cuda") / 16)
    pos = torch.randint(0, 4000, (3, 2, 9), device="cuda", generator=g)
    want, _ = ag.rope(q, None, pos, inv, [6, 5, 5])
    apart = pos.permute(1, 2, 0).contiguous().permute(2, 0, 1)
    assert torch.equal(ag.rope(q, None, apart, inv, [6, 5, 5])[0], want)
    same = pos[:1].expand(3, -1, -1)
    one, _ = ag.rope(q, None, pos[0], inv, [16])
    assert torch.equal(ag.rope(q, None, same, inv, [6, 5, 5])[0], one)
    flat, _ = ag.rope(q[0], None, same[:, 0], inv, [6, 5, 5])
    assert torch.equal(flat, one[0])


@gpu
def test_last_tokens_of_long_sequences():
    # rows far apart: their gradient takes the rows' own memory, not the stride's
    x = torch.randn(2, 1500, 1001, device="cuda")
    t = torch.tensor([5, 900], device="cuda")
    rows = x[:, -1].detach().requires_grad_(True)
    before = torch.cuda.memory_allocated()
    d, = torch.autograd.grad(ag.token_logprobs(rows, t).sum(), rows)
    assert torch.cuda.memory_allocated() - before < 1 << 17
    p = torch.softmax(rows.double(), -1)
    want = torch.nn.functional.one_hot(t, 1001) - p
    # an exponent below 32 in two roundings, and the sum behind rel_lse: some 120 x 2^-24
    assert bool(((d - want).abs() <= 2.0 ** -17 * p + 2.0 ** -22 * want.abs()).all())


@gpu
def test_wrong_shapes_are_refused():
    q, k = torch.randn(5, 4, 8, device="cuda"), torch.randn(5, 2, 8, device="cuda")
    pos, inv = torch.zeros(2, 5, dtype=torch.int64, device="cuda"), torch.ones(4, device="cuda")
    w = torch.ones(8, device="cuda")
    for bad in (lambda: ag.rope(q, k[:4], pos, inv, [2, 2]),
                lambda: ag.rope(q, k.half(), pos, inv, [2, 2]),
                lambda: ag.rope(q, k, pos[:, :4], inv, [2, 2]),
                lambda: ag.rope(q, k, pos, inv, [2, 1]),
                lambda: ag.rope(q, k, pos.cpu(), inv, [2, 2]),
                lambda: ag.rms_norm_rope(q, k, w[:4], w, pos, inv, [2, 2]),
                lambda: ag.rms_norm_rope(q, k, w, w.bfloat16(), pos, inv, [2, 2])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ValueError):
        ag.rms_norm_rope(q, k, None, w, pos, inv, [2, 2])
    with pytest.raises(rn.RMSNormError):
        ag.rms_norm_rope(q, k, w, None, pos, inv, [2, 2])
    x, t = torch.randn(3, 8, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")
    for bad in (lambda: ag.token_logprobs(x, t.int()), lambda: ag.token_logprobs(x, t[:2]),
                lambda: ag.policy_loss(x, t, x[:2, 0], x[:, 0]),
                lambda: ag.preference_loss(x, t, t[:2])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        ag.token_logprobs(x.half(), t)
