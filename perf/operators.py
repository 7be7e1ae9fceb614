"""The rotary and token-loss operators at the sizes they are used at: inputs, plain forms, exact values.

Five operators: rotary positions with several axes over the heads of q and k ("rope"), the
same behind the per-head q/k RMSNorm ("norm_rope"), the log-probability of each row's target token
("logprob"), the clipped policy loss with a KL term ("policy") and the preference loss of paired log
ratios ("preference").  `own` selects who computes them: elementary torch operations in 32 bits, or
this package's kernels through its Python binding of the C ABI.
"""
import math

import torch

own = False

_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}
_EPS = 1e-6


def _rope_case(name, op, passes, T, hq, hk, D, R, axes, pairs, order, dtype, packed):
    return {"name": name, "op": op, "passes": passes, "T": T, "hq": hq, "hk": hk, "D": D, "R": R,
            "axes": axes, "pairs": pairs, "order": order, "dtype": dtype, "packed": packed}


def _loss_case(name, op, passes, M, V, dtype, pairs=0, kl=0.0, temperature=1.0):
    return {"name": name, "op": op, "passes": passes, "M": M, "V": V, "dtype": dtype,
            "pairs": pairs, "kl": kl, "temperature": temperature}


def listed():
    return [
        # one sequence's next token, q and k inside the fused QKV projection's row: pure latency
        _rope_case("rope decode 1", "rope", "fwd", 1, 32, 8, 128, 128, 3, "halves", "blocks",
                   "bf16", True),
        # prefill of a long clip: frames x rows x columns behind a text prefix
        _rope_case("rope video prefill", "rope", "fwd", 16384, 32, 8, 128, 128, 3, "halves",
                   "interleaved", "bf16", True),
        # an image tower's gradient: two axes, partial rotation, adjacent pairs, odd token count
        _rope_case("rope image gradient f32", "rope", "bwd", 4097, 16, 16, 80, 64, 2, "adjacent",
                   "blocks", "f32", False),
        # a serving batch's next tokens through q/k norm and rotation in one call
        _rope_case("norm rope decode 64", "norm_rope", "fwd", 64, 32, 8, 128, 128, 3, "halves",
                   "interleaved", "bf16", True),
        # a training step's q/k norm and rotation, forward and backward with both weights' gradients
        _rope_case("norm rope training", "norm_rope", "fwd+bwd", 32768, 32, 8, 128, 128, 3,
                   "halves", "blocks", "bf16", True),
        # scoring the next token of a few sequences
        _loss_case("logprob 8 tokens", "logprob", "fwd", 8, 32768, "bf16"),
        # scoring a rollout under the old policy or the reference model
        _loss_case("logprob scoring", "logprob", "fwd", 8192, 131072, "bf16"),
        # odd vocabulary in 32 bits: rows that start off 16 bytes, sampled at a temperature
        _loss_case("logprob gradient odd f32", "logprob", "fwd+bwd", 1023, 50257, "f32",
                   temperature=0.7),
        # a policy update's loss and the logits' gradient
        _loss_case("policy step", "policy", "fwd+bwd", 4096, 131072, "bf16", kl=0.05),
        # a small model's update without the reference model, odd vocabulary
        _loss_case("policy step odd f32", "policy", "fwd+bwd", 255, 32003, "f32"),
        # preference training on eight pairs of answers
        _loss_case("preference step", "preference", "fwd+bwd", 8192, 65536, "bf16", pairs=8),
        # two short pairs in 32 bits
        _loss_case("preference short f32", "preference", "fwd+bwd", 77, 16384, "f32", pairs=2),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "norm_rope", "logprob", "policy", "preference"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("rope", "norm_rope"):
        D = rng.choice([64, 80, 96, 128, 128, 192, 256, 36])
        R = rng.choice([D, D, D // 2])
        R -= R % 2
        hk = rng.choice([1, 2, 4, 8])
        hq = hk * rng.choice([1, 3, 4, 7])
        most = 32768 * 40 * 128 * 2 // (_SIZE[dtype] * (hq + hk) * D)
        c = _rope_case("", op, rng.choice(["fwd", "bwd", "fwd+bwd"]),
                       _log_int(rng, 1, min(32768, most)), hq, hk, D, R, rng.choice([1, 2, 3]),
                       rng.choice(["halves", "adjacent"]), rng.choice(["blocks", "interleaved"]),
                       dtype, rng.random() < 0.5)
    else:
        V = _log_int(rng, 1000, 131072)
        if rng.random() < 0.5:
            V -= V % 64
        pairs = rng.randint(1, 16) if op == "preference" else 0
        most = 4096 * 131072 * 2 // (_SIZE[dtype] * V)
        M = _log_int(rng, max(1, 2 * pairs), min(32768, most))
        c = _loss_case("", op, rng.choice(["fwd", "fwd+bwd"]) if op == "logprob" else "fwd+bwd",
                       M, V, dtype, pairs, rng.choice([0.0, 0.05]) if op == "policy" else 0.0,
                       rng.choice([1.0, 0.7]))
    del c["name"]
    return c


def work(case):
    es = _SIZE[case["dtype"]]
    fwd, bwd = "fwd" in case["passes"], "bwd" in case["passes"]
    if "T" in case:
        n = case["T"] * (case["hq"] + case["hk"]) * case["D"]
        norm = case["op"] == "norm_rope"
        side = 8 * case["axes"] * case["T"] + 2 * case["R"]
        bytes_ = (2 * es * n + side) * fwd + ((3 if norm else 2) * es * n + side) * bwd
        if fwd and bwd and norm:
            bytes_ -= es * n          # the backward reads the input again: counted once
        return {"bytes": bytes_, "flops": n * ((8 if norm else 3) * fwd + (16 if norm else 3) * bwd)}
    n = case["M"] * case["V"]
    bytes_ = es * n * (2 if bwd else 1) + 40 * case["M"]
    return {"bytes": bytes_, "flops": n * (4 + 4 * bwd)}


# ---------------------------------------------------------------- inputs

def _axis_of(case):
    """The axis each frequency turns by."""
    half, A = case["R"] // 2, case["axes"]
    sec = _sections(case)
    if case["order"] == "blocks":
        return [a for a in range(A) for _ in range(sec[a])]
    return [i % A if i < sec[i % A] * A else 0 for i in range(half)]


def _sections(case):
    half, A = case["R"] // 2, case["axes"]
    rest = [half // A] * (A - 1)
    return [half - sum(rest)] + rest


def _prepare_rope(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    T, hq, hk, D, R = (case[k] for k in ("T", "hq", "hk", "D", "R"))
    dt = _DTYPE[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=dev) * scale).to(dtype)

    st = {"case": case, "T": T, "D": D, "R": R, "sections": _sections(case)}
    if case["packed"]:       # q, k (and v) side by side in the projection's output row
        qkv = normal(T, hq + 2 * hk, D)
        st["q"], st["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
    else:
        st["q"], st["k"] = normal(T, hq, D), normal(T, hk, D)
    st["dq_out"], st["dk_out"] = normal(T, hq, D), normal(T, hk, D)
    # text up to a far position, then frames of 32 x 32 patches
    base = torch.randint(0, 1 << 20, (1,), generator=g, device=dev)
    i = torch.arange(T, device=dev)
    grid = [i // 1024, i // 32 % 32, i % 32] if case["axes"] == 3 else [i // 64, i % 64, i]
    st["positions"] = torch.stack([base + grid[a] for a in range(case["axes"])]).contiguous()
    st["inv_freq"] = (10000.0 ** (-torch.arange(0, R, 2, device=dev, dtype=torch.float64) / R)
                      ).float()
    st["axis"] = torch.tensor(_axis_of(case), device=dev)
    if case["op"] == "norm_rope":
        st["q_gamma"] = (1 + 0.1 * torch.randn(D, generator=g, device=dev)).to(dt)
        st["k_gamma"] = (1 + 0.1 * torch.randn(D, generator=g, device=dev)).to(dt)
    # what the calls write, kept by the program from step to step
    for n in ("q", "k"):
        h = hq if n == "q" else hk
        st[n + "_out"] = torch.empty(T, h, D, device=dev, dtype=dt)
        st["d" + n] = torch.empty_like(st[n + "_out"])
        st["d" + n + "_gamma"] = torch.empty(D, device=dev)
    if own:
        import row_wise_normalization_02_gb300 as rn
        st["rope"] = rn.Rope(st["positions"], st["inv_freq"], st["sections"], R, case["pairs"],
                             case["order"])
        st["views"] = {n: rn.Heads.of(st[n]) for n in ("q", "k", "dq_out", "dk_out", "q_out",
                                                       "k_out", "dq", "dk")}
        st["workspace_bytes"] = rn.rmsnorm_rope_bwd_workspace_size(
            T, hq, hk, D, case["dtype"], case["dtype"])
        st["workspace"] = torch.empty(max(16, st["workspace_bytes"]), dtype=torch.uint8,
                                      device=dev)
        st["stream"] = torch.cuda.current_stream()
    return st


def _prepare_loss(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    M, V = case["M"], case["V"]
    dt = _DTYPE[case["dtype"]]
    logits = torch.empty(M, V, device=dev, dtype=dt)
    logits.normal_(0.0, 2.0, generator=g)
    targets = torch.randint(0, V, (M,), generator=g, device=dev)
    # the target is a likely token more often than not
    rows = torch.arange(M, device=dev)
    lift = 9 + 3 * torch.randn(M, generator=g, device=dev)
    logits[rows, targets] = (logits[rows, targets].float() + lift).to(dt)
    # prompt and padding tokens take no part
    masked = torch.rand(M, generator=g, device=dev) < 0.2
    targets = torch.where(masked & (rows > 0), torch.full_like(targets, -100), targets)
    st = {"case": case, "M": M, "V": V, "logits": logits, "targets": targets,
          "inv_temperature": 1.0 / case["temperature"]}
    st["dlogp_in"] = torch.randn(M, generator=g, device=dev) / M
    if case["op"] == "policy":
        # the old policy's ratio spreads around 1 and passes the clip borders (0.8, 1.28); a token
        # within 1e-4 of a border has a gradient no 32-bit sum decides, so none is put there
        ratio = torch.exp(0.15 * torch.randn(M, generator=g, device=dev, dtype=torch.float64))
        for border in (0.8, 1.28):
            near = (ratio - border).abs() < 1e-4
            ratio = torch.where(near, ratio + 3e-4, ratio)
        st["clip_low"], st["clip_high"] = 0.2, 0.28
        logp = _row_logp(st)
        st["old_logp"] = (logp - ratio.log()).float()
        st["ref_logp"] = (logp + 0.3 * torch.randn(M, generator=g, device=dev,
                                                   dtype=torch.float64)).float()
        if not case["kl"]:
            st["ref_logp"] = None
        st["advantages"] = torch.randn(M, generator=g, device=dev)
        live = targets >= 0
        st["weights"] = live.float() / live.sum()
    if case["op"] == "preference":
        # answers of uneven length packed end to end, the chosen ones first; a few rows behind the
        # last belong to none
        S = 2 * case["pairs"]
        cuts = torch.rand(S, generator=g, device=dev, dtype=torch.float64) + 0.25
        ends = (cuts.cumsum(0) / cuts.sum() * (M - M // 50)).long()
        st["cu_seqlens"] = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), ends])
        st["ref_logp"] = (_row_logp(st) + 0.05 * torch.randn(M, generator=g, device=dev,
                                                             dtype=torch.float64)).float()
        st["beta"], st["label_smoothing"] = 0.1, 0.1
        st["margins"] = torch.empty(case["pairs"], device=dev)
    st["loss"] = torch.empty((), device=dev)
    for n in ("logp", "lse", "dlogp", "token_loss"):
        st[n] = torch.empty(M, device=dev)
    st["dlogits"] = torch.empty_like(logits)
    if own:
        st["stream"] = torch.cuda.current_stream()
    return st


def _row_logp(st):
    """The targets' log-probabilities for making inputs, a few rows at a time."""
    out = []
    t = st["targets"].clamp(min=0)
    step = max(1, (1 << 27) // st["V"])
    for a in range(0, st["M"], step):
        z = st["logits"][a:a + step].float() * st["inv_temperature"]
        m = z.amax(1, keepdim=True)
        lse = m[:, 0].double() + (z - m).exp().sum(1).double().log()
        out.append(z.gather(1, t[a:a + step, None])[:, 0].double() - lse)
    return torch.cat(out)


def prepare(case, seed):
    return (_prepare_rope if "T" in case else _prepare_loss)(case, seed)


# ---------------------------------------------------------------- plain forms

def _rotate(x, cos, sin, pairs, R):
    """x [T, H, D] in 32 bits, its first R columns turned by the angles of cos, sin [T, 1, R / 2]."""
    if pairs == "halves":
        u, v = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat([u * cos - v * sin, u * sin + v * cos], -1)
    else:
        u, v = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack([u * cos - v * sin, u * sin + v * cos], -1).flatten(-2)
    return torch.cat([y, x[..., R:]], -1)


def _plain_rope(st):
    case, R = st["case"], st["R"]
    dt, norm = _DTYPE[case["dtype"]], case["op"] == "norm_rope"
    angle = (st["positions"][st["axis"]].double() * st["inv_freq"].double()[:, None]).t()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def forward(x, gamma):
        x = x.float()
        if norm:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS) * gamma.float()
        return _rotate(x, cos, sin, case["pairs"], R).to(dt)

    def backward(dy, x, gamma):
        g = _rotate(dy.float(), cos, -sin, case["pairs"], R)
        if not norm:
            return g.to(dt), None
        x, w = x.float(), gamma.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS)
        c = r * r * (w * g * x).mean(-1, keepdim=True)
        return (r * (w * g - x * c)).to(dt), (g * x * r).sum((0, 1))

    out = {}
    qg, kg = st.get("q_gamma"), st.get("k_gamma")
    if "fwd" in case["passes"]:
        out["q"], out["k"] = forward(st["q"], qg), forward(st["k"], kg)
    if "bwd" in case["passes"]:
        out["dq"], out["dq_gamma"] = backward(st["dq_out"], st["q"], qg)
        out["dk"], out["dk_gamma"] = backward(st["dk_out"], st["k"], kg)
    return out


def _plain_loss(st):
    case = st["case"]
    live = st["targets"] >= 0
    t = st["targets"].clamp(min=0)[:, None]
    z = st["logits"].float() * st["inv_temperature"]
    m = z.amax(1, keepdim=True)
    lse = m[:, 0].double() + (z - m).exp().sum(1).double().log()
    logp = torch.where(live, z.gather(1, t)[:, 0].double() - lse, 0.0)
    out = {"logp": logp.float()}
    if case["op"] == "logprob":
        dlogp = st["dlogp_in"].double()
    elif case["op"] == "policy":
        A = st["advantages"].double()
        r = (logp - st["old_logp"].double()).exp()
        lo, hi = 1 - st["clip_low"], 1 + st["clip_high"]
        s = torch.minimum(r * A, r.clamp(lo, hi) * A)
        clipped = torch.where(A >= 0, r > hi, r < lo)
        term, slope = -s, torch.where(clipped, 0.0, -A * r)
        if st["ref_logp"] is not None:
            d = st["ref_logp"].double() - logp
            term = term + case["kl"] * (torch.expm1(d) - d)
            slope = slope - case["kl"] * torch.expm1(d)
        w = torch.where(live, st["weights"].double(), 0.0)
        token_loss = torch.where(live, w * term, 0.0)
        out["loss"], out["token_loss"] = token_loss.sum().float(), token_loss.float()
        dlogp = w * slope
    else:
        rows = torch.arange(st["M"], device=logp.device)
        cu, B = st["cu_seqlens"], case["pairs"]
        seq = torch.searchsorted(cu, rows, right=True) - 1
        sign = torch.where(seq < B, 1.0, -1.0).double()
        inside = live & (seq < 2 * B)
        gap = torch.where(inside, sign * (logp - st["ref_logp"].double()), 0.0)
        h = torch.zeros(B, device=logp.device, dtype=torch.float64)
        h = st["beta"] * h.index_add(0, seq % B, gap)
        ls = st["label_smoothing"]
        soft = lambda v: torch.log1p(torch.exp(-v.abs())) + (-v).clamp(min=0)  # noqa: E731
        out["loss"] = ((1 - ls) * soft(h) + ls * soft(-h)).mean().float()
        out["margins"] = h.float()
        slope = (ls / (1 + torch.exp(-h)) - (1 - ls) / (1 + torch.exp(h))) / B
        dlogp = torch.where(inside, st["beta"] * sign * slope[seq % B], 0.0)
    if "bwd" in case["passes"]:
        d = torch.where(live, dlogp, 0.0).float()[:, None] * st["inv_temperature"]
        p = (z - lse.float()[:, None]).exp()
        grad = -d * p
        grad.scatter_add_(1, t, d)
        out["dlogits"] = grad.to(st["logits"].dtype)
    return out


# ---------------------------------------------------------------- the package's calls

def _own_rope(st):
    import row_wise_normalization_02_gb300 as rn
    case, v = st["case"], st["views"]
    dt, passes = case["dtype"], case["passes"]
    qg, kg = st.get("q_gamma"), st.get("k_gamma")
    out = {}
    if "fwd" in passes:
        rn.rmsnorm_rope_fwd(v["q"], v["k"], qg, kg, v["q_out"], v["k_out"], st["rope"], st["T"],
                            st["D"], _EPS, dt, dt, st["stream"])
        out["q"], out["k"] = st["q_out"], st["k_out"]
    if "bwd" in passes:
        norm = qg is not None
        rn.rmsnorm_rope_bwd(v["dq_out"], v["dk_out"], v["q"], v["k"], qg, kg, v["dq"], v["dk"],
                            st["dq_gamma"] if norm else None, st["dk_gamma"] if norm else None,
                            st["workspace"], st["workspace_bytes"], st["rope"], st["T"], st["D"],
                            _EPS, dt, dt, st["stream"])
        out["dq"], out["dk"] = st["dq"], st["dk"]
        if norm:
            out["dq_gamma"], out["dk_gamma"] = st["dq_gamma"], st["dk_gamma"]
    return out


def _own_loss(st):
    import row_wise_normalization_02_gb300 as rn
    case, M, V, dt = st["case"], st["M"], st["V"], st["case"]["dtype"]
    it, s = st["inv_temperature"], st["stream"]
    bwd = "bwd" in case["passes"]
    out = {"logp": st["logp"]}
    dlogp = st["dlogp"]
    if case["op"] == "logprob":
        rn.rmsnorm_token_logprob_fwd(st["logits"], V, st["targets"], it, st["logp"], st["lse"], M,
                                     V, dt, s)
        dlogp = st["dlogp_in"]
    elif case["op"] == "policy":
        rn.rmsnorm_policy_loss_fwd(st["logits"], V, st["targets"], it, st["old_logp"],
                                   st["ref_logp"], st["advantages"], st["weights"],
                                   st["clip_low"], st["clip_high"], case["kl"], st["loss"],
                                   st["token_loss"], st["logp"], st["lse"], dlogp,
                                   st["dlogits"], V, M, V, dt, s)
        out["loss"], out["token_loss"] = st["loss"], st["token_loss"]
    else:
        rn.rmsnorm_preference_loss_fwd(st["logits"], V, st["targets"], it, st["ref_logp"],
                                       st["cu_seqlens"], case["pairs"], st["beta"],
                                       st["label_smoothing"], st["loss"], st["margins"],
                                       st["logp"], st["lse"], dlogp, M, V, dt, s)
        out["loss"], out["margins"] = st["loss"], st["margins"]
    if bwd and case["op"] != "policy":
        rn.rmsnorm_token_logprob_bwd(st["logits"], V, st["targets"], it, st["lse"], dlogp, None,
                                     st["dlogits"], V, M, V, dt, s)
    if bwd:
        out["dlogits"] = st["dlogits"]
    return out


def run(state):
    rope = "T" in state["case"]
    if own:
        return _own_rope(state) if rope else _own_loss(state)
    return _plain_rope(state) if rope else _plain_loss(state)


# ---------------------------------------------------------------- exact values

def _exact_rope(case, seed):
    """Pairs as complex numbers times exp(i theta); gradients by differentiating that."""
    st = _prepare_rope(case, seed)
    R = case["R"]
    pos = st["positions"].double().cpu()
    freq = st["inv_freq"].double().cpu()
    theta = torch.stack([pos[a] * f for a, f in zip(_axis_of(case), freq)], -1).cuda()
    turn = torch.polar(torch.ones_like(theta), theta)[:, None, :]

    def value(x, gamma):
        if gamma is not None:
            x = gamma * x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + _EPS).sqrt()
        if case["pairs"] == "halves":
            c = torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:R].contiguous()) * turn
            y = torch.cat([c.real, c.imag], -1)
        else:
            c = torch.view_as_complex(x[..., :R].reshape(*x.shape[:-1], R // 2, 2)) * turn
            y = torch.view_as_real(c).reshape(*x.shape[:-1], R)
        return torch.cat([y, x[..., R:]], -1)

    out = {}
    for n in ("q", "k"):
        leaf = [st[n].double().requires_grad_()]
        if case["op"] == "norm_rope":
            leaf.append(st[n + "_gamma"].double().requires_grad_())
        y = value(leaf[0], leaf[1] if len(leaf) > 1 else None)
        if "fwd" in case["passes"]:
            out[n] = y.detach()
        if "bwd" in case["passes"]:
            grads = torch.autograd.grad(y, leaf, st["d" + n + "_out"].double())
            for key, gr in zip(("d" + n, "d" + n + "_gamma"), grads):
                out[key] = gr
        del y
    return out


def _exact_loss(case, seed):
    """The loss as a function of 64-bit log-probabilities, differentiated; rows in groups."""
    st = _prepare_loss(case, seed)
    M, V, temp = st["M"], st["V"], case["temperature"]
    t, live = st["targets"].clamp(min=0), st["targets"] >= 0
    step = max(1, (1 << 26) // V)

    def group(a):
        return torch.log_softmax(st["logits"][a:a + step].double() / temp, 1)

    logp = torch.cat([group(a).gather(1, t[a:a + step, None])[:, 0] for a in range(0, M, step)])
    logp = torch.where(live, logp, torch.zeros_like(logp)).requires_grad_()
    out = {"logp": logp.detach()}
    if case["op"] == "logprob":
        total = (logp * st["dlogp_in"].double())[live].sum()
    elif case["op"] == "policy":
        A, w = st["advantages"].double()[live], st["weights"].double()[live]
        lp = logp[live]
        r = torch.exp(lp - st["old_logp"].double()[live])
        s = torch.minimum(r * A, torch.clamp(r, 1 - st["clip_low"], 1 + st["clip_high"]) * A)
        each = -w * s
        if st["ref_logp"] is not None:
            ref = st["ref_logp"].double()[live]
            each = each + case["kl"] * w * (torch.exp(ref - lp) - (ref - lp) - 1)
        total = each.sum()
        out["loss"] = total.detach()
        out["token_loss"] = torch.zeros_like(logp).index_put((live,), each).detach()
    else:
        cu, B = st["cu_seqlens"].tolist(), case["pairs"]
        ratio = torch.where(live, logp - st["ref_logp"].double(), torch.zeros_like(logp))
        sums = [ratio[cu[s]:cu[s + 1]].sum() for s in range(2 * B)]
        h = st["beta"] * torch.stack([sums[b] - sums[B + b] for b in range(B)])
        ls = st["label_smoothing"]
        total = -((1 - ls) * torch.nn.functional.logsigmoid(h)
                  + ls * torch.nn.functional.logsigmoid(-h)).mean()
        out["loss"], out["margins"] = total.detach(), h.detach()
    if "bwd" in case["passes"]:
        d = torch.autograd.grad(total, logp)[0]
        d = torch.where(live, d, torch.zeros_like(d)) / temp
        grad = torch.empty(M, V, device=d.device, dtype=torch.float64)
        for a in range(0, M, step):
            one = torch.zeros_like(grad[a:a + step]).scatter_(1, t[a:a + step, None], 1.0)
            grad[a:a + step] = d[a:a + step, None] * (one - group(a).exp())
        out["dlogits"] = grad
    return out


def exact(case, seed):
    return (_exact_rope if "T" in case else _exact_loss)(case, seed)
