"""PyTorch training functions over the C ABI.

Forward and backward both run in this library's kernels; PyTorch allocates
the outputs, the tensors saved for the backward and the backward's
workspace, and supplies the current stream.

    y = rms_norm(x, gamma, eps)
    y, h = fused_add_rms_norm(x, residual, gamma, eps)     # h = residual + x
    y = layer_norm(x, gamma, beta, eps)                    # beta may be None
    q, k = rope(q, k, positions, inv_freq, sections)       # k may be None
    q, k = rms_norm_rope(q, k, q_gamma, k_gamma, positions, inv_freq, sections)
    logp = token_logprobs(logits, targets)
    loss, logp = policy_loss(logits, targets, old_logp, advantages, ref_logp)
    loss, margins = preference_loss(logits, targets, cu_seqlens, ref_logp)

Rows are the last dimension of x (contiguous, on a CUDA device); x and the
weights are bf16 or float32, and bf16 activations may take float32 weights.
The weight gradients come out of the kernels in float32 (the fused add
returns dgamma in the weight dtype, rounded once by its kernel); autograd
casts a float32 gradient to a bf16 weight's dtype.

fused_add_rms_norm is out of place: h is a new tensor (the residual is
copied into it and the kernel adds x over the copy), so that the h saved for
the backward is never modified by the next layer.  The C ABI's
rmsnorm_fused_add_fwd, which writes h over the residual itself, avoids that
copy where no backward is needed.

The rotary functions take q and k as [..., H, D] views with a contiguous last
dimension (slices of a fused projection are read in place) and the losses take
logits as [..., V] with the row stride they come with (a padded vocabulary's
slice is read in place); other layouts are copied first.

A step of these can be captured into a CUDA graph, backward included, after one run
on a side stream.  Let go of that run's losses first: an eager graph that still holds
the same parameters ties their gradients to its own stream, which a capture cannot
wait for.
"""
from __future__ import annotations

import torch

from . import (Heads, Rope, layernorm_bwd, layernorm_bwd_workspace_size, layernorm_fwd,
               rmsnorm_bwd, rmsnorm_bwd_workspace_size, rmsnorm_fused_add_bwd,
               rmsnorm_fused_add_fwd, rmsnorm_fwd, rmsnorm_policy_loss_fwd,
               rmsnorm_preference_loss_fwd, rmsnorm_rope_bwd, rmsnorm_rope_bwd_workspace_size,
               rmsnorm_rope_fwd, rmsnorm_token_logprob_bwd, rmsnorm_token_logprob_fwd)

__all__ = ["rms_norm", "fused_add_rms_norm", "layer_norm", "rope", "rms_norm_rope",
           "token_logprobs", "policy_loss", "preference_loss"]

_DT = {torch.bfloat16: "bf16", torch.float32: "f32"}


def _dt(t: torch.Tensor) -> str:
    try:
        return _DT[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}: bf16 or float32") from None


def _rows(x: torch.Tensor, *weights):
    if not x.is_cuda or not x.is_contiguous() or x.dim() < 1:
        raise ValueError("x must be a contiguous CUDA tensor with rows in its last dimension")
    N = x.shape[-1]
    for w in weights:
        if w is not None and (w.shape != (N,) or not w.is_contiguous() or w.device != x.device):
            raise ValueError(f"weights must be contiguous vectors of {N} on {x.device}")
    return (x.numel() // N if N else 0), N


def _stream(device) -> int:
    """The current stream of x's device: the C ABI launches on the current
    device, so every call below also makes x's device current."""
    return torch.cuda.current_stream(device).cuda_stream


def _workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)


class _RMSNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gamma, eps):
        M, N = _rows(x, gamma)
        y = torch.empty_like(x)
        rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        with torch.cuda.device(x.device):
            rmsnorm_fwd(x, gamma, y, rstd, M, N, eps, _dt(x), _dt(gamma), _stream(x.device))
        ctx.save_for_backward(x, gamma, rstd)
        ctx.eps = eps
        return y

    @staticmethod
    def backward(ctx, dy):
        x, gamma, rstd = ctx.saved_tensors
        M, N = _rows(x)
        dy = dy.contiguous()
        dx = torch.empty_like(x)
        dgamma, ws, nbytes = None, None, 0
        if ctx.needs_input_grad[1]:
            dgamma = torch.empty(N, dtype=torch.float32, device=x.device)
            nbytes = rmsnorm_bwd_workspace_size(M, N, _dt(x), _dt(gamma), x.device.index)
            ws = _workspace(nbytes, x.device)
        with torch.cuda.device(x.device):
            rmsnorm_bwd(dy, x, rstd, gamma, dx, dgamma, ws, nbytes, M, N, ctx.eps, _dt(x),
                        _dt(gamma), _stream(x.device))
        return dx, dgamma, None


class _FusedAddRMSNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, gamma, eps):
        M, N = _rows(x, gamma)
        if residual.shape != x.shape or residual.dtype != x.dtype:
            raise ValueError("residual must have the shape and dtype of x")
        if not residual.is_cuda or residual.device != x.device:
            raise ValueError(f"residual must be on x's device ({x.device})")
        h = residual.contiguous().clone()
        y = torch.empty_like(x)
        rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        with torch.cuda.device(x.device):
            rmsnorm_fused_add_fwd(x, h, gamma, y, rstd, M, N, eps, _dt(x), _dt(gamma),
                                  _stream(x.device))
        ctx.save_for_backward(h, gamma, rstd)
        ctx.eps = eps
        return y, h

    @staticmethod
    def backward(ctx, dy, dh):
        h, gamma, rstd = ctx.saved_tensors
        M, N = _rows(h)
        dy = dy.contiguous()
        # the gradient reaching h along the residual path; the kernel writes
        # dh_total = dx_norm + dh over it (the gradient of both x and residual)
        dres = dh.contiguous().clone()
        dgamma, ws, nbytes = None, None, 0
        if ctx.needs_input_grad[2]:
            dgamma = torch.empty(N, dtype=gamma.dtype, device=h.device)
            nbytes = rmsnorm_bwd_workspace_size(M, N, _dt(h), _dt(gamma), h.device.index)
            ws = _workspace(nbytes, h.device)
        with torch.cuda.device(h.device):
            rmsnorm_fused_add_bwd(dy, h, rstd, gamma, dres, dgamma, _dt(gamma), ws, nbytes, M,
                                  N, ctx.eps, _dt(h), _dt(gamma), _stream(h.device))
        return dres, dres, dgamma, None


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gamma, beta, eps):
        M, N = _rows(x, gamma, beta)
        y = torch.empty_like(x)
        mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
        with torch.cuda.device(x.device):
            layernorm_fwd(x, gamma, beta, y, mean, rstd, M, N, eps, _dt(x), _dt(gamma),
                          _stream(x.device))
        ctx.save_for_backward(x, gamma, mean, rstd)
        ctx.eps = eps
        ctx.has_beta = beta is not None
        return y

    @staticmethod
    def backward(ctx, dy):
        x, gamma, mean, rstd = ctx.saved_tensors
        M, N = _rows(x)
        dy = dy.contiguous()
        dx = torch.empty_like(x)
        want_g = ctx.needs_input_grad[1]
        want_b = ctx.has_beta and ctx.needs_input_grad[2]
        dgamma = torch.empty(N, dtype=torch.float32, device=x.device) if want_g else None
        dbeta = torch.empty(N, dtype=torch.float32, device=x.device) if want_b else None
        ws, nbytes = None, 0
        if want_g or want_b:
            nbytes = layernorm_bwd_workspace_size(M, N, _dt(x), _dt(gamma), x.device.index)
            ws = _workspace(nbytes, x.device)
        with torch.cuda.device(x.device):
            layernorm_bwd(dy, x, mean, rstd, gamma, dx, dgamma, dbeta, ws, nbytes, M, N,
                          ctx.eps, _dt(x), _dt(gamma), _stream(x.device))
        return dx, dgamma, dbeta, None


# ---------------------------------------------------------------- rotary positions

def _rows_of_heads(t: torch.Tensor) -> torch.Tensor:
    """t as [T, H, D] in a layout the kernels address: contiguous rows that do not
    overlap (a token's heads side by side, or a head's tokens); copied where it is not."""
    t = t.flatten(0, -3)
    T, H, D = t.shape
    st, sh, sd = t.stride()
    tokens_apart = (H < 2 or sh >= D) and (T < 2 or st >= (H - 1) * sh + D)
    heads_apart = (T < 2 or st >= D) and (H < 2 or sh >= (T - 1) * st + D)
    return t if (sd == 1 or D == 1) and (tokens_apart or heads_apart) else t.contiguous()


class _Rope(torch.autograd.Function):
    """[T, H, D] q and k (k None: alone); gammas None: the rotation alone."""

    @staticmethod
    def forward(ctx, q, k, q_gamma, k_gamma, positions, inv_freq, sections, rotary_dim, pairs,
                order, eps):
        T, _, D = q.shape
        turn = Rope(positions, inv_freq, sections, rotary_dim, pairs, order)
        qo = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        ko = None if k is None else torch.empty(k.shape, dtype=k.dtype, device=k.device)
        wd = _dt(q if q_gamma is None else q_gamma)
        with torch.cuda.device(q.device):
            rmsnorm_rope_fwd(Heads.of(q), None if k is None else Heads.of(k), q_gamma, k_gamma,
                             Heads.of(qo), None if k is None else Heads.of(ko), turn, T, D, eps,
                             _dt(q), wd, _stream(q.device))
        norm = q_gamma is not None
        ctx.save_for_backward(positions, inv_freq, q if norm else None, k if norm else None,
                              q_gamma, k_gamma)
        ctx.turn = (sections, rotary_dim, pairs, order)
        ctx.eps, ctx.wd = eps, wd
        return qo if k is None else (qo, ko)

    @staticmethod
    def backward(ctx, dqo, dko=None):
        positions, inv_freq, q, k, q_gamma, k_gamma = ctx.saved_tensors
        dqo = _rows_of_heads(dqo)
        dko = None if dko is None else _rows_of_heads(dko)
        T, Hq, D = dqo.shape
        Hk = 0 if dko is None else dko.shape[1]
        turn = Rope(positions, inv_freq, *ctx.turn)
        dev = dqo.device
        dq = torch.empty(dqo.shape, dtype=dqo.dtype, device=dev)
        dk = None if dko is None else torch.empty(dko.shape, dtype=dko.dtype, device=dev)
        dqg, dkg, ws, nbytes = None, None, None, 0
        if q is not None:
            if ctx.needs_input_grad[2]:
                dqg = torch.empty(D, dtype=torch.float32, device=dev)
            if dko is not None and ctx.needs_input_grad[3]:
                dkg = torch.empty(D, dtype=torch.float32, device=dev)
            if dqg is not None or dkg is not None:
                nbytes = rmsnorm_rope_bwd_workspace_size(T, Hq, Hk, D, _dt(dqo), ctx.wd, dev.index)
                ws = _workspace(nbytes, dev)
        of = lambda t: None if t is None else Heads.of(t)  # noqa: E731
        with torch.cuda.device(dev):
            rmsnorm_rope_bwd(of(dqo), of(dko), of(q), of(k), q_gamma, k_gamma, of(dq), of(dk),
                             dqg, dkg, ws, nbytes, turn, T, D, ctx.eps, _dt(dqo), ctx.wd,
                             _stream(dev))
        return dq, dk, dqg, dkg, None, None, None, None, None, None, None


def _apply_rope(q, k, q_gamma, k_gamma, positions, inv_freq, sections, pairs, order, eps):
    if not q.is_cuda or q.dim() < 3:
        raise ValueError("q must be a CUDA tensor [..., H, D]")
    for t in (k, q_gamma, k_gamma, positions, inv_freq):
        if t is not None and t.device != q.device:
            raise ValueError(f"every tensor must be on q's device ({q.device})")
    D, lead = q.shape[-1], q.shape[:-2]
    if k is not None and (k.shape[:-2] != lead or k.shape[-1] != D or k.dtype != q.dtype):
        raise ValueError("k must have q's dtype and shape, apart from its number of heads")
    for w in (q_gamma, k_gamma):
        if w is not None and (w.shape != (D,) or not w.is_contiguous()):
            raise ValueError(f"weights must be contiguous vectors of {D}")
    if k_gamma is not None and (q_gamma is None or k_gamma.dtype != q_gamma.dtype):
        raise ValueError("q_gamma and k_gamma must have the same dtype")
    sections = tuple(int(n) for n in sections)
    rotary_dim = 2 * sum(sections)
    if inv_freq.dim() != 1 or 2 * inv_freq.numel() != rotary_dim:
        raise ValueError(f"inv_freq must hold the sections' {rotary_dim // 2} frequencies")
    want = (len(sections), *lead)
    if positions.shape != want and not (len(sections) == 1 and positions.shape == lead):
        raise ValueError(f"positions must be {want}, a row for each axis")
    positions = positions.reshape(len(sections), -1)
    if positions.stride(1) != 1 or 0 < positions.stride(0) < positions.shape[1]:
        positions = positions.contiguous()
    out = _Rope.apply(_rows_of_heads(q), None if k is None else _rows_of_heads(k), q_gamma,
                      k_gamma, positions, inv_freq.contiguous(), sections, rotary_dim, pairs,
                      order, float(eps))
    if k is None:
        return out.view(q.shape), None
    return out[0].view(q.shape), out[1].view(k.shape)


# ---------------------------------------------------------------- token losses

def _logit_rows(logits, targets, *per_row):
    """logits as [M, V] rows (copied unless their rows are contiguous and apart),
    targets and the per-row values as contiguous vectors of M."""
    if not logits.is_cuda or logits.dim() < 2:
        raise ValueError("logits must be a CUDA tensor [..., V]")
    lead = logits.shape[:-1]
    if targets.shape != lead or targets.dtype != torch.int64:
        raise ValueError(f"targets must be int64 of shape {tuple(lead)}")
    for t in (targets, *per_row):
        if t is not None and t.device != logits.device:
            raise ValueError(f"every tensor must be on the logits' device ({logits.device})")
    rows = logits.flatten(0, -2)
    if (rows.stride(1) != 1 and rows.shape[1] > 1) or \
            (rows.shape[0] > 1 and rows.stride(0) < rows.shape[1]):
        rows = rows.contiguous()
    vectors = [targets.reshape(-1)]
    for t in per_row:
        if t is not None and t.shape != lead:
            raise ValueError(f"per-token values must have the shape {tuple(lead)}")
        vectors.append(None if t is None else t.detach().reshape(-1).float())
    return rows, [None if t is None else t.contiguous() for t in vectors]


def _row_stride(rows):
    return rows.stride(0) if rows.shape[0] > 1 else rows.shape[1]


def _gradient_rows(rows):
    """An empty [M, V] whose rows start where those of `rows` do modulo 16 bytes, so
    that reads and writes fall on the same vectors."""
    M, V = rows.shape
    per = 16 // rows.element_size()
    ld = V + (_row_stride(rows) - V) % per
    off = rows.data_ptr() % 16 // rows.element_size()
    flat = torch.empty(off + max(M * ld, 1), dtype=rows.dtype, device=rows.device)
    return flat[off:].as_strided((M, V), (ld, 1), off)


def _logit_gradient(ctx, rows, targets, rel_lse, dlogp, scale):
    M, V = rows.shape
    dlogits = _gradient_rows(rows)
    with torch.cuda.device(rows.device):
        rmsnorm_token_logprob_bwd(rows, _row_stride(rows), targets, ctx.inv_t, rel_lse, dlogp,
                                  scale, dlogits, _row_stride(dlogits), M, V, _dt(rows),
                                  _stream(rows.device))
    return dlogits


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, targets, inv_t):
        M, V = rows.shape
        logp, rel_lse = torch.empty(2, M, dtype=torch.float32, device=rows.device)
        with torch.cuda.device(rows.device):
            rmsnorm_token_logprob_fwd(rows, _row_stride(rows), targets, inv_t, logp, rel_lse, M, V,
                                      _dt(rows), _stream(rows.device))
        ctx.save_for_backward(rows, targets, rel_lse)
        ctx.inv_t = inv_t
        return logp

    @staticmethod
    def backward(ctx, dlogp):
        rows, targets, rel_lse = ctx.saved_tensors
        return _logit_gradient(ctx, rows, targets, rel_lse, dlogp.contiguous(), None), None, None


class _PolicyLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, targets, old_logp, ref_logp, advantages, weights, clip_low, clip_high,
                kl_coef, inv_t):
        M, V = rows.shape
        loss = torch.empty((), dtype=torch.float32, device=rows.device)
        token_loss, logp, rel_lse, dlogp = torch.empty(4, M, dtype=torch.float32,
                                                       device=rows.device)
        with torch.cuda.device(rows.device):
            rmsnorm_policy_loss_fwd(rows, _row_stride(rows), targets, inv_t, old_logp, ref_logp,
                                    advantages, weights, clip_low, clip_high, kl_coef, loss,
                                    token_loss, logp, rel_lse, dlogp, None, 0, M, V, _dt(rows),
                                    _stream(rows.device))
        ctx.save_for_backward(rows, targets, rel_lse, dlogp)
        ctx.inv_t = inv_t
        ctx.mark_non_differentiable(logp)
        return loss, logp

    @staticmethod
    def backward(ctx, dloss, _):
        rows, targets, rel_lse, dlogp = ctx.saved_tensors
        return (_logit_gradient(ctx, rows, targets, rel_lse, dlogp, dloss.contiguous()),
                *(None,) * 9)


class _PreferenceLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, targets, cu_seqlens, ref_logp, beta, label_smoothing, inv_t):
        M, V = rows.shape
        pairs = (cu_seqlens.numel() - 1) // 2
        loss = torch.empty((), dtype=torch.float32, device=rows.device)
        margins = torch.empty(pairs, dtype=torch.float32, device=rows.device)
        logp, rel_lse, dlogp = torch.empty(3, M, dtype=torch.float32, device=rows.device)
        with torch.cuda.device(rows.device):
            rmsnorm_preference_loss_fwd(rows, _row_stride(rows), targets, inv_t, ref_logp,
                                        cu_seqlens, pairs, beta, label_smoothing, loss, margins,
                                        logp, rel_lse, dlogp, M, V, _dt(rows), _stream(rows.device))
        ctx.save_for_backward(rows, targets, rel_lse, dlogp)
        ctx.inv_t = inv_t
        ctx.mark_non_differentiable(margins)
        return loss, margins

    @staticmethod
    def backward(ctx, dloss, _):
        rows, targets, rel_lse, dlogp = ctx.saved_tensors
        return (_logit_gradient(ctx, rows, targets, rel_lse, dlogp, dloss.contiguous()),
                *(None,) * 6)


def rms_norm(x: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-6) -> torch.Tensor:
    """y = x / sqrt(mean(x^2) + eps) * gamma over the last dimension."""
    return _RMSNorm.apply(x, gamma, float(eps))


def fused_add_rms_norm(x: torch.Tensor, residual: torch.Tensor, gamma: torch.Tensor,
                       eps: float = 1e-6):
    """h = residual + x (rounded to x's dtype) and y = rms_norm(h, gamma, eps);
    returns (y, h), h a new tensor."""
    return _FusedAddRMSNorm.apply(x, residual, gamma, float(eps))


def layer_norm(x: torch.Tensor, gamma: torch.Tensor, beta: torch.Tensor | None = None,
               eps: float = 1e-5) -> torch.Tensor:
    """y = (x - mean) / sqrt(var + eps) * gamma + beta over the last dimension."""
    return _LayerNorm.apply(x, gamma, beta, float(eps))


def rope(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor,
         inv_freq: torch.Tensor, sections, pairs: str = "halves", order: str = "blocks"):
    """Rotary positions with len(sections) axes over the heads of q [..., Hq, D] and k
    [..., Hk, D] (or None): the first 2 * sum(sections) columns turn.  positions: int64
    [axes, ...] (or [...] for one axis); inv_freq: float32, one per frequency; sections:
    frequencies per axis, laid out in "blocks" or "interleaved"; pairs of columns "halves"
    (i, i + R / 2) or "adjacent" (2i, 2i + 1).  Returns (q, k) rotated."""
    return _apply_rope(q, k, None, None, positions, inv_freq, sections, pairs, order, 0.0)


def rms_norm_rope(q: torch.Tensor, k: torch.Tensor | None, q_gamma: torch.Tensor,
                  k_gamma: torch.Tensor | None, positions: torch.Tensor, inv_freq: torch.Tensor,
                  sections, pairs: str = "halves", order: str = "blocks", eps: float = 1e-6):
    """rope(rms_norm(q, q_gamma), rms_norm(k, k_gamma)) over each head's D elements, in one
    pass and one rounding."""
    if q_gamma is None:
        raise ValueError("q_gamma is wanted: rope() is the rotation alone")
    return _apply_rope(q, k, q_gamma, k_gamma, positions, inv_freq, sections, pairs, order, eps)


def token_logprobs(logits: torch.Tensor, targets: torch.Tensor,
                   temperature: float = 1.0) -> torch.Tensor:
    """Log-probability (float32, the shape of targets) of each target under
    softmax(logits / temperature); 0, with no gradient, where the target is negative."""
    rows, (t,) = _logit_rows(logits, targets)
    return _TokenLogprobs.apply(rows, t, 1.0 / temperature).view(targets.shape)


def policy_loss(logits: torch.Tensor, targets: torch.Tensor, old_logp: torch.Tensor,
                advantages: torch.Tensor, ref_logp: torch.Tensor | None = None,
                weights: torch.Tensor | None = None, clip_low: float = 0.2,
                clip_high: float = 0.2, kl_coef: float = 0.0, temperature: float = 1.0):
    """Clipped policy loss with a KL term over the tokens whose target is not negative.
    weights: per token (their sum weighs the loss); None for the mean over those tokens.
    Gradients reach the logits only.  Returns (loss, logp), logp without a gradient."""
    rows, (t, old, adv, ref, w) = _logit_rows(logits, targets, old_logp, advantages, ref_logp,
                                              weights)
    if w is None:
        live = t >= 0
        w = live.float() / live.sum().clamp(min=1)
    loss, logp = _PolicyLoss.apply(rows, t, old, ref, adv, w, float(clip_low), float(clip_high),
                                   float(kl_coef), 1.0 / temperature)
    return loss, logp.view(targets.shape)


def preference_loss(logits: torch.Tensor, targets: torch.Tensor, cu_seqlens: torch.Tensor,
                    ref_logp: torch.Tensor | None = None, beta: float = 0.1,
                    label_smoothing: float = 0.0, temperature: float = 1.0):
    """Preference loss over pairs of sequences packed end to end in the rows of logits
    (chosen ones first, then the rejected ones): cu_seqlens int64 [2 * pairs + 1].  ref_logp:
    the reference model's log-probability per token.  Returns (loss, margins), margins
    without a gradient."""
    rows, (t, ref) = _logit_rows(logits, targets, ref_logp)
    if cu_seqlens.dtype != torch.int64 or cu_seqlens.dim() != 1 or cu_seqlens.numel() % 2 == 0 \
            or cu_seqlens.numel() < 3 or cu_seqlens.device != logits.device:
        raise ValueError("cu_seqlens must be int64 [2 * pairs + 1] on the logits' device")
    return _PreferenceLoss.apply(rows, t, cu_seqlens.contiguous(), ref, float(beta),
                                 float(label_smoothing), 1.0 / temperature)
