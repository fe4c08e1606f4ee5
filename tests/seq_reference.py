"""Plain 64-bit forms of the operators around the scan, token by token on the CPU in torch operations
that autograd can differentiate: the tests' reference for values and for the formulas' gradients."""

import torch


def up(t):
    return None if t is None else t.detach().double().cpu()


def silu(x):
    return x * torch.sigmoid(x)


def conv(x, weight, bias, state, lengths, act):
    """x [B, T, D], weight [D, K], state [B, K-1, D]: y (0 behind a length) and the last inputs."""
    B, T, D = x.shape
    K = weight.shape[1]
    state = x.new_zeros(B, K - 1, D) if state is None else state
    ys, states = [], []
    for b in range(B):
        n = T if lengths is None else min(max(int(lengths[b]), 0), T)
        ext = torch.cat((state[b], x[b, :n]), 0)
        rows = []
        for t in range(T):
            if t >= n:
                rows.append(x.new_zeros(D))
                continue
            pre = (ext[t:t + K] * weight.T).sum(0)
            pre = pre if bias is None else pre + bias
            rows.append(silu(pre) if act else pre)
        ys.append(torch.stack(rows) if rows else x.new_zeros(0, D))
        states.append(ext[n:n + K - 1])
    return torch.stack(ys), torch.stack(states)


def scan(u, delta, A, Bm, Cm, D, z, delta_bias, h0, lengths, softplus=True):
    """u [B, T, D], Bm [B, T, G, N]: y (0 behind a length) and the state at each row's length."""
    B, T, C = u.shape
    G, N = Bm.shape[2:]
    per = C // G
    x = delta if delta_bias is None else delta + delta_bias
    dt = torch.logaddexp(x, torch.zeros_like(x)) if softplus else x
    n = torch.full((B,), T) if lengths is None else lengths.long().clamp(0, T)
    h = u.new_zeros(B, C, N) if h0 is None else h0
    ys = []
    for t in range(T):
        on = (t < n)[:, None]
        Bt, Ct = (v[:, t].repeat_interleave(per, 1) for v in (Bm, Cm))
        new = torch.exp(dt[:, t, :, None] * A) * h + (dt[:, t] * u[:, t])[..., None] * Bt
        h = torch.where(on[..., None], new, h)
        r = (h * Ct).sum(-1)
        if D is not None:
            r = r + D * u[:, t]
        if z is not None:
            r = r * silu(z[:, t])
        ys.append(torch.where(on, r, torch.zeros_like(r)))
    return (torch.stack(ys, 1) if ys else u.new_zeros(B, 0, C)), h


def norm(x, weight, residual, eps):
    s = x if residual is None else x + residual
    return s / torch.sqrt((s * s).mean(-1, keepdim=True) + eps) * weight, s


def gradients(outputs, grads, leaves):
    """Gradients of sum <grad, output> for every leaf (None leaves and grads are skipped)."""
    loss = sum((o * g).sum() for o, g in zip(outputs, grads) if g is not None)
    wanted = [l for l in leaves if l is not None]
    got = iter(torch.autograd.grad(loss, wanted, allow_unused=True))
    return [None if l is None else (lambda g: torch.zeros_like(l) if g is None else g)(next(got))
            for l in leaves]


def rrms(got, ref):
    got, ref = up(got), up(ref)
    assert got.shape == ref.shape, (got.shape, ref.shape)
    assert torch.isfinite(got).all(), "non-finite values"
    if ref.numel() == 0:
        return 0.0
    n = ref.norm()
    return float((got - ref).norm() / n) if n > 0 else float(got.norm())


# A rounding to bf16 is off by at most half a step, 2^-8 of the value.
BF16 = 2.0 ** -8


def tol(dtype, steps, terms=1):
    """Relative RMS tolerance of values that carry `steps` dependent fp32 steps.

    A step of these recurrences multiplies by an exponential (ex2.approx: 2^-22, its argument
    rounded: 2^-24 of it) and rounds twice (2^-24 each): 2^-21 of the running magnitude covers it
    with room for the reads. Independent terms that cancel in a sum of n leave about 1 / sqrt(n) of
    that magnitude, hence the factor sqrt(terms). An output in bf16 adds its own rounding.
    """
    return (steps + 64) * 2.0 ** -21 * terms ** 0.5 + (BF16 if dtype == torch.bfloat16 else 0.0)
