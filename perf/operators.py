"""The operators around the scan that are measured: the short causal convolution in front of it, the
selective state space scan beside it, and the root-mean-square norm between two blocks.

``run`` computes them in elementary torch operations, or, with ``own``, through this package's calls.
``exact`` computes the same from the definitions in 64 bits, token by token.
"""

import math

import torch

own = False


# ---------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # One decoding step of a full batch: the convolution over the last inputs of every sequence.
        {"name": "conv, one token each", "op": "conv_step", "B": 512, "D": 2048, "K": 4, "dtype": "bf16"},
        # Queries or keys of the long-sequence workload: out of a projection, token by token, into heads.
        {"name": "conv, long prompt to heads", "op": "conv", "B": 2, "T": 32768, "H": 32, "D": 2048,
         "K": 4, "dtype": "bf16", "ragged": False},
        # A training step of a padded batch, forward and backward.
        {"name": "conv, training", "op": "conv_train", "B": 8, "T": 4096, "D": 768, "K": 4,
         "dtype": "bf16", "ragged": True},
        # A few short prompts of different lengths, one of them empty, that continue known states.
        {"name": "scan, short prompts", "op": "scan", "B": 4, "T": 509, "D": 256, "G": 1, "N": 16,
         "dtype": "fp32", "ragged": True},
        # Two long prompts.
        {"name": "scan, long prompts", "op": "scan", "B": 2, "T": 32768, "D": 2048, "G": 1, "N": 16,
         "dtype": "bf16", "ragged": False},
        # A training step, forward and backward.
        {"name": "scan, training", "op": "scan_train", "B": 8, "T": 4096, "D": 768, "G": 1, "N": 16,
         "dtype": "bf16", "ragged": False},
        # The same at odd sizes, in 32 bits, with two groups of channels and a padded batch.
        {"name": "scan, training, odd sizes", "op": "scan_train", "B": 3, "T": 777, "D": 202, "G": 2,
         "N": 8, "dtype": "fp32", "ragged": True},
        # One decoding step of a full batch; some rows have ended.
        {"name": "scan, one token each", "op": "scan_step", "B": 512, "D": 2048, "G": 1, "N": 16,
         "dtype": "bf16"},
        # One decoding step of a single sequence.
        {"name": "scan, one token", "op": "scan_step", "B": 1, "D": 1536, "G": 1, "N": 16,
         "dtype": "bf16"},
        # The norm in a decoding step: a row a sequence, 8 bits for the next product.
        {"name": "norm, tokens, 8 bits", "op": "norm8", "M": 64, "D": 2048, "group": 0, "dtype": "bf16"},
        # The norm over a long prompt, 8 bits with a scale for each 128 channels.
        {"name": "norm, prompt, 8 bits", "op": "norm8", "M": 65536, "D": 2048, "group": 128,
         "dtype": "bf16"},
        # The norm in a training step, forward and backward.
        {"name": "norm, training", "op": "norm_train", "M": 32768, "D": 1536, "dtype": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv_step", "conv", "conv_train", "scan", "scan_train", "scan_step", "norm8",
                     "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "norm8":
        D = _spread(rng, 64, 8192)
        return {"op": op, "M": _spread(rng, 1, min(65536, (1 << 27) // D)), "D": D,
                "group": rng.choice([0, 128]), "dtype": dtype}
    if op == "norm_train":
        D = _spread(rng, 64, 8192)
        return {"op": op, "M": _spread(rng, 1, min(65536, 50_000_000 // D)), "D": D, "dtype": dtype}
    H = rng.choice([1, 1, 4, 12])
    D = H * 64 if H > 1 else _spread(rng, 16, 2048)
    B = _spread(rng, 1, 512 if op.endswith("step") else 16)
    if op == "conv_step":
        return {"op": op, "B": B, "D": D, "K": rng.choice([2, 3, 4]), "dtype": dtype}
    if op == "conv":
        return {"op": op, "B": B, "T": _spread(rng, 1, min(32768, (1 << 26) // (B * D))), "H": H, "D": D,
                "K": rng.choice([2, 3, 4]), "dtype": dtype, "ragged": rng.random() < 0.5}
    if op == "conv_train":
        return {"op": op, "B": B, "T": _spread(rng, 1, min(8192, 25_000_000 // (B * D))), "D": D,
                "K": rng.choice([2, 3, 4]), "dtype": dtype, "ragged": rng.random() < 0.5}
    G = rng.choice([1, 1, H])
    N = rng.choice([8, 16, 16, 32])
    if op == "scan_step":
        return {"op": op, "B": B, "D": D, "G": G, "N": N, "dtype": dtype}
    if op == "scan":
        most = min(32768, (1 << 30) // (B * D * N))
    else:
        most = min(8192, 400_000_000 // (B * D * N))
    return {"op": op, "B": B, "T": _spread(rng, 1, max(1, most)), "D": D, "G": G, "N": N, "dtype": dtype,
            "ragged": rng.random() < 0.5}


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------

def _dtype(case):
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[case["dtype"]]


class _Make:
    """Seeded normal and uniform numbers on the GPU."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, *shape, dtype=torch.float32, scale=1.0, shift=0.0):
        return torch.randn(*shape, generator=self.g, device="cuda").mul_(scale).add_(shift).to(dtype)

    def uniform(self, lo, hi, *shape):
        return torch.rand(*shape, generator=self.g, device="cuda").mul_(hi - lo).add_(lo)

    def lengths(self, B, T):
        """Lengths up to T of a padded batch: the first row is full, the last of several is empty."""
        n = torch.randint(1, T + 1, (B,), generator=self.g, device="cuda", dtype=torch.int32)
        n[0] = T
        if B > 1:
            n[-1] = 0
        return n


def prepare(case, seed):
    m, op = _Make(seed), case["op"]
    s = {"op": op}
    if op in ("norm8", "norm_train"):
        dt, M, D = _dtype(case), case["M"], case["D"]
        s |= {"x": m.normal(M, D, dtype=dt), "residual": m.normal(M, D, dtype=dt, scale=3.0),
              "weight": m.normal(D, scale=0.1, shift=1.0), "eps": 1e-6}
        if op == "norm8":
            s["group"] = case["group"]
        else:
            s |= {"dy": m.normal(M, D, dtype=dt), "ds": m.normal(M, D, dtype=dt)}
        return s
    dt, B, D = _dtype(case), case["B"], case["D"]
    if op.startswith("conv"):
        K = case["K"]
        r = K ** -0.5
        s |= {"weight": m.uniform(-r, r, D, K), "bias": m.uniform(-r, r, D),
              "state": m.normal(B, K - 1, D, dtype=dt)}
        if op == "conv_step":
            return s | {"x": m.normal(B, D, dtype=dt)}
        T = case["T"]
        s["lengths"] = m.lengths(B, T) if case["ragged"] else None
        s["x"] = m.normal(B, T, D, dtype=dt)
        if op == "conv":
            s["H"] = case["H"]
        else:
            s["dy"] = m.normal(B, T, D, dtype=dt)
        return s
    G, N = case["G"], case["N"]
    # Step sizes between 1/1000 and 1/10, decays between 1 and N: how such layers are set up.
    step = torch.exp(m.uniform(math.log(1e-3), math.log(1e-1), D))
    s |= {"A": -torch.arange(1, N + 1, device="cuda", dtype=torch.float32) * m.uniform(0.8, 1.2, D, N),
          "D": m.normal(D, scale=0.1, shift=1.0), "bias": step + torch.log(-torch.expm1(-step)),
          "h": m.normal(B, D, N, scale=0.5)}
    lead = (B,) if op == "scan_step" else (B, case["T"])
    # u and z are halves of one projection, the step size and the two vectors slices of another.
    both = m.normal(*lead, 2 * D, dtype=dt)
    s |= {"u": both[..., :D], "z": both[..., D:], "delta": m.normal(*lead, D, dtype=dt, scale=0.5)}
    proj = m.normal(*lead, 2 * G * N, dtype=dt)
    s |= {"Bm": proj[..., :G * N].unflatten(-1, (G, N)), "Cm": proj[..., G * N:].unflatten(-1, (G, N))}
    if op == "scan_step":
        s["active"] = (m.uniform(0, 1, B) < 0.9).to(torch.uint8)
        s["active"][0] = 1
        return s
    s["lengths"] = m.lengths(B, case["T"]) if case["ragged"] else None
    if op == "scan_train":
        s |= {"dy": m.normal(*lead, D, dtype=dt), "dh_T": m.normal(B, D, N, scale=0.1)}
    return s


# ---------------------------------------------------------------------------------------------
# The calls of a user's program
# ---------------------------------------------------------------------------------------------

def _run_own(s):
    from test_sequence_layers_02_b200 import conv, norm, ssm
    op = s["op"]
    if op == "conv_step":
        return {"y": conv.causal_conv_step(s["x"], s["weight"], s["bias"], s["state"], silu=True),
                "state": s["state"]}
    if op == "conv":
        H, x = s["H"], s["x"]
        x = x.unflatten(-1, (H, x.shape[-1] // H)).transpose(1, 2)
        w = s["weight"].unflatten(0, x.shape[1::2])
        b = s["bias"].unflatten(0, x.shape[1::2])
        st = s["state"].unflatten(-1, x.shape[1::2]).transpose(1, 2)
        y, state = conv.causal_conv(x, w, b, silu=True, state=st, lengths=s["lengths"])
        return {"y": y, "state": state}
    if op == "conv_train":
        y, state = conv.causal_conv(s["x"], s["weight"], s["bias"], silu=True, state=s["state"],
                                    lengths=s["lengths"])
        g = conv.causal_conv_backward(s["x"], s["weight"], s["bias"], s["dy"], silu=True,
                                      state=s["state"], lengths=s["lengths"])
        return {"y": y, "state": state, "dx": g["dx"], "dweight": g["dweight"], "dbias": g["dbias"],
                "dstate": g["dstate"]}
    if op == "scan":
        y, h = ssm.selective_scan(s["u"], s["delta"], s["A"], s["Bm"], s["Cm"], s["D"], s["z"], s["bias"],
                                  h0=s["h"], lengths=s["lengths"])
        return {"y": y, "h": h}
    if op == "scan_train":
        a = (s["u"], s["delta"], s["A"], s["Bm"], s["Cm"], s["D"], s["z"], s["bias"])
        y, h, chunks = ssm.selective_scan(*a, h0=s["h"], lengths=s["lengths"], want_chunks=True)
        g = ssm.selective_scan_backward(*a, chunks, s["dy"], s["dh_T"], lengths=s["lengths"])
        return {"y": y, "h": h, **g}
    if op == "scan_step":
        y = ssm.selective_step(s["u"], s["delta"], s["A"], s["Bm"], s["Cm"], s["D"], s["z"], s["bias"],
                               s["h"], active=s["active"])
        return {"y": y, "h": s["h"]}
    if op == "norm8":
        y, scale, total = norm.rmsnorm_fp8(s["x"], s["weight"], s["residual"], eps=s["eps"],
                                           group=s["group"])
        return {"y": y, "scale": scale, "sum": total}
    y, total = norm.rmsnorm(s["x"], s["weight"], s["residual"], eps=s["eps"])
    g = norm.rmsnorm_backward(s["dy"], total, s["weight"], s["ds"], eps=s["eps"])
    return {"y": y, "sum": total, "dx": g["dx"], "dweight": g["dweight"]}


# ---------------------------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------------------------

def _inside(lengths, x):
    """Which tokens of x [B, T, ...] are there, as a mask [B, T, 1]; None for all."""
    if lengths is None:
        return None
    return (torch.arange(x.shape[1], device=x.device) < lengths[:, None])[..., None]


def _keep(mask, x):
    return x if mask is None else torch.where(mask, x, torch.zeros_like(x))


def _conv(s):
    """The convolution's windows [B, T, D, K], its values before the activation, and the last inputs."""
    x, w, K = s["x"], s["weight"], s["weight"].shape[1]
    mask = _inside(s["lengths"], x)
    past = torch.cat((s["state"].float(), _keep(mask, x.float())), 1)
    windows = past.unfold(1, K, 1)
    pre = (windows * w).sum(-1) + s["bias"]
    n = torch.full((x.shape[0],), x.shape[1], device=x.device) if mask is None else s["lengths"].long()
    at = (n[:, None] + torch.arange(K - 1, device=x.device))[..., None].expand(-1, -1, x.shape[2])
    return mask, windows, pre, past.gather(1, at).to(x.dtype)


def _plain_conv(s):
    mask, windows, pre, state = _conv(s)
    return {"y": _keep(mask, pre * torch.sigmoid(pre)).to(s["x"].dtype), "state": state}


def _plain_conv_to_heads(s):
    r, H = _plain_conv(s), s["H"]
    return {k: v.unflatten(-1, (H, v.shape[-1] // H)).transpose(1, 2).contiguous() for k, v in r.items()}


def _plain_conv_train(s):
    mask, windows, pre, state = _conv(s)
    w, dtype = s["weight"], s["x"].dtype
    K = w.shape[1]
    sig = torch.sigmoid(pre)
    dpre = _keep(mask, s["dy"].float() * sig * (1 + pre * (1 - sig)))
    edge = dpre.new_zeros(dpre.shape[0], K - 1, dpre.shape[2])
    dpast = (torch.cat((edge, dpre, edge), 1).unfold(1, K, 1) * w.flip(1)).sum(-1)
    # the sum over all tokens is a long one
    dw = (windows.double() * dpre.double()[..., None]).sum((0, 1))
    return {"y": _keep(mask, pre * sig).to(dtype), "state": state, "dx": _keep(mask, dpast[:, K - 1:]).to(dtype),
            "dweight": dw.float(), "dbias": dpre.double().sum((0, 1)).float(), "dstate": dpast[:, :K - 1].to(dtype)}


def _plain_conv_step(s):
    past = torch.cat((s["state"], s["x"][:, None]), 1)
    pre = (past.float().transpose(1, 2) * s["weight"]).sum(-1) + s["bias"]
    s["state"].copy_(past[:, 1:])
    return {"y": (pre * torch.sigmoid(pre)).to(s["x"].dtype), "state": s["state"]}


def _linear_scan(a, x):
    """h_t = a_t h_{t-1} + x_t along dimension 1, by doubling."""
    k = 1
    while k < x.shape[1]:
        x = torch.cat((x[:, :k], x[:, k:] + a[:, k:] * x[:, :-k]), 1)
        a = torch.cat((a[:, :k], a[:, k:] * a[:, :-k]), 1)
        k *= 2
    return x


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def _scan(s):
    """What forward and backward share: [B, T, D] and [B, T, D, N] values in 32 bits."""
    mask, D = _inside(s["lengths"], s["u"]), s["u"].shape[2]
    per = D // s["Bm"].shape[2]
    v = {"mask": mask, "u": _keep(mask, s["u"].float()), "z": _keep(mask, s["z"].float()),
         "raw": s["delta"].float() + s["bias"]}
    v["dt"] = _keep(mask, _softplus(v["raw"]))
    if mask is not None:
        m = mask[..., None]
        v["B"] = _keep(m, s["Bm"].float()).repeat_interleave(per, 2)
        v["C"] = _keep(m, s["Cm"].float()).repeat_interleave(per, 2)
    else:
        v["B"] = s["Bm"].float().repeat_interleave(per, 2)
        v["C"] = s["Cm"].float().repeat_interleave(per, 2)
    a = torch.exp(v["dt"][..., None] * s["A"])
    x = (v["dt"] * v["u"])[..., None] * v["B"]
    x[:, 0] += a[:, 0] * s["h"]
    v["a"], v["h"] = a, _linear_scan(a, x)
    v["sig"] = torch.sigmoid(v["z"])
    v["read"] = (v["h"] * v["C"]).sum(-1) + s["D"] * v["u"]
    return v


def _plain_scan(s):
    v = _scan(s)
    return {"y": _keep(v["mask"], v["read"] * v["z"] * v["sig"]).to(s["u"].dtype), "h": v["h"][:, -1].clone()}


def _plain_scan_train(s):
    v, A, dtype = _scan(s), s["A"], s["u"].dtype
    mask, u, dt, z, sig, a, h, B, C = (v[k] for k in ("mask", "u", "dt", "z", "sig", "a", "h", "B", "C"))
    Bsz, T, G, N = s["Bm"].shape
    dy = _keep(mask, s["dy"].float())
    dread = dy * z * sig
    g = dread[..., None] * C
    g[:, -1] += s["dh_T"]
    later = torch.cat((a[:, 1:], torch.ones_like(a[:, :1])), 1)
    g = _linear_scan(later.flip(1), g.flip(1)).flip(1)
    carried = a * torch.cat((s["h"][:, None], h[:, :-1]), 1)
    gc = g * carried
    gB = (g * B).sum(-1)
    ddt = (gc * A).sum(-1) + u * gB
    draw_ = _keep(mask, ddt * torch.sigmoid(v["raw"]))
    groups = lambda x: x.unflatten(2, (G, -1)).sum(3)  # noqa: E731
    return {
        "y": _keep(mask, v["read"] * z * sig).to(dtype), "h": h[:, -1].clone(),
        "du": _keep(mask, dt * gB + s["D"] * dread).to(dtype), "ddelta": draw_.to(dtype),
        "dz": (dy * v["read"] * sig * (1 + z * (1 - sig))).to(dtype),
        "dBm": groups(g * (dt * u)[..., None]).to(dtype), "dCm": groups(dread[..., None] * h).to(dtype),
        "dA": (gc * dt[..., None]).sum((0, 1)), "dD": (dread * u).sum((0, 1)), "ddelta_bias": draw_.sum((0, 1)),
        "dh0": a[:, 0] * g[:, 0]}


def _plain_scan_step(s):
    on = s["active"].bool()[:, None]
    u, z = s["u"].float(), s["z"].float()
    dt = _softplus(s["delta"].float() + s["bias"])
    per = u.shape[1] // s["Bm"].shape[1]
    B, C = (s[k].float().repeat_interleave(per, 1) for k in ("Bm", "Cm"))
    h = torch.exp(dt[..., None] * s["A"]) * s["h"] + (dt * u)[..., None] * B
    y = ((h * C).sum(-1) + s["D"] * u) * z * torch.sigmoid(z)
    s["h"].copy_(torch.where(on[..., None], h, s["h"]))
    return {"y": _keep(on, y).to(s["u"].dtype), "h": s["h"]}


def _norm(s):
    total = s["x"].float() + s["residual"].float()
    r = torch.rsqrt((total * total).mean(-1, keepdim=True) + s["eps"])
    return total, total * r * s["weight"]


def _plain_norm8(s):
    total, y = _norm(s)
    M, D = y.shape
    g = s["group"] or D
    n = -(-D // g)
    wide = torch.cat((y, y.new_zeros(M, n * g - D)), 1).view(M, n, g)
    scale = torch.clamp(wide.abs().amax(-1) / 448, min=torch.finfo(torch.float32).tiny)
    q = (wide / scale[..., None]).to(torch.float8_e4m3fn).view(M, n * g)[:, :D]
    return {"y": q.contiguous(), "scale": scale, "sum": total.to(s["x"].dtype)}


def _plain_norm_train(s):
    total, y = _norm(s)
    dtype, w = s["x"].dtype, s["weight"]
    kept = total.to(dtype)
    x, dy = kept.float(), s["dy"].float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"])
    hat, g = x * r, dy * w
    dx = r * (g - hat * (g * hat).mean(-1, keepdim=True)) + s["ds"].float()
    # the sum over all rows is a long one
    return {"y": y.to(dtype), "sum": kept, "dx": dx.to(dtype), "dweight": (dy * hat).double().sum(0).float()}


def run(s):
    if own:
        return _run_own(s)
    return {"conv_step": _plain_conv_step, "conv": _plain_conv_to_heads, "conv_train": _plain_conv_train,
            "scan": _plain_scan, "scan_train": _plain_scan_train, "scan_step": _plain_scan_step,
            "norm8": _plain_norm8, "norm_train": _plain_norm_train}[s["op"]](s)


# ---------------------------------------------------------------------------------------------
# Work
# ---------------------------------------------------------------------------------------------

def work(case):
    """Each input read once, each output written once; operations of the definitions (an exponential is one)."""
    op, D = case["op"], case["D"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op == "norm8":
        M, g = case["M"], case["group"] or case["D"]
        return {"bytes": M * D * (3 * e + 1) + 4 * D + 4 * M * -(-D // g), "flops": 8 * M * D}
    if op == "norm_train":
        return {"bytes": case["M"] * D * 7 * e + 8 * D, "flops": 18 * case["M"] * D}
    B, T = case["B"], case.get("T", 1)
    if op.startswith("conv"):
        K = case["K"]
        n, past, w = B * T * D, B * (K - 1) * D * e, 4 * D * (K + 1)
        if op == "conv_train":
            return {"bytes": 4 * n * e + 3 * past + 2 * w, "flops": n * (6 * K + 16)}
        return {"bytes": 2 * n * e + 2 * past + w, "flops": n * (2 * K + 5)}
    G, N = case["G"], case["N"]
    n, state, pars = B * T * D, 4 * B * D * N, 4 * D * (N + 2)
    bc = 2 * B * T * G * N * e
    if op == "scan_train":
        return {"bytes": n * e * 8 + 2 * bc + 4 * state + 2 * pars, "flops": n * (26 * N + 40)}
    return {"bytes": n * e * 4 + bc + 2 * state + pars, "flops": n * (7 * N + 16)}


# ---------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def _d(x):
    return x.double()


def _silu64(x):
    return x / (1 + torch.exp(-x))


def _dsilu64(x):
    p = 1 / (1 + torch.exp(-x))
    return p + x * p * (1 - p)


def _exact_conv(s, train):
    x, w, b, st = _d(s["x"]), _d(s["weight"]), _d(s["bias"]), _d(s["state"])
    B, T, D = x.shape
    K = w.shape[1]
    if s["lengths"] is not None:
        x = x.clone()
        for i, n in enumerate(s["lengths"].tolist()):
            x[i, n:] = 0
    # tap j looks K - 1 - j tokens back; older inputs are in the state
    taps = []
    for j in range(K):
        back = K - 1 - j
        taps.append(torch.cat((st[:, K - 1 - back:], x), 1)[:, :T] if back else x)
    pre = b + sum(w[:, j] * taps[j] for j in range(K))
    y = _silu64(pre)
    ends = s["lengths"].tolist() if s["lengths"] is not None else [T] * B
    state = torch.stack([torch.cat((st[i], x[i, :n]))[n:n + K - 1] for i, n in enumerate(ends)])
    for i, n in enumerate(ends):
        y[i, n:] = 0
    if not train:
        return {"y": y, "state": state}
    dp = _d(s["dy"]) * _dsilu64(pre)
    for i, n in enumerate(ends):
        dp[i, n:] = 0
    dx, dst = torch.zeros_like(x), torch.zeros_like(st)
    for j in range(K):
        back = K - 1 - j
        t = w[:, j] * dp
        if back < T:
            dx[:, :T - back] += t[:, back:]
        for k in range(min(back, T)):  # token k looked at the state's entry K - 1 - back + k
            dst[:, K - 1 - back + k] += t[:, k]
    for i, n in enumerate(ends):
        dx[i, n:] = 0
    dw = torch.stack([(dp * taps[j]).sum((0, 1)) for j in range(K)], 1)
    return {"y": y, "state": state, "dx": dx, "dweight": dw, "dbias": dp.sum((0, 1)), "dstate": dst}


def _exact_scan(s, train):
    u, z, A, skip = _d(s["u"]), _d(s["z"]), _d(s["A"]), _d(s["D"])
    raw = _d(s["delta"]) + _d(s["bias"])
    dt = torch.logaddexp(raw, torch.zeros_like(raw))
    Bsz, T, D = u.shape
    G, N = s["Bm"].shape[2:]
    per = D // G
    n = s["lengths"].long() if s["lengths"] is not None else torch.full((Bsz,), T, device=u.device)
    wide = lambda x, t: _d(x[:, t]).repeat_interleave(per, 1)  # noqa: E731
    h, hs, reads = _d(s["h"]), [], []
    for t in range(T):
        on = (t < n)[:, None, None]
        new = torch.exp(dt[:, t, :, None] * A) * h + (dt[:, t] * u[:, t])[..., None] * wide(s["Bm"], t)
        if train:
            hs.append(h)
        h = torch.where(on, new, h)
        reads.append((h * wide(s["Cm"], t)).sum(-1))
    there = (torch.arange(T, device=u.device) < n[:, None])[..., None]
    zero = u.new_zeros(())
    read = torch.stack(reads, 1) + skip * u
    y = torch.where(there, read * _silu64(z), zero)
    if not train:
        return {"y": y, "h": h}
    dy = torch.where(there, _d(s["dy"]), zero)
    dread = dy * _silu64(z)
    r = {"y": y, "h": h, "dz": dy * read * _dsilu64(z), "dD": (dread * u).sum((0, 1)), "dA": torch.zeros_like(A)}
    g, last = _d(s["dh_T"]), h
    du, ddt, dB, dC = [], [], [], []
    for t in range(T - 1, -1, -1):
        on = (t < n)[:, None, None]
        a, before = torch.exp(dt[:, t, :, None] * A), hs[t]
        B, C = wide(s["Bm"], t), wide(s["Cm"], t)
        gh = g + dread[:, t, :, None] * C
        dC.append((dread[:, t, :, None] * last).unflatten(1, (G, per)).sum(2))
        live = torch.where(on, gh, zero)
        dB.append((live * (dt[:, t] * u[:, t])[..., None]).unflatten(1, (G, per)).sum(2))
        lB, la = (live * B).sum(-1), live * a * before
        du.append(dt[:, t] * lB)
        ddt.append((la * A).sum(-1) + u[:, t] * lB)
        r["dA"] += (la * dt[:, t, :, None]).sum(0)
        g, last = torch.where(on, gh * a, g), before
    back = lambda v: torch.stack(v[::-1], 1)  # noqa: E731
    draw_ = back(ddt) / (1 + torch.exp(-raw))
    return r | {"du": back(du) + skip * dread, "ddelta": draw_, "ddelta_bias": draw_.sum((0, 1)), "dBm": back(dB),
                "dCm": back(dC), "dh0": g}


def _exact_norm(s):
    x, w = _d(s["x"]) + _d(s["residual"]), _d(s["weight"])
    return x, x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]) * w


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "conv_step":
        r = _exact_conv(s | {"x": s["x"][:, None], "lengths": None}, False)
        return {"y": r["y"][:, 0], "state": r["state"]}
    if op == "conv":
        H = s["H"]
        return {k: v.unflatten(-1, (H, v.shape[-1] // H)).transpose(1, 2).contiguous()
                for k, v in _exact_conv(s, False).items()}
    if op == "conv_train":
        return _exact_conv(s, True)
    if op in ("scan", "scan_train"):
        return _exact_scan(s, op == "scan_train")
    if op == "scan_step":
        one = {k: s[k][:, None] for k in ("u", "z", "delta", "Bm", "Cm")}
        r = _exact_scan(s | one | {"lengths": s["active"].int()}, False)
        return {"y": r["y"][:, 0], "h": r["h"]}
    total, y = _exact_norm(s)
    if op == "norm8":
        # the rounding to 8 bits is the operator's own: the value before it is what the codes stand for
        g = s["group"] or case["D"]
        parts = [y[:, i:i + g] for i in range(0, case["D"], g)]
        scale = torch.stack([p.abs().amax(-1) / 448 for p in parts], 1)
        return {"y": torch.cat([p / scale[:, i:i + 1] for i, p in enumerate(parts)], 1), "scale": scale,
                "sum": total}
    x, w, dy = _d(total.to(_dtype(case))), _d(s["weight"]), _d(s["dy"])
    ms = (x ** 2).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]
    g = dy * w
    dx = g / ms.sqrt() - x * (g * x).sum(-1, keepdim=True) / x.shape[-1] / ms ** 1.5 + _d(s["ds"])
    return {"y": y, "sum": total, "dx": dx, "dweight": (dy * x / ms.sqrt()).sum(0)}
