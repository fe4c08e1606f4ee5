"""The selective state space scan against a plain form in 64 bits: prompts, gradients, single tokens."""

import pytest
import torch

from tests import seq_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def ssm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from test_sequence_layers_02_b200 import build, ssm as module
    build.build()
    return module


NAMES = ("u", "delta", "A", "Bm", "Cm", "D", "z", "delta_bias")


def problem(B, T, C, N, dtype, G=1, seed=0, skip=True, gate=True, bias=True, h0=True, lengths=None):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    p = dict(u=r(B, T, C).to(dtype), delta=(r(B, T, C) * 0.7).to(dtype),
             A=-torch.rand(C, N, generator=g) * 4 - 0.05,
             Bm=r(B, T, G, N).to(dtype), Cm=r(B, T, G, N).to(dtype),
             D=r(C) if skip else None, z=r(B, T, C).to(dtype) if gate else None,
             delta_bias=r(C) - 2 if bias else None, h0=r(B, C, N) if h0 else None, lengths=None)
    if lengths is not None:
        p["lengths"] = torch.tensor(lengths, dtype=torch.int32)
        for b, n in enumerate(lengths):
            for k in ("u", "delta", "z", "Bm", "Cm"):
                if p[k] is not None:
                    p[k][b, min(max(n, 0), T):] = float("nan")   # nothing there may be read
    return p


def cuda(p):
    return {k: None if v is None else v.cuda() for k, v in p.items()}


def clean(p):
    """64-bit copies, with zeros in the place of what is behind a length."""
    return {k: v if k == "lengths" else None if v is None else torch.nan_to_num(ref.up(v), nan=0.0)
            for k, v in p.items()}


def args(p):
    return [p[k] for k in NAMES]


def check_forward(ssm, p, softplus=True, out_dtype=None):
    c, q = cuda(p), clean(p)
    y, h, chunks = ssm.selective_scan(*args(c), softplus=softplus, h0=c["h0"], lengths=c["lengths"],
                                      out_dtype=out_dtype, want_chunks=True)
    ry, rh = ref.scan(*args(q), q["h0"], q["lengths"], softplus)
    T = p["u"].shape[1]
    assert ref.rrms(y, ry) <= ref.tol(y.dtype, T)
    assert ref.rrms(h, rh) <= ref.tol(F32, T)
    # without snapshots: the same bits
    y2, h2 = ssm.selective_scan(*args(c), softplus=softplus, h0=c["h0"], lengths=c["lengths"],
                                out_dtype=out_dtype)
    assert torch.equal(y, y2) and torch.equal(h, h2)
    return y, h, chunks


@pytest.mark.parametrize("N", [8, 16, 32, 64])
@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF16, BF16), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("T", [1, 15, 16, 17, 49])
def test_prompt(ssm, T, N, dtype, out):
    check_forward(ssm, problem(2, T, 40, N, dtype, seed=T + N), out_dtype=out)


@pytest.mark.parametrize("C,G,N", [(1, 1, 16), (7, 1, 8), (33, 1, 16), (65, 1, 8), (130, 2, 16), (192, 3, 32),
                                   (24, 24, 8), (18, 2, 64)])
def test_channels_and_groups(ssm, C, G, N):
    check_forward(ssm, problem(2, 37, C, N, F32, G=G, seed=C))
    check_forward(ssm, problem(2, 37, C, N, BF16, G=G, seed=C))


@pytest.mark.parametrize("off", ["skip", "gate", "bias", "h0", "softplus"])
def test_options(ssm, off):
    kw = {} if off == "softplus" else {off: False}
    p = problem(2, 33, 24, 16, F32, seed=7, **kw)
    if off == "softplus":
        p["delta"] = torch.rand(2, 33, 24) * 0.5
        p["delta_bias"] = torch.rand(24) * 0.1
    check_forward(ssm, p, softplus=off != "softplus")


@pytest.mark.parametrize("T,C,B,N", [(1000, 8, 1, 16), (517, 40, 2, 8), (700, 20, 1, 64), (2049, 3, 1, 32)])
def test_long_prompts_are_split(ssm, T, C, B, N):
    """Few channels and many tokens: the tokens are shared by a cluster of CTAs."""
    check_forward(ssm, problem(B, T, C, N, F32, seed=T))


@pytest.mark.parametrize("N", [8, 16])
@pytest.mark.parametrize("T,lengths", [(40, [40, 0, 1, 17, 32]), (600, [600, 0, 1, 130, 599]),
                                       (20, [99, -3, 20, 5, 16])])
def test_lengths(ssm, T, lengths, N):
    p = problem(5, T, 12, N, F32, seed=5, lengths=lengths)
    y, h, _ = check_forward(ssm, p)
    for b, n in enumerate(lengths):
        n = min(max(n, 0), T)
        assert not y[b, n:].any()
        if n == 0:
            assert torch.equal(h[b].cpu(), p["h0"][b])
    c = cuda(p)
    mine = torch.full_like(y, 9.0)
    ssm.selective_scan(*args(c), h0=c["h0"], lengths=c["lengths"], y=mine)
    for b, n in enumerate(lengths):
        n = min(max(n, 0), T)
        assert (mine[b, n:] == 9).all() and torch.equal(mine[b, :n], y[b, :n])


@pytest.mark.parametrize("T,n", [(40, 17), (40, 1), (700, 300)])
def test_padding_leaves_the_state_bit_for_bit(ssm, T, n):
    """A row of n tokens in a longer batch ends in the bits that it ends in by itself, where both go
    through the tokens alike (one CTA: short, or without many SMs to spare)."""
    B = 1 if T < 100 else 80
    p = problem(B, T, 32, 16, F32, seed=n)
    c = cuda(p)
    full = torch.full((B,), n, dtype=torch.int32, device="cuda")
    y, h = ssm.selective_scan(*args(c), h0=c["h0"], lengths=full)
    q = {k: v[:, :n].contiguous() if k in ("u", "delta", "Bm", "Cm", "z") else v for k, v in c.items()}
    y2, h2 = ssm.selective_scan(*args(q), h0=c["h0"])
    assert torch.equal(h, h2) and torch.equal(y[:, :n], y2)


def test_no_tokens_and_no_rows(ssm):
    p = cuda(problem(2, 0, 6, 16, F32))
    y, h, ck = ssm.selective_scan(*args(p), h0=p["h0"], want_chunks=True)
    assert y.shape == (2, 0, 6) and torch.equal(h, p["h0"]) and ck.shape == (2, 0, 6, 16)
    r = ssm.selective_scan_backward(*args(p), ck, y, p["h0"])
    assert torch.equal(r["dh0"], p["h0"]) and not r["dA"].any() and not r["dD"].any()
    p = cuda(problem(0, 5, 6, 16, F32))
    y, h, ck = ssm.selective_scan(*args(p), h0=p["h0"], want_chunks=True)
    assert y.shape == (0, 5, 6)
    r = ssm.selective_scan_backward(*args(p), ck, y)
    assert not r["dA"].any() and not r["ddelta_bias"].any() and r["du"].shape == (0, 5, 6)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strides(ssm, dtype):
    """Slices of projections, at odd offsets, and broadcast inputs."""
    B, T, C, G, N = 2, 21, 10, 2, 8
    p = problem(B, T, C, N, dtype, G=G, seed=3)
    wide = torch.randn(B, T, 3 * C + 1).to(dtype)
    proj = torch.randn(T, B, 1 + 2 * G * N).to(dtype).transpose(0, 1)
    q = dict(p, u=wide[..., 1:C + 1], z=wide[..., 2 * C:3 * C],
             delta=p["delta"][:, :1].expand(B, T, C),                      # token stride 0
             Bm=proj[..., 1:1 + G * N].unflatten(-1, (G, N)),
             Cm=proj[..., 1 + G * N:].unflatten(-1, (G, N))[:, :, :1].expand(B, T, G, N))
    wc, pc, dc = wide.cuda(), proj.cuda(), p["delta"].cuda()
    c = dict(cuda(p), u=wc[..., 1:C + 1], z=wc[..., 2 * C:3 * C], delta=dc[:, :1].expand(B, T, C),
             Bm=pc[..., 1:1 + G * N].unflatten(-1, (G, N)),
             Cm=pc[..., 1 + G * N:].unflatten(-1, (G, N))[:, :, :1].expand(B, T, G, N))
    ry, rh = ref.scan(*(ref.up(q[k]) for k in NAMES), ref.up(p["h0"]), None)
    out = torch.zeros(B, T, 2 * C, dtype=dtype, device="cuda")
    y, h, ck = ssm.selective_scan(*args(c), h0=c["h0"], y=out[..., C:], want_chunks=True)
    assert ref.rrms(y, ry) <= ref.tol(dtype, T) and ref.rrms(h, rh) <= ref.tol(F32, T)
    assert not out[..., :C].any()
    # and the gradients, with a strided dy
    dy = torch.randn(B, T, 2 * C).to(dtype)
    leaves = [ref.up(q[k]).contiguous().requires_grad_() for k in NAMES]
    ry, _ = ref.scan(*leaves, ref.up(p["h0"]), None)
    want = ref.gradients((ry,), (ref.up(dy[..., :C]),), leaves)
    r = ssm.selective_scan_backward(*args(c), ck, dy.cuda()[..., :C])
    for k, w in zip(("du", "ddelta", "dA", "dBm", "dCm", "dD", "dz", "ddelta_bias"), want):
        assert ref.rrms(r[k], w) <= ref.tol(r[k].dtype, T, B * T), k


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N", [8, 16, 32, 64])
def test_prompt_in_parts_and_in_tokens(ssm, N, dtype):
    B, T, C = 3, 53, 20
    c = cuda(problem(B, T, C, N, dtype, G=2, seed=N))
    tok = ("u", "delta", "Bm", "Cm", "z")
    y, hT = ssm.selective_scan(*args(c), h0=c["h0"], out_dtype=F32)
    h, parts = c["h0"].clone(), []
    for a, b in ((0, 1), (1, 33), (33, 53)):
        q = {k: v[:, a:b] if k in tok else v for k, v in c.items()}
        o, h2 = ssm.selective_scan(*args(q), h0=h, h_T=h, out_dtype=F32)
        assert h2 is h
        parts.append(o)
    # the same recurrence in the same order: only the contraction of products may differ
    assert ref.rrms(torch.cat(parts, 1), y) <= ref.tol(F32, T) and ref.rrms(h, hT) <= ref.tol(F32, T)
    h, steps = c["h0"].clone(), []
    for t in range(T):
        q = {k: v[:, t] if k in tok else v for k, v in c.items()}
        steps.append(ssm.selective_step(*args(q), h, out_dtype=F32))
    assert ref.rrms(torch.stack(steps, 1), y) <= ref.tol(F32, T)
    assert ref.rrms(h, hT) <= ref.tol(F32, T)


@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("B,C,G,N", [(1, 1, 1, 8), (5, 33, 1, 16), (3, 130, 2, 32), (2, 17, 1, 64)])
def test_step(ssm, B, C, G, N, dtype, out):
    p = problem(B, 1, C, N, dtype, G=G, seed=C)
    one = {k: v[:, 0] if k in ("u", "delta", "Bm", "Cm", "z") else v for k, v in p.items()}
    on = torch.ones(B, dtype=torch.uint8)
    on[1::2] = 0
    ry, rh = ref.scan(*args(clean(p)), ref.up(p["h0"]), on.int())
    c = cuda(one)
    h, y = c["h0"].clone(), torch.full((B, C), 5.0, dtype=out, device="cuda")
    ssm.selective_step(*args(c), h, active=on.cuda(), y=y)
    for b in range(B):
        if on[b]:
            assert ref.rrms(y[b], ry[b, 0]) <= ref.tol(out, 1)
            assert ref.rrms(h[b], rh[b]) <= ref.tol(F32, 1)
        else:
            assert (y[b] == 5).all() and torch.equal(h[b], c["h0"][b])
    # every option off
    h = c["h0"].clone()
    y = ssm.selective_step(c["u"], c["delta"].abs(), c["A"], c["Bm"], c["Cm"], None, None, None, h,
                           softplus=False)
    q = clean(p)
    ry, rh = ref.scan(q["u"], q["delta"].abs(), q["A"], q["Bm"], q["Cm"], None, None, None, q["h0"], None,
                      False)
    assert ref.rrms(y, ry[:, 0]) <= ref.tol(dtype, 1) and ref.rrms(h, rh) <= ref.tol(F32, 1)


GRADS = ("du", "ddelta", "dA", "dBm", "dCm", "dD", "dz", "ddelta_bias", "dh0")


def check_backward(ssm, p, out=None, softplus=True, dh=True, seed=1):
    B, T, C = p["u"].shape
    G, N = p["Bm"].shape[2:]
    g = torch.Generator().manual_seed(seed)
    dy = torch.randn(B, T, C, generator=g).to(out or p["u"].dtype)
    dhT = torch.randn(B, C, N, generator=g) if dh else None
    q = clean(p)
    leaves = [None if q[k] is None else q[k].requires_grad_() for k in NAMES + ("h0",)]
    ry, rh = ref.scan(*leaves[:8], leaves[8], q["lengths"], softplus)
    want = ref.gradients((ry, rh), (ref.up(dy), ref.up(dhT)), leaves)
    if p["lengths"] is not None:
        for b, n in enumerate(p["lengths"].tolist()):
            dy[b, min(max(n, 0), T):] = float("nan")
    c = cuda(p)
    _, _, ck = ssm.selective_scan(*args(c), softplus=softplus, h0=c["h0"], lengths=c["lengths"],
                                  want_chunks=True)
    run = lambda: ssm.selective_scan_backward(  # noqa: E731
        *args(c), ck, dy.cuda(), None if dhT is None else dhT.cuda(), softplus=softplus,
        lengths=c["lengths"])
    r = run()
    sums = {"dA": B * T, "dD": B * T, "ddelta_bias": B * T, "dBm": C // G, "dCm": C // G}
    for k, w in zip(GRADS, want):
        if w is None:
            assert k == "dh0" or r[k] is None
            continue
        # du, ddelta and dz sum over N states, the others over rows and tokens or channels
        assert ref.rrms(r[k], w) <= ref.tol(r[k].dtype, T, sums.get(k, N)), k
    again = run()
    assert all(r[k] is None or torch.equal(r[k], again[k]) for k in r)
    return r


@pytest.mark.parametrize("N", [8, 16, 32, 64])
@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF16, BF16), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("T", [1, 8, 16, 17, 41])
def test_backward(ssm, T, N, dtype, out):
    check_backward(ssm, problem(2, T, 24, N, dtype, seed=T + N), out)


@pytest.mark.parametrize("C,G,N", [(1, 1, 16), (7, 1, 8), (65, 1, 16), (130, 2, 8), (150, 1, 16), (192, 3, 32),
                                   (24, 24, 8), (34, 2, 64)])
def test_backward_channels_and_groups(ssm, C, G, N):
    check_backward(ssm, problem(2, 19, C, N, F32, G=G, seed=C))


@pytest.mark.parametrize("off", ["skip", "gate", "bias", "h0", "softplus", "dh"])
def test_backward_options(ssm, off):
    kw = {off: False} if off in ("skip", "gate", "bias", "h0") else {}
    p = problem(2, 33, 24, 16, F32, seed=9, **kw)
    if off == "softplus":   # taken as they are, step sizes are positive
        p["delta"], p["delta_bias"] = torch.rand(2, 33, 24) * 0.5, torch.rand(24) * 0.1
    check_backward(ssm, p, softplus=off != "softplus", dh=off != "dh")


@pytest.mark.parametrize("T,C,B,N", [(500, 8, 1, 16), (300, 40, 2, 8), (290, 20, 1, 64), (700, 3, 2, 32)])
def test_backward_long_prompts_are_split(ssm, T, C, B, N):
    check_backward(ssm, problem(B, T, C, N, F32, seed=T))


@pytest.mark.parametrize("T,lengths", [(40, [40, 0, 1, 17, 32]), (400, [400, 0, 1, 130, 399]), (3, [0, 0, 0, 0, 0]),
                                       (20, [99, -3, 20, 5, 16])])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_backward_lengths(ssm, T, lengths, dtype):
    p = problem(5, T, 12, 16, dtype, seed=6, lengths=lengths)
    r = check_backward(ssm, p)
    for b, n in enumerate(lengths):
        for k in ("du", "ddelta", "dz", "dBm", "dCm"):
            assert not r[k][b, min(max(n, 0), T):].any(), k


def test_backward_against_differences(ssm):
    """<gradient, direction> against central differences of the 64-bit loss."""
    B, T, C, N = 2, 23, 6, 8
    p = problem(B, T, C, N, F32, G=2, seed=13)
    g = torch.Generator().manual_seed(4)
    dy, dhT = torch.randn(B, T, C, generator=g), torch.randn(B, C, N, generator=g)
    c = cuda(p)
    _, _, ck = ssm.selective_scan(*args(c), h0=c["h0"], want_chunks=True)
    r = ssm.selective_scan_backward(*args(c), ck, dy.cuda(), dhT.cuda())
    at = [ref.up(p[k]) for k in NAMES + ("h0",)]
    for i, key in enumerate(GRADS):
        v = torch.randn(at[i].shape, generator=g, dtype=torch.float64)

        def loss(e):
            a = list(at)
            a[i] = a[i] + e * v
            y, h = ref.scan(*a[:8], a[8], None)
            return (y * dy.double()).sum() + (h * dhT.double()).sum()
        e = 1e-5   # e^2 of truncation, 1e-16 / e of rounding
        diff = float((loss(e) - loss(-e)) / (2 * e))
        got = float((ref.up(r[key]) * v).sum())
        assert abs(got - diff) <= ref.tol(F32, T) * float(ref.up(r[key]).norm() * v.norm()), key


def test_values_at_the_edges(ssm):
    """Step sizes near 0 and large ones, fast decays, large gates."""
    B, T, C, N = 1, 40, 8, 16
    p = problem(B, T, C, N, F32, seed=17)
    p["delta"] = torch.linspace(-25, 25, T)[None, :, None].expand(B, T, C).contiguous()
    p["delta_bias"] = None
    p["A"] = -torch.logspace(-4, 3, C * N).view(C, N)
    p["z"] = torch.linspace(-90, 90, T)[None, :, None].expand(B, T, C).contiguous()
    c, q = cuda(p), clean(p)
    y, h = ssm.selective_scan(*args(c), h0=c["h0"])
    ry, rh = ref.scan(*args(q), q["h0"], None)
    assert ref.rrms(y, ry) <= ref.tol(F32, T) and ref.rrms(h, rh) <= ref.tol(F32, T)
    # token by token: a small value is not drowned by the others'
    for t in range(T):
        assert ref.rrms(y[:, t], ry[:, t]) <= ref.tol(F32, T) * 4 or ry[:, t].abs().max() < 1e-30, t


def test_streams_and_graphs(ssm):
    p = cuda(problem(2, 150, 24, 16, BF16, seed=41))
    dy = torch.randn(2, 150, 24, device="cuda").to(BF16)

    def both(**kw):
        y, h, ck = ssm.selective_scan(*args(p), h0=p["h0"], want_chunks=True, **kw)
        return dict(ssm.selective_scan_backward(*args(p), ck, dy, h, **kw), y=y, h=h)
    r = both()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    r2 = both(stream=side)
    side.synchronize()
    assert all(torch.equal(r[k], r2[k]) for k in r)
    # two captured passes, replayed in turn and together
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(both())
        graphs.append(g)
    for g in (graphs[0], graphs[1], graphs[0]):
        g.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(r[k], o[k]) for k in r)
    # a captured step moves its state at every replay
    h = p["h0"].clone()
    one = {k: v[:, 0] if k in ("u", "delta", "Bm", "Cm", "z") else v for k, v in p.items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = ssm.selective_step(*args(one), h)
    h.copy_(p["h0"])
    for _ in range(3):
        g.replay()
    want = p["h0"].clone()
    for _ in range(3):
        wy = ssm.selective_step(*args(one), want)
    torch.cuda.synchronize()
    assert torch.equal(h, want) and torch.equal(y, wy)


def test_refusals(ssm):
    p = cuda(problem(2, 20, 16, 16, F32))
    a = args(p)
    change = lambda **kw: args(dict(p, **kw))  # noqa: E731
    bad = [
        change(u=p["u"].cpu()), change(u=p["u"].half()), change(u=p["u"][0]),
        change(delta=p["delta"].to(BF16)), change(delta=p["delta"][:, :5]), change(A=p["A"][:8]),
        change(A=p["A"].to(BF16)), change(Bm=p["Bm"][..., :8]), change(Cm=p["Cm"][:, :, :0]),
        change(D=p["D"][:3]), change(z=p["z"][..., :8]), change(delta_bias=p["D"].double()),
    ]
    for x in bad:
        with pytest.raises(ValueError):
            ssm.selective_scan(*x)
    with pytest.raises(ValueError):
        ssm.selective_scan(*a, h0=p["h0"][:1])
    with pytest.raises(ValueError):
        ssm.selective_scan(*a, lengths=torch.tensor([3, 4], device="cuda"))
    with pytest.raises(ValueError):
        ssm.selective_scan_backward(*a, torch.zeros(2, 1, 16, 16, device="cuda"), p["u"])
    with pytest.raises(ValueError):
        ssm.selective_step(*a, p["h0"])
    from test_sequence_layers_02_b200.ttt_scan import TTTScanError
    with pytest.raises(TTTScanError):     # N
        ssm.selective_scan(*change(A=p["A"][:, :4].contiguous(), Bm=p["Bm"][..., :4], Cm=p["Cm"][..., :4]))
    with pytest.raises(TTTScanError):     # groups that do not divide the channels
        ssm.selective_scan(*change(Bm=p["Bm"].expand(2, 20, 3, 16), Cm=p["Cm"].expand(2, 20, 3, 16)))
    with pytest.raises(TTTScanError):     # the output over an input
        ssm.selective_scan(*a, y=p["z"])
    with pytest.raises(TTTScanError):     # rows of an output on top of one another
        ssm.selective_scan(*a, y=torch.empty(1, 20, 16, device="cuda").expand(2, 20, 16))
    _, _, ck = ssm.selective_scan(*a, want_chunks=True)
    with pytest.raises(TTTScanError):     # too small a workspace
        ssm.selective_scan_backward(*a, ck, p["u"].clone(), workspace=torch.empty(4, device="cuda"))


LOWEST = torch.finfo(F32).min


@pytest.mark.parametrize("N", [8, 16, 64])
@pytest.mark.parametrize("T,lengths", [(20, None), (20, [20, 5, 0]), (16, None), (300, [300, 129, 7])])
def test_states_that_are_switched_off(ssm, T, lengths, N):
    """The lowest fp32 value in A (and one that only a factor of log2 e takes out of range): exp(dt A) is 0 at a
    step and 1 where there is none, behind a length, in a tile's last tokens or in an empty span."""
    p = problem(3, T, 12, N, F32, seed=T + N, lengths=lengths)
    p["A"][:, 3] = LOWEST
    p["A"][5] = -2.5e38
    y, h, _ = check_forward(ssm, p)
    assert torch.isfinite(y).all() and torch.isfinite(h).all()
    check_backward(ssm, p)


@pytest.mark.parametrize("N", [8, 16, 64])
def test_step_of_no_length_with_a_state_switched_off(ssm, N):
    """A step size of 0 (softplus of a large negative number) leaves every state as it is."""
    p = problem(3, 1, 12, N, F32, seed=N)
    p["A"][:, 3] = LOWEST
    p["delta"][1] = -300.0
    one = cuda({k: v[:, 0] if k in ("u", "delta", "Bm", "Cm", "z") else v for k, v in p.items()})
    h = one["h0"].clone()
    y = ssm.selective_step(*args(one), h)
    q = clean(p)
    ry, rh = ref.scan(*args(q), q["h0"], None)
    assert ref.rrms(y, ry[:, 0]) <= ref.tol(F32, 1) and ref.rrms(h, rh) <= ref.tol(F32, 1)
    assert torch.equal(h[1], one["h0"][1])
    y, h = ssm.selective_scan(*args(cuda(p)), h0=one["h0"])
    assert ref.rrms(y, ry) <= ref.tol(F32, 1) and ref.rrms(h, rh) <= ref.tol(F32, 1)


@pytest.mark.parametrize("N", [8, 16, 32])
def test_growth_beyond_range_over_a_span_of_nothing(ssm, N):
    """States that would grow by more than fp32 holds over a span of a split prompt, but have nothing to
    grow from: they stay 0, as in a prompt that is not split. Likewise a gradient of 0 on its way back."""
    B, T, C = 1, 400, 8
    p = problem(B, T, C, N, F32, seed=N, h0=False, bias=False)
    p["A"], p["delta"] = torch.full((C, N), 2.0), torch.ones(B, T, C)
    p["u"][:, :T - 6] = 0                  # the states start in the last span, and grow by e^12
    y, h, ck = check_forward(ssm, p, softplus=False)
    assert not h.isnan().any() and not y[:, :T - 6].any()
    # and back: gradients that start in the first span, below states of 0
    p["u"].zero_()
    dy = torch.zeros(B, T, C)
    dy[:, :3] = torch.randn(B, 3, C, generator=torch.Generator().manual_seed(3))
    c, q = cuda(p), clean(p)
    _, _, ck = ssm.selective_scan(*args(c), softplus=False, want_chunks=True)
    r = ssm.selective_scan_backward(*args(c), ck, dy.cuda(), softplus=False)
    leaves = [None if q[k] is None else q[k].requires_grad_() for k in NAMES]
    want = ref.gradients(ref.scan(*leaves, None, None, False)[:1], (ref.up(dy),), leaves)
    for k, w in zip(GRADS, want):
        if w is not None:
            assert ref.rrms(r[k], w) <= ref.tol(F32, T, C * T), k


def test_growth_beyond_range_of_a_small_state(ssm):
    """1e-20 e^100 = 2.7e23 is a number of fp32, e^100 is not; the second half of the tokens leave it as it is."""
    B, T, C, N = 1, 160, 4, 16
    p = problem(B, T, C, N, F32, seed=1, bias=False)
    p["u"].zero_()
    p["h0"] = torch.full((B, C, N), 1e-20)
    p["A"] = torch.full((C, N), 100 / 80)
    p["delta"] = torch.cat((torch.ones(B, 80, C), torch.zeros(B, 80, C)), 1)
    y, h, _ = check_forward(ssm, p, softplus=False)
    assert torch.isfinite(h).all()


def test_one_token_of_a_token_major_batch(ssm):
    """T = 1: the distance between tokens does not matter, however long."""
    B, C, N = 3, 16, 16
    p = problem(B, 1, C, N, F32, seed=2)
    c = cuda(p)
    y, h, ck = ssm.selective_scan(*args(c), h0=c["h0"], want_chunks=True)
    dy = torch.randn(B, 1, C, device="cuda")
    r = ssm.selective_scan_backward(*args(c), ck, dy, h)
    wide = torch.zeros(B, 3 * C, device="cuda")
    far = dict(c)
    for i, k in enumerate(("u", "delta", "z")):   # slices of a projection [1, B, 3 C] of a larger batch
        wide[:, i * C:(i + 1) * C] = c[k][:, 0]
        far[k] = torch.as_strided(wide, (B, 1, C), (3 * C, 1 << 25, 1), i * C)
    assert not far["u"].is_contiguous()
    y2, h2, ck2 = ssm.selective_scan(*args(far), h0=c["h0"], want_chunks=True)
    r2 = ssm.selective_scan_backward(*args(far), ck2, dy, h)
    assert torch.equal(y, y2) and torch.equal(h, h2) and all(torch.equal(r[k], r2[k]) for k in r)


@pytest.mark.parametrize("N", [8, 16, 32, 64])
@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF16, BF16), (F32, BF16)])
def test_step_of_a_large_batch(ssm, N, dtype, out):
    """Enough rows for several of them a thread (a batch that leaves a remainder): every row by itself."""
    B, C, G = 303, 520, 2
    p = problem(B, 1, C, N, dtype, G=G, seed=N)
    one = cuda({k: v[:, 0] if k in ("u", "delta", "Bm", "Cm", "z") else v for k, v in p.items()})
    on = (torch.rand(B, generator=torch.Generator().manual_seed(N)) < 0.7).to(torch.uint8)
    on[-3:] = torch.tensor([1, 0, 1], dtype=torch.uint8)
    ry, rh = ref.scan(*args(clean(p)), ref.up(p["h0"]), on.int())
    h, y = one["h0"].clone(), torch.full((B, C), 5.0, dtype=out, device="cuda")
    ssm.selective_step(*args(one), h, active=on.cuda(), y=y)
    h2 = one["h0"].clone()
    y2 = ssm.selective_step(*args(one), h2, active=on.cuda(), out_dtype=out)
    assert torch.equal(h, h2)
    for b in range(B):
        if on[b]:
            assert ref.rrms(y[b], ry[b, 0]) <= ref.tol(out, 1), b
            assert ref.rrms(h[b], rh[b]) <= ref.tol(F32, 1), b
            assert torch.equal(y[b], y2[b])
        else:
            assert (y[b] == 5).all() and not y2[b].any() and torch.equal(h[b], one["h0"][b]), b
    # all rows, no options, and a single element off the packs
    h3 = one["h0"].clone()
    wide = torch.zeros(B, G * N + 1, dtype=dtype, device="cuda")
    wide[:, 1:] = one["Bm"].flatten(1)
    y3 = ssm.selective_step(one["u"], one["delta"], one["A"], wide[:, 1:].unflatten(1, (G, N)), one["Cm"], None, None, None,
                            h3, out_dtype=out)
    q = clean(p)
    ry, rh = ref.scan(q["u"], q["delta"], q["A"], q["Bm"], q["Cm"], None, None, None, q["h0"], None)
    for b in range(B):
        assert ref.rrms(y3[b], ry[b, 0]) <= ref.tol(out, 1) and ref.rrms(h3[b], rh[b]) <= ref.tol(F32, 1), b


@pytest.mark.parametrize("C,G,N", [(24, 3, 16), (21, 3, 16), (40, 2, 8), (16, 2, 32)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_split_prompts_with_groups_strides_and_lengths(ssm, C, G, N, dtype):
    """Tokens over a cluster of CTAs, with slices of projections for inputs, groups and a ragged batch."""
    B, T = 3, 411
    p = problem(B, T, C, N, dtype, G=G, seed=C, lengths=[411, 130, 3])
    c = cuda(p)
    wide = torch.empty(B, T, 3 * C, dtype=dtype, device="cuda")
    proj = torch.empty(B, T, 2 * G * N, dtype=dtype, device="cuda")
    for i, k in enumerate(("u", "z", "delta")):
        wide[..., i * C:(i + 1) * C] = c[k]
        c[k] = wide[..., i * C:(i + 1) * C]
    for i, k in enumerate(("Bm", "Cm")):
        proj[..., i * G * N:(i + 1) * G * N] = c[k].flatten(2)
        c[k] = proj[..., i * G * N:(i + 1) * G * N].unflatten(2, (G, N))
    y, h, ck = ssm.selective_scan(*args(c), h0=c["h0"], lengths=c["lengths"], want_chunks=True)
    q = clean(p)
    leaves = [q[k].requires_grad_() for k in NAMES + ("h0",)]
    ry, rh = ref.scan(*leaves, q["lengths"])
    for b, n in enumerate(p["lengths"].tolist()):
        assert ref.rrms(y[b, :n], ry[b, :n]) <= ref.tol(dtype, n) and not y[b, n:].any()
        assert ref.rrms(h[b], rh[b]) <= ref.tol(F32, n)
    g = torch.Generator().manual_seed(1)
    dy, dh = torch.randn(B, T, C, generator=g).to(dtype), torch.randn(B, C, N, generator=g)
    want = ref.gradients((ry, rh), (ref.up(dy), ref.up(dh)), leaves)
    two = torch.full((B, T, 2 * C), float("nan"), dtype=dtype)
    for b, n in enumerate(p["lengths"].tolist()):
        two[b, :n, C:] = dy[b, :n]
    r = ssm.selective_scan_backward(*args(c), ck, two.cuda()[..., C:], dh.cuda(), lengths=c["lengths"])
    terms = {"dA": B * T, "dD": B * T, "ddelta_bias": B * T, "dBm": C // G, "dCm": C // G}
    for k, w in zip(GRADS, want):
        assert ref.rrms(r[k], w) <= ref.tol(r[k].dtype, T, terms.get(k, N)), k


def straight(p, grads=None):
    """The reference's form in fp32, and its error against 64 bits: outputs, and gradients for ``grads``."""
    res = []
    for up in (lambda t: t.detach().clone(), ref.up):
        leaves = [None if p[k] is None else up(p[k]).requires_grad_(grads is not None) for k in NAMES + ("h0",)]
        out = ref.scan(*leaves[:8], leaves[8], None)
        if grads is not None:
            out = tuple(out) + tuple(ref.gradients(out, [up(g) for g in grads], leaves))
        res.append(out)
    return res[1], [ref.rrms(a, b) for a, b in zip(*res)]


# Eight times the error of a straight fp32 evaluation (a decay here is one ex2, four times as far off as exp
# may be, of a rounded argument, and sums are taken in another order), and 2^-21 where that one
# happens to be exact. Steps or states held in bf16 or tf32 are off by 2^-9 or 2^-12.
def close_as_fp32(got, want, error, what):
    assert ref.rrms(got, want) <= 8 * error + 2.0 ** -21, (what, ref.rrms(got, want), error)


@pytest.mark.parametrize("B,T,C,N", [(2, 100, 40, 16), (2, 1500, 24, 8), (80, 300, 33, 16), (1, 9001, 8, 16), (2, 700, 12, 64)])
def test_as_exact_as_fp32(ssm, B, T, C, N):
    p = problem(B, T, C, N, F32, seed=T)
    c = cuda(p)
    y, h = ssm.selective_scan(*args(c), h0=c["h0"])
    want, error = straight(p)
    close_as_fp32(y, want[0], error[0], "y")
    close_as_fp32(h, want[1], error[1], "h")


@pytest.mark.parametrize("B,T,C,N", [(2, 90, 40, 16), (1, 500, 24, 8), (2, 333, 12, 32)])
def test_gradients_as_exact_as_fp32(ssm, B, T, C, N):
    p = problem(B, T, C, N, F32, seed=T)
    g = torch.Generator().manual_seed(1)
    dy, dh = torch.randn(B, T, C, generator=g), torch.randn(B, C, N, generator=g)
    c = cuda(p)
    _, _, ck = ssm.selective_scan(*args(c), h0=c["h0"], want_chunks=True)
    r = ssm.selective_scan_backward(*args(c), ck, dy.cuda(), dh.cuda())
    want, error = straight(p, (dy, dh))
    for k, w, e in zip(GRADS, want[2:], error[2:]):
        close_as_fp32(r[k], w, e, k)


def test_decays_have_no_bias(ssm):
    """A state without input, 112 tokens of one decay: the mean error of a decay between 0.7 and 1 stays within 0.2
    units of 2^-24. 16384 decays in each of six ranges: their mean is known to 0.01 units (each
    is off by up to 2 units and the products by half a unit a token, of either sign)."""
    T, C, N = 112, 1024, 16
    for lo, hi in ((0.70, 0.75), (0.75, 0.80), (0.80, 0.85), (0.85, 0.90), (0.90, 0.95), (0.95, 0.999)):
        a = torch.rand(C, N, generator=torch.Generator().manual_seed(int(lo * 100)), dtype=torch.float64) * (hi - lo) + lo
        A = torch.log(a).float()
        one, zero = torch.ones(1, T, C, device="cuda"), torch.zeros(1, T, C, device="cuda")
        v = torch.zeros(1, T, N, device="cuda")
        _, h = ssm.selective_scan(zero, one, A.cuda(), v, v, softplus=False, h0=torch.ones(1, C, N, device="cuda"))
        units = (torch.log(ref.up(h)[0]) - T * A.double()).mean() / T * 2 ** 24
        assert abs(units) <= 0.2 + 0.01, (lo, float(units))
