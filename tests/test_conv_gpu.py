"""The short causal convolution against a plain form in 64 bits: prompts, gradients, single tokens."""

import pytest
import torch

from tests import seq_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def conv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from test_sequence_layers_02_b200 import build, conv as module
    build.build()
    return module


def problem(B, T, D, K, dtype, seed=0, state=True, bias=True, lengths=None):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = r(B, T, D).to(dtype)
    if lengths is not None:
        lengths = torch.tensor(lengths, dtype=torch.int32)
        for b, n in enumerate(lengths.tolist()):
            x[b, max(n, 0):] = float("nan")    # nothing behind a length may be read
    return dict(x=x, weight=r(D, K) * 0.5, bias=r(D) * 0.5 if bias else None,
                state=r(B, K - 1, D).to(dtype) if state else None, lengths=lengths)


def cuda(p):
    return {k: None if v is None else v.cuda() for k, v in p.items()}


def bound(out_dtype, K):
    """K + 1 roundings and the SiLU's special functions (each below 2^-21), and the output's own."""
    return (K + 8) * 2.0 ** -21 + (ref.BF16 if out_dtype == BF16 else 0.0)


def check_forward(conv, p, silu, out_dtype=None):
    c = cuda(p)
    y, st = conv.causal_conv(c["x"], c["weight"], c["bias"], silu=silu, state=c["state"],
                             lengths=c["lengths"], out_dtype=out_dtype)
    ry, rst = ref.conv(*(ref.up(p[k]) for k in ("x", "weight", "bias", "state")), p["lengths"], silu)
    K = p["weight"].shape[1]
    assert ref.rrms(y, ry) <= bound(y.dtype, K)
    assert torch.equal(ref.up(st), rst)   # moved, not computed
    return y, st


@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF16, BF16), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("T", [1, 2, 3, 16, 17, 45])
def test_prompt(conv, T, K, dtype, out):
    check_forward(conv, problem(2, T, 24, K, dtype, seed=T), True, out)


@pytest.mark.parametrize("D", [1, 7, 8, 200, 1032])
@pytest.mark.parametrize("state,bias,silu", [(True, True, True), (False, True, False),
                                             (True, False, True), (False, False, False)])
def test_prompt_channels_and_options(conv, D, state, bias, silu):
    check_forward(conv, problem(2, 37, D, 4, F32, seed=D, state=state, bias=bias), silu)
    check_forward(conv, problem(2, 37, D, 4, BF16, seed=D, state=state, bias=bias), silu)


@pytest.mark.parametrize("K", [2, 4])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_lengths(conv, K, dtype):
    p = problem(6, 40, 16, K, dtype, seed=3, lengths=[40, 0, 1, 2, 17, 39])
    check_forward(conv, p, True)
    # a given y keeps what it holds behind a length; lengths beyond the range are clipped
    c = cuda(p)
    y = torch.full((6, 40, 16), 7.0, dtype=dtype, device="cuda")
    conv.causal_conv(c["x"], c["weight"], c["bias"], lengths=c["lengths"], state=c["state"], y=y)
    for b, n in enumerate(p["lengths"].tolist()):
        assert (y[b, n:] == 7).all() and torch.isfinite(y[b, :n].float()).all()
    q = problem(2, 12, 16, K, dtype, seed=4)
    q["lengths"] = torch.tensor([99, -5], dtype=torch.int32)
    check_forward(conv, q, True)


def test_no_tokens_and_no_rows(conv):
    p = cuda(problem(2, 0, 8, 4, F32))
    y, st = conv.causal_conv(p["x"], p["weight"], p["bias"], state=p["state"])
    assert y.shape == (2, 0, 8) and torch.equal(st, p["state"])
    g = conv.causal_conv_backward(p["x"], p["weight"], p["bias"], y, p["state"], state=p["state"])
    assert torch.equal(g["dstate"], p["state"]) and not g["dweight"].any() and not g["dbias"].any()
    p = cuda(problem(0, 5, 8, 4, F32))
    y, st = conv.causal_conv(p["x"], p["weight"], p["bias"], state=p["state"])
    assert y.shape == (0, 5, 8) and st.shape == (0, 3, 8)
    g = conv.causal_conv_backward(p["x"], p["weight"], p["bias"], y, state=p["state"])
    assert not g["dweight"].any() and not g["dbias"].any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [8, 5])
def test_heads_and_strides(conv, dtype, d):
    """A slice of a token-major projection, read in place and written as heads."""
    B, T, H, K = 2, 21, 3, 4
    p = problem(B, T, 3 * H * d + 1, K, dtype, seed=9)
    x = p["x"][..., H * d:2 * H * d]                       # strided; unaligned for d = 5
    w, b = p["weight"][:H * d].contiguous(), p["bias"][:H * d].contiguous()
    st = p["state"][..., 1:1 + H * d]
    ry, rst = ref.conv(ref.up(x), ref.up(w), ref.up(b), ref.up(st), None, True)
    heads = lambda t: t.unflatten(-1, (H, d)).transpose(1, 2)  # noqa: E731
    xc, sc = p["x"].cuda()[..., H * d:2 * H * d], p["state"].cuda()[..., 1:1 + H * d]
    y, s2 = conv.causal_conv(heads(xc), w.cuda().view(H, d, K), b.cuda().view(H, d), silu=True,
                             state=heads(sc))
    assert y.is_contiguous() and y.shape == (B, H, T, d)
    assert ref.rrms(y, heads(ry)) <= bound(dtype, K)
    assert torch.equal(ref.up(s2), heads(rst))
    # into a strided output
    wide = torch.zeros(B, T, 2 * H * d, dtype=dtype, device="cuda")
    conv.causal_conv(heads(xc), w.cuda().view(H, d, K), b.cuda().view(H, d), silu=True,
                     state=heads(sc), y=heads(wide[..., H * d:]))
    assert ref.rrms(wide[..., H * d:], ry) <= bound(dtype, K) and not wide[..., :H * d].any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("K", [2, 3, 4])
def test_prompt_in_parts_and_in_tokens(conv, K, dtype):
    """A prompt, the same in three parts with the state in place, and token by token: the same bits."""
    p = cuda(problem(3, 39, 40, K, dtype, seed=11))
    args = (p["weight"], p["bias"])
    y, st = conv.causal_conv(p["x"], *args, silu=True, state=p["state"])
    parts, s = [], p["state"].clone()
    for a, b in ((0, 1), (1, 20), (20, 39)):
        o, s2 = conv.causal_conv(p["x"][:, a:b], *args, silu=True, state=s, state_T=s)
        assert s2 is s
        parts.append(o)
    assert torch.equal(torch.cat(parts, 1), y) and torch.equal(s, st)
    s = p["state"].clone()
    steps = [conv.causal_conv_step(p["x"][:, t], *args, s, silu=True) for t in range(39)]
    assert torch.equal(torch.stack(steps, 1), y) and torch.equal(s, st)


def test_step_heads_and_active(conv):
    B, H, d, K = 5, 2, 9, 3
    g = torch.Generator().manual_seed(5)
    x = torch.randn(B, H, d, generator=g)
    w, bias = torch.randn(H, d, K, generator=g), torch.randn(H, d, generator=g)
    st = torch.randn(B, H, K - 1, d, generator=g)
    on = torch.tensor([1, 0, 1, 1, 0], dtype=torch.uint8)
    s, y = st.cuda(), torch.full((B, H, d), 3.0, device="cuda")
    conv.causal_conv_step(x.cuda(), w.cuda(), bias.cuda(), s, silu=True, active=on.cuda(), y=y)
    flat = lambda t: t.transpose(1, 2).reshape(B, -1, H * d)  # noqa: E731
    ry, rs = ref.conv(x.reshape(B, 1, H * d).double(), w.view(H * d, K).double(),
                      bias.view(-1).double(), flat(st).double(), None, True)
    for b in range(B):
        if on[b]:
            assert ref.rrms(y[b].reshape(1, -1), ry[b]) <= bound(F32, K)
            assert torch.equal(ref.up(flat(s.cpu())[b]), rs[b])
        else:
            assert (y[b] == 3).all() and torch.equal(s[b].cpu(), st[b])
    made = conv.causal_conv_step(x.cuda(), w.cuda(), bias.cuda(), s, active=on.cuda())
    assert not made[1].any() and not made[4].any()


def reference_gradients(p, dy, dst, silu):
    names = ("x", "weight", "bias", "state")
    x = p["x"]
    if p["lengths"] is not None:
        x = torch.nan_to_num(x, nan=0.0)
    leaves = [None if t is None else ref.up(t).requires_grad_() for t in
              (x, *(p[k] for k in names[1:]))]
    y, st = ref.conv(*leaves, p["lengths"], silu)
    return ref.gradients((y, st), (ref.up(dy), None if dst is None else ref.up(dst)), leaves)


@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("T,D,lengths", [(1, 8, None), (2, 5, None), (31, 24, None), (70, 12, [70, 0, 33]),
                                         (300, 8, [300, 1, 257]), (40, 200, [3, 2, 40])])
def test_backward(conv, T, D, lengths, K, dtype, out):
    B = 3 if lengths else 2
    p = problem(B, T, D, K, dtype, seed=T + D, lengths=lengths)
    g = torch.Generator().manual_seed(1)
    dy = torch.randn(B, T, D, generator=g).to(out)
    dst = torch.randn(B, K - 1, D, generator=g).to(dtype)
    want = reference_gradients(p, dy if lengths is None else torch.where(
        torch.arange(T)[None, :, None] < p["lengths"][:, None, None], dy, torch.zeros_like(dy)), dst, True)
    if lengths:
        for b, n in enumerate(lengths):
            dy[b, n:] = float("nan")
    c = cuda(p)
    r = conv.causal_conv_backward(c["x"], c["weight"], c["bias"], dy.cuda(), dst.cuda(), silu=True,
                                  state=c["state"], lengths=c["lengths"])
    terms = B * T
    for name, w, n in (("dx", want[0], 1), ("dweight", want[1], terms), ("dbias", want[2], terms),
                       ("dstate", want[3], 1)):
        # as forward, and the sums over n terms
        assert ref.rrms(r[name], w) <= bound(r[name].dtype, K) * (1 + n ** 0.5), name
    again = conv.causal_conv_backward(c["x"], c["weight"], c["bias"], dy.cuda(), dst.cuda(), silu=True,
                                      state=c["state"], lengths=c["lengths"])
    assert all(torch.equal(r[k], again[k]) for k in r)


@pytest.mark.parametrize("silu,bias,state", [(False, True, True), (True, False, False)])
def test_backward_options_strides_and_heads(conv, silu, bias, state):
    B, T, H, d, K = 2, 50, 3, 8, 4
    p = problem(B, T, H * d, K, F32, seed=2, bias=bias, state=state)
    g = torch.Generator().manual_seed(3)
    dy = torch.randn(B, T, H * d, generator=g)
    want = reference_gradients(p, dy, None, silu)
    c = cuda(p)
    heads = lambda t: None if t is None else t.unflatten(-1, (H, d)).transpose(1, 2)  # noqa: E731
    r = conv.causal_conv_backward(
        heads(c["x"]), c["weight"].view(H, d, K), None if not bias else c["bias"].view(H, d),
        heads(dy.cuda()), silu=silu, state=heads(c["state"]))
    assert ref.rrms(r["dx"], heads(want[0])) <= bound(F32, K) * 2
    assert ref.rrms(r["dweight"].view(H * d, K), want[1]) <= bound(F32, K) * (1 + (B * T) ** 0.5)
    assert (r["dbias"] is None) == (not bias)
    if bias:
        assert ref.rrms(r["dbias"].view(-1), want[2]) <= bound(F32, K) * (1 + (B * T) ** 0.5)
    if state:
        assert ref.rrms(r["dstate"], heads(want[3])) <= bound(F32, K) * 2


def test_backward_against_differences(conv):
    """<gradient, direction> against central differences of the 64-bit loss."""
    B, T, D, K = 2, 19, 6, 4
    p = problem(B, T, D, K, F32, seed=21)
    g = torch.Generator().manual_seed(4)
    dy, dst = torch.randn(B, T, D, generator=g), torch.randn(B, K - 1, D, generator=g)
    c = cuda(p)
    r = conv.causal_conv_backward(c["x"], c["weight"], c["bias"], dy.cuda(), dst.cuda(), silu=True,
                                  state=c["state"])
    names = ("x", "weight", "bias", "state")
    at = [ref.up(p[k]) for k in names]
    for i, key in enumerate(("dx", "dweight", "dbias", "dstate")):
        v = torch.randn(at[i].shape, generator=g, dtype=torch.float64)

        def loss(eps):
            a = list(at)
            a[i] = a[i] + eps * v
            y, st = ref.conv(*a, None, True)
            return (y * dy.double()).sum() + (st * dst.double()).sum()
        e = 1e-5   # central differences in 64 bits: e^2 of truncation, 1e-16 / e of rounding
        diff = float((loss(e) - loss(-e)) / (2 * e))
        got = float((ref.up(r[key]) * v).sum())
        size = float(ref.up(r[key]).norm() * v.norm())
        assert abs(got - diff) <= 1e-5 * size, key


def test_stream_graph_and_workspace(conv):
    """On a side stream, and captured: replays follow the inputs and repeat the bits."""
    p = cuda(problem(2, 130, 64, 4, BF16, seed=31))
    dy = torch.randn(2, 130, 64, device="cuda").to(BF16)
    args = (p["x"], p["weight"], p["bias"])
    y, st = conv.causal_conv(*args, silu=True, state=p["state"])
    r = conv.causal_conv_backward(*args, dy, silu=True, state=p["state"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y2, _ = conv.causal_conv(*args, silu=True, state=p["state"], stream=side)
    ws = torch.empty(conv.backward_workspace_bytes(2, 1, 130, 64, 4), dtype=torch.uint8, device="cuda")
    r2 = conv.causal_conv_backward(*args, dy, silu=True, state=p["state"], stream=side, workspace=ws)
    side.synchronize()
    assert torch.equal(y, y2) and all(torch.equal(r[k], r2[k]) for k in r)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y3, st3 = conv.causal_conv(*args, silu=True, state=p["state"])
        r3 = conv.causal_conv_backward(*args, dy, silu=True, state=p["state"])
    x0 = p["x"].clone()
    p["x"].mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(y3, y)
    p["x"].copy_(x0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y3, y) and torch.equal(st3, st) and all(torch.equal(r[k], r3[k]) for k in r)


def test_refusals(conv):
    p = cuda(problem(2, 8, 16, 4, F32))
    x, w, b = p["x"], p["weight"], p["bias"]
    bad = [
        lambda: conv.causal_conv(x.cpu(), w, b),
        lambda: conv.causal_conv(x.half(), w, b),
        lambda: conv.causal_conv(x[0], w, b),
        lambda: conv.causal_conv(x, w[:8], b),
        lambda: conv.causal_conv(x, w.half(), b),
        lambda: conv.causal_conv(x, w, b[:8]),
        lambda: conv.causal_conv(x.transpose(1, 2).contiguous().transpose(1, 2), w, b),
        lambda: conv.causal_conv(x, w, b, state=p["state"][:, :2]),
        lambda: conv.causal_conv(x, w, b, state=p["state"].to(BF16)),
        lambda: conv.causal_conv(x, w, b, lengths=torch.tensor([1, 2], device="cuda")),
        lambda: conv.causal_conv(x, w, b, y=torch.empty(2, 8, 8, device="cuda")),
        lambda: conv.causal_conv(x, w, b, out_dtype=torch.float16),
        lambda: conv.causal_conv_step(x, w, b, p["state"]),
        lambda: conv.causal_conv_step(x[:, 0], w, b, p["state"], active=torch.ones(2, device="cuda")),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    lib = [
        lambda: conv.causal_conv(x, torch.zeros(16, 5, device="cuda"), b),            # K
        lambda: conv.causal_conv(x, w, b, y=x),                                        # over its input
        lambda: conv.causal_conv(x, w, b, state=p["state"], state_T=x[:, 1:4]),
        lambda: conv.causal_conv(x, w, b, y=torch.empty(1, 8, 16, device="cuda").expand(2, 8, 16)),
        lambda: conv.causal_conv_backward(x, w, b, x.clone(), workspace=torch.empty(16, device="cuda")),
    ]
    for f in lib:
        with pytest.raises(conv.raise_for.__globals__["TTTScanError"]):
            f()


@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("T,lengths", [(24, None), (83, [83, 40, 9])])
def test_an_infinite_input_stays_in_its_own_products(conv, T, lengths, K):
    """The last token reaches the weight gradient of its own tap alone: an infinity there leaves the others."""
    B, D = 3, 12
    p = problem(B, T, D, K, F32, seed=K, lengths=lengths)
    n = lengths or [T] * B
    p["x"][0, n[0] - 1, 5] = float("inf")
    dy = torch.randn(B, T, D, generator=torch.Generator().manual_seed(2)) ** 2 + 0.5
    c = cuda(p)
    r = conv.causal_conv_backward(c["x"], c["weight"], c["bias"], dy.cuda(), silu=False, state=c["state"],
                                  lengths=c["lengths"])
    want = torch.zeros(D, K, dtype=torch.float64)
    for b in range(B):
        ext = torch.cat((ref.up(p["state"])[b], ref.up(p["x"])[b, :n[b]]))
        for j in range(K):
            want[:, j] += (ref.up(dy)[b, :n[b]] * ext[j:j + n[b]]).sum(0)
    assert want[5, K - 1] == float("inf") and torch.isfinite(want[5, :K - 1]).all()
    assert r["dweight"][5, K - 1] == float("inf")
    got, want = r["dweight"].clone(), want.clone()
    got[5, K - 1] = want[5, K - 1] = 0
    assert ref.rrms(got, want) <= bound(F32, K) * (1 + (B * T) ** 0.5)


def plain(p, silu):
    """The 64-bit form over whole tensors, on the GPU: windows of [state, x]. y, and the padded inputs."""
    x, T, K = p["x"].double(), p["x"].shape[1], p["weight"].shape[1]
    if p["lengths"] is not None:
        x = torch.where((torch.arange(T, device="cuda") < p["lengths"][:, None])[..., None], x, torch.zeros_like(x))
    ext = torch.cat((p["state"].double(), x), 1)
    pre = p["bias"].double() + sum(p["weight"].double()[:, j] * ext[:, j:j + T] for j in range(K))
    return (ref.silu(pre) if silu else pre), ext


@pytest.mark.parametrize("D", [256, 65])
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_tokens(conv, dtype, K, D):
    """Enough tokens for runs of 32 a thread, four batches of loads each, with a ragged end."""
    B, T = 3, 12643
    assert D // (4 if D % 4 == 0 else 1) * B * T >= 148 * 16 * 32 * 32     # the rule of those runs
    lengths = [T, 12000, 6677]
    p = cuda(problem(B, T, D, K, dtype, seed=K, lengths=lengths))
    y, st = conv.causal_conv(p["x"], p["weight"], p["bias"], silu=True, state=p["state"], lengths=p["lengths"])
    want, ext = plain(p, True)
    for b, n in enumerate(lengths):
        # every stretch of tokens by itself: an error in one run is not averaged over the others
        for a in range(0, n, 997):
            e = min(n, a + 997)
            assert ref.rrms(y[b, a:e], want[b, a:e]) <= bound(dtype, K), (b, a)
        assert not y[b, n:].any()
        assert torch.equal(st[b].double(), ext[b, n:n + K - 1])
    # into heads
    if D == 256:
        heads = lambda t: t.unflatten(-1, (4, 64)).transpose(1, 2)  # noqa: E731
        y2, st2 = conv.causal_conv(heads(p["x"]), p["weight"].view(4, 64, K), p["bias"].view(4, 64), silu=True,
                                   state=heads(p["state"]), lengths=p["lengths"])
        assert torch.equal(y2, heads(y)) and torch.equal(st2, heads(st))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T,D,K", [(2, 6007, 512, 4), (3, 4003, 387, 3), (8, 4099, 768, 2), (4, 4099, 767, 4)])
def test_backward_in_longer_segments(conv, B, T, D, K, dtype):
    """Sizes whose segments are longer than 8 tokens and not a whole number of load batches."""
    blocks = conv.backward_workspace_bytes(B, 1, T, D, K) // (4 * B * D * (K + 1))
    segments = [s for s in range(8, 65) if -(-T // (8 * s)) == blocks]
    assert segments and min(segments) > 8
    lengths = [T] + [max(1, T * (B - i) // (B + 1) - 1) for i in range(B - 1)]
    p = cuda(problem(B, T, D, K, dtype, seed=T, lengths=lengths))
    g = torch.Generator().manual_seed(1)
    dy = torch.randn(B, T, D, generator=g).to(dtype).cuda()
    dst = torch.randn(B, K - 1, D, generator=g).to(dtype).cuda()
    leaves = {k: torch.nan_to_num(p[k].double(), nan=0.0).requires_grad_() for k in ("x", "weight", "bias", "state")}
    y, ext = plain(dict(leaves, lengths=p["lengths"]), True)
    there = (torch.arange(T, device="cuda") < p["lengths"][:, None])[..., None]
    loss = (y * torch.where(there, dy.double(), torch.zeros_like(y))).sum()
    loss = loss + sum((ext[b, n:n + K - 1] * dst[b].double()).sum() for b, n in enumerate(lengths))
    want = dict(zip(("dx", "dweight", "dbias", "dstate"), torch.autograd.grad(loss, list(leaves.values()))))
    for b, n in enumerate(lengths):
        dy[b, n:] = float("nan")
    r = conv.causal_conv_backward(p["x"], p["weight"], p["bias"], dy, dst, silu=True, state=p["state"],
                                  lengths=p["lengths"])
    for b, n in enumerate(lengths):
        for a in range(0, n, 499):
            e = min(n, a + 499)
            assert ref.rrms(r["dx"][b, a:e], want["dx"][b, a:e]) <= bound(dtype, K) * 2, (b, a)
        assert not r["dx"][b, n:].any()
    assert ref.rrms(r["dstate"], want["dstate"]) <= bound(dtype, K) * 2
    for k in ("dweight", "dbias"):
        assert ref.rrms(r[k], want[k]) <= bound(F32, K) * (1 + (B * T) ** 0.5), k


@pytest.mark.parametrize("D", [8, 5])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_the_slope_of_silu_over_its_whole_range(conv, dtype, D):
    """Values before the activation from 1e-3 to 1e30, of either sign, element by element: the slope is
    s (1 + x (1 - s)), 1 for a large x. With s from an ex2 whose argument is rounded, s is off by up to
    2^-21 + |x| 2^-23 of itself for x < 0; its two terms and their sum round three times more."""
    T = 400
    mag = torch.logspace(-3, 30, T // 2)
    x = torch.cat((mag, -mag))[None, :, None].expand(1, T, D).to(dtype).contiguous()
    x[:, ::7] = x[:, ::7].clamp(-12, 12)
    weight = torch.zeros(D, 2)
    weight[:, 1] = 1                                     # pre = x
    g = torch.Generator().manual_seed(6)
    dy = torch.randn(1, T, D, generator=g)
    r = conv.causal_conv_backward(x.cuda(), weight.cuda(), None, dy.cuda(), silu=True)
    v, gy = ref.up(x), ref.up(dy)
    s = torch.sigmoid(v)
    want = gy * s * (1 + v * (1 - s))
    room = 2.0 ** -21 + v.clamp(min=-200, max=0).abs() * 2.0 ** -23 + 3 * 2.0 ** -24
    # For x > 0, s = 1 / (1 + e) is off by the rounding of 1 + e (2^-24) and the reciprocal (2^-23), and x (1 - s) by
    # x times that; from x = 17 on e < 2^-24, so that s is 1 and the term, at most 17 e^-17, is 0.
    room = room + v.clamp(min=0, max=17) * (2.0 ** -23 + 2.0 ** -24)
    if dtype == BF16:
        room = room + ref.BF16
    size = gy.abs() * s * (1 + v.abs() * (1 - s))        # of the terms: they cancel at x = -1.28
    # (below the smallest normal numbers s is 0)
    assert ((ref.up(r["dx"]) - want).abs() <= room * size + 1e-35).all()
