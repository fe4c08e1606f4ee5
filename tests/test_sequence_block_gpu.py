"""The operators in a run, as a model uses them: norm, projection, convolution, scan, and back; a
prompt in one pass and continued token by token; and the convolution in front of the TTT scan."""

import numpy as np
import pytest
import torch

from tests import seq_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from test_sequence_layers_02_b200 import build, conv, norm, ssm, ttt_scan
    build.build()
    return conv, norm, ssm, ttt_scan


class Block:
    """One layer's parameters (64-bit, on the CPU) and its two forms. ``R`` inputs a channel's step size
    is made from."""

    def __init__(self, M, D, N, K, R, seed):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s, scale=1.0: (torch.randn(*s, generator=g, dtype=torch.float64) * scale).float().double()  # noqa: E731
        self.N, self.R = N, R
        self.p = dict(gain=r(M, scale=0.1) + 1, w_in=r(M, 2 * D, scale=M ** -0.5), cw=r(D, K, scale=0.5), cb=r(D, scale=0.1),
                      w_x=r(D, R + 2 * N, scale=D ** -0.5), w_dt=r(R, D, scale=R ** -0.5),
                      A=-torch.arange(1, N + 1, dtype=torch.float64).repeat(D, 1), skip=r(D, scale=0.1) + 1,
                      dt_bias=r(D, scale=0.5) - 3, w_out=r(D, M, scale=D ** -0.5))

    def plain(self, x, residual, lengths):
        """64-bit: the layer's output, the residual stream, the states after it."""
        p, D = self.p, self.p["cw"].shape[0]
        n, s = ref.norm(x, p["gain"], residual, 1e-6)
        uz = n @ p["w_in"]
        u, cst = ref.conv(uz[..., :D], p["cw"], p["cb"], None, lengths, True)
        proj = u @ p["w_x"]
        delta = proj[..., :self.R] @ p["w_dt"]
        Bm, Cm = proj[..., self.R:].unsqueeze(-2).chunk(2, -1)
        y, h = ref.scan(u, delta, p["A"], Bm, Cm, p["skip"], uz[..., D:], p["dt_bias"], None, lengths)
        return y @ p["w_out"], s, cst, h

    def run(self, ops, x, residual, lengths=None, states=None):
        """fp32 on the GPU; ``states`` (convolution's, scan's) are moved on in place when given."""
        conv, norm, ssm, _ = ops
        p = {k: v.float().cuda() for k, v in self.p.items()}
        D = p["cw"].shape[0]
        step = x.dim() == 2
        n, s = norm.rmsnorm(x, p["gain"], residual)
        uz = n @ p["w_in"]
        xin, z = uz[..., :D], uz[..., D:]
        if step:
            u = conv.causal_conv_step(xin, p["cw"], p["cb"], states[0], silu=True)
        else:
            cs = None if states is None else states[0]
            u, cst = conv.causal_conv(xin, p["cw"], p["cb"], silu=True, state=cs, state_T=cs, lengths=lengths)
        proj = u @ p["w_x"]
        delta = proj[..., :self.R] @ p["w_dt"]
        Bm, Cm = proj[..., self.R:self.R + self.N], proj[..., self.R + self.N:]
        args = (u, delta, p["A"], Bm, Cm, p["skip"], z, p["dt_bias"])
        if step:
            return ssm.selective_step(*args, states[1]) @ p["w_out"], s
        h0 = None if states is None else states[1]
        y, h = ssm.selective_scan(*args, h0=h0, h_T=h0, lengths=lengths)
        return y @ p["w_out"], s, cst, h


# A layer's two projections in fp32 add sqrt(D) 2^-24 each to what its operators leave (ref.tol).
def close(got, want, steps):
    assert ref.rrms(got, want) <= 4 * ref.tol(F32, steps)


@pytest.fixture(autouse=True)
def exact_products():
    before = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    yield
    torch.backends.cuda.matmul.allow_tf32 = before


def test_two_layers_prompt_then_tokens(ops):
    """A ragged batch of prompts through two layers, then tokens one by one, against the whole sequences."""
    B, T, M, D, N, K, more = 3, 41, 48, 64, 16, 4, 5
    layers = [Block(M, D, N, K, 8, seed) for seed in (1, 2)]
    g = torch.Generator().manual_seed(3)
    x = torch.randn(B, T + more, M, generator=g, dtype=torch.float64).float().double()
    n = torch.tensor([T, 1, 17], dtype=torch.int32)
    # what a row sees: its prompt, then its tokens
    rows = [torch.cat((x[b, :n[b]], x[b, T:])) for b in range(B)]
    want = []
    for row in rows:
        out, s = row[None], torch.zeros_like(row)[None]
        for layer in layers:
            out, s, _, _ = layer.plain(out, s, None)
        want.append((out[0], s[0]))
    dev = x.float().cuda()
    out, s, states = dev[:, :T].contiguous(), torch.zeros(B, T, M, device="cuda"), []
    for layer in layers:
        st = [torch.zeros(B, K - 1, D, device="cuda"), torch.zeros(B, D, N, device="cuda")]
        out, s, cst, h = layer.run(ops, out, s, n.cuda(), st)
        assert cst is st[0] and h is st[1]
        states.append(st)
    for b in range(B):
        close(out[b, :n[b]], want[b][0][:n[b]], T)
        close(s[b, :n[b]], want[b][1][:n[b]], T)
    for t in range(more):
        out, s = dev[:, T + t].contiguous(), torch.zeros(B, M, device="cuda")
        for layer, st in zip(layers, states):
            out, s = layer.run(ops, out, s, None, st)
        for b in range(B):
            close(out[b], want[b][0][n[b] + t], T + more)
            close(s[b], want[b][1][n[b] + t], T + more)


def test_training_step_of_a_layer(ops):
    """The gradients of a layer's parameters and inputs, chained through the backward calls."""
    conv, norm, ssm, _ = ops
    B, T, M, D, N, K, R = 2, 37, 40, 56, 8, 3, 4
    layer = Block(M, D, N, K, R, 5)
    g = torch.Generator().manual_seed(6)
    x, res, dout, ds_out = (torch.randn(B, T, M, generator=g) for _ in range(4))
    leaves = {k: v.clone().requires_grad_() for k, v in layer.p.items()}
    leaves |= {"x": x.double().requires_grad_(), "res": res.double().requires_grad_()}
    layer.p, saved = leaves, layer.p
    out, s, _, _ = layer.plain(leaves["x"], leaves["res"], None)
    layer.p = saved
    want = dict(zip(leaves, torch.autograd.grad((out * dout.double()).sum() + (s * ds_out.double()).sum(),
                                                list(leaves.values()))))
    p = {k: v.float().cuda() for k, v in saved.items()}
    flat = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
    n, s = norm.rmsnorm(x.cuda(), p["gain"], res.cuda())
    uz = n @ p["w_in"]
    xin, z = uz[..., :D], uz[..., D:]
    u, _ = conv.causal_conv(xin, p["cw"], p["cb"], silu=True)
    proj = u @ p["w_x"]
    delta = proj[..., :R] @ p["w_dt"]
    args = (u, delta, p["A"], proj[..., R:R + N], proj[..., R + N:], p["skip"], z, p["dt_bias"])
    y, _, chunks = ssm.selective_scan(*args, want_chunks=True)
    got = {"w_out": flat(y).T @ flat(dout.cuda())}
    r = ssm.selective_scan_backward(*args, chunks, dout.cuda() @ p["w_out"].T)
    got |= {"A": r["dA"], "skip": r["dD"], "dt_bias": r["ddelta_bias"], "w_dt": flat(proj[..., :R]).T @ flat(r["ddelta"])}
    dproj = torch.cat((r["ddelta"] @ p["w_dt"].T, r["dBm"], r["dCm"]), -1)
    got["w_x"] = flat(u).T @ flat(dproj)
    c = conv.causal_conv_backward(xin, p["cw"], p["cb"], r["du"] + dproj @ p["w_x"].T, silu=True)
    got |= {"cw": c["dweight"], "cb": c["dbias"]}
    duz = torch.cat((c["dx"], r["dz"]), -1)
    got["w_in"] = flat(n).T @ flat(duz)
    e = norm.rmsnorm_backward(duz @ p["w_in"].T, s, p["gain"], ds_out.cuda())
    got |= {"gain": e["dweight"], "x": e["dx"], "res": e["dx"]}
    for k, v in got.items():
        # sums over B T tokens whose terms cancel
        assert ref.rrms(v, want[k]) <= 4 * ref.tol(F32, T, B * T), k


def test_convolution_in_front_of_the_ttt_scan(ops):
    """Queries and keys out of one token-major projection, through the convolution into heads, into the
    TTT scan, against the oracle on the plain convolution's values."""
    import oracle
    from tests.helpers import assert_fp32_close
    conv, _, _, ttt_scan = ops
    B, T, H, d, K = 2, 45, 3, 64, 4
    g = torch.Generator().manual_seed(8)
    r = lambda *s, scale=1.0: torch.randn(*s, generator=g) * scale  # noqa: E731
    proj = r(B, T, 3 * H * d)
    wq, wk = r(H * d, K, scale=0.5), r(H * d, K, scale=0.5)
    eta, gate, W0 = r(B, H, T), r(B, H, T), r(B, H, d, d, scale=0.02)
    gamma, beta = 1 + r(H, d, scale=0.1), r(H, d, scale=0.1)
    heads = lambda t: t.unflatten(-1, (H, d)).transpose(1, 2)  # noqa: E731
    p = proj.cuda()
    q, _ = conv.causal_conv(heads(p[..., :H * d]), wq.cuda().view(H, d, K), silu=True)
    k, _ = conv.causal_conv(heads(p[..., H * d:2 * H * d]), wk.cuda().view(H, d, K), silu=True)
    k = k / (k.norm(dim=-1, keepdim=True) + 1e-6)
    v = heads(p[..., 2 * H * d:]).contiguous()
    o, W_T = ttt_scan.scan(q, k, v, eta.cuda(), gate.cuda(), W0.cuda(), gamma.cuda(), beta.cuda(), lnjac=True)
    torch.cuda.synchronize()
    assert ttt_scan.check_device_status() == ttt_scan.TTT_OK
    rq = heads(ref.conv(proj[..., :H * d].double(), wq.double(), None, None, None, True)[0])
    rk = heads(ref.conv(proj[..., H * d:2 * H * d].double(), wk.double(), None, None, None, True)[0])
    rk = rk / (rk.norm(dim=-1, keepdim=True) + 1e-6)
    f = lambda t: np.ascontiguousarray(t.double().numpy())  # noqa: E731
    ro, rW = oracle.forward(f(rq), f(rk), f(heads(proj[..., 2 * H * d:])), f(eta), f(gate), f(W0), f(gamma), f(beta),
                            eps=1e-6, mode=2, b=16)
    assert_fp32_close(o.cpu().numpy(), ro, "o")
    assert_fp32_close(W_T.cpu().numpy(), rW, "W_T")


def test_eight_bit_norm_feeds_a_product(ops):
    """The codes and scales stand for the norm's values in the product behind it."""
    _, norm, _, _ = ops
    g = torch.Generator().manual_seed(9)
    x, res, w = torch.randn(33, 512, generator=g), torch.randn(33, 512, generator=g), torch.randn(512, 64, generator=g)
    gain = 1 + 0.1 * torch.randn(512, generator=g)
    want = ref.norm(x.double(), gain.double(), res.double(), 1e-6)[0] @ w.double()
    for group in (0, 128):
        q, scale, s = norm.rmsnorm_fp8(x.cuda(), gain.cuda(), res.cuda(), group=group)
        wide = scale.repeat_interleave(group or 512, 1)
        got = (q.float() * wide) @ w.cuda()
        # a code is off by at most 2^-4 of its value
        assert ref.rrms(got, want) <= 2.0 ** -4
        assert torch.equal(s.cpu(), x + res)


def test_more_rows_than_a_grid_is_high(ops):
    """Over 65535 batch rows: the kernels walk them."""
    conv, _, ssm, _ = ops
    B, D, N, K = 65535 + 70, 8, 8, 2
    g = torch.Generator(device="cuda").manual_seed(10)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, w, st = r(B, 2, D), r(D, K), r(B, K - 1, D)
    y, st2 = conv.causal_conv(x, w, state=st)
    taps = torch.cat((st, x), 1).double()
    want = sum(w[:, j].double() * taps[:, j:j + 2] for j in range(K))
    assert ref.rrms(y, want) <= 1e-6 and torch.equal(st2, x[:, 1:])
    c = conv.causal_conv_backward(x, w, None, y, state=st)
    assert ref.rrms(c["dweight"], torch.stack([(taps[:, j:j + 2] * y.double()).sum((0, 1)) for j in range(K)], 1)) <= 1e-5
    s = st.clone()
    assert torch.equal(conv.causal_conv_step(x[:, 0], w, None, s), y[:, 0])
    A, dt, h0 = -torch.rand(D, N, device="cuda", generator=g), torch.rand(B, 2, D, device="cuda", generator=g), r(B, D, N)
    Bm, Cm = r(B, 2, N), r(B, 2, N)
    y, h, ck = ssm.selective_scan(x, dt, A, Bm, Cm, softplus=False, h0=h0, want_chunks=True)
    hd, ys = h0.double(), []
    for t in range(2):
        hd = torch.exp(dt[:, t, :, None].double() * A.double()) * hd + (dt * x)[:, t, :, None].double() * Bm[:, t, None].double()
        ys.append((hd * Cm[:, t, None].double()).sum(-1))
    assert ref.rrms(y, torch.stack(ys, 1)) <= 1e-5 and ref.rrms(h, hd) <= 1e-5
    b = ssm.selective_scan_backward(x, dt, A, Bm, Cm, None, None, None, ck, y, softplus=False)
    for lo, hi in ((0, 40), (65500, B)):
        q = lambda t: t[lo:hi].contiguous()  # noqa: E731
        p = ssm.selective_scan_backward(q(x), q(dt), A, q(Bm), q(Cm), None, None, None, q(ck), q(y), softplus=False)
        assert all(torch.equal(p[k], b[k][lo:hi]) for k in ("du", "ddelta", "dBm", "dCm", "dh0"))
    hs = h0.clone()
    for t in range(2):
        o = ssm.selective_step(x[:, t], dt[:, t], A, Bm[:, t], Cm[:, t], None, None, None, hs, softplus=False)
        assert ref.rrms(o, ys[t]) <= 1e-5
