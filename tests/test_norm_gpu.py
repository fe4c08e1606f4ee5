"""The root-mean-square norm against a plain form in 64 bits: with and without a residual, in 8 bits,
and its gradients."""

import pytest
import torch

from tests import seq_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16, FP8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
TINY = torch.finfo(F32).tiny


@pytest.fixture(scope="module")
def norm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from test_sequence_layers_02_b200 import build, norm as module
    build.build()
    return module


def bound(dtype, D):
    """Sums of D squares in strands of at most 64 (2^-24 each step), rsqrt (2^-22) and a few roundings."""
    return 80 * 2.0 ** -24 + (ref.BF16 if dtype == BF16 else 0.0)


def inputs(M, D, dtype, res, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, D, generator=g).to(dtype)
    r = None if res is None else (torch.randn(M, D, generator=g) * 3).to(res)
    return x, torch.randn(D, generator=g) * 0.3 + 1, r


DIMS = [1, 7, 64, 128, 200, 256, 264, 513, 1024, 1536, 2048, 2056, 4096, 8200, 16384]


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("dtype,res,out", [(F32, F32, F32), (BF16, BF16, BF16), (BF16, F32, BF16),
                                           (BF16, None, F32), (F32, BF16, BF16)])
def test_norm(norm, D, dtype, res, out):
    x, w, r = inputs(9, D, dtype, res, seed=D)
    y, s = norm.rmsnorm(x.cuda(), w.cuda(), None if r is None else r.cuda(), out_dtype=out, eps=1e-5)
    ry, rs = ref.norm(ref.up(x), ref.up(w), ref.up(r), 1e-5)
    assert y.dtype == out and ref.rrms(y, ry) <= bound(out, D)
    if r is None:
        assert s.shape == x.shape and torch.equal(s.cpu(), x)
    else:
        assert s.dtype == res and torch.equal(s.cpu(), (x.float() + r.float()).to(res))


@pytest.mark.parametrize("M", [0, 1, 2, 5, 1000])
def test_rows(norm, M):
    for D in (96, 100, 3000):
        x, w, r = inputs(M, D, BF16, BF16, seed=M)
        y, s = norm.rmsnorm(x.cuda(), w.cuda(), r.cuda())
        ry, _ = ref.norm(ref.up(x), ref.up(w), ref.up(r), 1e-6)
        assert ref.rrms(y, ry) <= bound(BF16, D)


def check_codes(y, scale, want, group):
    """Codes are e4m3 roundings of want / scale: half a step, 2^-4 of the value, or 2^-10 (half of the
    smallest subnormal); 1 + 2^-16 allows for the fp32 steps in front of it."""
    M, D = want.shape
    wide = scale.repeat_interleave(group or D, 1)[:, :D].double().cpu()
    v, w = ref.up(y.float()), want / wide
    assert ((v - w).abs() <= (w.abs() * 2.0 ** -4).clamp(min=2.0 ** -10) * (1 + 2.0 ** -16) + 1e-5).all()


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("dtype,res", [(BF16, BF16), (F32, F32), (BF16, None), (F32, BF16)])
def test_norm_8_bits(norm, D, group, dtype, res):
    x, w, r = inputs(7, D, dtype, res, seed=D)
    y, scale, s = norm.rmsnorm_fp8(x.cuda(), w.cuda(), None if r is None else r.cuda(), group=group)
    want, rs = ref.norm(ref.up(x), ref.up(w), ref.up(r), 1e-6)
    n = -(-D // 128) if group else 1
    assert y.dtype == FP8 and y.shape == x.shape and scale.shape == (7, n)
    parts = [want[:, i * 128:(i + 1) * 128] if group else want for i in range(n)]
    rscale = torch.stack([p.abs().amax(1) for p in parts], 1) / 448
    assert ref.rrms(scale, rscale) <= bound(F32, D)
    check_codes(y, scale, want, group)
    assert y.float().abs().max() <= 448
    # the values are those of the unquantised form
    y32, _ = norm.rmsnorm(x.cuda(), w.cuda(), None if r is None else r.cuda(), out_dtype=F32)
    check_codes(y, scale, ref.up(y32), group)


def test_rows_of_zeros_and_of_nan(norm):
    x = torch.randn(4, 300, device="cuda")
    x[1] = 0
    x[2, 17] = float("nan")
    x[3, 5] = float("inf")
    w = torch.ones(300, device="cuda")
    y, scale, _ = norm.rmsnorm_fp8(x, w)
    assert not y[1].float().any() and scale[1] == TINY
    assert y[2].float().isnan().all() and torch.isfinite(scale[:2]).all()
    assert y[3].float()[5].isnan()                     # inf * 0, as in the formula
    z, _ = norm.rmsnorm(x, w)
    assert not z[1].any() and z[2].isnan().all() and z[3, 5].isnan() and torch.isfinite(z[:2]).all()
    q, sc, _ = norm.rmsnorm_fp8(x[:, :256].contiguous(), w[:256], group=128)
    assert (sc[1] == TINY).all() and not q[1].float().any()


def test_in_place_strides_and_shapes(norm):
    x, w, r = inputs(6, 264, BF16, BF16, seed=3)
    xc, wc, rc = x.cuda(), w.cuda(), r.cuda()
    y, s = norm.rmsnorm(xc, wc, rc)
    # the residual stream in place, and over x
    r2 = rc.clone()
    y2, s2 = norm.rmsnorm(xc, wc, r2, s=r2)
    assert s2 is r2 and torch.equal(r2, s) and torch.equal(y2, y)
    x2 = xc.clone()
    y2, s2 = norm.rmsnorm(x2, wc, rc, s=x2)
    assert torch.equal(x2, s) and torch.equal(y2, y)
    # strided rows, at an odd offset (single columns) and at an even one
    for off, pad in ((1, 3), (8, 16)):
        wide = torch.zeros(6, 264 + pad, dtype=BF16, device="cuda")
        xs = wide[:, off:off + 264] if pad > off else wide[:, :264]
        xs.copy_(xc)
        out = torch.zeros(6, 2 * 264 + 1, dtype=BF16, device="cuda")
        y2, s2 = norm.rmsnorm(xs, wc, rc, y=out[:, 264:528])
        # the two forms add the squares in different orders
        assert ref.rrms(y2, ref.norm(ref.up(x), ref.up(w), ref.up(r), 1e-6)[0]) <= bound(BF16, 264)
        assert torch.equal(s2, s) and not out[:, :264].any() and not out[:, 528:].any()
    # more dimensions
    y3, s3 = norm.rmsnorm(xc.view(2, 3, 264), wc, rc.view(2, 3, 264))
    assert y3.shape == (2, 3, 264) and torch.equal(y3.view(6, 264), y)
    q, sc, _ = norm.rmsnorm_fp8(xc.view(2, 3, 264), wc, rc.view(2, 3, 264), group=128)
    assert q.shape == (2, 3, 264) and sc.shape == (2, 3, 3)
    v, _ = norm.rmsnorm(xc[0], wc)
    assert v.shape == (264,)


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("M", [1, 13])
def test_backward(norm, M, D, dtype, out):
    x, w, _ = inputs(M, D, dtype, None, seed=D + M)
    g = torch.Generator().manual_seed(1)
    dy, ds = torch.randn(M, D, generator=g).to(out), torch.randn(M, D, generator=g).to(dtype)
    for e in (ds, None):
        leaves = [ref.up(x).requires_grad_(), ref.up(w).requires_grad_()]
        y, s = ref.norm(*leaves, None, 1e-3)
        want = ref.gradients((y, s), (ref.up(dy), ref.up(e)), leaves)
        r = norm.rmsnorm_backward(dy.cuda(), x.cuda(), w.cuda(), None if e is None else e.cuda(), eps=1e-3)
        # with D = 1 the two terms of dx cancel to eps of their size
        room = bound(F32, D) * ref.up(dy).abs().max().item() * 4 * D ** 0.5 * M ** 0.5 if D < 8 else 0.0
        diff = (ref.up(r["dx"]) - want[0]).norm()
        assert diff <= bound(dtype, D) * 4 * want[0].norm() + room
        assert ref.rrms(r["dweight"], want[1]) <= bound(F32, D) * (1 + M ** 0.5)
        again = norm.rmsnorm_backward(dy.cuda(), x.cuda(), w.cuda(), None if e is None else e.cuda(), eps=1e-3)
        assert torch.equal(r["dx"], again["dx"]) and torch.equal(r["dweight"], again["dweight"])


@pytest.mark.parametrize("M", [0, 1183, 1184, 1185, 3000])
def test_backward_rows(norm, M):
    x, w, _ = inputs(M, 72, BF16, None, seed=M)
    dy = torch.randn(M, 72)
    leaves = [ref.up(x).requires_grad_(), ref.up(w).requires_grad_()]
    y, _ = ref.norm(*leaves, None, 1e-6)
    want = ref.gradients((y,), (ref.up(dy),), leaves)
    r = norm.rmsnorm_backward(dy.cuda(), x.cuda(), w.cuda())
    assert ref.rrms(r["dx"], want[0]) <= bound(BF16, 72) * 4
    assert ref.rrms(r["dweight"], want[1]) <= bound(F32, 72) * (1 + M ** 0.5)


def test_backward_in_place_and_differences(norm):
    x, w, _ = inputs(5, 48, F32, None, seed=2)
    g = torch.Generator().manual_seed(4)
    dy, ds = torch.randn(5, 48, generator=g), torch.randn(5, 48, generator=g)
    r = norm.rmsnorm_backward(dy.cuda(), x.cuda(), w.cuda(), ds.cuda())
    e = ds.cuda()
    ws = torch.empty(norm.backward_workspace_bytes(5, 48), dtype=torch.uint8, device="cuda")
    r2 = norm.rmsnorm_backward(dy.cuda(), x.cuda(), w.cuda(), e, dx=e, workspace=ws)
    assert r2["dx"] is e and torch.equal(e, r["dx"]) and torch.equal(r2["dweight"], r["dweight"])
    at = [ref.up(x), ref.up(w)]
    for i, key in enumerate(("dx", "dweight")):
        v = torch.randn(at[i].shape, generator=g, dtype=torch.float64)

        def loss(h):
            a = list(at)
            a[i] = a[i] + h * v
            y, s = ref.norm(*a, None, 1e-6)
            return (y * dy.double()).sum() + (s * ds.double()).sum()
        h = 1e-5   # h^2 of truncation, 1e-16 / h of rounding
        diff = float((loss(h) - loss(-h)) / (2 * h))
        got = float((ref.up(r[key]) * v).sum())
        assert abs(got - diff) <= 1e-5 * float(ref.up(r[key]).norm() * v.norm()), key


def test_streams_and_graphs(norm):
    x, w, r = (t.cuda() for t in inputs(300, 1536, BF16, BF16, seed=5))
    dy = torch.randn(300, 1536, device="cuda").to(BF16)

    def both(**kw):
        y, s = norm.rmsnorm(x, w, r, **kw)
        q, sc, _ = norm.rmsnorm_fp8(x, w, r, group=128, **kw)
        return dict(norm.rmsnorm_backward(dy, s, w, dy, **kw), y=y, s=s, q=q.view(torch.uint8), sc=sc)
    a = both()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    b = both(stream=side)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c = both()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a[k], b[k]) and torch.equal(a[k], c[k]) for k in a)


def test_refusals(norm):
    x, w, r = (t.cuda() for t in inputs(4, 64, F32, F32))
    bad = [
        lambda: norm.rmsnorm(x.cpu(), w, r), lambda: norm.rmsnorm(x.half(), w, r),
        lambda: norm.rmsnorm(x, w[:32], r), lambda: norm.rmsnorm(x, w.to(BF16), r),
        lambda: norm.rmsnorm(x, w, r[:2]), lambda: norm.rmsnorm(x, w, s=x.clone()),
        lambda: norm.rmsnorm(x, w, r, out_dtype=torch.float16), lambda: norm.rmsnorm_fp8(x, w, r, group=64),
        lambda: norm.rmsnorm(x.t().contiguous().t(), w, r),
        lambda: norm.rmsnorm_fp8(x, w, r, y=torch.empty_like(x)),
        lambda: norm.rmsnorm_backward(x, x, w, ds=x.to(BF16)),
        lambda: norm.rmsnorm_backward(x[:2], x, w),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    from test_sequence_layers_02_b200.ttt_scan import TTTScanError
    big = torch.zeros(1, 16392, device="cuda")
    lib = [
        lambda: norm.rmsnorm(big, big[0].contiguous()), lambda: norm.rmsnorm(x, w, r, eps=-1.0),
        lambda: norm.rmsnorm(x, w, r, eps=float("nan")), lambda: norm.rmsnorm(x, w, r, y=x),
        lambda: norm.rmsnorm(x, w, r, y=r), lambda: norm.rmsnorm(x, w, r, y=torch.empty(1, 64, device="cuda").expand(4, 64)),
        lambda: norm.rmsnorm_backward(x, x.clone(), w, dx=x),
        lambda: norm.rmsnorm_backward(x, x.clone(), w, workspace=torch.empty(1, device="cuda")),
    ]
    for f in lib:
        with pytest.raises(TTTScanError):
            f()


@pytest.mark.parametrize("D,group", [(2048, 0), (2048, 128), (1000, 128), (1001, 0), (1001, 128)])
@pytest.mark.parametrize("size", [1.0, 1e-36, 1e30])
def test_codes_are_those_of_the_quotient(norm, D, group, size):
    """A code is e4m3(y / scale), the quotient rounded once to fp32, for every value: also where it lies next
    to the middle between two codes (two values in a million), and where the scale is the smallest
    normal number."""
    x, w, r = inputs(2048, D, BF16, BF16, seed=D)
    a = (x.cuda(), (w * size).cuda(), r.cuda())
    q, scale, _ = norm.rmsnorm_fp8(*a, group=group)
    y, _ = norm.rmsnorm(*a, out_dtype=F32)     # the values before their codes, bit for bit
    wide = scale.cpu().repeat_interleave(group or D, 1)[:, :D]
    want = (y.cpu() / wide).to(FP8).view(torch.uint8)
    assert torch.equal(q.cpu().view(torch.uint8), want)


# Rows off 8 columns that take from 3 to 32 warps, a column a lane; beyond 8192 a CTA of 1024 threads.
ODD = [1023, 1535, 4099, 8191, 8193, 12289, 16383]


@pytest.mark.parametrize("D", ODD)
@pytest.mark.parametrize("dtype,res,out", [(F32, F32, F32), (BF16, BF16, BF16), (BF16, F32, BF16), (F32, BF16, BF16)])
def test_long_rows_off_8_columns(norm, D, dtype, res, out):
    x, w, r = inputs(9, D, dtype, res, seed=D)
    y, s = norm.rmsnorm(x.cuda(), w.cuda(), r.cuda(), out_dtype=out, eps=1e-5)
    ry, _ = ref.norm(ref.up(x), ref.up(w), ref.up(r), 1e-5)
    assert y.dtype == out and ref.rrms(y, ry) <= bound(out, D)
    assert torch.equal(s.cpu(), (x.float() + r.float()).to(res))
    for group in (0, 128):
        q, scale, _ = norm.rmsnorm_fp8(x.cuda(), w.cuda(), r.cuda(), group=group, eps=1e-5)
        parts = [ry[:, i:i + (group or D)] for i in range(0, D, group or D)]
        assert ref.rrms(scale, torch.stack([p.abs().amax(1) for p in parts], 1) / 448) <= bound(F32, D)
        check_codes(q, scale, ry, group)


@pytest.mark.parametrize("D", ODD)
@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
def test_backward_of_long_rows_off_8_columns(norm, D, dtype, out):
    M = 11
    x, w, _ = inputs(M, D, dtype, None, seed=D + M)
    g = torch.Generator().manual_seed(1)
    dy, ds = torch.randn(M, D, generator=g).to(out), torch.randn(M, D, generator=g).to(dtype)
    leaves = [ref.up(x).requires_grad_(), ref.up(w).requires_grad_()]
    y, s = ref.norm(*leaves, None, 1e-3)
    want = ref.gradients((y, s), (ref.up(dy), ref.up(ds)), leaves)
    r = norm.rmsnorm_backward(dy.cuda(), x.cuda(), w.cuda(), ds.cuda(), eps=1e-3)
    assert ref.rrms(r["dx"], want[0]) <= bound(dtype, D) * 4
    assert ref.rrms(r["dweight"], want[1]) <= bound(F32, D) * (1 + M ** 0.5)


@pytest.mark.parametrize("D", [256, 300, 257, 4096, 1501])
@pytest.mark.parametrize("group", [0, 128])
def test_the_scale_of_nan_is_nan(norm, D, group):
    """max |y| / 448 over values with a NaN among them is NaN, for a row as for 128 columns."""
    x = torch.randn(4, D, device="cuda")
    x[2, D - 1] = float("nan")                 # through the sum of squares, all of row 2
    w = torch.ones(D, device="cuda")
    y, scale, _ = norm.rmsnorm_fp8(x, w, group=group)
    assert scale[2].isnan().all() and y[2].float().isnan().all()
    keep = [0, 1, 3]
    assert scale[keep].isfinite().all() and y[keep].float().isfinite().all()
    w[130] = float("nan")                      # one column of every row
    y, scale, _ = norm.rmsnorm_fp8(x[keep], w, group=group)
    assert y[:, 130].float().isnan().all()
    assert scale[:, 1 if group else 0].isnan().all()
    if group:
        assert scale[:, 0].isfinite().all() and y[:, :128].float().isfinite().all()
