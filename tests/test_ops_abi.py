"""The C entry points of the operators around the scan reject bad arguments before any CUDA call
(these run without a GPU: the addresses are made up and never dereferenced)."""

import ctypes

import pytest

from test_sequence_layers_02_b200 import build as pkg_build

INVALID, UNSUPPORTED = -1, -2
IN_BF16, OUT_BF16, SILU, SOFTPLUS, SUM_BF16, E4M3 = 1 << 3, 1 << 4, 1 << 16, 1 << 17, 1 << 18, 1 << 19


def addr(i, off=0):
    """Made-up, 16-byte aligned addresses, 4 GiB apart."""
    return (1 << 40) + i * (1 << 32) + off


def strides(*v):
    return (ctypes.c_longlong * len(v))(*v)


@pytest.fixture(scope="module")
def libs():
    pkg_build.build()
    from test_sequence_layers_02_b200 import conv, norm, ssm  # noqa: F401
    return {"conv": conv._lib, "ssm": ssm._lib, "norm": norm._lib}


CONV = dict(x=addr(0), weight=addr(1), bias=addr(2), state=addr(3), lengths=addr(4), B=2, H=3, T=40, d=8,
            K=4, mode=0, strides=None, y=addr(5), state_T=addr(6))
BAD_CONV = [dict(x=None), dict(weight=None), dict(y=None), dict(x=addr(0, 2)), dict(weight=addr(1, 4)),
            dict(y=addr(5, 1)), dict(lengths=addr(4, 2)), dict(bias=addr(2, 3)), dict(state=addr(3, 2)),
            dict(B=-1), dict(H=-1), dict(T=-1), dict(d=0), dict(K=0), dict(mode=1), dict(mode=1 << 21),
            dict(y=addr(0)), dict(y=addr(0, 400)), dict(y=addr(3)), dict(y=addr(1)), dict(state_T=addr(0)),
            dict(state_T=addr(5, 64)), dict(state_T=addr(3, 4)),
            dict(strides=strides(-960, 320, 8, 960, 320, 8, 72, 24, 8, 72, 24, 8)),
            dict(strides=strides(960, 320, 8, 960, 320, 0, 72, 24, 8, 72, 24, 8)),     # y on top of itself
            dict(strides=strides(960, 320, 8, 960, 4, 24, 72, 24, 8, 72, 24, 8)),
            dict(strides=strides(960, 320, 8, 960, 320, 8, 72, 24, 8, 72, 24, 4)),
            dict(state_T=addr(3), strides=strides(960, 320, 8, 960, 320, 8, 72, 24, 8, 72, 8, 24))]


@pytest.mark.parametrize("over,want", [(o, INVALID) for o in BAD_CONV] +
                         [(dict(K=1), UNSUPPORTED), (dict(K=5), UNSUPPORTED),
                          (dict(H=1 << 20, d=1 << 11, T=0), UNSUPPORTED),
                          (dict(T=(1 << 30) + 1), UNSUPPORTED)])
def test_conv_forward(libs, over, want):
    assert libs["conv"].ttt_conv_forward(*dict(CONV, **over).values(), None) == want


CONV_BWD = dict(x=addr(0), weight=addr(1), bias=addr(2), state=addr(3), lengths=None, B=2, H=3, T=40, d=8,
                K=4, mode=0, strides=None, dy=addr(4), dstate_T=addr(5), dx=addr(6), dweight=addr(7),
                dbias=addr(8), dstate=addr(9), ws=addr(10), ws_bytes=1 << 20)


@pytest.mark.parametrize("over,want", [(o, INVALID) for o in (
    dict(x=None), dict(dy=None), dict(dx=None), dict(dweight=None), dict(dbias=None), dict(ws=None),
    dict(ws_bytes=100), dict(ws=addr(10, 8)), dict(dx=addr(0)), dict(dx=addr(4)), dict(dstate=addr(3)),
    dict(dweight=addr(1)), dict(dbias=addr(7, 64)), dict(ws=addr(6)), dict(dx=addr(6, 1)), dict(T=-1),
    dict(strides=strides(960, 320, 8, 960, 320, -8, 72, 24, 8)))] +
    [(dict(K=7), UNSUPPORTED), (dict(T=1 << 30, B=1, H=1, d=1, ws_bytes=1 << 50, x=addr(0), dx=addr(60),
                                     ws=addr(100)), UNSUPPORTED)])
def test_conv_backward(libs, over, want):
    a = dict(CONV_BWD, **over)
    if want == UNSUPPORTED and a["T"] == 1 << 30:
        a |= {k: addr(20 + 8 * i) for i, k in enumerate(("x", "dy"))}
    assert libs["conv"].ttt_conv_backward(*a.values(), None) == want


@pytest.mark.parametrize("over,want", [(o, INVALID) for o in (
    dict(x=None), dict(state=None), dict(y=None), dict(y=addr(0)), dict(state=addr(0)), dict(y=addr(3, 16)),
    dict(B=-1), dict(mode=2), dict(strides=strides(24, 8, 24, 4, 72, 24, 8)))] + [(dict(K=9), UNSUPPORTED)])
def test_conv_step(libs, over, want):
    a = dict(x=addr(0), weight=addr(1), bias=addr(2), state=addr(3), active=addr(4, 1), B=2, H=3, d=8, K=4,
             mode=0, strides=None, y=addr(5))
    assert libs["conv"].ttt_conv_step(*dict(a, **over).values(), None) == want


SSM = dict(u=addr(0), delta=addr(1), A=addr(2), Bm=addr(3), Cm=addr(4), skip=addr(5), z=addr(6),
           bias=addr(7), h0=addr(8), lengths=addr(9), B=2, T=40, D=12, G=2, N=16, mode=SOFTPLUS,
           strides=None, y=addr(10), h_T=addr(11), chunks=addr(12))
FULL = [480, 12, 480, 12, 480, 12, 1280, 32, 16, 1280, 32, 16, 480, 12]


def with_stride(i, v):
    s = list(FULL)
    s[i] = v
    return strides(*s)


@pytest.mark.parametrize("over,want", [(o, INVALID) for o in (
    dict(u=None), dict(delta=None), dict(A=None), dict(Bm=None), dict(Cm=None), dict(y=None), dict(h_T=None),
    dict(A=addr(2, 4)), dict(h0=addr(8, 8)), dict(h_T=addr(11, 4)), dict(chunks=addr(12, 4)),
    dict(u=addr(0, 2)), dict(lengths=addr(9, 1)), dict(skip=addr(5, 2)), dict(B=-1), dict(T=-1), dict(D=0),
    dict(G=0), dict(G=5), dict(N=0), dict(mode=1), dict(y=addr(0)), dict(y=addr(6, 4)), dict(h_T=addr(8, 16)),
    dict(h_T=addr(10)), dict(chunks=addr(11)), dict(chunks=addr(3)), dict(strides=with_stride(1, -1)),
    dict(strides=with_stride(13, 11)), dict(strides=with_stride(12, 0)),
    dict(strides=with_stride(3, (1 << 24) + 4)))] +
    [(dict(N=n), UNSUPPORTED) for n in (1, 4, 12, 24, 128)] +
    [(dict(T=(1 << 30) + 1), UNSUPPORTED), (dict(D=1 << 25), UNSUPPORTED)])
def test_ssm_forward(libs, over, want):
    assert libs["ssm"].ttt_ssm_forward(*dict(SSM, **over).values(), None) == want


SSM_BWD = dict(u=addr(0), delta=addr(1), A=addr(2), Bm=addr(3), Cm=addr(4), skip=addr(5), z=addr(6),
               bias=addr(7), lengths=addr(9), B=2, T=40, D=12, G=2, N=16, mode=SOFTPLUS, strides=None,
               chunks=addr(12), dy=addr(13), dh_T=addr(14), du=addr(15), ddelta=addr(16), dA=addr(17),
               dBm=addr(18), dCm=addr(19), dskip=addr(20), dz=addr(21), dbias=addr(22), dh0=addr(23),
               ws=addr(24), ws_bytes=1 << 30)


@pytest.mark.parametrize("over,want", [(o, INVALID) for o in (
    dict(u=None), dict(A=None), dict(chunks=None), dict(dy=None), dict(du=None), dict(ddelta=None),
    dict(dA=None), dict(dBm=None), dict(dCm=None), dict(dz=None), dict(z=None), dict(ws=None), dict(ws_bytes=64),
    dict(ws=addr(24, 4)), dict(chunks=addr(12, 4)), dict(dh0=addr(23, 4)), dict(du=addr(0)), dict(dz=addr(13)),
    dict(dBm=addr(18 + 1)), dict(dA=addr(2)), dict(dh0=addr(14)), dict(dskip=addr(22)), dict(ws=addr(15)),
    dict(G=7), dict(mode=1 << 16), dict(strides=with_stride(12, -480)))] + [(dict(N=20), UNSUPPORTED)])
def test_ssm_backward(libs, over, want):
    assert libs["ssm"].ttt_ssm_backward(*dict(SSM_BWD, **over).values(), None) == want


@pytest.mark.parametrize("over,want", [(o, INVALID) for o in (
    dict(u=None), dict(A=None), dict(h=None), dict(y=None), dict(h=addr(8, 4)), dict(y=addr(0)), dict(h=addr(2)),
    dict(y=addr(8)), dict(G=5), dict(strides=strides(12, 12, 12, 32, 16, 32, 16, 11)))] +
    [(dict(N=48), UNSUPPORTED)])
def test_ssm_step(libs, over, want):
    a = dict(u=addr(0), delta=addr(1), A=addr(2), Bm=addr(3), Cm=addr(4), skip=addr(5), z=addr(6), bias=addr(7),
             h=addr(8), active=addr(9, 1), B=2, D=12, G=2, N=16, mode=SOFTPLUS, strides=None, y=addr(10))
    assert libs["ssm"].ttt_ssm_step(*dict(a, **over).values(), None) == want


@pytest.mark.parametrize("over,want", [(o, INVALID) for o in (
    dict(x=None), dict(w=None), dict(y=None), dict(M=-1), dict(D=0), dict(eps=-1.0), dict(eps=float("inf")),
    dict(mode=1), dict(mode=E4M3 | OUT_BF16), dict(mode=E4M3), dict(group=128), dict(group=7, mode=E4M3),
    dict(scale=addr(5)), dict(residual=None), dict(y=addr(0)), dict(y=addr(1, 64)), dict(s=addr(3)),
    dict(s=addr(1, 4)), dict(s=addr(0), mode=IN_BF16), dict(x=addr(0, 2)), dict(y=addr(3, 2)),
    dict(strides=strides(99, 100, 100, 100)), dict(strides=strides(100, 100, 100, 50)),
    dict(s=addr(1), strides=strides(100, 100, 100, 128)), dict(mode=E4M3, scale=addr(3, 64)))] +
    [(dict(D=16385), UNSUPPORTED)])
def test_norm_forward(libs, over, want):
    a = dict(x=addr(0), residual=addr(1), w=addr(2), M=4, D=100, eps=1e-6, mode=0, group=0, strides=None,
             y=addr(3), s=addr(4), scale=None)
    assert libs["norm"].ttt_norm_forward(*dict(a, **over).values(), None) == want


@pytest.mark.parametrize("over,want", [(o, INVALID) for o in (
    dict(dy=None), dict(s=None), dict(w=None), dict(dx=None), dict(dweight=None), dict(ws=None), dict(ws_bytes=8),
    dict(ws=addr(6, 4)), dict(dx=addr(0)), dict(dx=addr(1)), dict(dx=addr(3, 4)), dict(dweight=addr(4, 16)),
    dict(ws=addr(4)), dict(mode=E4M3), dict(eps=float("nan")), dict(strides=strides(100, 100, 100, 4)),
    dict(dx=addr(3), strides=strides(100, 100, 100, 128)))] + [(dict(D=20000, ws_bytes=1 << 30), UNSUPPORTED)])
def test_norm_backward(libs, over, want):
    a = dict(dy=addr(0), s=addr(1), w=addr(2), ds=addr(3), M=4, D=100, eps=1e-6, mode=0, strides=None,
             dx=addr(4), dweight=addr(5), ws=addr(6), ws_bytes=1 << 20)
    assert libs["norm"].ttt_norm_backward(*dict(a, **over).values(), None) == want


def test_workspace_sizes(libs):
    conv, ssm, norm = (libs[k] for k in ("conv", "ssm", "norm"))
    assert conv.ttt_conv_backward_workspace_bytes(0, 1, 5, 8, 4) == 0
    assert conv.ttt_conv_backward_workspace_bytes(2, 3, 0, 8, 4) == 2 * 24 * 5 * 4
    # whole rows of partial sums, more of them for more tokens
    many = conv.ttt_conv_backward_workspace_bytes(2, 3, 257, 8, 4)
    assert many % (2 * 24 * 5 * 4) == 0 and many >= 2 * 24 * 5 * 4
    assert conv.ttt_conv_backward_workspace_bytes(2, 3, 100000, 8, 4) > many
    assert ssm.ttt_ssm_backward_workspace_bytes(2, 5, 12, 5, 16) == 0
    assert ssm.ttt_ssm_backward_workspace_bytes(2, 5, 12, 2, 12) == 0
    assert ssm.ttt_ssm_backward_workspace_bytes(1, 100000, 64, 1, 16) > 100000 * 32 * 4
    assert norm.ttt_norm_backward_workspace_bytes(0, 64) == 0
    assert norm.ttt_norm_backward_workspace_bytes(3, 64) == 3 * 64 * 4


@pytest.mark.parametrize("rows,want", [((1 << 30) + 1, UNSUPPORTED), ((1 << 31) - 1, UNSUPPORTED)])
def test_rows_beyond_what_the_kernels_count(libs, rows, want):
    """Row numbers and the rows of a grid beyond them fit an int."""
    far = lambda i: (i + 1) << 56  # noqa: E731  (room for tensors of that many rows)
    one = dict(B=rows, H=1, T=1, d=1)
    a = dict(CONV, **one, x=far(0), state=None, lengths=None, weight=far(1), bias=None, y=far(2), state_T=None)
    assert libs["conv"].ttt_conv_forward(*a.values(), None) == want
    a = dict(CONV_BWD, **one, x=far(0), weight=far(1), bias=None, state=None, dy=far(2), dstate_T=None, dx=far(3),
             dweight=far(4), dbias=None, dstate=None, ws=far(5), ws_bytes=1 << 50)
    assert libs["conv"].ttt_conv_backward(*a.values(), None) == want
    a = dict(x=far(0), weight=far(1), bias=None, state=far(2), active=None, B=rows, H=1, d=1, K=4, mode=0,
             strides=None, y=far(3))
    assert libs["conv"].ttt_conv_step(*a.values(), None) == want
    names = ("u", "delta", "A", "Bm", "Cm", "skip", "z", "bias", "h0", "lengths")
    a = dict(SSM, **{k: far(i) for i, k in enumerate(names)}, B=rows, T=1, D=1, G=1, N=8, y=far(10), h_T=far(11),
             chunks=None)
    assert libs["ssm"].ttt_ssm_forward(*a.values(), None) == want
    keys = [k for k, v in SSM_BWD.items() if v is not None and k not in ("B", "T", "D", "G", "N", "mode", "ws_bytes")]
    a = dict(SSM_BWD, **{k: far(i) for i, k in enumerate(keys)}, B=rows, T=1, D=1, G=1, N=8, ws_bytes=1 << 60)
    assert libs["ssm"].ttt_ssm_backward(*a.values(), None) == want
    a = dict(u=far(0), delta=far(1), A=far(2), Bm=far(3), Cm=far(4), skip=None, z=None, bias=None, h=far(5),
             active=None, B=rows, D=1, G=1, N=8, mode=0, strides=None, y=far(6))
    assert libs["ssm"].ttt_ssm_step(*a.values(), None) == want


def test_partial_sums_beyond_what_their_reduction_counts(libs):
    """Rows times blocks along the tokens: the reduction's row number and a step beyond it fit an int."""
    far = lambda i: (i + 1) << 56  # noqa: E731
    for B, T in (((1 << 30) - 1, 600), (1 << 24, 40000)):
        a = dict(CONV_BWD, B=B, H=1, T=T, d=1, K=2, x=far(0), weight=far(1), bias=None, state=None, dy=far(2),
                 dstate_T=None, dx=far(3), dweight=far(4), dbias=None, dstate=None, ws=far(5), ws_bytes=1 << 50)
        parts = libs["conv"].ttt_conv_backward_workspace_bytes(B, 1, T, 1, 2) // 12
        assert 1 << 30 < parts < 1 << 31
        assert libs["conv"].ttt_conv_backward(*a.values(), None) == UNSUPPORTED


def test_bindings_without_torch_s_private_calls(monkeypatch):
    """Where a torch release has not the two private calls that shorten a call, its public ones are taken."""
    import importlib.util
    import types

    import torch

    from test_sequence_layers_02_b200 import _binding
    spec = importlib.util.spec_from_file_location("test_sequence_layers_02_b200._binding_public", _binding.__file__)
    module = importlib.util.module_from_spec(spec)
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    spec.loader.exec_module(module)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: types.SimpleNamespace(cuda_stream=700 + dev))
    with module.On(3, None, ()) as stream:
        assert stream == 703


def test_sizes_beyond_an_int_are_refused_by_the_bindings(monkeypatch):
    """ctypes would cut 2^32 + 5 to 5: a call on 5 tokens that reports success. (Expanded tensors: no memory.)"""
    import torch

    from test_sequence_layers_02_b200 import conv, norm, ssm
    for m in (conv, norm, ssm):
        monkeypatch.setattr(m, "cuda_index", lambda name, x: -1)
    for module in (conv._lib, norm._lib, ssm._lib):
        for name in module._functions:
            monkeypatch.setattr(module, name, lambda *a: pytest.fail("reached the library"), raising=False)
    big = (1 << 32) + 5
    row, w = torch.zeros(8), torch.zeros(8, 4)
    A, bc = torch.zeros(8, 8), torch.zeros(8)
    calls = [lambda: norm.rmsnorm(row.expand(big, 8), row), lambda: norm.rmsnorm_fp8(row.expand(1 << 16, 1 << 16, 8), row),
             lambda: norm.rmsnorm_backward(row.expand(big, 8), row.expand(big, 8), row)]
    for shape in ((1, big, 8), (big, 1, 8)):
        x, v = row.expand(shape), bc.expand(shape)
        calls += [lambda x=x: conv.causal_conv(x, w), lambda x=x: conv.causal_conv_backward(x, w, None, x),
                  lambda x=x, v=v: ssm.selective_scan(x, x, A, v, v),
                  lambda x=x, v=v: ssm.selective_scan_backward(x, x, A, v, v, None, None, None, None, x)]
    x, v = row.expand(big, 8), bc.expand(big, 8)
    calls += [lambda: conv.causal_conv_step(x, w, None, row.expand(big, 3, 8)),
              lambda: ssm.selective_step(x, x, A, v, v, None, None, None, row.expand(big, 8, 8))]
    for f in calls:
        with pytest.raises(ValueError, match="2147483647"):
            f()
