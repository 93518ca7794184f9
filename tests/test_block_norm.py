"""pa_gate_residual_norm against the fp64 oracle on the GPU, and its refusals on
the CPU.

Tolerances: one rounding to the output's type, half a step relative (bf16 2^-8,
fp32 2^-24), and fp32 arithmetic in between: sums of D terms in a tree err by
less than 2^-20 relative for D <= 16384 (12 levels and the terms of a thread),
rsqrtf and the products by a few 2^-23.  What is subtracted (the mean, the
residual) can make a result small beside its terms, so the absolute part counts
from the largest term of the row, `size`.
"""

import math

import numpy as np
import pytest
import torch

import context_blocks_b200 as pa
from context_blocks_b200 import _binding as B
from oracle import block_norm as oracle

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _bf16(shape, seed, std=1.0, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (mean + std * torch.randn(shape, generator=g, device="cuda")).bfloat16()


def _check(got, want, size):
    g = got.float().cpu().double().numpy() if got.dtype != torch.float32 else got.cpu().double().numpy()
    tol = HALF[got.dtype] * np.abs(want) + 2.0 ** -18 * size
    assert (np.abs(g - want) <= tol).all(), np.abs(g - want).max()


def _case(Bn, N, D, x32, seed, mean=0.0, check=True, **kw):
    y, x = _bf16((Bn, N, D), seed, 2.0, mean), _bf16((Bn, N, D), seed + 1, 3.0, mean)
    if x32:
        x = x.float() + 1e-3 * _bf16((Bn, N, D), seed + 2).float()
    args = dict(kw)
    wide = _bf16((Bn, 4 * D), seed + 3, 0.5)
    for i, n in enumerate(("gate", "scale", "shift")):
        if args.get(n):
            args[n] = wide[:, i * D:(i + 1) * D]
    for n in ("post_weight", "norm_weight"):
        if args.get(n):
            args[n] = _bf16((D,), seed + 4, 0.2, 1.0)
    xo, h = pa.gate_residual_norm(y, x, check=True, **args)
    xr, hr = oracle.gate_residual_norm(y, x if not x32 else x.cpu().double().numpy(), **args)
    big = np.abs(xr).max() + abs(mean)
    _check(xo, xr, big)
    assert xo.dtype == x.dtype
    if hr is None:
        assert h is None
    else:
        # an error e of x_new becomes e / rms(x_new) in h; rows here have rms >= 1
        _check(h, hr, big * max(1.0, np.abs(hr).max()))
    return y, x, args, xo, h


@pytest.mark.gpu
@pytest.mark.parametrize("D", [8, 64, 248, 256, 264, 504, 1000, 1024, 1032, 1536, 2048, 2056, 4096, 4104, 8192, 8200, 16384])
@pytest.mark.parametrize("x32", [False, True])
def test_widths(D, x32):
    _case(2, 5, D, x32, seed=D, post="rms", post_weight=True, norm="layer", gate=True, scale=True, shift=True)


@pytest.mark.gpu
@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("norm", ["none", "rms", "layer"])
@pytest.mark.parametrize("kw", [dict(), dict(gate=True), dict(post_weight=True, residual_scale=0.5)], ids=str)
def test_kinds(post, norm, kw):
    for Bn, N in ((1, 1), (3, 7), (1, 9)):
        _case(Bn, N, 320, False, seed=N, post=post, norm=norm, **kw)
        if norm != "none":
            _case(Bn, N, 2560, True, seed=N, post=post, norm=norm, norm_weight=True, shift=True, **kw)


@pytest.mark.gpu
def test_rows_far_from_zero_keep_their_variance():
    _case(1, 16, 4096, True, seed=3, mean=200.0, post="layer", norm="layer")


@pytest.mark.gpu
def test_zero_rows_and_one_value_rows():
    """A row of zeros has rms 0 and stays 0; a constant row has variance 0."""
    z = torch.zeros((1, 3, 512), dtype=torch.bfloat16, device="cuda")
    xo, h = pa.gate_residual_norm(z, z, post="rms", norm="rms", check=True)
    assert (xo == 0).all() and (h == 0).all()
    xo, h = pa.gate_residual_norm(z, z + 4, norm="layer", check=True)
    assert (xo == 4).all() and (h == 0).all()


@pytest.mark.gpu
def test_many_rows():
    y, x, args, xo, h = _case(2, 4481, 1536, False, seed=9, norm="layer", gate=True, scale=True, shift=True)


@pytest.mark.gpu
@pytest.mark.parametrize("x32", [False, True])
def test_in_place_and_neighbours(x32):
    """x_out = x, and rows around the outputs stay as they are."""
    y, x, args, xo, h = _case(1, 37, 1000, x32, seed=10, post="rms", gate=True)
    xw = torch.full((39, 1000), 5.0, dtype=x.dtype, device="cuda")
    hw = torch.full((39, 1000), 5.0, dtype=torch.bfloat16, device="cuda")
    xw[1:38] = x[0]
    xi = xw[1:38].view(1, 37, 1000)
    a, b = pa.gate_residual_norm(y, xi, x_out=xi, out=hw[1:38].view(1, 37, 1000), check=True, **args)
    assert a.data_ptr() == xi.data_ptr() and torch.equal(xi, xo) and torch.equal(hw[1:38], h[0])
    for w in (xw, hw):
        assert (w[0] == 5).all() and (w[38] == 5).all()


@pytest.mark.gpu
def test_captured_and_on_another_stream():
    y, x, args, xo, h = _case(2, 33, 2048, False, seed=12, post="rms", post_weight=True, gate=True, norm_weight=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a, b = pa.gate_residual_norm(y, x, stream=s, **args)
    torch.cuda.synchronize()
    assert torch.equal(a, xo) and torch.equal(b, h)
    ga, gb = torch.empty_like(xo), torch.empty_like(h)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.gate_residual_norm(y, x, x_out=ga, out=gb, **args)
    for _ in range(2):
        ga.zero_(), gb.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(ga, xo) and torch.equal(gb, h)


@pytest.mark.gpu
def test_nan_and_inf_stay_in_their_rows():
    y, x, args, xo, h = _case(1, 9, 1536, False, seed=13, post="rms", norm="layer")
    y2 = y.clone()
    y2[0, 4, 7] = float("nan")
    y2[0, 2, 1] = float("inf")
    a, b = pa.gate_residual_norm(y2, x, check=True, **args)
    rows = [0, 1, 3, 5, 6, 7, 8]
    assert torch.equal(a[:, rows], xo[:, rows]) and torch.equal(b[:, rows], h[:, rows])
    assert torch.isnan(b[0, 4]).all()


@pytest.mark.gpu
def test_a_layer_with_its_attention():
    """The operators together: norm, attention over the normed rows, gated
    residual with the next norm; against the same steps in fp64 on the values
    each step was given."""
    y, x, args, xo, h = _case(1, 200, 256, True, seed=14, post="rms", gate=True, norm="rms", norm_weight=True)
    q = h.view(1, 200, 4, 64).transpose(1, 2)
    o, lse = pa.attn_fwd_mod(q, q, q, causal=True, softcap=20.0)
    from oracle import score_mod
    from tests.test_score_mod import check_close
    o_ref, l_ref = score_mod.attention(q.cpu(), q.cpu(), q.cpu(), 0.125, softcap=20.0, causal=True)
    check_close(o, lse, o_ref, l_ref, float(h.abs().max()))
    y2 = o.transpose(1, 2).reshape(1, 200, 256)
    assert y2.data_ptr() == o.data_ptr()  # o has q's layout: no copy on the way
    x2, h2 = pa.gate_residual_norm(y2, xo, x_out=xo.clone(), norm="layer", check=True)
    xr, hr = oracle.gate_residual_norm(y2, xo.cpu().double().numpy(), norm="layer")
    _check(x2, xr, np.abs(xr).max())
    _check(h2, hr, np.abs(xr).max() * np.abs(hr).max())


@pytest.mark.gpu
def test_refusals_of_the_binding():
    y, w = _bf16((2, 3, 64), 1), _bf16((64,), 2)
    g = _bf16((2, 64), 3)
    for bad in (dict(y=y.float()), dict(x=y.half()), dict(x=y[:1]), dict(post="batch"), dict(gate=w), dict(gate=g.float()),
                dict(post_weight=g), dict(norm_weight=w.float()), dict(norm="none", out=torch.empty_like(y)),
                dict(x_out=torch.empty((2, 3, 64), device="cuda")), dict(out=torch.empty((2, 3, 72), device="cuda")),
                dict(gate=g.cpu()), dict(x=y.transpose(1, 2)), dict(norm="none", norm_weight=w), dict(eps=-1.0),
                dict(residual_scale=math.nan), dict(out=y), dict(x_out=y), dict(gate=_bf16((2, 68), 3)[:, :64])):
        with pytest.raises((TypeError, ValueError, pa.PaError)):
            pa.gate_residual_norm(**dict(dict(y=y, x=y.clone()), **bad))
    with pytest.raises(pa.PaError, match="multiple of 8"):
        pa.gate_residual_norm(_bf16((1, 1, 12), 1), _bf16((1, 1, 12), 1))
    a, b = pa.gate_residual_norm(y[:, :0].contiguous(), y[:, :0].contiguous())
    assert a.numel() == 0 and b.numel() == 0


A, MB = 1 << 20, 1 << 24


@pytest.mark.parametrize("kw,code", [
    (dict(y=0), B.PA_ERR_INVALID_ARG), (dict(x=0), B.PA_ERR_INVALID_ARG), (dict(xo=0), B.PA_ERR_INVALID_ARG),
    (dict(h=0), B.PA_ERR_INVALID_ARG), (dict(norm=0), B.PA_ERR_INVALID_ARG), (dict(norm=3), B.PA_ERR_INVALID_ARG),
    (dict(post=-1), B.PA_ERR_INVALID_ARG), (dict(Bn=0), B.PA_ERR_INVALID_ARG), (dict(N=-1), B.PA_ERR_INVALID_ARG),
    (dict(D=0), B.PA_ERR_UNSUPPORTED), (dict(D=12), B.PA_ERR_UNSUPPORTED), (dict(D=16392), B.PA_ERR_UNSUPPORTED),
    (dict(y=A + 8), B.PA_ERR_MISALIGNED), (dict(gate=A + 5 * MB + 2), B.PA_ERR_MISALIGNED),
    (dict(gate=A + 5 * MB, gs=68), B.PA_ERR_MISALIGNED), (dict(gate=A + 5 * MB, gs=-64), B.PA_ERR_INVALID_ARG),
    (dict(h=A), B.PA_ERR_INVALID_ARG), (dict(xo=A + 16), B.PA_ERR_INVALID_ARG), (dict(xo=A + MB + 16), B.PA_ERR_INVALID_ARG),
    (dict(h=A + 2 * MB), B.PA_ERR_INVALID_ARG), (dict(gate=A + 3 * MB, gs=64), B.PA_ERR_INVALID_ARG),
    (dict(eps=math.inf), B.PA_ERR_INVALID_ARG), (dict(a=math.inf), B.PA_ERR_INVALID_ARG), (dict(cfg=None), B.PA_ERR_INVALID_ARG),
    (dict(N=0), B.PA_OK),
])
def test_argument_checks(kw, code):
    import ctypes
    a = dict(dict(y=A, x=A + MB, xo=A + 2 * MB, h=A + 3 * MB, Bn=2, N=3, D=64, post=1, norm=1, gate=None, gs=0, eps=1e-6,
                  a=1.0), **kw)
    cfg = B.BlockNorm(a["post"], a["norm"], gate=a["gate"], gate_stride=a["gs"], residual_scale=a["a"], eps=a["eps"])
    rc = B.load_library().pa_gate_residual_norm(a["y"], a["x"], a["xo"], a["h"] or None, a["Bn"], a["N"], a["D"], 0,
                                                 None if "cfg" in kw else ctypes.byref(cfg), None)
    assert rc == code, B.last_error()


def test_norm_codes_match_header():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "pa_attn.h")).read()
    for name, value in B.PA_NORM.items():
        assert int(re.search(r"#define PA_NORM_%s (\d)" % name.upper(), text).group(1)) == value


def test_oracle_by_hand():
    x, h = oracle.gate_residual_norm(np.array([[[3.0, 4.0]]]), np.array([[[1.0, 1.0]]]), gate=np.array([[2.0, 0.0]]),
                                     post="rms", norm="layer", residual_scale=0.5, eps=0.0)
    r = math.sqrt(12.5)
    assert np.allclose(x, [[[0.5 + 2 * 3 / r, 0.5]]], atol=1e-15) and np.allclose(h, [[[1.0, -1.0]]], atol=1e-15)
