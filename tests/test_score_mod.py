"""pa_attn_fwd_mod against the fp64 oracle on the GPU, and its refusals on the
CPU: caps, distance bias, causal, prefix and document masks, grouped heads,
strides, rows that see nothing, and NaN and Inf in hidden keys.

Tolerances.  O: P and O are rounded to bf16 (half a step, 2^-8 relative, each)
and everything else is fp32, so elementwise |o - o_ref| <= 2^-8 sum_j p_j |v_j|
+ 2^-8 |o_ref| + fp32 noise <= 2^-7 max|v| of the row's keys; over a tensor the
errors of the weights average out, and relative L2 <= 1e-2 as tests/_parity.py
derives.  LSE: the scores carry fp32 rounding (|s| <= 64 in these tests, so
2^-24 * 64 * a few) and, capped, c * 2^-21 * 2; the polynomial exponentials err
by 1.4e-4 relative at most, all of them in one direction at worst: 1.4e-4 + 1e-4
absolute, checked as 3e-4.
"""

import math

import numpy as np
import pytest
import torch

import context_blocks_b200 as pa
from context_blocks_b200 import _binding as B
from oracle import score_mod as oracle

LSE_ABS = 3e-4
REL_L2 = 1e-2


def _rand(shape, seed, std=1.0, layout="bhnd", device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    if layout == "bnhd":
        b, h, n, d = shape
        return (std * torch.randn((b, n, h, d), generator=g, device=device)).bfloat16().transpose(1, 2)
    return (std * torch.randn(shape, generator=g, device=device)).bfloat16()


def _slopes(H):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=torch.float32, device="cuda")


def check_close(o, lse, o_ref, l_ref, v_max):
    o, lse = o.float().cpu().double().numpy(), lse.cpu().double().numpy()
    none = np.isneginf(l_ref)
    assert np.array_equal(none, np.isneginf(lse))
    assert np.array_equal(o[none], np.zeros_like(o[none]))
    assert np.isfinite(o).all() and np.isfinite(lse[~none]).all()
    assert np.abs(o - o_ref).max() <= 2.0 ** -7 * v_max
    if np.linalg.norm(o_ref) > 0:
        assert np.linalg.norm(o - o_ref) <= REL_L2 * np.linalg.norm(o_ref)
    if (~none).any():
        assert np.abs(lse[~none] - l_ref[~none]).max() <= LSE_ABS


def _case(Bn, Hq, Hkv, Nq, Nk, d, seed, layout="bhnd", qstd=1.0, **kw):
    q, k, v = (_rand((Bn, Hq, Nq, d), seed, qstd, layout), _rand((Bn, Hkv, Nk, d), seed + 1, 1.0, layout),
               _rand((Bn, Hkv, Nk, d), seed + 2, 1.0, layout))
    args = dict(kw)
    host = dict(kw)
    for n in ("prefix_lens", "doc_offsets"):
        if kw.get(n) is not None:
            args[n] = torch.tensor(kw[n], dtype=torch.int32, device="cuda")
    if kw.get("slopes"):
        args["slopes"] = _slopes(Hq)
        host["slopes"] = args["slopes"].cpu().numpy()
    else:
        args.pop("slopes", None)
        host.pop("slopes", None)
    o, lse = pa.attn_fwd_mod(q, k, v, check=True, **args)
    o_ref, l_ref = oracle.attention(q.cpu(), k.cpu(), v.cpu(), d ** -0.5, **host)
    check_close(o, lse, o_ref, l_ref, float(v.abs().max()))
    return q, k, v, o, lse


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,Nk", [(1, 1), (1, 129), (2, 300), (127, 127), (128, 128), (129, 131), (257, 257), (300, 517)])
@pytest.mark.parametrize("kw", [dict(), dict(causal=True), dict(causal=True, softcap=5.0), dict(softcap=1.0),
                                dict(causal=True, slopes=True), dict(slopes=True),
                                dict(causal=True, slopes=True, softcap=5.0)], ids=str)
def test_small(d, Nq, Nk, kw):
    _case(2, 4, 2, Nq, Nk, d, seed=Nq + Nk, qstd=3.0, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("cap", [0.5, 5.0, 30.0, 50.0, 52.5, 80.0, 1e4])
@pytest.mark.parametrize("qstd", [0.1, 3.0, 20.0])
@pytest.mark.parametrize("slopes", [False, True])
def test_caps(cap, qstd, slopes):
    """Scores well inside the cap, around it and far outside; caps that take the
    fixed reference maximum and caps that do not; rows that see nothing."""
    _case(1, 2, 1, 260, 391, 64, seed=int(cap * 10), qstd=qstd, causal=True, softcap=cap, slopes=slopes,
          doc_offsets=[[0, 140, 200, 380]])


@pytest.mark.gpu
def test_capped_scores_at_the_far_end():
    """Every score of a row at -c: the weights are small beside the fixed
    reference, and the result is as if they were not."""
    q = torch.ones((1, 1, 130, 64), dtype=torch.bfloat16, device="cuda")
    k = -100.0 * torch.ones((1, 1, 200, 64), dtype=torch.bfloat16, device="cuda")
    for scale_v in (1.0, 1e-4, 1e6):
        v = (scale_v * _rand((1, 1, 200, 64), 5)).bfloat16()
        o, lse = pa.attn_fwd_mod(q, k, v, softcap=50.0, check=True)
        want = v.double().mean(2)
        assert (o[0, 0].double() - want[0]).abs().max() <= 2.0 ** -7 * v.double().abs().max()
        assert (lse - (math.log(200) - 50.0)).abs().max() <= LSE_ABS


@pytest.mark.gpu
@pytest.mark.parametrize("prefix", [0, 1, 127, 128, 129, 200, 300, 1000])
def test_prefix(prefix):
    _case(2, 2, 1, 300, 300, 64, seed=prefix, causal=True, prefix_lens=[prefix, max(0, prefix - 3)])


DOCS = {
    "one": [[0, 300]], "padded": [[0, 211]], "late start": [[37, 290]], "halves": [[0, 128, 300]],
    "short": [[0, 1, 2, 3, 7, 100, 101, 260, 300]], "empty ones": [[0, 0, 0, 90, 90, 300, 300]],
    "nothing": [[0, 0]], "nothing at the end": [[300, 300]], "tiles": [[0, 128, 256]],
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", DOCS)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("layout", ["bhnd", "bnhd"])
def test_documents(name, causal, layout):
    _case(1, 3, 1, 300, 300, 128, seed=5, layout=layout, causal=causal, doc_offsets=DOCS[name])


@pytest.mark.gpu
def test_documents_of_a_batch_with_prefixes_cap_and_bias():
    docs = [[0, 10, 200, 517], [100, 300, 300, 400]]
    _case(2, 4, 2, 517, 517, 64, seed=8, causal=True, doc_offsets=docs, prefix_lens=[[3, 150, 0], [40, 5, 1000]],
          softcap=10.0, slopes=True)


@pytest.mark.gpu
@pytest.mark.parametrize("q_offset", [-50, -300, 0, 100, 217, 500, 2000])
@pytest.mark.parametrize("docs", [None, [[5, 200, 450]]])
def test_query_positions(q_offset, docs):
    _case(1, 2, 2, 300, 517, 64, seed=9, causal=True, q_offset=q_offset, doc_offsets=docs, slopes=True)


@pytest.mark.gpu
def test_many_items_and_long_keys():
    """More items than CTAs and many key tiles, against the package's own merge
    of unmasked chunks where the mask is a plain one (rows behind all keys)."""
    q, k, v = _rand((2, 24, 700, 128), 1), _rand((2, 24, 4603, 128), 2), _rand((2, 24, 4603, 128), 3)
    o, lse = pa.attn_fwd_mod(q, k, v, causal=True, q_offset=5000, check=True)
    o2, lse2 = pa.attn_fwd(q, k, v)
    assert (o.float() - o2.float()).abs().max() <= 2.0 ** -7 * 5
    assert (lse - lse2).abs().max() <= LSE_ABS


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf"), 3e38])
@pytest.mark.parametrize("kw", [dict(causal=True), dict(causal=True, softcap=20.0),
                                dict(causal=True, slopes=True, softcap=20.0)], ids=str)
def test_hidden_keys_do_not_matter(bad, kw):
    """NaN, Inf and the type's largest values in keys and values that a row does
    not see leave the row as it is: behind the last document, and one document's
    in another's rows."""
    q, k, v = _rand((1, 2, 300, 128), 1), _rand((1, 2, 300, 128), 2), _rand((1, 2, 300, 128), 3)
    docs = torch.tensor([[0, 100, 170, 290]], dtype=torch.int32, device="cuda")
    sl = _slopes(2) if kw.get("slopes") else None
    args = dict(kw, slopes=sl, doc_offsets=docs)
    o, lse = pa.attn_fwd_mod(q, k, v, **args)
    k2, v2 = k.clone(), v.clone()
    k2[:, :, 290:], v2[:, :, 290:] = bad, bad          # behind the last document
    k2[:, :, 165:170], v2[:, :, 165:170] = bad, bad    # the end of the second one
    o2, lse2 = pa.attn_fwd_mod(q, k2, v2, check=True, **args)
    rows = torch.ones(300, dtype=torch.bool, device="cuda")
    rows[165:170] = False
    assert (lse2[:, :, rows] - lse[:, :, rows]).nan_to_num(0, 0, 0).abs().max() <= LSE_ABS
    assert torch.isfinite(o2[:, :, rows]).all()
    # recomputed rows do not round their weights to bf16: both are 2^-8 from exact
    assert (o2[:, :, rows].float() - o[:, :, rows].float()).abs().max() <= 2.0 ** -6 * float(v.abs().max())


@pytest.mark.gpu
def test_two_streams_at_once():
    """Calls that overlap on the GPU share nothing."""
    ops = [(_rand((1, 8, 2000, 64), 10 * i), _rand((1, 8, 2000, 64), 10 * i + 1), _rand((1, 8, 2000, 64), 10 * i + 2))
           for i in range(2)]
    want = [pa.attn_fwd_mod(*o, causal=True, softcap=10.0) for o in ops]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ops]
    got = [[pa.attn_fwd_mod(*o, causal=True, softcap=10.0, stream=s) for _ in range(5)] for o, s in zip(ops, streams)]
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for o, lse in g:
            assert torch.equal(o, w[0]) and torch.equal(lse, w[1])
    assert pa.poll_device_status() == pa.PA_OK


@pytest.mark.gpu
def test_long_keys_with_a_short_wait_limit():
    """A warp that waits while another works through a long item is not taken
    for one that is stuck: one query tile sees the last key only, the other all
    200 000."""
    pa.set_wait_limit_ms(1)
    try:
        q, k, v = _rand((1, 1, 256, 64), 1), _rand((1, 1, 200000, 64), 2), _rand((1, 1, 200000, 64), 3)
        docs = torch.tensor([[0, 199872, 199873]], dtype=torch.int32, device="cuda")
        o, lse = pa.attn_fwd_mod(q, k, v, q_offset=199872 - 128, doc_offsets=docs, check=True)
        assert torch.isfinite(o[:, :, :129]).all() and torch.equal(o[:, :, 128], v[:, :, 199872])
        assert (o[:, :, 129:] == 0).all()
    finally:
        pa.set_wait_limit_ms(5000)


@pytest.mark.gpu
def test_offsets_that_decrease_do_no_harm():
    """Undefined results, as documented, but no fault and no stuck wait."""
    q, k, v = _rand((2, 2, 600, 64), 1), _rand((2, 2, 600, 64), 2), _rand((2, 2, 600, 64), 3)
    g = torch.Generator(device="cuda").manual_seed(4)
    for _ in range(5):
        docs = torch.randint(-1000, 2000, (2, 9), generator=g, device="cuda", dtype=torch.int32)
        lens = torch.randint(-(1 << 31), (1 << 31) - 1, (2, 8), generator=g, device="cuda", dtype=torch.int32)
        pa.attn_fwd_mod(q, k, v, causal=True, doc_offsets=docs, prefix_lens=lens, check=True)


@pytest.mark.gpu
def test_strided_operands_and_outputs():
    """q, k and v as slices of one projection, o into a slice of a wider buffer;
    what lies around it stays."""
    qkv = _rand((2, 1, 300, (4 + 2 + 2) * 64), 4).view(2, 300, 8, 64)
    q, k, v = (t.transpose(1, 2) for t in (qkv[:, :, :4], qkv[:, :, 4:6], qkv[:, :, 6:]))
    wide = torch.full((2, 300, 6, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, :, 1:5].transpose(1, 2)
    o, lse = pa.attn_fwd_mod(q, k, v, causal=True, out=out, check=True)
    assert o.data_ptr() == out.data_ptr()
    o_ref, l_ref = oracle.attention(q.cpu(), k.cpu(), v.cpu(), 0.125, causal=True)
    check_close(o, lse, o_ref, l_ref, float(v.abs().max()))
    assert (wide[:, :, 0] == 7.0).all() and (wide[:, :, 5] == 7.0).all()


@pytest.mark.gpu
def test_captured_replayed_and_on_another_stream():
    q, k, v = _rand((1, 4, 300, 64), 1), _rand((1, 2, 300, 64), 2), _rand((1, 2, 300, 64), 3)
    want = pa.attn_fwd_mod(q, k, v, causal=True, softcap=8.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = pa.attn_fwd_mod(q, k, v, causal=True, softcap=8.0, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    o, lse = torch.empty_like(q), torch.empty_like(want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.attn_fwd_mod(q, k, v, causal=True, softcap=8.0, out=o, lse=lse)
    for _ in range(2):
        o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.gpu
def test_refusals_of_the_binding():
    q, k = _rand((1, 4, 8, 64), 1), _rand((1, 2, 8, 64), 2)
    ids = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    for bad in (dict(q=q.float()), dict(k=_rand((1, 3, 8, 64), 1)), dict(slopes=_slopes(3)),
                dict(doc_offsets=ids.long()), dict(doc_offsets=ids[:, :1]), dict(out=torch.empty_like(k)),
                dict(lse=torch.empty((1, 4, 8), device="cuda", dtype=torch.float64)), dict(q=q.transpose(2, 3)),
                dict(prefix_lens=ids)):
        with pytest.raises((TypeError, ValueError, pa.PaError)):
            pa.attn_fwd_mod(**dict(dict(q=q, k=k, v=k), **bad))
    with pytest.raises(pa.PaError, match="causal"):
        pa.attn_fwd_mod(q, k, k, prefix_lens=ids[:, 0].contiguous())
    with pytest.raises(pa.PaError, match="overlap"):
        pa.attn_fwd_mod(q, k, k, out=q)
    with pytest.raises(pa.PaError, match="stride"):
        pa.attn_fwd_mod(q, k, k, out=q[:, :1].expand(1, 4, 8, 64))
    with pytest.raises(pa.PaError):
        pa.attn_fwd_mod(q[:, :1].expand(1, 4, 8, 64), k, k)  # stride 0
    o, lse = pa.attn_fwd_mod(q[:, :, :0], k, k)
    assert o.numel() == 0 and lse.numel() == 0


A, MB = 1 << 20, 1 << 24


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), B.PA_ERR_INVALID_ARG), (dict(lse=0), B.PA_ERR_INVALID_ARG), (dict(mod=None), B.PA_ERR_INVALID_ARG),
    (dict(Hkv=3), B.PA_ERR_INVALID_ARG), (dict(Hkv=0), B.PA_ERR_INVALID_ARG), (dict(Nk=0), B.PA_ERR_INVALID_ARG),
    (dict(Nq=-1), B.PA_ERR_INVALID_ARG), (dict(d=96), B.PA_ERR_UNSUPPORTED), (dict(Bn=40000), B.PA_ERR_UNSUPPORTED),
    (dict(Nk=(1 << 30) + 1), B.PA_ERR_UNSUPPORTED), (dict(softcap=-1.0), B.PA_ERR_INVALID_ARG),
    (dict(softcap=math.inf), B.PA_ERR_INVALID_ARG), (dict(softcap=1e-20), B.PA_ERR_INVALID_ARG),
    (dict(softcap=1e20), B.PA_ERR_INVALID_ARG), (dict(softcap=1e14, scale=1e-20), B.PA_ERR_INVALID_ARG), (dict(softcap=math.nan), B.PA_ERR_INVALID_ARG),
    (dict(scale=0.0), B.PA_ERR_INVALID_ARG), (dict(prefix=A), B.PA_ERR_INVALID_ARG),
    (dict(docs=A), B.PA_ERR_INVALID_ARG), (dict(docs=A + 2, n_docs=1), B.PA_ERR_MISALIGNED),
    (dict(slopes=A + 1), B.PA_ERR_MISALIGNED), (dict(k=A + MB + 8), B.PA_ERR_MISALIGNED),
    (dict(q_offset=-(1 << 30) - 1), B.PA_ERR_UNSUPPORTED), (dict(o=A), B.PA_ERR_INVALID_ARG),
    (dict(lse=A + 3 * MB), B.PA_ERR_INVALID_ARG), (dict(slopes=A + 4 * MB), B.PA_ERR_INVALID_ARG),
    (dict(strides=[0] * 12), B.PA_ERR_INVALID_ARG), (dict(strides=[4096, 1024, 68] * 4), B.PA_ERR_MISALIGNED),
    (dict(strides=[4096, 1024, 64] * 4), B.PA_ERR_INVALID_ARG),  # o's rows overlap: 8 rows of 128 in 1024
    (dict(Nq=0), B.PA_OK),
])
def test_argument_checks(kw, code):
    import ctypes
    lib = B.load_library()
    a = dict(dict(q=A, k=A + MB, v=A + 2 * MB, o=A + 3 * MB, lse=A + 4 * MB, Bn=2, Hq=4, Hkv=2, Nq=8, Nk=8, d=128,
                  strides=None, scale=0.125, softcap=0.0, causal=0, slopes=None, prefix=None, docs=None, n_docs=0,
                  q_offset=0), **kw)
    mod = B.ScoreMod(a["softcap"], a["causal"], a["slopes"], a["prefix"], a["docs"], a["n_docs"], a["q_offset"])
    st = (ctypes.c_longlong * 12)(*a["strides"]) if a["strides"] else None
    rc = lib.pa_attn_fwd_mod(a["q"], a["k"], a["v"], a["o"], a["lse"], a["Bn"], a["Hq"], a["Hkv"], a["Nq"], a["Nk"],
                             a["d"], st, a["scale"], None if "mod" in kw else ctypes.byref(mod), None)
    assert rc == code, B.last_error()
    assert rc == B.PA_OK or B.last_error() != ""


def test_oracle_masks_by_hand():
    t = oracle.visible(4, 4, causal=True)
    assert t.tolist() == np.tril(np.ones((4, 4), bool)).tolist()
    t = oracle.visible(2, 4, causal=True, prefix=4)
    assert t.all()
    t = oracle.visible(5, 5, offsets=[1, 3, 4])
    assert t.astype(int).tolist() == [[0] * 5, [0, 1, 1, 0, 0], [0, 1, 1, 0, 0], [0, 0, 0, 1, 0], [0] * 5]
    # one visible key: its value and score
    q = np.array([[2.0]])
    o, lse = oracle.rows(q, np.array([[3.0], [9.0]]), np.array([[5.0], [np.nan]]), np.array([[True, False]]), [1],
                         np.array([0, 1]), 0.5, softcap=2.0, slope=0.25)
    assert o[0, 0] == 5.0 and abs(lse[0] - (2.0 * math.tanh(1.5) - 0.25)) < 1e-15


@pytest.mark.gpu
@pytest.mark.parametrize("Bn,Hq,Nq,Nk,d", [(2, 20, 2100, 2100, 64), (7, 8, 2300, 2300, 64), (1, 36, 2400, 3001, 128)])
@pytest.mark.parametrize("kw", [dict(), dict(causal=True), dict(causal=True, softcap=4.0), dict(slopes=True)], ids=str)
def test_many_heads_take_the_same_values_as_few(Bn, Hq, Nq, Nk, d, kw):
    """The order in which items are worked on (longest first with many items and
    few documents) changes no bit: all heads at once against the first two alone,
    which is too few items to order."""
    q, k, v = _rand((Bn, Hq, Nq, d), 31, 2.0), _rand((Bn, Hq // 2, Nk, d), 32), _rand((Bn, Hq // 2, Nk, d), 33)
    cuts = [[0, 0, 5 + 37 * b, 700, 700 + 130 * b, Nk - 700, Nk - 40 * b] for b in range(Bn)]
    kw = dict(kw, doc_offsets=torch.tensor(cuts, dtype=torch.int32, device="cuda"))
    few = dict(kw)
    if kw.pop("slopes", False):
        kw["slopes"] = _slopes(Hq)
        few["slopes"] = kw["slopes"][:2].contiguous()
    o, lse = pa.attn_fwd_mod(q, k, v, check=True, **kw)
    o2, lse2 = pa.attn_fwd_mod(q[:, :2], k[:, :1], v[:, :1], check=True, **few)
    assert torch.equal(o[:, :2], o2) and torch.equal(lse[:, :2], lse2)
    assert torch.isfinite(o.float()).all()
    some = torch.isfinite(lse[:, 0]).sum(-1).tolist()
    at = [range(Nk - Nq, Nk)] * Bn
    assert some == [sum(c[0] <= p < c[-1] for p in r) for c, r in zip(cuts, at)]


def test_tanh_polynomial_matches_its_fit_and_bound():
    import os
    import re
    import sys
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "context_blocks_b200", "csrc")
    sys.path.insert(0, csrc)
    import gen_tanh_poly as gen
    text = re.search(r"kTanhC\[6\] = \{([^}]*)\}", open(os.path.join(csrc, "score_mod.cuh")).read()).group(1)
    k = np.array([float(x.strip().rstrip("f")) for x in text.split(",")], dtype=np.float32)
    c, err = gen.fit(5)
    assert err < 6e-7 and np.allclose(k, c.astype(np.float32), rtol=1e-6, atol=0)
    u = np.linspace(-1.0, 1.0, 200001)
    u = u[u != 0]
    rel = np.abs(gen.simulate(k, u).astype(np.float64) - np.tanh(u)) / np.abs(np.tanh(u))
    assert rel.max() < 8e-7  # the fit, and the roundings of w, p and the product: a few 2^-24
