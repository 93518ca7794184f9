"""NaN, Inf and very large numbers in the operands of attn_fwd_mod and
attn_shared_prefix: they reach the rows that see them, as in the formulas, and
no others.

Tolerances as derived in tests/test_score_mod.py: 2^-7 max|v| of the visible
values on O, 3e-4 on LSE.
"""

import numpy as np
import pytest
import torch

import context_blocks_b200 as pa
from oracle import score_mod as oracle
from tests.test_score_mod import LSE_ABS, _rand, _slopes

NAN, INF = float("nan"), float("inf")

# Plain, capped against the fixed reference, capped with a running maximum, biased, both.
FORMS = [dict(), dict(softcap=4.0), dict(softcap=60.0), dict(slopes=True), dict(softcap=4.0, slopes=True)]


def check_same(o, lse, o_ref, l_ref, v_max):
    """Equal to the oracle within the tolerances where it is finite, NaN where it
    is NaN, the same infinity where it is infinite."""
    o, lse = o.float().cpu().double().numpy(), lse.cpu().double().numpy()
    for got, want, tol in ((o, o_ref, 2.0 ** -7 * v_max), (lse, l_ref, LSE_ABS)):
        fin = np.isfinite(want)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.array_equal(got[np.isinf(want)], want[np.isinf(want)])
        assert np.isfinite(got[fin]).all()
        assert not fin.any() or np.abs(got[fin] - want[fin]).max() <= tol


def _shared(q, kp, vp, kt, vt, lens, kw, v_max):
    Hq, d = q.shape[1], q.shape[3]
    args = dict(kw, slopes=_slopes(Hq)) if kw.get("slopes") else kw
    host = dict(args, slopes=args["slopes"].cpu().numpy()) if kw.get("slopes") else kw
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = pa.attn_shared_prefix(q, kp, vp, kt, vt, n, check=True, **args)
    with np.errstate(invalid="ignore"):
        o_ref, l_ref = oracle.shared_prefix(q, kp, vp, kt, vt, lens, d ** -0.5, **host)
    check_same(o, lse, o_ref, l_ref, v_max)
    return o, lse


# Rows of a request under one K/V head, and of a row tile, in 4, 2 and 1 copies;
# two row tiles (a pair), three (a pair and an odd one).
ROWS = [(3, 4, 1), (3, 16, 1), (2, 48, 1), (2, 80, 1), (1, 100, 1), (30, 8, 1), (40, 8, 1), (5, 4, 3), (2, 7, 14)]


@pytest.mark.gpu
@pytest.mark.parametrize("kw", FORMS, ids=str)
@pytest.mark.parametrize("Bn,G,Nq", ROWS)
@pytest.mark.parametrize("Np", [0, 300])
def test_nan_in_queries_and_new_keys_of_a_decoding_step(Np, Bn, G, Nq, kw):
    """A NaN query row; a request whose only key of its own is NaN; one whose last
    key is, alone in its key tile.  The other requests are as without them."""
    q, kp, vp = _rand((Bn, 2 * G, Nq, 64), 1, 2.0), _rand((2, Np, 64), 2), _rand((2, Np, 64), 3)
    kt, vt = _rand((Bn, 2, 140, 64), 4), _rand((Bn, 2, 140, 64), 5)
    lens = [max(Nq, (1, 129, 70)[b % 3]) for b in range(Bn)]
    _shared(q, kp, vp, kt, vt, lens, kw, 6.0)
    q2 = q.clone()
    q2[Bn // 2, 1, Nq - 1] = NAN
    _shared(q2, kp, vp, kt, vt, lens, kw, 6.0)
    for b in range(min(Bn, 2)):
        k2 = kt.clone()
        k2[b, 1, lens[b] - 1] = NAN
        _shared(q, kp, vp, k2, vt, lens, kw, 6.0)


@pytest.mark.gpu
@pytest.mark.parametrize("kw", FORMS, ids=str)
@pytest.mark.parametrize("Bn,G,Nq", ROWS)
def test_nan_key_in_the_prefix(Bn, G, Nq, kw):
    """All rows under its K/V head are NaN, wherever it stands: alone in the last
    key tile, among others, and alone in the prefix."""
    for Np, at in ((257, 256), (257, 40), (1, 0)):
        q, kp, vp = _rand((Bn, 2 * G, Nq, 64), 1, 2.0), _rand((2, Np, 64), 2), _rand((2, Np, 64), 3)
        kt, vt = _rand((Bn, 2, 16, 64), 4), _rand((Bn, 2, 16, 64), 5)
        kp[1, at] = NAN
        o, lse = _shared(q, kp, vp, kt, vt, [min(16, Nq + b % 3) for b in range(Bn)], kw, 6.0)
        assert torch.isnan(lse[:, G:]).all() and not torch.isnan(lse[:, :G]).any()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kw", FORMS, ids=str)
@pytest.mark.parametrize("Bn,G,Nq", ROWS)
def test_infinite_values_of_a_decoding_step(Bn, G, Nq, kw, d):
    """Inf in a value column that a row sees is Inf in its O, both signs and NaN
    are NaN; the other columns, heads, requests and earlier tokens are as without."""
    Np = 300
    q, kp, vp = _rand((Bn, 2 * G, Nq, d), 1, 2.0), _rand((2, Np, d), 2), _rand((2, Np, d), 3)
    kt, vt = _rand((Bn, 2, 16, d), 4), _rand((Bn, 2, 16, d), 5)
    lens = [min(16, Nq + b % 3) for b in range(Bn)]
    vp[1, Np - 3, 5], vp[1, Np - 9, 20] = INF, -INF
    vp[1, Np - 4, 9], vp[1, Np - 2, 9], vp[1, Np - 7, 33] = INF, -INF, NAN
    for b in range(0, Bn, 3):
        vt[b, 0, lens[b] - 1, 40] = INF   # the last new token's own
        vt[b, 0, lens[b]:] = NAN          # behind the tail
    _shared(q, kp, vp, kt, vt, lens, kw, 6.0)


CAPS = [0.0, 1.0, 20.0, 50.0, 52.0, 60.0]


@pytest.mark.gpu
@pytest.mark.parametrize("size", [1e-17, 1e27, 5e37])
@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("d", [64, 128])
def test_large_and_small_values(d, cap, size):
    """Weights that sum to one leave O within the values, whatever their size."""
    q, k, v = _rand((1, 4, 200, d), 1, 3.0), _rand((1, 2, 333, d), 2), (size * _rand((1, 2, 333, d), 3).clamp(-5, 5)).bfloat16()
    o, lse = pa.attn_fwd_mod(q, k, v, softcap=cap, causal=True, check=True)
    check_same(o, lse, *oracle.attention(q.cpu(), k.cpu(), v.cpu(), d ** -0.5, softcap=cap, causal=True), 5 * size)
    for Bn, G, Nq in ROWS:
        q = _rand((Bn, 2 * G, Nq, d), 4, 3.0)
        kt, vt = _rand((Bn, 2, 20, d), 5), (size * _rand((Bn, 2, 20, d), 6).clamp(-5, 5)).bfloat16()
        _shared(q, k[0], v[0], kt, vt, [min(20, Nq + b % 7) for b in range(Bn)], dict(softcap=cap), 5 * size)


@pytest.mark.gpu
@pytest.mark.parametrize("size", [1e-17, 1e27, 5e37])
@pytest.mark.parametrize("cap", CAPS[1:])
def test_large_and_small_values_at_the_far_end_of_the_cap(cap, size):
    """Every score at -c."""
    q, k = torch.ones((1, 2, 130, 64), dtype=torch.bfloat16, device="cuda"), \
        -100.0 * torch.ones((1, 1, 200, 64), dtype=torch.bfloat16, device="cuda")
    v = (size * _rand((1, 1, 200, 64), 5).clamp(-5, 5)).bfloat16()
    o, lse = pa.attn_fwd_mod(q, k, v, softcap=cap, check=True)
    check_same(o, lse, *oracle.attention(q.cpu(), k.cpu(), v.cpu(), 0.125, softcap=cap), 5 * size)
    for Bn, G in ((2, 4), (2, 80), (300, 1)):
        q = torch.ones((Bn, G, 1, 64), dtype=torch.bfloat16, device="cuda")
        _shared(q, k[0], v[0], k[:, :, :0].expand(Bn, 1, 0, 64), v[:, :, :0].expand(Bn, 1, 0, 64), [0] * Bn,
                dict(softcap=cap), 5 * size)


@pytest.mark.gpu
@pytest.mark.parametrize("kw", FORMS, ids=str)
@pytest.mark.parametrize("mask", [dict(), dict(causal=True), dict(doc_offsets=[[0, 100, 170, 290]]),
                                  dict(causal=True, doc_offsets=[[0, 100, 170, 290]], prefix_lens=[[30, 0, 50]])], ids=str)
@pytest.mark.parametrize("d", [64, 128])
def test_infinite_values_reach_the_rows_that_see_them(d, mask, kw):
    """Inf and NaN in single columns: the same infinity, or NaN, in the rows that
    see them; rows and columns that do not are as without them."""
    q, k, v = _rand((1, 4, 300, d), 1, 2.0), _rand((1, 2, 300, d), 2), _rand((1, 2, 300, d), 3)
    q[:, 0, 150:] *= 0.1
    v[0, 0, 280, 3], v[0, 0, 160, 7], v[0, 0, 165, 7], v[0, 0, 20, 50] = INF, INF, -INF, -INF
    v[0, 1, 99, 0], v[0, 1, 295, 1], v[0, 1, 0, 63] = NAN, NAN, INF
    v[0, 1, 250, :] = INF
    args, host = dict(kw, **mask), dict(kw, **mask)
    if kw.get("slopes"):
        # no weight of a visible key falls out of float32
        args["slopes"] = torch.tensor([0.05, 0.1, 0.15, 0.2], dtype=torch.float32, device="cuda")
        host["slopes"] = args["slopes"].cpu().numpy()
    for n in ("doc_offsets", "prefix_lens"):
        if n in mask:
            args[n] = torch.tensor(mask[n], dtype=torch.int32, device="cuda")
    o, lse = pa.attn_fwd_mod(q, k, v, check=True, **args)
    with np.errstate(invalid="ignore"):
        ref = oracle.attention(q.cpu(), k.cpu(), v.cpu(), d ** -0.5, **host)
    check_same(o, lse, *ref, 6.0)


@pytest.mark.gpu
@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_repaired_rows_keep_a_short_wait_from_running_out(softcap):
    """More items than SMs, values that are not finite hidden from most rows of
    their tile: others wait while a warp does 32 rows again, which the limit allows for."""
    q, k, v = (_rand((2, 30, 4096, 64), s) for s in (1, 2, 3))
    o, lse = pa.attn_fwd_mod(q, k, v, causal=True, softcap=softcap)
    bad = v.clone()
    bad[:, :, 1023::1024] = NAN
    bad[:, :, 1535::1024, ::2] = -INF
    pa.set_wait_limit_ms(1)
    try:
        o2, lse2 = pa.attn_fwd_mod(q, k, bad, causal=True, softcap=softcap, check=True)
    finally:
        pa.set_wait_limit_ms(5000)
    assert (lse2 - lse).abs().max() <= LSE_ABS
    # recomputed rows do not round their weights to bf16: both are 2^-8 from exact
    assert (o2[:, :, :1023].float() - o[:, :, :1023].float()).abs().max() <= 2.0 ** -6 * float(v.abs().max())
    assert torch.isnan(o2[:, :, 1023:]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kw", FORMS, ids=str)
@pytest.mark.parametrize("d", [64, 128])
def test_keys_behind_all_rows_reach_are_left_out(d, kw):
    """What padding and the free end of a cache were left with changes no bit of
    rows that share a key tile with it: it is not even repaired."""
    args = dict(kw, slopes=_slopes(4)) if kw.get("slopes") else kw
    for Nq, Nk, docs, off, end in ((300, 300, [0, 100, 170, 290], 0, 290), (300, 300, [0, 211], 0, 211),
                                   (40, 517, None, 100, 140), (1, 517, None, 127, 128), (1, 517, None, 128, 129),
                                   (1, 517, None, 144, 145), (600, 700, [70, 75], 0, 75), (517, 517, [17, 30, 500], 0, 500)):
        q, k, v = _rand((2, 4, Nq, d), 1, 2.0), _rand((2, 2, Nk, d), 2), _rand((2, 2, Nk, d), 3)
        more = {} if docs is None else dict(doc_offsets=torch.tensor([docs] * 2, dtype=torch.int32, device="cuda"))
        for causal in ((True,) if docs is None else (False, True)):
            o, lse = pa.attn_fwd_mod(q, k, v, causal=causal, q_offset=off, check=True, **args, **more)
            k2, v2 = k.clone(), v.clone()
            k2[:, :, end:], v2[:, :, end:] = NAN, INF
            o2, lse2 = pa.attn_fwd_mod(q, k2, v2, causal=causal, q_offset=off, check=True, **args, **more)
            # causal: rows before the item's last see less than it does, but those keys are real
            assert torch.equal(o, o2) and torch.equal(lse, lse2)
