"""Seeded random shapes, masks, layouts and modifications of attn_fwd_mod and
attn_shared_prefix against a plain float64 evaluation on the GPU (scores, cap,
bias, truth table, softmax, product; the tables from oracle.score_mod's rules,
written with tensor comparisons).  Tolerances as derived in test_score_mod.py.
"""

import random

import pytest
import torch

import context_blocks_b200 as pa
from tests.test_score_mod import LSE_ABS, REL_L2, _rand, _slopes

pytestmark = pytest.mark.gpu


def _attend(q, k, v, seen, pos, key_pos, softcap, slopes):
    """q [H,n,d], k, v [H,m,d], seen [n,m] -> (o, lse) in float64."""
    s = q.double() @ k.double().transpose(1, 2) * q.shape[2] ** -0.5
    if softcap:
        s = softcap * torch.tanh(s / softcap)
    if slopes is not None:
        s = s - slopes.double()[:, None, None] * (pos[:, None] - key_pos[None]).abs().double()
    s = s.masked_fill(~seen, float("-inf"))
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse.masked_fill(lse == float("-inf"), 0.0)[..., None])
    return p @ v.double(), lse


def _close(o, lse, o_ref, l_ref, v_max, what):
    none = l_ref == float("-inf")
    assert torch.equal(none, lse == float("-inf")), what
    assert (o[none] == 0).all(), what
    assert (o.double() - o_ref).abs().max() <= 2.0 ** -7 * v_max, what
    assert (o.double() - o_ref).norm() <= REL_L2 * o_ref.norm() + 1e-30, what
    if (~none).any():
        assert (lse.double() - l_ref)[~none].abs().max() <= LSE_ABS, what


@pytest.mark.parametrize("seed", range(40))
def test_mod(seed):
    r = random.Random(seed)
    Bn, Hkv, G, d = r.choice((1, 2, 3)), r.choice((1, 2, 3)), r.choice((1, 2, 5)), r.choice((64, 128))
    Nk = r.choice((1, 64, 127, 128, 129, 300, 640, 1500))
    Nq = r.choice((1, Nk, max(1, Nk // 3), min(Nk, 257), Nk + 7))
    causal, n_docs = r.random() < 0.6, r.choice((0, 0, 1, 4, 30))
    off = r.choice((Nk - Nq, Nk - Nq, 0, r.randint(-200, 200)))
    softcap, layout = r.choice((0.0, 0.0, 3.0, 30.0, 70.0)), r.choice(("bhnd", "bnhd"))
    q = _rand((Bn, Hkv * G, Nq, d), seed, r.choice((0.5, 3.0)), layout)
    k, v = _rand((Bn, Hkv, Nk, d), seed + 1, 1.0, layout), _rand((Bn, Hkv, Nk, d), seed + 2, 1.0, layout)
    slopes = _slopes(Hkv * G) if r.random() < 0.4 else None
    kw, docs, pre = {}, None, None
    if n_docs:
        end = r.randint(0, Nk)
        docs = [sorted([r.choice((0, r.randint(0, end))), end] + [r.randint(0, end) for _ in range(n_docs - 1)])
                for _ in range(Bn)]
        kw["doc_offsets"] = torch.tensor(docs, dtype=torch.int32, device="cuda")
    if causal and r.random() < 0.4:
        pre = [[r.randint(0, Nk) for _ in range(max(n_docs, 1))] for _ in range(Bn)]
        kw["prefix_lens"] = torch.tensor(pre, dtype=torch.int32, device="cuda")
    o, lse = pa.attn_fwd_mod(q, k, v, softcap=softcap, slopes=slopes, causal=causal, q_offset=off, check=True, **kw)
    pos, key = torch.arange(Nq, device="cuda") + off, torch.arange(Nk, device="cuda")
    what = (Bn, Hkv, G, Nq, Nk, d, causal, n_docs, off, softcap, layout, slopes is not None, pre is not None)
    for b in range(Bn):
        seen = torch.zeros((Nq, Nk), dtype=torch.bool, device="cuda")
        for t, (a, e) in enumerate(zip(docs[b], docs[b][1:]) if docs else [(0, Nk)]):
            inside = (key >= a) & (key < e)
            rows = (pos >= a) & (pos < e) if docs else torch.ones_like(pos, dtype=torch.bool)
            ok = torch.ones((Nq, Nk), dtype=torch.bool, device="cuda")
            if causal:
                ok = (key[None] <= pos[:, None]) | (key < a + (pre[b][t] if pre else 0))[None]
            seen |= rows[:, None] & inside[None] & ok
        o_ref, l_ref = _attend(q[b], k[b].repeat_interleave(G, 0), v[b].repeat_interleave(G, 0), seen, pos, key, softcap,
                               slopes)
        _close(o[b], lse[b], o_ref, l_ref, float(v.abs().max()), what)


@pytest.mark.parametrize("seed", range(40))
def test_shared(seed):
    r = random.Random(1000 + seed)
    Bn, Hkv, G = r.choice((1, 2, 5, 17, 64, 130, 200)), r.choice((1, 2, 3)), r.choice((1, 2, 3, 4, 7, 9))
    Nq, d = r.choice((1, 1, 2, 5, 14)), r.choice((64, 128))
    Np, Nt = r.choice((0, 1, 100, 128, 513, 3000)), r.choice((0, 1, 17, 64, 129, 700))
    softcap, slopes = r.choice((0.0, 0.0, 4.0, 30.0, 70.0)), _slopes(Hkv * G) if r.random() < 0.4 else None
    lens = [r.choice((0, Nt, r.randint(0, Nt))) for _ in range(Bn)]
    q, kp, vp = _rand((Bn, Hkv * G, Nq, d), seed, 2.0), _rand((Hkv, Np, d), seed + 1), _rand((Hkv, Np, d), seed + 2)
    kt, vt = _rand((Bn, Hkv, Nt, d), seed + 3), _rand((Bn, Hkv, Nt, d), seed + 4)
    o, lse = pa.attn_shared_prefix(q, kp, vp, kt, vt, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                   softcap=softcap, slopes=slopes, check=True)
    what = (Bn, Hkv, G, Nq, d, Np, Nt, softcap, slopes is not None)
    for b in range(Bn):
        n = lens[b]
        pos, key = Np + n - Nq + torch.arange(Nq, device="cuda"), torch.arange(Np + n, device="cuda")
        seen = (key[None] < Np) | (key[None] <= pos[:, None])
        k, v = (torch.cat([x, y[b, :, :n]], 1).repeat_interleave(G, 0) for x, y in ((kp, kt), (vp, vt)))
        o_ref, l_ref = _attend(q[b], k, v, seen, pos, key, softcap, slopes)
        _close(o[b], lse[b], o_ref, l_ref, 6.0, what)
