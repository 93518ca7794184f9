"""fp64 oracle of attention with modified scores and interval masks.

NumPy, from the definitions alone: scores, cap, bias, truth table of the mask,
softmax, product.  Hidden keys are dropped by indexing, so whatever they hold
never enters.  Rows that see nothing: o = 0, lse = -inf.
"""

from __future__ import annotations

import numpy as np


def _f64(t):
    return t.detach().float().cpu().double().numpy() if hasattr(t, "detach") else np.asarray(t, dtype=np.float64)


def visible(Nq, Nk, causal=False, prefix=None, offsets=None, q_offset=None):
    """[Nq, Nk] truth table for one batch entry.  ``prefix``: one length, or one
    per document; ``offsets``: the n_docs + 1 document offsets."""
    q_offset = Nk - Nq if q_offset is None else q_offset
    seen = np.zeros((Nq, Nk), dtype=bool)
    docs = [(0, Nk)] if offsets is None else list(zip(offsets[:-1], offsets[1:]))
    pre = [0] * len(docs) if prefix is None else list(np.atleast_1d(prefix))
    for i in range(Nq):
        p = i + q_offset
        for (a, b), n in zip(docs, pre):
            if offsets is not None and not a <= p < b:
                continue
            for j in range(a, b):
                seen[i, j] = (not causal) or j <= p or j < a + n
    return seen


def rows(q, k, v, seen, pos, key_pos, scale, softcap=0.0, slope=None):
    """One head: q [n,d], k, v [m,d], seen [n,m]; (o [n,d], lse [n])."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    o, lse = np.zeros((len(q), v.shape[1])), np.full(len(q), -np.inf)
    for i in range(len(q)):
        j = np.flatnonzero(seen[i])
        if not len(j):
            continue
        s = scale * (k[j] @ q[i])
        if softcap:
            s = softcap * np.tanh(s / softcap)
        if slope is not None:
            s = s - float(slope) * np.abs(pos[i] - key_pos[j])
        m = s.max()
        w = np.exp(s - m)
        lse[i] = m + np.log(w.sum())
        o[i] = (w / w.sum()) @ v[j]
    return o, lse


def attention(q, k, v, scale, softcap=0.0, slopes=None, causal=False, prefix_lens=None, doc_offsets=None,
              q_offset=None):
    """q [B,Hq,Nq,d], k, v [B,Hkv,Nk,d] -> (o, lse) in fp64."""
    B, Hq, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    off = Nk - Nq if q_offset is None else q_offset
    o, lse = np.zeros((B, Hq, Nq, d)), np.zeros((B, Hq, Nq))
    for b in range(B):
        seen = visible(Nq, Nk, causal, None if prefix_lens is None else np.asarray(prefix_lens[b]),
                       None if doc_offsets is None else [int(x) for x in doc_offsets[b]], off)
        for h in range(Hq):
            kv = h // (Hq // Hkv)
            o[b, h], lse[b, h] = rows(q[b, h], k[b, kv], v[b, kv], seen, np.arange(Nq) + off, np.arange(Nk), scale,
                                      softcap, None if slopes is None else slopes[h])
    return o, lse


def shared_prefix(q, k_prefix, v_prefix, k_tail, v_tail, tail_lens, scale, softcap=0.0, slopes=None):
    """q [B,Hq,Nq,d], prefix [Hkv,Np,d], tails [B,Hkv,Nt,d] -> (o, lse): token t
    of request b stands at Np + tail_lens[b] - Nq + t and sees the prefix and
    its own tail up to itself."""
    B, Hq, Nq, d = q.shape
    Hkv, Np = k_prefix.shape[0], k_prefix.shape[1]
    kp, vp, kt, vt = _f64(k_prefix), _f64(v_prefix), _f64(k_tail), _f64(v_tail)
    o, lse = np.zeros((B, Hq, Nq, d)), np.zeros((B, Hq, Nq))
    for b in range(B):
        n = int(tail_lens[b])
        pos = Np + n - Nq + np.arange(Nq)
        key = np.arange(Np + n)
        seen = (key[None] < Np) | (key[None] <= pos[:, None])
        for h in range(Hq):
            kv = h // (Hq // Hkv)
            o[b, h], lse[b, h] = rows(q[b, h], np.concatenate([kp[kv], kt[b, kv, :n]]),
                                      np.concatenate([vp[kv], vt[b, kv, :n]]), seen, pos, key, scale, softcap,
                                      None if slopes is None else slopes[h])
    return o, lse
