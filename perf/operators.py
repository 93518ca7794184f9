"""Cases of the language-model operators, for timing and comparing them.

Three operators stand here, each in a plain form (elementary torch operations
in float32) and as the calls of this package:

``mod``     attention with modified scores (``attn_fwd_mod``): scores capped
            by a tanh, a bias that grows with distance, causal, prefix and
            document masks, grouped heads;
``shared``  attention of a batch of requests that share a long prefix
            (``attn_shared_prefix``): a few new tokens of each request against
            one prefix K/V and the request's own tail K/V;
``norm``    a block's gated residual update with the norms around it
            (``gate_residual_norm``).

``own`` selects: False runs the plain form, True the package's kernels.
"""

import math
import random

import torch

own = False


# --------------------------------------------------------------------- cases
def _mod(name, B, Hq, Hkv, Nq, Nk, d, causal, prefix, docs, pad, softcap, bias, layout, pattern=0):
    """One attention case.  ``prefix``: tokens at the start of each document
    (of the sequence, without documents) that all its tokens see; ``docs``:
    documents packed into each sequence (0: no document mask), ``pad``: keys
    behind the last one; ``layout`` "bhnd" or "bnhd": the order in memory."""
    c = dict(op="mod", B=B, Hq=Hq, Hkv=Hkv, Nq=Nq, Nk=Nk, d=d, causal=causal, prefix=prefix, docs=docs, pad=pad,
             softcap=softcap, bias=bias, layout=layout, pattern=pattern)
    return dict(c, name=name) if name else c


def _shared(name, B, Hq, Hkv, Nq, Np, Nt, d, softcap, bias, pattern=0):
    """One decoding case: Np shared tokens, room for Nt own tokens a request."""
    c = dict(op="shared", B=B, Hq=Hq, Hkv=Hkv, Nq=Nq, Np=Np, Nt=Nt, d=d, softcap=softcap, bias=bias, pattern=pattern)
    return dict(c, name=name) if name else c


def _norm(name, B, N, D, x32, post, norm, gate, modulated, residual_scale):
    c = dict(op="norm", B=B, N=N, D=D, x32=x32, post=post, norm=norm, gate=gate, modulated=modulated,
             residual_scale=residual_scale)
    return dict(c, name=name) if name else c


def listed():
    return [
        # A short prompt of a small model: launch and call latency.
        _mod("mod prompt 67", 1, 8, 2, 67, 67, 64, True, 0, 0, 0, 30.0, False, "bhnd"),
        # FLUX-sized sequence whose 512 text tokens all tokens see, the 4096
        # image tokens generated one after another.
        _mod("mod prefix 4608", 1, 24, 24, 4608, 4608, 128, True, 512, 0, 0, 0.0, False, "bhnd"),
        # Documents packed into one sequence, distance bias instead of positions.
        _mod("mod packed 8192", 1, 24, 8, 8192, 8192, 128, True, 0, 24, 0, 0.0, True, "bnhd", 3),
        # A long prompt with capped scores and grouped heads: the largest.
        _mod("mod capped 8192", 1, 24, 8, 8192, 8192, 128, True, 0, 0, 0, 20.0, False, "bhnd"),
        # A piece of a batch of padded packed sequences, both directions
        # visible inside a document; odd lengths, rows that see nothing.
        _mod("mod piece 1151 of 4603", 2, 24, 4, 1151, 4603, 64, False, 0, 3, 453, 0.0, False, "bnhd", 5),
        # One request, a short shared prompt: latency of a decoding step.
        _shared("shared 1 request", 1, 8, 1, 1, 129, 16, 64, 0.0, False),
        # A serving batch on a common instruction.
        _shared("shared 32 requests", 32, 24, 8, 1, 4608, 1152, 128, 0.0, False, 1),
        # Many requests on one long document, capped scores.
        _shared("shared 128 requests", 128, 32, 8, 1, 32768, 1024, 128, 30.0, False, 2),
        # A HunyuanVideo-long prefix continued seven ways, three drafted tokens a step.
        _shared("shared long prefix", 7, 24, 24, 3, 119056, 333, 128, 0.0, True, 3),
        # One decoding step of a batch: 32 rows.
        _norm("norm 32 rows", 32, 1, 2048, False, "rms", "rms", False, False, 1.0),
        # An image model's block (FLUX 1008^2 tokens), adaptive modulation.
        _norm("norm 2 x 4481", 2, 4481, 1536, False, "none", "layer", True, True, 1.0),
        # A HunyuanVideo-long sequence, residual stream in float32.
        _norm("norm 119056 rows", 1, 119056, 2048, True, "rms", "rms", True, False, 1.0),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("mod", "mod", "shared", "shared", "norm"))
    if op == "mod":
        while True:
            B, Hkv, G = rng.choice((1, 1, 2, 3)), rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4))
            d, Nk = rng.choice((64, 128)), _log(rng, 1, 8192)
            Nq = Nk if rng.random() < 0.6 else _log(rng, 1, Nk)
            if B * Hkv * G * Nq * Nk <= 24 * 8192 * 8192 // 2:
                break
        docs = rng.choice((0, 0, 1, _log(rng, 1, 40)))
        causal = rng.random() < 0.7
        return _mod(None, B, Hkv * G, Hkv, Nq, Nk, d, causal, rng.randint(1, Nk) if causal and rng.random() < 0.4 else 0,
                    docs, rng.randint(0, Nk // 3) if docs else 0, rng.choice((0.0, 0.0, 15.0, 50.0)),
                    rng.random() < 0.3, rng.choice(("bhnd", "bnhd")), rng.randint(0, 1 << 20))
    if op == "shared":
        while True:
            B, Hkv, G = _log(rng, 1, 128), rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 7))
            Nq, Np, Nt = rng.choice((1, 1, 1, 2, 4)), _log(rng, 1, 40000), _log(rng, 4, 2048)
            if Hkv * Np <= 8 * 32768 and B * Hkv * Nt <= 128 * 8 * 1024:
                break
        return _shared(None, B, Hkv * G, Hkv, Nq, Np, Nt, rng.choice((64, 128)), rng.choice((0.0, 0.0, 30.0)),
                       rng.random() < 0.3, rng.randint(0, 1 << 20))
    while True:
        B, N, D = rng.choice((1, 2, 5)), _log(rng, 1, 60000), 8 * _log(rng, 8, 1024)
        if B * N * D <= 119056 * 2048 // 2:
            break
    return _norm(None, B, N, D, rng.random() < 0.4, rng.choice(("none", "rms", "layer")), rng.choice(("rms", "layer")),
                 rng.random() < 0.7, rng.random() < 0.5, rng.choice((1.0, 1.0, 0.5)))


# -------------------------------------------------------------------- inputs
def _doc_offsets(case):
    """[B][docs + 1]: where each packed document begins, cut at random places
    (some documents are short, a few empty); the last ends at Nk - pad."""
    r = random.Random(case["pattern"])
    end = case["Nk"] - case["pad"]
    return [sorted([0, end] + [r.randint(0, end) for _ in range(case["docs"] - 1)]) for _ in range(case["B"])]


def _tail_lens(case):
    """[B]: tokens in each request's tail, the new ones among them; one in
    sixteen requests has none (it left the batch)."""
    r = random.Random(case["pattern"])
    return [0 if r.random() < 1 / 16 else r.randint(min(case["Nq"], case["Nt"]), case["Nt"]) for _ in range(case["B"])]


def _slopes(H, device):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=torch.float32, device=device)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def rows(*shape, gain=1.0):
        """Rows normalised to rms 1, as attention gets its queries and keys."""
        x = torch.randn(shape, generator=g, device=dev)
        return (gain * x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()

    def normal(*shape, std=1.0):
        return (std * torch.randn(shape, generator=g, device=dev)).bfloat16()

    s = dict(case=case)
    if case["op"] == "mod":
        B, Hq, Hkv, Nq, Nk, d = (case[n] for n in ("B", "Hq", "Hkv", "Nq", "Nk", "d"))
        if case["layout"] == "bnhd":  # as a projection leaves them: heads inside tokens
            q, k, v = (t.transpose(1, 2) for t in (rows(B, Nq, Hq, d, gain=3.0), rows(B, Nk, Hkv, d), normal(B, Nk, Hkv, d)))
        else:
            q, k, v = rows(B, Hq, Nq, d, gain=3.0), rows(B, Hkv, Nk, d), normal(B, Hkv, Nk, d)
        s.update(q=q, k=k, v=v, slopes=_slopes(Hq, dev) if case["bias"] else None, doc_offsets=None, prefix_lens=None)
        if case["docs"]:
            s["doc_offsets"] = torch.tensor(_doc_offsets(case), dtype=torch.int32, device=dev)
        if case["prefix"]:
            s["prefix_lens"] = torch.full((B, max(1, case["docs"])), case["prefix"], dtype=torch.int32, device=dev)
    elif case["op"] == "shared":
        B, Hq, Hkv, Nq, Np, Nt, d = (case[n] for n in ("B", "Hq", "Hkv", "Nq", "Np", "Nt", "d"))
        s.update(q=rows(B, Hq, Nq, d, gain=3.0), kp=rows(Hkv, Np, d), vp=normal(Hkv, Np, d), kt=rows(B, Hkv, Nt, d),
                 vt=normal(B, Hkv, Nt, d), tail_lens=torch.tensor(_tail_lens(case), dtype=torch.int32, device=dev),
                 slopes=_slopes(Hq, dev) if case["bias"] else None)
    else:
        B, N, D = case["B"], case["N"], case["D"]
        y, x = normal(B, N, D, std=2.0), 3.0 * torch.randn((B, N, D), generator=g, device=dev)
        s.update(y=y, x=x if case["x32"] else x.bfloat16(), gate=None, scale=None, shift=None, post_weight=None,
                 norm_weight=None)
        table = normal(B, 3 * D, std=0.5)  # the modulation, as one projection leaves it
        if case["gate"]:
            s["gate"] = table[:, :D]
        if case["modulated"]:
            s["scale"], s["shift"] = table[:, D:2 * D], table[:, 2 * D:]
        if case["post"] == "rms":
            s["post_weight"] = (1.0 + 0.2 * torch.randn(D, generator=g, device=dev)).bfloat16()
        if case["norm"] == "rms":
            s["norm_weight"] = (1.0 + 0.2 * torch.randn(D, generator=g, device=dev)).bfloat16()
    return s


# --------------------------------------------------------------- plain forms
def _softmax_v(s, v):
    """(o, lse) of scores s [.., n, keys] whose hidden entries are -inf."""
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(l > 0, l, torch.ones_like(l))
    return o, torch.where(l > 0, m + l.log(), torch.full_like(l, -math.inf)).squeeze(-1)


def _visible(case, st):
    """[B, 1, Nq, Nk] truth values: which keys a query sees; None: all."""
    B, Nq, Nk = case["B"], case["Nq"], case["Nk"]
    dev = st["q"].device
    key = torch.arange(Nk, device=dev)
    row = torch.arange(Nq, device=dev) + (Nk - Nq)
    seen = None
    if st["doc_offsets"] is not None:
        off = st["doc_offsets"].long()
        doc = (key[None, :, None] >= off[:, None, :]).sum(-1) - 1  # [B, Nk]; behind the last one: docs
        start = off.gather(1, doc.clamp(max=case["docs"]))
        real = doc < case["docs"]
        seen = (doc[:, row][:, :, None] == doc[:, None, :]) & real[:, None, :]
    else:
        start = torch.zeros((B, Nk), dtype=torch.long, device=dev)
        doc = torch.zeros((B, Nk), dtype=torch.long, device=dev)
    if case["causal"]:
        past = (key[None, :] <= row[:, None])[None]
        if st["prefix_lens"] is not None:
            n = st["prefix_lens"].long().gather(1, doc.clamp(max=max(1, case["docs"]) - 1))  # [B, Nk]
            past = past | (key[None] < start + n)[:, None, :]
        seen = past if seen is None else seen & past
    return None if seen is None else seen[:, None]


def _plain_mod(st):
    c = st["case"]
    B, Hq, Hkv, Nq, Nk, d = (c[n] for n in ("B", "Hq", "Hkv", "Nq", "Nk", "d"))
    G = Hq // Hkv
    q = st["q"].float().reshape(B, Hkv, G * Nq, d)
    k, v = st["k"].float(), st["v"].float()
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).view(B, Hq, Nq, Nk)
    if c["softcap"]:
        s = s.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    if st["slopes"] is not None:
        row = torch.arange(Nq, device=s.device, dtype=torch.float32) + (Nk - Nq)
        far = (row[:, None] - torch.arange(Nk, device=s.device, dtype=torch.float32)[None, :]).abs()
        s = s.sub_(st["slopes"][:, None, None] * far)
    seen = _visible(c, st)
    if seen is not None:
        s = s.masked_fill_(~seen, -math.inf)
    o, lse = _softmax_v(s.view(B, Hkv, G * Nq, Nk), v)
    return o.view(B, Hq, Nq, d).bfloat16(), lse.view(B, Hq, Nq)


def _plain_shared(st):
    c = st["case"]
    B, Hq, Hkv, Nq, Np, Nt, d = (c[n] for n in ("B", "Hq", "Hkv", "Nq", "Np", "Nt", "d"))
    G = Hq // Hkv
    q = st["q"].float().view(B, Hkv, G * Nq, d)
    dev = q.device
    scale = 1.0 / math.sqrt(d)
    # Scores against the prefix, once for all requests: one product a K/V head.
    sp = torch.matmul(q.transpose(0, 1).reshape(Hkv, B * G * Nq, d), st["kp"].float().transpose(-1, -2))
    sp = sp.view(Hkv, B, G, Nq, Np).mul_(scale)
    s_t = torch.matmul(q, st["kt"].float().transpose(-1, -2)).view(B, Hkv, G, Nq, Nt).mul_(scale)
    if c["softcap"]:
        sp = sp.div_(c["softcap"]).tanh_().mul_(c["softcap"])
        s_t = s_t.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    # A new token's own index in the tail; the last one is the tail's last.
    at = st["tail_lens"].long()[:, None] - Nq + torch.arange(Nq, device=dev)  # [B, Nq]
    if st["slopes"] is not None:
        sl = st["slopes"].view(Hkv, G)
        far = (at + Np)[:, :, None].float() - torch.arange(Np, device=dev, dtype=torch.float32)  # [B, Nq, Np]
        sp = sp.sub_(sl[:, None, :, None, None] * far.abs()[None, :, None])
        far = at[:, :, None].float() - torch.arange(Nt, device=dev, dtype=torch.float32)
        s_t = s_t.sub_(sl[None, :, :, None, None] * far.abs()[:, None, None])
    hidden = torch.arange(Nt, device=dev) > at[:, :, None]  # [B, Nq, Nt]
    s_t = s_t.masked_fill_(hidden[:, None, None], -math.inf)
    o_p, l_p = _softmax_v(sp.view(Hkv, B * G * Nq, Np), st["vp"].float())
    o_p = o_p.view(Hkv, B, G, Nq, d).transpose(0, 1)
    l_p = l_p.view(Hkv, B, G, Nq).transpose(0, 1)
    o_t, l_t = _softmax_v(s_t.view(B, Hkv, G * Nq, Nt), st["vt"].float())
    o_t, l_t = o_t.view(B, Hkv, G, Nq, d), l_t.view(B, Hkv, G, Nq)
    m = torch.maximum(l_p, l_t)
    w_p, w_t = (l_p - m).exp(), (l_t - m).exp()
    o = (w_p[..., None] * o_p + w_t[..., None] * o_t) / (w_p + w_t)[..., None]
    return o.reshape(B, Hq, Nq, d).bfloat16(), (m + (w_p + w_t).log()).reshape(B, Hq, Nq)


EPS = 1e-6


def _plain_normed(x, kind, weight):
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    if kind != "none":
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x if weight is None else x * weight.float()


def _plain_norm(st):
    c = st["case"]
    t = _plain_normed(st["y"].float(), c["post"], st["post_weight"])
    if st["gate"] is not None:
        t = t * st["gate"].float()[:, None]
    x = c["residual_scale"] * st["x"].float() + t
    h = _plain_normed(x, c["norm"], st["norm_weight"])
    if st["scale"] is not None:
        h = h * (1.0 + st["scale"].float()[:, None]) + st["shift"].float()[:, None]
    return x.to(st["x"].dtype), h.bfloat16()


def run(state):
    c = state["case"]
    if own:
        import context_blocks_b200 as pa
        if c["op"] == "mod":
            return pa.attn_fwd_mod(state["q"], state["k"], state["v"], softcap=c["softcap"], slopes=state["slopes"],
                                   causal=c["causal"], prefix_lens=state["prefix_lens"],
                                   doc_offsets=state["doc_offsets"])
        if c["op"] == "shared":
            return pa.attn_shared_prefix(state["q"], state["kp"], state["vp"], state["kt"], state["vt"],
                                         state["tail_lens"], softcap=c["softcap"], slopes=state["slopes"])
        return pa.gate_residual_norm(state["y"], state["x"], gate=state["gate"], post=c["post"],
                                     post_weight=state["post_weight"], norm=c["norm"],
                                     norm_weight=state["norm_weight"], scale=state["scale"], shift=state["shift"],
                                     residual_scale=c["residual_scale"], eps=EPS)
    if c["op"] == "mod":
        return _plain_mod(state)
    if c["op"] == "shared":
        return _plain_shared(state)
    return _plain_norm(state)


# ---------------------------------------------------------------------- work
def _pairs(case):
    """Query-key pairs that count, over the batch, for one query head."""
    Nq, Nk = case["Nq"], case["Nk"]
    docs = _doc_offsets(case) if case["docs"] else [[0, Nk]] * case["B"]
    pairs = 0
    for off in docs:
        for a, b in zip(off, off[1:]):
            lo, hi = max(a, Nk - Nq), b  # rows of this document that are asked for
            if hi <= lo:
                continue
            if not case["causal"]:
                pairs += (hi - lo) * (b - a)
            else:
                w = min(b, a + case["prefix"])  # rows before w see [a, w), later ones [a, row]
                first = max(lo, w)
                pairs += max(0, min(hi, w) - lo) * (w - a)
                pairs += (hi - first) * (first + hi - 1 + 2 * (1 - a)) // 2 if hi > first else 0
    return pairs


def work(case):
    if case["op"] == "mod":
        B, Hq, Hkv, Nq, Nk, d = (case[n] for n in ("B", "Hq", "Hkv", "Nq", "Nk", "d"))
        return {"bytes": 2.0 * B * d * (2 * Hq * Nq + 2 * Hkv * Nk) + 4.0 * B * Hq * Nq,
                "flops": 4.0 * d * Hq * _pairs(case)}
    if case["op"] == "shared":
        B, Hq, Hkv, Nq, Np, d = (case[n] for n in ("B", "Hq", "Hkv", "Nq", "Np", "d"))
        lens = _tail_lens(case)
        return {"bytes": 4.0 * d * Hkv * (Np + sum(lens)) + B * Hq * Nq * (4.0 * d + 4),
                "flops": 4.0 * d * Hq * Nq * (B * Np + sum(lens))}
    n = case["B"] * case["N"] * case["D"]
    return {"bytes": n * (12.0 if case["x32"] else 8.0), "flops": 10.0 * n}


# --------------------------------------------------------------------- exact
def _exact_rows(q, k, v, lo, hi, pos, key_pos, softcap, slope):
    """One head in 64 bits: row i of q sees keys lo[i] <= j < hi[i]."""
    s = torch.einsum("id,jd->ij", q.double(), k.double()) * (q.shape[1] ** -0.5)
    if softcap:
        s = softcap * torch.tanh(s / softcap)
    if slope is not None:
        s = s - slope.double() * (pos[:, None] - key_pos[None, :]).abs().double()
    j = torch.arange(k.shape[0], device=q.device)
    s[(j[None] < lo[:, None]) | (j[None] >= hi[:, None])] = -math.inf
    lse = torch.logsumexp(s, 1)
    p = torch.exp(s - lse[:, None]).nan_to_num_(0.0)  # a row that sees nothing: -inf - -inf
    return p @ v.double(), lse


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        y, x = st["y"].double(), st["x"].double()

        def normed(t, kind, w):
            if kind == "layer":
                t = (t - t.mean(-1, keepdim=True)) / torch.sqrt(t.var(-1, unbiased=False, keepdim=True) + EPS)
            elif kind == "rms":
                t = t / torch.sqrt((t * t).mean(-1, keepdim=True) + EPS)
            return t if w is None else t * w.double()

        t = normed(y, case["post"], st["post_weight"])
        x = x * case["residual_scale"] + (t if st["gate"] is None else t * st["gate"].double()[:, None, :])
        h = normed(x, case["norm"], st["norm_weight"])
        if case["modulated"]:
            h = h + h * st["scale"].double()[:, None, :] + st["shift"].double()[:, None, :]
        return x, h
    q, dev = st["q"], st["q"].device
    B, Hq, Nq, d = q.shape
    G = Hq // case["Hkv"]
    o = torch.empty((B, Hq, Nq, d), dtype=torch.float64, device=dev)
    lse = torch.empty((B, Hq, Nq), dtype=torch.float64, device=dev)
    lens = _tail_lens(case) if case["op"] == "shared" else None
    for b in range(B):
        if case["op"] == "shared":
            Np, n = case["Np"], lens[b]
            pos = Np + n - Nq + torch.arange(Nq, device=dev)
            lo = torch.zeros(Nq, dtype=torch.long, device=dev)
            hi = torch.clamp(pos + 1, min=Np)
            key_pos = torch.arange(Np + n, device=dev)
        else:
            Nk = case["Nk"]
            pos = torch.arange(Nk - Nq, Nk, device=dev)
            key_pos = torch.arange(Nk, device=dev)
            lo, hi = torch.zeros(Nq, dtype=torch.long), torch.zeros(Nq, dtype=torch.long)
            off = _doc_offsets(case)[b] if case["docs"] else [0, Nk]
            for s0, s1 in zip(off, off[1:]):  # rows of this document: [s0, s1)
                r = torch.arange(max(s0, Nk - Nq), max(s1, Nk - Nq))
                at = r - (Nk - Nq)
                lo[at] = s0
                hi[at] = torch.clamp(r + 1, min=min(s1, s0 + case["prefix"])) if case["causal"] else s1
            lo, hi = lo.to(dev), hi.to(dev)
        for h in range(Hq):
            if case["op"] == "shared":
                k = torch.cat([st["kp"][h // G], st["kt"][b, h // G, :lens[b]]])
                v = torch.cat([st["vp"][h // G], st["vt"][b, h // G, :lens[b]]])
            else:
                k, v = st["k"][b, h // G], st["v"][b, h // G]
            o[b, h], lse[b, h] = _exact_rows(q[b, h], k, v, lo, hi, pos, key_pos, case["softcap"],
                                             None if st["slopes"] is None else st["slopes"][h])
    return o, lse
