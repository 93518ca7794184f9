"""pa_attn_shared_prefix against the fp64 oracle on the GPU, its refusals on the
CPU, and prefill and decoding together.  Tolerances as derived in
tests/test_score_mod.py: the partial results are joined in fp32, which adds
nothing that counts beside the roundings of P and O.
"""

import ctypes

import pytest
import torch

import context_blocks_b200 as pa
from context_blocks_b200 import _binding as B
from oracle import score_mod as oracle
from tests.test_score_mod import LSE_ABS, _rand, _slopes, check_close


def _case(Bn, Hq, Hkv, Nq, Np, Nt, d, lens, seed, softcap=0.0, slopes=False):
    q, kp, vp = _rand((Bn, Hq, Nq, d), seed, 2.0), _rand((Hkv, Np, d), seed + 1), _rand((Hkv, Np, d), seed + 2)
    kt, vt = _rand((Bn, Hkv, Nt, d), seed + 3), _rand((Bn, Hkv, Nt, d), seed + 4)
    sl = _slopes(Hq) if slopes else None
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = pa.attn_shared_prefix(q, kp, vp, kt, vt, n, softcap=softcap, slopes=sl, check=True)
    o_ref, l_ref = oracle.shared_prefix(q, kp, vp, kt, vt, lens, d ** -0.5, softcap,
                                        None if sl is None else sl.cpu().numpy())
    check_close(o, lse, o_ref, l_ref, 6.0)
    return q, kp, vp, kt, vt, n, o, lse


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Bn,Hq,Hkv,Nq", [(1, 1, 1, 1), (3, 4, 2, 1), (5, 8, 1, 3), (2, 16, 1, 8), (40, 4, 1, 1)])
@pytest.mark.parametrize("Np,Nt", [(1, 1), (130, 20), (300, 129), (517, 300)])
def test_sizes(d, Bn, Hq, Hkv, Nq, Np, Nt):
    lens = [(37 * b + Nt) % (Nt + 1) for b in range(Bn)]
    _case(Bn, Hq, Hkv, Nq, Np, Nt, d, lens, seed=Np + Nt + Bn)


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(softcap=4.0), dict(slopes=True), dict(softcap=4.0, slopes=True)], ids=str)
@pytest.mark.parametrize("d", [64, 128])
def test_modified_scores(kw, d):
    _case(7, 6, 2, 2, 700, 260, d, [260, 0, 1, 2, 128, 129, 200], seed=3, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[0, 0, 0], [0, 5, 0], [128, 127, 129], [1, 1, 1], [300, 0, 256]])
@pytest.mark.parametrize("Np", [0, 200])
def test_lengths(lens, Np):
    """Empty tails, no prefix, rows that see nothing (no prefix and no tail)."""
    _case(3, 4, 2, 1, Np, 300, 64, lens, seed=11)
    _case(3, 4, 2, 4, Np, 300, 128, lens, seed=12, slopes=True)


@pytest.mark.gpu
def test_no_tail_at_all():
    _case(3, 4, 2, 2, 300, 0, 64, [0, 0, 0], seed=13)
    _case(3, 4, 2, 2, 0, 0, 64, [0, 0, 0], seed=14)


@pytest.mark.gpu
@pytest.mark.parametrize("Bn,G,Nq", [(1, 128, 1), (3, 8, 16), (70, 1, 1), (257, 1, 1), (33, 4, 2), (5, 25, 1)])
def test_row_tiles(Bn, G, Nq):
    """One row tile, a pair, an odd number of them, tiles that are not full."""
    _case(Bn, 2 * G if Bn < 10 else G, 2 if Bn < 10 else 1, Nq, 400, 140, 64, [(13 * b) % 141 for b in range(Bn)], seed=15)


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(), dict(softcap=4.0), dict(softcap=60.0), dict(slopes=True),
                                dict(softcap=4.0, slopes=True)], ids=str)
@pytest.mark.parametrize("Bn,G", [(40, 4), (70, 4), (100, 7)])
def test_pairs_of_row_tiles(Bn, G, kw):
    """Two row tiles, five (two pairs and an odd one), six; several key tiles."""
    _case(Bn, 2 * G, 2, 1, 900, 70, 128, [(7 * b) % 71 for b in range(Bn)], seed=16, **kw)


@pytest.mark.gpu
def test_more_pairs_than_ctas():
    """300 row tiles of 128 rows: every CTA has a pair or more to itself.  All rows
    see the whole prefix, so the unmasked forward is the reference."""
    q, kp, vp = _rand((300, 8, 16, 64), 1, 2.0), _rand((1, 300, 64), 2), _rand((1, 300, 64), 3)
    none = torch.zeros((300, 1, 0, 64), dtype=torch.bfloat16, device="cuda")
    o, lse = pa.attn_shared_prefix(q, kp, vp, none, none, torch.zeros(300, dtype=torch.int32, device="cuda"), check=True)
    o2, lse2 = pa.attn_fwd(q.view(1, 1, -1, 64), kp[None], vp[None])
    assert (lse.view(-1) - lse2.view(-1)).abs().max() <= LSE_ABS
    assert (o.view(-1, 64).float() - o2.view(-1, 64).float()).abs().max() <= 2.0 ** -6 * float(vp.abs().max())


@pytest.mark.gpu
@pytest.mark.parametrize("Bn,Hkv,Nt", [(20, 8, 16), (37, 4, 40), (3, 2, 700), (61, 8, 129)])
@pytest.mark.parametrize("Np", [0, 150, 8000])
def test_short_tails_in_many_parts(Bn, Hkv, Nt, Np):
    """About as many units of work as parts, and with the long prefix the tails'
    starts among them: parts that hold a start alone, tails that are cut before
    each of their tiles."""
    _case(Bn, Hkv, Hkv, 1, Np, Nt, 64, [(b * 17) % Nt + 1 for b in range(Bn)], seed=18)


@pytest.mark.gpu
def test_two_streams_at_once():
    """Calls that overlap on the GPU, each with a workspace of its own."""
    cases = [(_rand((20, 4, 1, 64), 10 * i, 2.0), *(_rand((2, 3000, 64), 10 * i + j) for j in (1, 2)),
              *(_rand((20, 2, 300, 64), 10 * i + j) for j in (3, 4)),
              torch.tensor([(31 * b) % 301 for b in range(20)], dtype=torch.int32, device="cuda")) for i in range(2)]
    want = [pa.attn_shared_prefix(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[pa.attn_shared_prefix(*c, stream=s) for _ in range(5)] for c, s in zip(cases, streams)]
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for o, lse in g:
            assert torch.equal(o, w[0]) and torch.equal(lse, w[1])
    assert pa.poll_device_status() == pa.PA_OK


@pytest.mark.gpu
def test_long_keys_over_many_ctas():
    """Few rows, long keys: every segment is cut over several CTAs.  Against the
    package's unmasked attention over the same keys."""
    q, kp, vp = _rand((1, 4, 1, 128), 1, 2.0), _rand((4, 40000, 128), 2), _rand((4, 40000, 128), 3)
    kt, vt = _rand((1, 4, 3001, 128), 4), _rand((1, 4, 3001, 128), 5)
    n = torch.tensor([3000], dtype=torch.int32, device="cuda")
    o, lse = pa.attn_shared_prefix(q, kp, vp, kt, vt, n, check=True)
    o2, lse2 = pa.attn_fwd(q, torch.cat([kp[None], kt[:, :, :3000]], 2), torch.cat([vp[None], vt[:, :, :3000]], 2))
    assert (lse - lse2).abs().max() <= LSE_ABS
    # both round P and O to bf16: twice the bound of one
    assert (o.float() - o2.float()).norm() <= 2e-2 * o2.float().norm()


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 3e38])
@pytest.mark.parametrize("Nq", [1, 3])
def test_what_lies_behind_a_tail_does_not_matter(bad, Nq):
    lens = [17, 128, 0, 250, 3]
    q, kp, vp, kt, vt, n, o, lse = _case(5, 4, 2, Nq, 200, 300, 128, lens, seed=21)
    for b, m in enumerate(lens):
        kt[b, :, m:] = bad
        vt[b, :, m:] = bad
    o2, lse2 = pa.attn_shared_prefix(q, kp, vp, kt, vt, n, check=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.gpu
def test_a_later_token_does_not_reach_an_earlier_one():
    lens = [17, 129, 250]
    q, kp, vp, kt, vt, n, o, lse = _case(3, 4, 2, 3, 200, 300, 64, lens, seed=22)
    for b, m in enumerate(lens):
        kt[b, :, m - 1] = float("nan")
        vt[b, :, m - 1] = float("inf")
    o2, lse2 = pa.attn_shared_prefix(q, kp, vp, kt, vt, n, check=True)
    assert (lse2[:, :, :2] - lse[:, :, :2]).abs().max() <= LSE_ABS
    assert (o2[:, :, :2].float() - o[:, :, :2].float()).abs().max() <= 2.0 ** -6 * 6.0


@pytest.mark.gpu
def test_prefill_then_decode():
    """A run as it is used: the prompt through attn_fwd_mod, then each request's
    tokens through attn_shared_prefix, equals one causal pass over everything;
    and a partial over the prefix merges with one over the tail."""
    Hq, Hkv, d, Np, T = 6, 2, 128, 333, 5
    sl = _slopes(Hq)
    seq = [_rand((1, h, Np + T, d), s, g) for h, s, g in ((Hq, 1, 2.0), (Hkv, 2, 1.0), (Hkv, 3, 1.0))]
    q, k, v = seq
    want, lwant = pa.attn_fwd_mod(q, k, v, causal=True, softcap=15.0, slopes=sl)
    kt = torch.zeros((1, Hkv, 16, d), dtype=torch.bfloat16, device="cuda")
    vt = torch.zeros_like(kt)
    for t in range(T):
        kt[:, :, t], vt[:, :, t] = k[:, :, Np + t], v[:, :, Np + t]
        n = torch.tensor([t + 1], dtype=torch.int32, device="cuda")
        o, lse = pa.attn_shared_prefix(q[:, :, Np + t:Np + t + 1].contiguous(), k[0, :, :Np], v[0, :, :Np], kt, vt, n,
                                       softcap=15.0, slopes=sl, check=True)
        assert (lse[:, :, 0] - lwant[:, :, Np + t]).abs().max() <= LSE_ABS
        assert (o[:, :, 0].float() - want[:, :, Np + t].float()).abs().max() <= 2.0 ** -6 * 6.0
    # the last T tokens at once, and as two parts joined by attn_merge
    n = torch.tensor([T], dtype=torch.int32, device="cuda")
    qs = q[:, :, Np:].contiguous()
    o, lse = pa.attn_shared_prefix(qs, k[0, :, :Np], v[0, :, :Np], kt, vt, n, softcap=15.0, slopes=sl, check=True)
    assert (lse - lwant[:, :, Np:]).abs().max() <= LSE_ABS
    parts = [pa.attn_fwd_mod(qs, kk, vv, causal=True, softcap=15.0, slopes=sl, q_offset=off)
             for kk, vv, off in ((k[:, :, :Np], v[:, :, :Np], Np), (k[:, :, Np:], v[:, :, Np:], 0))]
    om, lm = pa.attn_merge(torch.stack([a.contiguous() for a, _ in parts]), torch.stack([b for _, b in parts]))
    assert (lm - lse).abs().max() <= LSE_ABS
    assert (om.float() - o.float()).abs().max() <= 2.0 ** -6 * 6.0


@pytest.mark.gpu
def test_strided_caches():
    """Tails as [B, Nt, Hkv, d] and the prefix as a slice of a longer cache."""
    q, cache = _rand((3, 4, 1, 64), 1, 2.0), _rand((2, 2, 500, 64), 2)
    kp, vp = cache[0][:, 100:400], cache[1][:, 100:400]
    kt, vt = _rand((3, 2, 50, 64), 3, layout="bnhd"), _rand((3, 2, 50, 64), 4, layout="bnhd")
    lens = [50, 7, 0]
    o, lse = pa.attn_shared_prefix(q, kp, vp, kt, vt, torch.tensor(lens, dtype=torch.int32, device="cuda"), check=True)
    o_ref, l_ref = oracle.shared_prefix(q, kp, vp, kt, vt, lens, 0.125)
    check_close(o, lse, o_ref, l_ref, 6.0)


@pytest.mark.gpu
def test_captured_replayed_with_new_lengths_and_on_another_stream():
    q, kp, vp, kt, vt, n, o, lse = _case(3, 4, 2, 1, 300, 200, 64, [10, 100, 200], seed=31)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o2, lse2 = pa.attn_shared_prefix(q, kp, vp, kt, vt, n, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    ws = torch.empty(pa.shared_prefix_workspace_bytes(3, 4, 2, 1, 300, 200, 64), dtype=torch.uint8, device="cuda")
    og, lg = torch.empty_like(o), torch.empty_like(lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.attn_shared_prefix(q, kp, vp, kt, vt, n, out=og, lse=lg, workspace=ws)
    for lens in ([10, 100, 200], [11, 0, 129], [200, 200, 1]):
        n.copy_(torch.tensor(lens, dtype=torch.int32))
        ws.fill_(0xff)
        g.replay()
        want = pa.attn_shared_prefix(q, kp, vp, kt, vt, n)
        torch.cuda.synchronize()
        assert torch.equal(og, want[0]) and torch.equal(lg, want[1])


@pytest.mark.gpu
def test_lengths_out_of_range_are_reported():
    q, kp, vp, kt, vt, n, o, lse = _case(3, 4, 2, 1, 300, 200, 64, [0, 100, 200], seed=32)
    n.copy_(torch.tensor([-5, 100, 1 << 30], dtype=torch.int32))
    o2, lse2 = pa.attn_shared_prefix(q, kp, vp, kt, vt, n)
    torch.cuda.synchronize()
    assert pa.poll_device_status() == pa.PA_ERR_BAD_INPUT
    assert torch.equal(o, o2) and torch.equal(lse, lse2)  # clamped to [0, Nt]


@pytest.mark.gpu
def test_refusals_of_the_binding():
    q, kp, kt = _rand((2, 4, 1, 64), 1), _rand((2, 8, 64), 2), _rand((2, 2, 8, 64), 3)
    n = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    ok = dict(q=q, k_prefix=kp, v_prefix=kp, k_tail=kt, v_tail=kt, tail_lens=n)
    for bad in (dict(q=q.float()), dict(tail_lens=n.long()), dict(tail_lens=n[:1]), dict(k_tail=kt[:1]),
                dict(v_prefix=kp[:, :4]), dict(slopes=_slopes(2)), dict(q=q[:, :3].contiguous()),
                dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
                dict(q=_rand((2, 4, 65, 64), 1)), dict(out=kt), dict(tail_lens=n.cpu()),
                dict(q=_rand((2, 4, 2, 64), 1, layout="bnhd"))):
        with pytest.raises((TypeError, ValueError, pa.PaError)):
            pa.attn_shared_prefix(**dict(ok, **bad))
    o, lse = pa.attn_shared_prefix(**dict(ok, q=q[:, :, :0].contiguous()))
    assert o.numel() == 0 and lse.numel() == 0


A, MB = 1 << 20, 1 << 24


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), B.PA_ERR_INVALID_ARG), (dict(kp=0), B.PA_ERR_INVALID_ARG), (dict(vt=0), B.PA_ERR_INVALID_ARG),
    (dict(lens=0), B.PA_ERR_INVALID_ARG), (dict(lse=0), B.PA_ERR_INVALID_ARG), (dict(ws=0), B.PA_ERR_INVALID_ARG),
    (dict(wsb=1000), B.PA_ERR_INVALID_ARG), (dict(ws=A + 8 * MB + 8), B.PA_ERR_MISALIGNED),
    (dict(kt=A + 3 * MB + 8), B.PA_ERR_MISALIGNED), (dict(lens=A + 5 * MB + 2), B.PA_ERR_MISALIGNED),
    (dict(Hkv=3), B.PA_ERR_INVALID_ARG), (dict(Np=-1), B.PA_ERR_INVALID_ARG), (dict(Nt=-1), B.PA_ERR_INVALID_ARG),
    (dict(Nq=65), B.PA_ERR_UNSUPPORTED), (dict(d=32), B.PA_ERR_UNSUPPORTED), (dict(Np=1 << 30), B.PA_ERR_UNSUPPORTED),
    (dict(Bn=20000), B.PA_ERR_UNSUPPORTED), (dict(cap=-1.0), B.PA_ERR_INVALID_ARG), (dict(cap=1e-20), B.PA_ERR_INVALID_ARG),
    (dict(slopes=A + 1), B.PA_ERR_MISALIGNED), (dict(o=A), B.PA_ERR_INVALID_ARG), (dict(ws=A + MB), B.PA_ERR_INVALID_ARG),
    (dict(strides=[1024, 0, 1024, 128, 2048, 1024, 128, 2048, 1024, 128]), B.PA_ERR_INVALID_ARG),
    (dict(strides=[1024, 128, 1024, 128, 2048, 1024, 132, 2048, 1024, 128]), B.PA_ERR_MISALIGNED),
    (dict(Nq=0), B.PA_OK),
])
def test_argument_checks(kw, code):
    lib = B.load_library()
    a = dict(dict(q=A, kp=A + MB, vp=A + 2 * MB, kt=A + 3 * MB, vt=A + 4 * MB, lens=A + 5 * MB, o=A + 6 * MB,
                  lse=A + 7 * MB, Bn=2, Hq=4, Hkv=2, Nq=1, Np=8, Nt=8, d=128, strides=None, cap=0.0, slopes=None,
                  ws=A + 8 * MB, wsb=1 << 23), **kw)
    st = (ctypes.c_longlong * 10)(*a["strides"]) if a["strides"] else None
    rc = lib.pa_attn_shared_prefix(a["q"], a["kp"], a["vp"], a["kt"], a["vt"], a["lens"], a["o"], a["lse"], a["Bn"],
                                   a["Hq"], a["Hkv"], a["Nq"], a["Np"], a["Nt"], a["d"], st, 0.125, a["cap"],
                                   a["slopes"], a["ws"], a["wsb"], None)
    assert rc == code, B.last_error()


def test_workspace_sizes():
    size = B.shared_prefix_workspace_bytes
    assert size(2, 4, 2, 1, 8, 8, 128) > 0
    assert size(2, 4, 2, 1, 0, 0, 128) == 0
    assert size(2, 4, 3, 1, 8, 8, 128) == 0 and size(2, 4, 2, 65, 8, 8, 128) == 0 and size(0, 4, 2, 1, 8, 8, 128) == 0
    assert size(2, 4, 2, 1, 8, 8, 128) > size(2, 4, 2, 1, 8, 0, 128) > 0
    assert size(2, 4, 2, 1, 8, 8, 128) < 1 << 23


def _line(total_tiles, ctas):
    parts = max(min(total_tiles, ctas), 1)
    q, r = divmod(total_tiles, parts)
    return [(c * q + min(c, r), (c + 1) * q + min(c + 1, r)) for c in range(parts)]


@pytest.mark.parametrize("start", [0, 1])
@pytest.mark.parametrize("segs", [[3, 1, 4, 1, 5], [0, 0, 7, 0], [1] * 400, [1000], [37, 0, 2, 511, 1]])
@pytest.mark.parametrize("ctas", [1, 5, 148])
def test_pieces_have_slots_of_their_own(segs, ctas, start):
    """The arithmetic that places partial results: cut the line of key tiles (with
    ``start`` units before each segment that has any) into equal parts, name a
    piece by segment + part, and no two pieces share a name, none is past
    segments + parts, every tile is in one piece, and the parts that hold a
    segment's first and last tile and those between are those with a piece of it."""
    total, at, seen, tiles = sum(n + start for n in segs if n), 0, set(), 0
    line = _line(total, ctas)
    for s, n in enumerate(segs):
        at += start if n else 0
        with_piece = []
        for c, (u0, u1) in enumerate(line):
            t0, t1 = max(u0 - at, 0), min(u1 - at, n)
            if t0 < t1:
                assert s + c not in seen and s + c < len(segs) + ctas
                seen.add(s + c)
                tiles += t1 - t0
                with_piece.append(c)
        if n:
            holder = [next(c for c, (u0, u1) in enumerate(line) if u0 <= u < u1) for u in (at, at + n - 1)]
            assert with_piece == list(range(holder[0], holder[1] + 1))
        at += n
    assert tiles == sum(segs)
