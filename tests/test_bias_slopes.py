"""Distance bias with slopes of any finite size.  Tolerances as derived in
tests/test_score_mod.py; a bias that is large beside a score leaves the score of
the row's own key as it is.
"""

import pytest
import torch

import context_blocks_b200 as pa
from oracle import score_mod as oracle
from tests.test_score_mod import _rand, check_close


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kw", [dict(), dict(softcap=20.0)], ids=str)
def test_large_slopes_keep_the_score_at_distance_zero(d, kw):
    sl = torch.tensor([1.0, 1e4, 1e6, 1e10, 1e30, 0.0], dtype=torch.float32, device="cuda")
    host = sl.cpu().numpy()
    q, k, v = _rand((1, 6, 300, d), 1, 3.0), _rand((1, 2, 300, d), 2), _rand((1, 2, 300, d), 3)
    for args in (dict(causal=True), dict(), dict(causal=True, doc_offsets=[[0, 100, 170, 290]])):
        dev = dict(args)
        if "doc_offsets" in args:
            dev["doc_offsets"] = torch.tensor(args["doc_offsets"], dtype=torch.int32, device="cuda")
        o, lse = pa.attn_fwd_mod(q, k, v, slopes=sl, check=True, **dev, **kw)
        check_close(o, lse, *oracle.attention(q.cpu(), k.cpu(), v.cpu(), d ** -0.5, slopes=host, **args, **kw),
                    float(v.abs().max()))
    for Bn, G in ((3, 3), (2, 12), (2, 36), (30, 6)):  # rows in copies, pairs
        H = 2 * G
        sl2 = sl.repeat(H // 6).contiguous()
        q, kt, vt = _rand((Bn, H, 1, d), 4, 3.0), _rand((Bn, 2, 140, d), 5), _rand((Bn, 2, 140, d), 6)
        lens = [1 + (37 * b) % 140 for b in range(Bn)]
        o, lse = pa.attn_shared_prefix(q, k[0], v[0], kt, vt, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                       slopes=sl2, check=True, **kw)
        check_close(o, lse, *oracle.shared_prefix(q, k[0], v[0], kt, vt, lens, d ** -0.5, slopes=sl2.cpu().numpy(), **kw),
                    6.0)
