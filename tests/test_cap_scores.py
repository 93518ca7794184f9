"""The score cap of attn_fwd_mod and attn_shared_prefix: small scores under a
large cap, and rows whose bits depend on nothing but what they see.

Tolerances as derived in tests/test_score_mod.py.
"""

import pytest
import torch

import context_blocks_b200 as pa
from oracle import score_mod as oracle
from tests.test_score_mod import _rand, _slopes, check_close


@pytest.mark.gpu
@pytest.mark.parametrize("cap", [1e3, 1e5, 1e6])
@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_small_scores_beside_one_past_a_large_cap(d, slopes, cap):
    """One key far past the cap (its weight is 0) leaves the others' scores as exact
    as they are without it."""
    q, k, v = _rand((1, 4, 300, d), 1), _rand((1, 2, 300, d), 2), _rand((1, 2, 300, d), 3)
    q[..., 0] = 8.0
    k[:, :, ::60, 0] = -3.0 * cap * d ** 0.5 / 8.0
    sl = _slopes(4) if slopes else None
    host = None if sl is None else sl.cpu().numpy()
    o, lse = pa.attn_fwd_mod(q, k, v, softcap=cap, slopes=sl, causal=True, check=True)
    ref = oracle.attention(q.cpu(), k.cpu(), v.cpu(), d ** -0.5, softcap=cap, causal=True, slopes=host)
    # rows 1 .. : the first sees the far key alone
    check_close(o[:, :, 1:], lse[:, :, 1:], ref[0][:, :, 1:], ref[1][:, :, 1:], float(v.abs().max()))
    for G, Bn in ((2, 3), (20, 2), (40, 2), (2, 100)):
        q, kt, vt = _rand((Bn, 2 * G, 1, d), 4), _rand((Bn, 2, 40, d), 5), _rand((Bn, 2, 40, d), 6)
        q[..., 0] = 8.0
        lens = [1 + b % 40 for b in range(Bn)]
        sl = _slopes(2 * G) if slopes else None
        host = None if sl is None else sl.cpu().numpy()
        o, lse = pa.attn_shared_prefix(q, k[0], v[0], kt, vt, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                       softcap=cap, slopes=sl, check=True)
        check_close(o, lse, *oracle.shared_prefix(q, k[0], v[0], kt, vt, lens, d ** -0.5, cap, host), 6.0)


@pytest.mark.gpu
@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("G", [1, 4, 20, 40])
@pytest.mark.parametrize("cap", [8.0, 60.0])
def test_a_decoding_step_takes_the_same_bits_whatever_ran_before(cap, G, slopes):
    """Rows that stand for nothing hold what an earlier kernel left in shared
    memory: it changes nothing."""
    def step(std):
        q, kp, vp = _rand((3, 2 * G, 1, 64), 1, std), _rand((2, 500, 64), 2), _rand((2, 500, 64), 3)
        kt, vt = _rand((3, 2, 200, 64), 4), _rand((3, 2, 200, 64), 5)
        n = torch.tensor([200, 1, 77], dtype=torch.int32, device="cuda")
        return pa.attn_shared_prefix(q, kp, vp, kt, vt, n, softcap=cap, slopes=_slopes(2 * G) if slopes else None)

    def fill(std):  # full tiles of queries of this size on every SM
        q = _rand((40, 64, 2, 64), 6, std)
        k = _rand((1, 4000, 64), 7)
        pa.attn_shared_prefix(q, k, k, k[None, :, :0].expand(40, 1, 0, 64), k[None, :, :0].expand(40, 1, 0, 64),
                              torch.zeros(40, dtype=torch.int32, device="cuda"), softcap=cap)
        pa.attn_fwd_mod(q.view(1, 1, -1, 64).expand(1, 1, -1, 64), k[None, :, :64], k[None, :, :64])

    fill(0.0)
    o, lse = step(1.0)
    for std in (1.0, 100.0, 1e4):
        fill(std)
        o2, lse2 = step(1.0)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    torch.cuda.synchronize()
    assert pa.poll_device_status() == pa.PA_OK


@pytest.mark.gpu
@pytest.mark.parametrize("cap", [8.0, 60.0])
@pytest.mark.parametrize("slopes", [False, True])
def test_hidden_keys_change_no_bit(slopes, cap):
    """Keys behind the tails, hidden by the mask or of other documents may have scores
    past the cap."""
    q, k, v = _rand((1, 2, 300, 64), 1), _rand((1, 2, 300, 64), 2), _rand((1, 2, 300, 64), 3)
    sl = _slopes(2) if slopes else None
    docs = torch.tensor([[0, 100, 170, 290]], dtype=torch.int32, device="cuda")
    args = dict(softcap=cap, slopes=sl, causal=True, doc_offsets=docs)
    o, lse = pa.attn_fwd_mod(q, k, v, **args)
    k2 = k.clone()
    k2[:, :, 290:] *= 1e3
    k2[:, :, 120] *= 1e3  # seen by its own document's later rows, another warp's than the first's
    o2, lse2 = pa.attn_fwd_mod(q, k2, v, check=True, **args)
    rows = torch.ones(300, dtype=torch.bool, device="cuda")
    rows[96:170] = False
    assert torch.equal(o[:, :, rows], o2[:, :, rows]) and torch.equal(lse[:, :, rows], lse2[:, :, rows])

    q, kt, vt = _rand((5, 4, 1, 64), 4), _rand((5, 2, 300, 64), 5), _rand((5, 2, 300, 64), 6)
    lens = [17, 128, 0, 250, 3]
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    args = dict(softcap=cap, slopes=_slopes(4) if slopes else None)
    o, lse = pa.attn_shared_prefix(q, k[0], v[0], kt, vt, n, **args)
    for b, m in enumerate(lens):
        kt[b, :, m:] *= 1e3
    o2, lse2 = pa.attn_shared_prefix(q, k[0], v[0], kt, vt, n, check=True, **args)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
