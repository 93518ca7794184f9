"""Where the partial results of attn_shared_prefix lie: the library's own
arithmetic, compiled on the host, over random shapes and numbers of CTAs; and on
the GPU a workspace of exactly the size asked for, with something behind it.
"""

import os
import shutil
import subprocess

import pytest
import torch

import context_blocks_b200 as pa
from tests.test_score_mod import LSE_ABS, _rand, _slopes

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("slots") / "shared_slots")
    gxx = shutil.which("g++")
    assert gxx, "g++ not found"
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-x", "c++",
                        f"-I{os.path.join(ROOT, 'context_blocks_b200', 'csrc')}",
                        os.path.join(ROOT, "tests", "c", "shared_slots.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return exe


@pytest.mark.parametrize("seed", range(4))
def test_pieces_and_slots_of_random_calls(program, seed):
    r = subprocess.run([program, str(seed), "400"], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "slots checked" in r.stdout, r.stderr


@pytest.mark.gpu
@pytest.mark.parametrize("Np", [0, 128])
def test_as_many_requests_as_there_may_be(Np):
    """65535 requests with the shortest wait: looking for pieces among their lengths
    is part of the limit.  Against a float64 evaluation of all of them; tolerances as
    derived in tests/test_score_mod.py."""
    Bn, Nt, d = 65535, 8, 64
    q, kp, vp = _rand((Bn, 1, 1, d), 1, 2.0), _rand((1, Np, d), 2), _rand((1, Np, d), 3)
    kt, vt = _rand((Bn, 1, Nt, d), 4), _rand((Bn, 1, Nt, d), 5)
    n = (torch.arange(Bn, device="cuda") * 7 % (Nt + 1)).to(torch.int32)
    pa.set_wait_limit_ms(1)
    try:
        o, lse = pa.attn_shared_prefix(q, kp, vp, kt, vt, n, check=True)
    finally:
        pa.set_wait_limit_ms(5000)
    s_p = (q[:, 0].double() @ kp[0].double().t()).view(Bn, 1, Np) * d ** -0.5
    s_t = torch.einsum("bd,bnd->bn", q[:, 0, 0].double(), kt[:, 0].double()) * d ** -0.5
    s_t = s_t.masked_fill(torch.arange(Nt, device="cuda") >= n[:, None], float("-inf"))
    s = torch.cat([s_p[:, 0], s_t], 1)
    want = torch.logsumexp(s, 1)
    none = want == float("-inf")
    p = torch.exp(s - want.masked_fill(none, 0.0)[:, None])
    ref = p[:, :Np] @ vp[0].double() + torch.einsum("bn,bnd->bd", p[:, Np:], vt[:, 0].double())
    got = lse[:, 0, 0].double()
    assert torch.equal(none, got == float("-inf")) and (o[none] == 0).all()
    assert (got - want)[~none].abs().max() <= LSE_ABS
    assert (o[:, 0, 0].double() - ref).abs().max() <= 2.0 ** -7 * 6.0


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Bn,G,Nq,Np,Nt", [(1, 1, 1, 1, 1), (3, 7, 1, 40000, 16), (40, 4, 1, 900, 300), (100, 8, 1, 5000, 129),
                                           (300, 1, 1, 0, 700), (61, 40, 1, 2000, 20), (5, 5, 14, 300, 2000), (7, 3, 1, 300, 0)])
def test_nothing_behind_the_workspace_is_written(Bn, G, Nq, Np, Nt, d):
    q, kp, vp = _rand((Bn, 2 * G, Nq, d), 1, 2.0), _rand((2, Np, d), 2), _rand((2, Np, d), 3)
    kt, vt = _rand((Bn, 2, Nt, d), 4), _rand((Bn, 2, Nt, d), 5)
    size = pa.shared_prefix_workspace_bytes(Bn, 2 * G, 2, Nq, Np, Nt, d)
    room = torch.full((256 + size + 65536,), 0x5a, dtype=torch.uint8, device="cuda")
    for kw in (dict(), dict(softcap=10.0), dict(slopes=_slopes(2 * G))):
        for lens in ([Nt] * Bn, [(37 * b) % (Nt + 1) for b in range(Bn)], [Nt if b == Bn - 1 else 0 for b in range(Bn)]):
            n = torch.tensor(lens, dtype=torch.int32, device="cuda")
            want = pa.attn_shared_prefix(q, kp, vp, kt, vt, n, **kw)
            got = pa.attn_shared_prefix(q, kp, vp, kt, vt, n, workspace=room[256:256 + size], check=True, **kw)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (room[:256] == 0x5a).all() and (room[256 + size:] == 0x5a).all()
    if size:
        with pytest.raises(pa.PaError, match="workspace"):
            pa.attn_shared_prefix(q, kp, vp, kt, vt, n, workspace=room[256:256 + size - 1])
