"""Row positions past a C int are refused, not wrapped round."""

import pytest

import context_blocks_b200 as pa
from tests.test_score_mod import _rand


@pytest.mark.gpu
@pytest.mark.parametrize("q_offset", [1 << 32, (1 << 32) + 7, -(1 << 32), (1 << 31), (1 << 30) + 1, -(1 << 40)])
def test_positions_past_the_limit_are_refused(q_offset):
    q, k = _rand((1, 2, 8, 64), 1), _rand((1, 2, 8, 64), 2)
    with pytest.raises(ValueError, match="q_offset"):
        pa.attn_fwd_mod(q, k, k, causal=True, q_offset=q_offset)


@pytest.mark.gpu
def test_positions_at_the_limit_are_taken():
    q, k = _rand((1, 2, 8, 64), 1), _rand((1, 2, 8, 64), 2)
    o, lse = pa.attn_fwd_mod(q, k, k, causal=True, q_offset=-(1 << 30), check=True)
    assert (o == 0).all() and (lse == float("-inf")).all()
    o, lse = pa.attn_fwd_mod(q, k, k, causal=True, q_offset=1 << 30, check=True)
    o2, lse2 = pa.attn_fwd_mod(q, k, k)
    assert (o == o2).all() and (lse == lse2).all()
