"""Rows that reach behind the tables are refused where the host knows of them (no GPU)."""

import pytest

from tests.test_training_args import INVALID, _embed, pytestmark, sba  # noqa: F401


@pytest.mark.parametrize("T,max_pos", [(10, 9), (1 << 20, 1), (2, 1)])
def test_rows_longer_than_the_tables(sba, T, max_pos):  # noqa: F811
    """Without positions token t of a row sits at t."""
    strides = dict(q_stride=256, k_stride=128, q_out_stride=256, k_out_stride=128)
    code, text = _embed(sba, B=1, T=T, max_pos=max_pos, **strides)
    assert code == INVALID and "max_pos" in text, (code, text)


def test_a_row_of_their_length_is_taken(sba):  # noqa: F811
    """A refusal of something else: a row that the tables hold is no fault."""
    assert "max_pos" not in _embed(sba, B=1, T=10, max_pos=10, q_stride=255)[1]
    assert "max_pos" not in _embed(sba, B=1, T=10, max_pos=9, positions=8 << 32, q_stride=255)[1]
