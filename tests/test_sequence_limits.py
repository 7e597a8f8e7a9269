"""Sizes and call forms of the sequence operators' C entries that only a C program can ask for, without a GPU.

Every call below is refused, or has nothing to do, before any HIP call.
"""
from __future__ import annotations

import pytest

from tests.test_sequence_abi import ERR_NULL, ERR_SHAPE, OK, lib, norm_rotate, norm_rotate_backward  # noqa: F401

NO_HEADS = dict(H=0, Hk=0, q=None, k=None)


@pytest.mark.parametrize("E,T", [(2 ** 62, 4), (2 ** 40, 2 ** 20), (2 ** 46 + 1, 1), (2 ** 27, 2 ** 20 - 1)])
def test_tokens_are_counted_where_there_are_no_heads(lib, E, T):  # noqa: F811
    # 2^46 elements at most, whatever the number of heads: E T must not leave the range of 64 bits
    assert norm_rotate(lib, E=E, T=T, qo=None, ko=None, **NO_HEADS) == ERR_SHAPE
    assert norm_rotate_backward(lib, E=E, T=T, gq=None, gk=None, dq=None, dk=None, bytes=1 << 30,
                                **NO_HEADS) == ERR_SHAPE
    assert lib.rlscan_norm_rotate_heads_workspace(E, T, 0, 0, 64) == -1


def test_no_heads_need_no_positions(lib):  # noqa: F811
    assert norm_rotate(lib, pos=None, qo=None, ko=None, **NO_HEADS) == OK
    none = dict(pos=None, gq=None, gk=None, dq=None, dk=None, **NO_HEADS)
    assert norm_rotate_backward(lib, dqw=None, dkw=None, **none) == OK
    # sums of the weights' gradients take memory all the same
    assert norm_rotate_backward(lib, ws=None, **none) == ERR_NULL
    assert lib.rlscan_norm_rotate_heads_workspace(2 ** 20, 2 ** 19, 0, 0, 64) == 2 * 64 * 4
