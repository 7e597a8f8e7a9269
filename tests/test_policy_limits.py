"""Launch limits of the policy operators: refused on the host, before any HIP call."""
from tests.test_policy_abi import ERR_SHAPE, backward, lib  # noqa: F401 (a fixture)


def test_heads_without_rows(lib):  # noqa: F811
    """No rows: only the gradient of one decay for each head is written, by a block each."""
    assert backward(lib, E=0, H=2 ** 24, Hkv=2 ** 24, per_step=0) == ERR_SHAPE
    assert backward(lib, E=0, H=2 ** 32 + 1, Hkv=2 ** 32 + 1, per_step=0) == ERR_SHAPE
