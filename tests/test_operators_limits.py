"""What the decoding step's operators refuse at the ends of their ranges: through
the C ABI, whose checks run on the host before anything is launched."""
import pytest

pytest.importorskip("torch")

import __graft_entry__  # noqa: E402

__graft_entry__.build()
from dynamic_sparsity_spmspv_gb300 import _lib  # noqa: E402

OK, BAD = 0, 1


def test_limits_of_the_waits():
    lib = _lib.load()
    for limit, block in ((0, -1), (-5, 0), (2_000_000_001, -1), (1000, -3)):
        assert lib.dbs_debug_operator_waits(limit, block) == BAD
    assert lib.dbs_debug_operator_waits(2_000_000_000, -1) == OK
