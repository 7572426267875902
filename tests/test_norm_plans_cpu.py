"""How the backward pass of the norms shares its rows out, as its workspace shows (no GPU): a row
of sums for each chunk of rows and vector."""
from __future__ import annotations

import pytest

from test_operators_cpu import OK, grad_size


def chunks(M, D, groups=1):
    """Chunks of rows whose sums are kept, of a bfloat16 pass with one vector's gradient."""
    strides = {k: D for k in ("ldx", "ldh", "lddr", "lddy", "lddx", "lddh")}
    st, size = grad_size(M=M, D=D, groups=groups, db=0, dg=0, dpw=0, dpb=0, **strides)
    assert st == OK
    return size // (D * 4)


# rows that a workgroup takes at once
@pytest.mark.parametrize("D,rows", [(64, 32), (128, 32), (192, 8), (512, 8), (1024, 2), (2048, 2),
                                    (4096, 1)])
@pytest.mark.parametrize("M", [1, 7, 33, 512, 1000, 4096, 65536])
def test_chunks_are_of_whole_rounds(M, D, rows):
    # no more chunks than rounds of rows, and workgroups enough to fill the CUs where there are
    # that many rounds
    rounds = -(-M // rows)
    assert chunks(M, D) <= max(1, rounds) + (256 // (D * 4))      # (sizes are in 256 bytes)
    assert chunks(M, D) >= min(rounds, 256)


def test_chunks_of_groups():
    for M, D, groups, rows in ((1000, 128, 4, 32), (4096, 64, 4096, 32), (512, 512, 8, 8)):
        per = -(-(M // groups) // rows)
        assert chunks(M, D, groups) == groups * per
