"""Resizes whose number in the accounts' workspace runs past 32 bits, against the sequential reference."""
import numpy as np
import pytest

from test_gpu_pages import Both

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("short", [False, True], ids=["all served", "one refused"])
@pytest.mark.parametrize("before", [1, 2, 3, 4, 5, 6])
def test_the_number_of_calls_wraps(before, short):
    """Two rounds of three resizes of more than 1024 entries (the ones that are numbered), the first
    number `before` calls short of 2^32: pages shared by three, of which one is cut back and written
    behind (its copies are taken), one ends, and at last both others. With a fourth sequence that always
    asks for more pages than there are the call takes its general form."""
    P, N = 1600, 2700
    b = Both(5, P, N)
    b.work[:-64].view(torch.int32)[4 * N] = -before  # behind three marks per page, 16 bytes
    more = P * 64 if short else 0
    for _ in range(2):
        b.resize([0] * 5, [1300 * 64 - 5, 0, 0, 70, more])
        b.fork([0, 0], [1, 2], [1300 * 64 - 5, 1300 * 64])
        b.resize([1300 * 64 - 5, 100 * 64 + 9, 0, 70, 0], [1300 * 64, 1310 * 64, 0, 70, more])
        b.ref.check()
        b.resize([0] * 5, [0, 0, 0, 0, more])
        assert b.ref.count == N
    assert b.ref.no_page == short
    # (2^32 - 1 is followed by 1)
    assert int(b.work[:-64].view(torch.int32)[4 * N]) == 7 - before
