"""Further CPU checks of the calls on a cache's pages (include/paged_pages.h)."""
import pytest

from linear_recurrent_rnn_gb300 import librglru as R
from test_paged_abi import lib, shape  # noqa: F401  (lib: a fixture)
from test_paged_pages_abi import copy


@pytest.mark.parametrize("n", [2 ** 30 + 1, 2 ** 31 - 1])
def test_lists_of_moves_past_32_bits_are_refused(lib, n):  # noqa: F811
    """Their entries' places would overflow the kernel's indexes.  (Without caches nothing is launched.)"""
    assert copy(lib, shape(), n, caches=(), strides=(), sizes=(), arrays=False) == R.ERR_UNSUPPORTED
    assert copy(lib, shape(), 2 ** 30, caches=(), strides=(), sizes=(), arrays=False) == R.OK
