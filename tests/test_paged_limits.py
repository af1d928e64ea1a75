"""Sizes and numbers at the ends of what the paged-cache calls take: what is beyond is refused on
the host (fake, never dereferenced addresses)."""
import pytest

from linear_recurrent_rnn_gb300 import librglru as R
from test_paged_abi import attend, lib, plan, shape, write  # noqa: F401  (lib: a fixture)


@pytest.mark.parametrize("kw", [dict(tokens=2 ** 30 + 1), dict(tokens=2 ** 31 - 1),
                                dict(num_seqs=8192, table_width=2 ** 18), dict(num_seqs=2, table_width=2 ** 30)])
def test_counts_that_pass_32_bits_are_refused(lib, kw):  # noqa: F811
    """Row and page counters of the kernels are 32 bits wide."""
    for f in (plan, write, attend):
        assert f(lib, shape(**kw)) == R.ERR_UNSUPPORTED
    assert R.paged_attention_workspace_bytes(shape(**kw)) == 0


def test_the_largest_sizes_are_taken(lib):  # noqa: F811
    for kw in (dict(tokens=2 ** 30), dict(num_seqs=8192, table_width=2 ** 18 - 1)):
        assert R.paged_attention_workspace_bytes(shape(**kw)) > 0


@pytest.mark.parametrize("scale", [2.4e38, 3.4028235e38])
def test_scales_that_overflow_in_log2_units_are_refused(lib, scale):  # noqa: F811
    """Scores are held times log2 e: such a scale would be infinite there, and every weight NaN."""
    assert attend(lib, shape(), scale=scale) == R.ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["num_seqs", "tokens", "Hq", "Hkv", "D", "num_pages", "page_size", "table_width", "io", "window"])
def test_sizes_beyond_32_bits_are_refused(name):
    """Not taken for their low 32 bits (a window of 2^32 + 64 would be one of 64)."""
    for v in (2 ** 32 + 64, 2 ** 31, -2 ** 31 - 1):
        with pytest.raises(ValueError, match=f"^{name}: "):
            shape(**{name: v})
