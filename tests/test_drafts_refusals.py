"""Host-side refusals of the drafts' operators beyond test_drafts_host.py: no GPU, no device work queued."""
import pytest

from test_drafts_host import EINVAL, cache, call, lib, shared_args  # noqa: F401


@pytest.mark.parametrize("bits", [-1, 2, 256])
def test_all_bits_is_a_truth_value(lib, bits):  # noqa: F811
    assert call(lib, "nbw_kv_attend_shared", cache(), shared_args(all_bits=bits)) == EINVAL
