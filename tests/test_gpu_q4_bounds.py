"""The 4-bit cache's kernels in the debug-bounds build: every index that the decode derives for its
cos/sin rows is checked on the device, and each case must still agree with its reference."""
import pytest

import test_gpu_q4 as Q
from test_gpu_bounds import jlb  # noqa: F401  (the fixture: the binding on libjetlong_bounds.so)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,hq,hkv", [(64, 8, 2), (128, 32, 8), (128, 3, 3), (128, 16, 2), (64, 16, 1), (128, 12, 4)])
@pytest.mark.parametrize("w0,w_pre", [(0, 64), (50, 100), (33, 37)])
def test_bounds_build_q4_decode(jlb, d, hq, hkv, w0, w_pre):  # noqa: F811
    Q.test_decode_against_the_definition(jlb, d, hq, hkv, w0, w_pre)


def test_bounds_build_q4_paged_and_long(jlb):  # noqa: F811
    Q.test_paged_decode_equals_contiguous(jlb, 48, 128, 32, 8)
    Q.test_batches_and_lengths_share_the_ctas(jlb, 70, 40)
    Q.test_a_long_cache(jlb, 128, 32, 8)


def test_bounds_build_q4_writers_and_reader(jlb):  # noqa: F811
    Q.test_fill_writes_the_reference_codes(jlb, 128, 3, (130, 1), (2, 0), 48)
    Q.test_append_equals_fill_of_one_token(jlb, 64, 8, 2, 32)
    Q.test_read_returns_what_rows_stand_for(jlb, 128, 8, 40)
