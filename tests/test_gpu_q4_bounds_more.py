"""More of the 4-bit cache in the debug-bounds build: windows that end anywhere, a lone key, value scales of any
size, lengths of one to many tiles a CTA, pages of the writers that the decode does not take."""
import pytest

import test_gpu_q4 as Q
import test_gpu_q4_batches as B
import test_gpu_q4_sums as S
import test_gpu_q4_window as W
from test_gpu_bounds import jlb  # noqa: F401  (the fixture: the binding on libjetlong_bounds.so)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,hq,hkv", [(128, 32, 8), (128, 12, 2), (64, 16, 1), (128, 16, 1)])
def test_bounds_build_windows_and_lengths(jlb, d, hq, hkv):  # noqa: F811
    W.test_the_windows_edge(jlb, d, hq, hkv, 33)
    S.test_a_lone_key_gives_its_values(jlb, d, hq, hkv)
    S.test_value_scales_of_any_size(jlb, d, hq, hkv, "both")


@pytest.mark.parametrize("batch,L", [(1, 4737), (3, 2000), (300, 9)])
def test_bounds_build_shares_of_the_ctas(jlb, batch, L):  # noqa: F811
    Q.test_batches_and_lengths_share_the_ctas(jlb, batch, L)


@pytest.mark.parametrize("name", ["tiny", "odd heads", "head blocks", "one long among many", "long ones"])
def test_bounds_build_large_batches(jlb, name):  # noqa: F811
    B.test_large_batches(jlb, name)


def test_bounds_build_writers_and_reader(jlb):  # noqa: F811
    Q.test_fill_writes_the_reference_codes(jlb, 64, 8, (37, 0, 5), (0, 3, 64), 32)
    Q.test_append_equals_fill_of_one_token(jlb, 128, 32, 8, 7)
    Q.test_read_returns_what_rows_stand_for(jlb, 64, 2, 32)
    Q.test_read_returns_what_rows_stand_for(jlb, 128, 3, 0)
