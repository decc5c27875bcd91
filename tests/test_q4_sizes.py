"""Sizes whose products pass 64 bits, or a launch's grid, are refused before any launch (no GPU)."""
import pytest

from test_q4_host import _append, _decode, _fill, _read, jl  # noqa: F401

MOST = (1 << 31) - 1


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("call,over", [
    (_fill, dict(T=MOST, Hkv=MOST)), (_fill, dict(T=1 << 30, Hkv=1 << 30)), (_fill, dict(T=MOST, Hkv=65)),
    (_append, dict(B=MOST, Hq=MOST, Hkv=MOST)), (_append, dict(B=1 << 30, Hq=1 << 29, Hkv=1 << 30)),
    (_append, dict(B=MOST, Hq=16)), (_read, dict(rows=MOST, Hkv=1 << 30)), (_read, dict(B=65535, rows=32768, Hkv=MOST)),
    (_read, dict(B=65535, rows=1 << 62)),
])
def test_writers_and_reader_refuse_sizes_past_a_grid(jl, call, over, paged):  # noqa: F811
    assert call(jl, paged, **over) == jl.JL_ERR_UNSUPPORTED
    assert jl.jl_last_error()


def test_decode_refuses_strides_past_32_bits(jl):  # noqa: F811
    for over in (dict(B=4, stride=1 << 62), dict(B=2, stride=(1 << 63) - 1), dict(B=65535, stride=1 << 48),
                 dict(B=1, stride=1 << 31)):
        assert _decode(jl, **over) == jl.JL_ERR_UNSUPPORTED
        assert "cache_stride" in jl.jl_last_error()
