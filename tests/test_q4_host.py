"""Host-side checks of the 4-bit cache's entry points (no GPU): what they refuse before any launch,
the workspace size, and the binding's checks of shapes, types and devices."""
import numpy as np
import pytest
import torch

import _q4_ref as R


@pytest.fixture(scope="module")
def jl():
    from rope_context_extension_sm_b200 import build
    build.build()
    from rope_context_extension_sm_b200 import jetlong
    return jetlong


# The pointers are fake host addresses: a launch would fail, so a refusal came first.
def _decode(jl, paged=False, **over):
    a = dict(q=16, kc=16, vc=16, sc=16, table=16, sl=16, B=1, stride=1024, max_pages=8, page=128, pages=8, max_seqlen=1024,
             Hq=32, Hkv=8, d=128, w0=64, w_pre=256, cos=16, sin=16, n_tab=1024, scale=0.0, out=16, lse=16, ws=16,
             ws_bytes=1 << 30)
    a.update(over)
    tail = (a["max_seqlen"], a["Hq"], a["Hkv"], a["d"], a["w0"], a["w_pre"], a["cos"], a["sin"], a["n_tab"],
            a["scale"], a["out"], a["lse"], a["ws"], a["ws_bytes"], None)
    if paged:
        return jl._lib.jl_bifocal_decode_q4_paged(a["q"], a["kc"], a["vc"], a["sc"], a["table"], a["sl"], a["B"],
                                                  a["max_pages"], a["page"], a["pages"], *tail)
    return jl._lib.jl_bifocal_decode_q4(a["q"], a["kc"], a["vc"], a["sc"], a["sl"], a["B"], a["stride"], *tail)


@pytest.mark.parametrize("over,status", [
    (dict(B=-1), 1), (dict(d=80), 2), (dict(Hq=30), 1), (dict(Hkv=0), 1), (dict(Hq=34, Hkv=2), 2), (dict(w0=-1), 1),
    (dict(w_pre=0), 1), (dict(max_seqlen=0), 1), (dict(stride=1000), 1), (dict(n_tab=1023), 1),
    (dict(B=3, stride=1 << 30), 2), (dict(B=65536), 2), (dict(q=None), 1), (dict(sc=None), 1), (dict(kc=24), 1),
    (dict(sc=8), 1), (dict(out=4), 1), (dict(ws=None), 1), (dict(ws=24), 1), (dict(ws_bytes=1000), 1),
])
def test_decode_refuses_before_launching(jl, over, status):
    assert _decode(jl, **over) == status
    assert jl.jl_last_error()


@pytest.mark.parametrize("over,status", [
    (dict(page=100), 2), (dict(page=8), 2), (dict(page=0), 2), (dict(max_pages=7), 1), (dict(max_pages=0), 1),
    (dict(pages=0), 1), (dict(pages=1 << 24), 1), (dict(table=None), 1), (dict(vc=8), 1),
])
def test_paged_decode_refuses_before_launching(jl, over, status):
    assert _decode(jl, paged=True, **over) == status


def test_an_empty_batch_is_a_no_op(jl):
    assert _decode(jl, B=0, q=None, ws=None) == 0
    assert _decode(jl, paged=True, B=0, q=None, ws=None) == 0
    assert _fill(jl, T=0, k=None) == 0 and _fill(jl, batch=0) == 0
    assert _append(jl, B=0, q=None) == 0
    assert _read(jl, B=0) == 0 and _read(jl, rows=0) == 0


def _fill(jl, paged=False, **over):
    a = dict(k=16, v=16, cu=16, past=None, batch=1, T=8, Hkv=2, d=128, cos=16, sin=16, n_tab=64, kc=16, vc=16, sc=16,
             stride=64, table=16, max_pages=2, page=32, pages=2)
    a.update(over)
    head = (a["k"], a["v"], a["cu"], a["past"], a["batch"], a["T"], a["Hkv"], a["d"], a["cos"], a["sin"], a["n_tab"],
            a["kc"], a["vc"], a["sc"])
    if paged:
        return jl._lib.jl_kv_cache_fill_q4_paged(*head, a["table"], a["max_pages"], a["page"], a["pages"], None)
    return jl._lib.jl_kv_cache_fill_q4(*head, a["stride"], None)


def _append(jl, paged=False, **over):
    a = dict(q=16, k=16, v=16, sl=16, B=1, Hq=4, Hkv=2, d=128, cos=16, sin=16, n_tab=64, qo=16, kc=16, vc=16, sc=16,
             stride=64, table=16, max_pages=2, page=32, pages=2)
    a.update(over)
    head = (a["q"], a["k"], a["v"], a["sl"], a["B"], a["Hq"], a["Hkv"], a["d"], a["cos"], a["sin"], a["n_tab"],
            a["qo"], a["kc"], a["vc"], a["sc"])
    if paged:
        return jl._lib.jl_decode_append_q4_paged(*head, a["table"], a["max_pages"], a["page"], a["pages"], None)
    return jl._lib.jl_decode_append_q4(*head, a["stride"], None)


def _read(jl, paged=False, **over):
    a = dict(kc=16, vc=16, sc=16, stride=64, starts=None, lens=16, B=1, Hkv=2, d=128, ko=16, vo=16, rows=64, table=16,
             max_pages=2, page=32, pages=2)
    a.update(over)
    tail = (a["starts"], a["lens"], a["B"], a["Hkv"], a["d"], a["ko"], a["vo"], a["rows"], None)
    if paged:
        return jl._lib.jl_kv_cache_read_q4_paged(a["kc"], a["vc"], a["sc"], a["table"], a["max_pages"], a["page"],
                                                 a["pages"], *tail)
    return jl._lib.jl_kv_cache_read_q4(a["kc"], a["vc"], a["sc"], a["stride"], *tail)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("call,over,status", [
    (_fill, dict(d=96), 2), (_fill, dict(batch=-1), 1), (_fill, dict(T=-1), 1), (_fill, dict(Hkv=0), 1),
    (_fill, dict(n_tab=0), 1), (_fill, dict(k=None), 1), (_fill, dict(cu=None), 1), (_fill, dict(sc=None), 1),
    (_fill, dict(kc=8), 1), (_fill, dict(cos=4), 1), (_fill, dict(T=1 << 31), 2),
    (_append, dict(d=32), 2), (_append, dict(B=-1), 1), (_append, dict(Hq=0), 1), (_append, dict(q=None), 1),
    (_append, dict(qo=None), 1), (_append, dict(sl=None), 1), (_append, dict(vc=24), 1), (_append, dict(qo=8), 1),
    (_read, dict(d=100), 2), (_read, dict(B=-1), 1), (_read, dict(rows=-1), 1), (_read, dict(ko=None), 1),
    (_read, dict(lens=None), 1), (_read, dict(vo=8), 1), (_read, dict(B=3, rows=1 << 30), 2),
])
def test_writers_and_reader_refuse_before_launching(jl, call, over, status, paged):
    assert call(jl, paged, **over) == status
    assert jl.jl_last_error()


@pytest.mark.parametrize("call", [_fill, _append, _read])
def test_bad_cache_shapes_are_refused(jl, call):
    assert call(jl, stride=0) == 1
    for over in (dict(page=0), dict(max_pages=0), dict(pages=0), dict(table=None)):
        assert call(jl, True, **over) == 1


def test_workspace_holds_two_partials_for_each_cta(jl):
    assert jl.jl_bifocal_decode_q4_workspace_size(32, 128) == 148 * 2 * 32 * (128 + 2) * 4
    assert jl.jl_bifocal_decode_q4_workspace_size(0, 128) == 0


def test_binding_refuses_cpu_tensors_and_wrong_types(jl):
    codes, scales = torch.zeros(1, 8, 2, 64, dtype=torch.uint8), torch.zeros(1, 8, 2, 8, dtype=torch.bfloat16)
    lens = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        jl.jl_kv_cache_read_q4(codes, codes, scales, lens)
    with pytest.raises(ValueError, match="CUDA tensor"):
        jl.jl_bifocal_decode_q4(torch.zeros(1, 2, 128, dtype=torch.bfloat16), codes, codes, scales, lens, 8, 0, 8, lens, lens)


@pytest.mark.parametrize("d", [64, 128])
def test_every_code_has_a_place_of_its_own(d):
    for place in (R.key_place, R.value_place):
        assert len({place(d, c) for c in range(d)}) == d
        assert all(0 <= b < d // 2 and s in (0, 4) for b, s in (place(d, c) for c in range(d)))
    for c in range(d // 2):  # both channels of a rotate-half pair share a byte and a scale
        assert R.key_place(d, c)[0] == R.key_place(d, c + d // 2)[0]
        assert R.key_group(d, c) == R.key_group(d, c + d // 2)


def test_reference_rounding_is_within_half_a_scale():
    x = np.random.default_rng(0).standard_normal((50, 128)).astype(np.float32)
    code, scale = R.quantise(x, R.value_group)
    g = np.array([R.value_group(128, c) for c in range(128)])
    # half a step, and where the scale was rounded down (by 2^-8 of itself at most) the clamp at 7 steps
    assert (np.abs((code - 8.0) * scale[..., g] - x) <= scale[..., g] * (0.5 + 7 * 2.0**-8)).all()
    assert code.min() >= 1 and code.max() <= 15
