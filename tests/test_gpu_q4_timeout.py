"""A 4-bit decode that gives up, in the time-out test build (a cos/sin warp gives up at its CTA's fourth tile,
as a wait that ran out would have it): every warp ends, the load warp after its last copies have landed, the
call reports the time-out and writes NaN, and the same context goes on with right results."""
import ctypes

import pytest
import torch

import test_gpu_q4 as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def jll():
    from rope_context_extension_sm_b200 import build
    build.build()
    path = build.build_give_up()
    from rope_context_extension_sm_b200 import jetlong
    lib = ctypes.CDLL(path)
    for name, (res, args) in jetlong.SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    saved = jetlong._lib
    jetlong._lib = lib
    try:
        yield jetlong
    finally:
        jetlong._lib = saved


# 148 CTAs, tiles of 32, 128 and 256 keys: the first length gives no CTA more than one tile, the second four or
# five, which is about the ring of stages, the third more.
@pytest.mark.parametrize("d,hq,hkv,lengths", [(128, 32, 8, (4000, 19000, 60000)), (128, 16, 1, (4000, 60000, 150000)),
                                              (64, 8, 2, (4000, 120000, 300000))])
def test_giving_up_is_reported_and_leaves_the_context_usable(jll, d, hq, hkv, lengths):
    short, *longer = lengths
    cos, sin = Q.tables(max(lengths), d)
    q = Q.normal(82, 1, hq, d)
    cache = Q.random_cache(81, 1, max(lengths), hkv, d)

    def call(L, w0):
        out = jll.jl_bifocal_decode_q4(q, *cache, Q.dev([L], torch.int32), max(lengths), w0, 1500, cos, sin)
        torch.cuda.synchronize()
        return out

    for L in longer:
        for w0 in (0, L):  # all remote, all local
            out, lse = call(L, w0)
            assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())
            out, _ = call(short, 0)  # until the status is read, later calls do nothing but say so
            assert bool(torch.isnan(out).all())
            with pytest.raises(jll.JetLongError) as err:
                jll.jl_sync_status()
            assert err.value.status == jll.JL_ERR_TIMEOUT
            jll.jl_sync_status()  # cleared
            out, lse = call(short, 100)
            jll.jl_sync_status()
            Q.close(out, lse, Q.expect(q, [x[:, :short] for x in cache], [short], 100, 1500))
