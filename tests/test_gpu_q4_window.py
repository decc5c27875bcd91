"""The edge of the local window and of an entry in the 4-bit decode, key by key: lse to 2e-5 and each channel to
what its weights and values allow, at windows that end inside a sixteen of keys.  A window off by one key shows in
every case, which the last test holds on the CPU."""
import numpy as np
import pytest
import torch

import test_gpu_q4 as Q
from test_gpu_q4 import jl  # noqa: F401  (the fixture)
from test_gpu_q4_sums import expect_gpu

SHAPES = [(128, 32, 8), (128, 3, 3), (64, 8, 2), (128, 12, 2), (128, 16, 1), (64, 10, 2), (64, 16, 1), (128, 8, 4)]
WINDOWS = [1, 7, 16, 33, 50, 203]
LENS, W_PRE = (700, 349, 2048), 300  # G = 3, 2, 7


def make(d, hq, hkv, w0):
    g = np.random.default_rng(d + 10 * hq + hkv + w0)
    nib = lambda: g.integers(1, 16, (3, 2048, hkv, d // 2)).astype(np.uint8)  # noqa: E731
    k, v = (torch.from_numpy(nib() | nib() << 4) for _ in range(2))
    scales = torch.from_numpy(g.uniform(0.15, 0.31, (3, 2048, hkv, 8))).to(torch.bfloat16)
    q = torch.from_numpy(2 * g.standard_normal((3, hq, d), dtype=np.float32)).to(torch.bfloat16)
    return (k, v, scales), q


@pytest.mark.gpu
@pytest.mark.parametrize("d,hq,hkv", SHAPES)
@pytest.mark.parametrize("w0", WINDOWS)
def test_the_windows_edge(jl, d, hq, hkv, w0):  # noqa: F811
    """A key's score is off by 1e-5 in the root mean square for queries of unit variance (a turned channel by 7.7e-5
    of a code at the most, see test_gpu_q4.py), by twice that here; the lse averages it over the keys, and 4e-5 covers
    a row of one key.  Channels: weights times scales to 2^-11, the scores' error six deviations, half a bf16 step."""
    cache, q = make(d, hq, hkv, w0)
    cache, q = [x.cuda() for x in cache], q.cuda()
    cos, sin = Q.tables(2048, d)
    out, lse = jl.jl_bifocal_decode_q4(q, *cache, Q.dev(LENS, torch.int32), 2048, w0, W_PRE, cos, sin)
    jl.jl_sync_status()
    for b, L in enumerate(LENS):
        want, want_lse, size, _ = expect_gpu(q[b], [x[b] for x in cache], L, w0, W_PRE)
        assert (lse[b] - want_lse).abs().max().item() <= 4e-5
        step = torch.exp2(torch.floor(torch.log2(want.abs().clamp(min=2.0**-60))) - 8)
        assert bool(((out[b].double() - want).abs() <= step + (2.0**-11 + 1.2e-4) * size).all())


@pytest.mark.gpu
@pytest.mark.parametrize("d,hq,hkv", [(128, 32, 8), (128, 16, 1), (64, 8, 1), (128, 3, 3)])
def test_one_remote_key(jl, d, hq, hkv):  # noqa: F811
    """All keys but one are zero and have the score 0, the one is remote and its score large: the lse shows its error
    alone.  A turned channel is off by 7.7e-5 of a code at the most (44 steps of cos and sin, 14 * 44 * 2^-24, and the
    remainders' roundings, 3 * 14 * 2^-8 * 2^-12), so the score by the scale times the sum of the query's channels
    times that; the fp32 sums by 2^-20 of the score."""
    B, L, w_pre = 32, 4096, 700
    g = torch.Generator(device="cuda").manual_seed(8)
    kc = torch.randint(0, 256, (B, L, hkv, d // 2), generator=g, device="cuda", dtype=torch.uint8)
    kc = torch.where(kc & 15 == 0, kc | 1, kc)
    kc = torch.where(kc >> 4 == 0, kc | 16, kc)
    scales = torch.zeros(B, L, hkv, 8, dtype=torch.bfloat16, device="cuda")
    at = torch.randint(0, L, (B,), generator=g, device="cuda")
    scales[torch.arange(B, device="cuda"), at, :, :4] = 0.25
    q = (8 * torch.randn(B, hq, d, generator=g, device="cuda")).bfloat16()
    cos, sin = Q.tables(L, d)
    out, lse = jl.jl_bifocal_decode_q4(q, kc, kc, scales, Q.dev([L] * B, torch.int32), L, 0, w_pre, cos, sin)
    jl.jl_sync_status()
    assert bool((out == 0).all())
    for b in range(B):
        _, want, _, _ = expect_gpu(q[b], (kc[b], kc[b], scales[b]), L, 0, w_pre)
        bound = 0.25 * 7.7e-5 * q[b].double().abs().sum(-1) / d**0.5
        assert bool(((lse[b] - want).abs() <= bound + 2.0**-20 * want.abs()).all())


@pytest.mark.parametrize("d,hq,hkv", SHAPES)
@pytest.mark.parametrize("w0", WINDOWS)
def test_a_window_off_by_one_would_show(d, hq, hkv, w0):
    """In one entry at least, by twice the tolerance.  (Without a window the query's own key is remote, at the
    distance 0: the same score as with a window of 1.)"""
    cache, q = make(d, hq, hkv, w0)
    off = {w: 0.0 for w in (w0 - 1, w0 + 1)}
    for b, L in enumerate(LENS):
        k, v = Q.R.values(*(x[b] for x in cache))
        x = Q.R.f32(q[b]).astype(np.float64)
        lse = Q.R.decode(x, k[:L], v[:L], w0, W_PRE, Q.BASE)[1]
        for w in off:
            off[w] = max(off[w], np.abs(Q.R.decode(x, k[:L], v[:L], w, W_PRE, Q.BASE)[1] - lse).max())
    assert all(x > 2 * 4e-5 for w, x in off.items() if w > 0)
