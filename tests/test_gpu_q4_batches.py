"""Large batches of the 4-bit decode: more entries than CTAs, with empty ones, ones of one key, ones that several
CTAs share, and lengths outside the contract among them."""
import numpy as np
import pytest
import torch

import test_gpu_q4 as Q
from test_gpu_q4 import jl  # noqa: F401  (the fixture)
from test_gpu_q4_sums import key_rows, rope64, uniform_codes, value_rows

pytestmark = pytest.mark.gpu


def check(q, cache, lens, w0, w_pre, out, lse):
    """Every entry against the definition in 64 bits, all entries of a length at once.  Tolerances as in
    test_gpu_q4_window.py for queries of unit variance: weights times scales to 2^-11, scores to six times 1e-5."""
    hq, d = q.shape[1:]
    lens = np.array(lens)
    for L in sorted(set(lens.tolist())):
        at = torch.from_numpy(np.flatnonzero(lens == L)).cuda()
        if L == 0:
            assert bool((out[at] == 0).all()) and bool(torch.isneginf(lse[at]).all())
            continue
        k, v = (f(c[at, :L], cache[2][at, :L]).double().transpose(0, 1) for f, c in ((key_rows, cache[0]), (value_rows, cache[1])))
        grow, i = max(1, -(-L // w_pre)), L - 1
        edge = max(0, min(L, i - w0 + 1)) if grow > 1 else 0
        j = torch.arange(edge, device="cuda")
        k[:edge] = rope64(k[:edge], j // grow - j)  # [L][entries][hkv][d]
        near = q[at].double()
        far = rope64(near[None], torch.tensor([i // grow - i], device="cuda"))[0]
        kv = torch.arange(hq, device="cuda") // (hq // k.shape[2])
        k, v = k[:, :, kv], v[:, :, kv]
        s = torch.cat([(k[:edge] * far).sum(-1), (k[edge:] * near).sum(-1)]) / d**0.5  # [L][entries][hq]
        w = torch.softmax(s, 0)[..., None]
        want, size = (w * v).sum(0), (w * v.abs()).sum(0)
        step = torch.exp2(torch.floor(torch.log2(want.abs().clamp(min=2.0**-60))) - 8)
        assert bool(((out[at].double() - want).abs() <= step + (2.0**-11 + 6e-5) * size).all())
        assert (lse[at] - torch.logsumexp(s, 0)).abs().max().item() <= 4e-5


def case(seed, lens, stride, hq, hkv, d):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B = len(lens)
    cache = (uniform_codes(g, B, stride, hkv, d // 2), uniform_codes(g, B, stride, hkv, d // 2),
             torch.empty(B, stride, hkv, 8, device="cuda").uniform_(0.15, 0.31, generator=g).bfloat16())
    return cache, torch.randn(B, hq, d, generator=g, device="cuda").bfloat16()


BATCHES = {  # lengths, hq, hkv, d
    "tiny": (lambda g: g.integers(0, 18, 3000), 1, 1, 64),
    "most": (lambda g: g.choice([0, 1, 2, 17], 65535), 1, 1, 64),
    "grouped": (lambda g: g.choice([0, 1, 30, 31, 40], 1000), 8, 2, 64),
    "odd heads": (lambda g: g.choice([1, 130, 257, 0], 400), 9, 3, 128),
    "head blocks": (lambda g: g.choice([1, 300, 33, 0], 60), 20, 20, 64),
    "few heads, a block of channels each": (lambda g: g.choice([0, 1, 300, 517], 230), 1, 1, 128),
    "wide groups": (lambda g: g.choice([0, 5, 129], 270), 16, 1, 128),
    "one long among many": (lambda g: np.concatenate([np.full(200, 3), [6000], np.full(99, 0), [2500], np.full(60, 1)]), 8, 2, 128),
    "long ones": (lambda g: g.choice([1000, 1500], 251), 4, 4, 128),
    "all empty but one": (lambda g: np.concatenate([np.zeros(500, int), [700], np.zeros(300, int)]), 4, 1, 128),
    "all empty": (lambda g: np.zeros(300, int), 4, 1, 128),
}


@pytest.mark.parametrize("name", BATCHES)
def test_large_batches(jl, name):  # noqa: F811
    make, hq, hkv, d = BATCHES[name]
    lens = [int(x) for x in make(np.random.default_rng(5))]
    top = max(max(lens), 1)
    cache, q = case(101, lens, top, hq, hkv, d)
    cos, sin = Q.tables(top, d)
    w0, w_pre = (5, 12) if top < 50 else (40, 150)
    out, lse = jl.jl_bifocal_decode_q4(q, *cache, Q.dev(lens, torch.int32), top, w0, w_pre, cos, sin)
    jl.jl_sync_status()
    check(q, cache, lens, w0, w_pre, out, lse)
    again, _ = jl.jl_bifocal_decode_q4(q, *cache, Q.dev(lens, torch.int32), top, w0, w_pre, cos, sin, want_lse=False)
    assert torch.equal(out, again)


def test_lengths_outside_in_a_large_batch(jl):  # noqa: F811
    hq, hkv, d, top = 6, 2, 64, 90
    g = np.random.default_rng(6)
    lens = g.integers(0, top + 1, 500)
    wrong = np.array([0, 3, 147, 148, 149, 300, 499])
    lens[wrong] = [-1, top + 1, -(1 << 31), (1 << 31) - 1, 1000, -5, top + 1]
    cache, q = case(102, lens, top, hq, hkv, d)
    cos, sin = Q.tables(top, d)
    out, lse = jl.jl_bifocal_decode_q4(q, *cache, Q.dev(lens, torch.int32), top, 10, 30, cos, sin)
    with pytest.raises(jl.JetLongError, match="outside"):
        jl.jl_sync_status()
    assert bool(torch.isnan(out[wrong]).all()) and bool(torch.isnan(lse[wrong]).all())
    right = np.setdiff1d(np.arange(500), wrong)
    check(q[right], [x[right] for x in cache], lens[right], 10, 30, out[right], lse[right])
    jl.jl_sync_status()


@pytest.mark.parametrize("w_pre", [1, 2, (1 << 31) - 1])
@pytest.mark.parametrize("w0", [0, 1, (1 << 31) - 1])
def test_the_smallest_and_largest_windows(jl, w0, w_pre):  # noqa: F811
    lens = (1, 2, 3, 33, 300, 0, 259)
    cache, q = case(103, lens, 300, 8, 2, 128)
    cos, sin = Q.tables(300, 128)
    out, lse = jl.jl_bifocal_decode_q4(q, *cache, Q.dev(lens, torch.int32), 300, w0, w_pre, cos, sin)
    jl.jl_sync_status()
    check(q, cache, lens, w0, w_pre, out, lse)


def test_a_nan_query_stays_in_its_head(jl):  # noqa: F811
    """NaN and infinity in one query head, and a cache of zeros in another KV head."""
    lens = (300, 40)
    for hq, hkv, d in ((8, 2, 128), (12, 2, 64), (32, 2, 128)):
        cache, q = case(104, lens, 300, hq, hkv, d)
        cos, sin = Q.tables(300, d)
        args = (Q.dev(lens, torch.int32), 300, 20, 70, cos, sin)
        clean = jl.jl_bifocal_decode_q4(q, *cache, *args)
        bad = q.clone()
        bad[0, 1, 5], bad[1, 2, 0] = float("nan"), float("inf")
        out, lse = jl.jl_bifocal_decode_q4(bad, *cache, *args)
        keep = torch.ones(2, hq, dtype=torch.bool, device="cuda")
        keep[0, 1] = keep[1, 2] = False
        assert bool(torch.isnan(out[~keep]).all()) and bool(torch.isnan(lse[~keep]).all())
        torch.testing.assert_close(out[keep].float(), clean[0][keep].float(), rtol=2.0**-7, atol=1e-3)
        torch.testing.assert_close(lse[keep], clean[1][keep], rtol=0, atol=4e-5)
        cache[0][:, :, 1], cache[1][:, :, 1], cache[2][:, :, 1] = 0x88, 0x88, 0
        out, lse = jl.jl_bifocal_decode_q4(q, *cache, *args)
        jl.jl_sync_status()
        assert bool((out[:, hq // 2:] == 0).all())
        for b, L in enumerate(lens):
            assert (lse[b, hq // 2:] - np.log(L)).abs().max().item() <= 1e-5


def test_calls_on_two_streams_at_once(jl):  # noqa: F811
    """Two decodes of their own workspaces in flight together, each also captured and replayed."""
    runs = []
    for seed, lens in ((105, [5000, 3]), (106, [int(x) for x in np.random.default_rng(7).integers(0, 60, 400)])):
        top = max(lens)
        cache, q = case(seed, lens, top, 8, 2, 128)
        cos, sin = Q.tables(top, 128)
        sl, out, lse = Q.dev(lens, torch.int32), torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        ws = torch.empty(jl.jl_bifocal_decode_q4_workspace_size(8, 128), dtype=torch.uint8, device="cuda")
        stream = torch.cuda.Stream()
        call = lambda q=q, cache=cache, sl=sl, top=top, cos=cos, sin=sin, out=out, lse=lse, ws=ws: jl.jl_bifocal_decode_q4(  # noqa: E731
            q, *cache, sl, top, 30, 40, cos, sin, out=out, lse=lse, workspace=ws)
        runs.append((stream, call, q, cache, lens, out, lse))
    torch.cuda.synchronize()
    graphs = []
    for stream, call, *_ in runs:
        with torch.cuda.stream(stream):
            call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            call()
        graphs.append(graph)
    for _ in range(20):
        for (stream, *_), graph in zip(runs, graphs):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    jl.jl_sync_status()
    for _, _, q, cache, lens, out, lse in runs:
        check(q, cache, lens, 30, 40, out, lse)
