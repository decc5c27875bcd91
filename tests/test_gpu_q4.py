"""The 4-bit cache on the GPU: writers and reader bit for bit against the fp32 reference, the decode
against the definition in 64 bits, and all of them together as a user calls them.

Decode tolerances are the framework's own for a decode (out max-abs 2e-2 and mean-abs 2e-3 for values
of unit variance, lse 1e-2).  The one rounding of the kernel that shows in them is that of the weights
times the value scales to fp16, 2^-12 of each, which averages over the keys; the lse, which it does not
touch, has a test of its own."""
import numpy as np
import pytest
import torch

import _q4_ref as R

pytestmark = pytest.mark.gpu
BASE = 1e4


@pytest.fixture(scope="module")
def jl():
    from rope_context_extension_sm_b200 import build
    build.build()
    from rope_context_extension_sm_b200 import jetlong
    yield jetlong
    jetlong.jl_sync_status()


def dev(x, dtype=None):
    t = torch.as_tensor(x)
    return (t if dtype is None else t.to(dtype)).cuda()


def tables(n, d):
    c, s = R.tables(max(n, 1), d, BASE)
    return dev(c), dev(s)


def normal(seed, *shape):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape, dtype=np.float32)).to(torch.bfloat16).cuda()


def paged(x, page, seed=0):
    """[B][stride][..] -> (pool, block table) with the pages in a mixed order and two spare ones."""
    B, stride = x.shape[:2]
    per = -(-stride // page)
    perm = np.random.default_rng(seed).permutation(B * per + 2)[: B * per].reshape(B, per)
    pool = torch.zeros((B * per + 2, page, *x.shape[2:]), dtype=x.dtype, device=x.device)
    for b in range(B):
        for n in range(per):
            part = x[b, n * page:(n + 1) * page]
            pool[perm[b, n], : part.shape[0]] = part
    return pool, dev(perm, torch.int32)


def random_cache(seed, B, stride, hkv, d):
    """A cache of random codes (1 .. 15) and scales such that keys and values have unit variance."""
    g = np.random.default_rng(seed)
    nib = lambda: g.integers(1, 16, (B, stride, hkv, d // 2)).astype(np.uint8)  # noqa: E731
    kc, vc = (dev(nib() | nib() << 4) for _ in range(2))
    scales = dev(g.uniform(0.15, 0.31, (B, stride, hkv, 8)), torch.bfloat16)
    return kc, vc, scales


def expect(q, cache, lens, w0, w_pre):
    k, v = R.values(*cache)
    q = R.f32(q).astype(np.float64)
    got = [R.decode(q[b], k[b, :n], v[b, :n], w0, w_pre, BASE) for b, n in enumerate(lens)]
    return np.stack([o for o, _ in got]), np.stack([x for _, x in got])


def close(out, lse, want):
    err = np.abs(R.f32(out) - want[0])
    assert np.isfinite(err).all() and err.max() <= 2e-2 and err.mean() <= 2e-3, (err.max(), err.mean())
    if lse is not None:
        l, w = R.f32(lse), want[1]
        assert np.array_equal(np.isneginf(l), np.isneginf(w))
        fine = np.isfinite(w)
        assert not fine.any() or np.abs(l[fine] - w[fine]).max() <= 1e-2, np.abs(l[fine] - w[fine]).max()


# ------------------------------------------------------------ writing, reading --

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv,lens,past", [(1, (1,), (0,)), (8, (37, 0, 5), (0, 3, 64)), (3, (130, 1), (2, 0))])
@pytest.mark.parametrize("page", [0, 32, 48])
def test_fill_writes_the_reference_codes(jl, d, hkv, lens, past, page):
    T, B, stride = sum(lens), len(lens), 144
    k, v = normal(1, T, hkv, d), normal(2, T, hkv, d)
    cos, sin = tables(stride, d)
    cu = dev(np.concatenate([[0], np.cumsum(lens)]), torch.int32)
    cache = [torch.full((B, stride, hkv, d // 2), 0x5a, dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache.append(torch.full((B, stride, hkv, 8), 3.0, dtype=torch.bfloat16, device="cuda"))
    if page:
        pools = [paged(x, page) for x in cache]
        table = pools[0][1]
        jl.jl_kv_cache_fill_q4_paged(k, v, cu, cos, sin, *(x for x, _ in pools), table, past_lens=dev(past, torch.int32))
        got = [x[table.long()].flatten(1, 2) for x, _ in pools]
    else:
        jl.jl_kv_cache_fill_q4(k, v, cu, cos, sin, *cache, past_lens=dev(past, torch.int32))
        got = cache
    jl.jl_sync_status()
    c, s = R.tables(stride, d, BASE)
    for b in range(B):
        rows = slice(past[b], past[b] + lens[b])
        x = R.rotate_f32(R.f32(k[cu[b]:cu[b + 1]]), c[rows, None], s[rows, None])
        for which, x, group, place, at in ((0, x, R.key_group, R.key_place, 0),
                                           (1, R.f32(v[cu[b]:cu[b + 1]]), R.value_group, R.value_place, 4)):
            code, scale = R.quantise(x, group)
            assert np.array_equal(R.codes(got[which][b, rows].cpu().numpy(), d, place), code)
            assert np.array_equal(R.f32(got[2][b, rows, :, at:at + 4]), scale)
            behind = got[which][b, past[b] + lens[b]:stride]  # rows behind the last token stay
            assert bool((behind == 0x5a).all()) and bool((got[which][b, :past[b]] == 0x5a).all())


@pytest.mark.parametrize("d", [64, 128])
def test_many_rows_have_the_reference_codes(jl, d):
    """Roundings that depend on the order of a key's products and sums show in some ten groups of four
    million: a rotation whose products are fused into its sums is not the one that the codes are defined by."""
    T, hkv = 40000, 8
    k, v = normal(61, T, hkv, d), normal(62, T, hkv, d)
    cos, sin = tables(T, d)
    cache = jl.jl_kv_cache_q4_empty(1, T, hkv, d)
    jl.jl_kv_cache_fill_q4(k, v, dev([0, T], torch.int32), cos, sin, *cache)
    jl.jl_sync_status()
    c, s = R.tables(T, d, BASE)
    code, scale = R.quantise(R.rotate_f32(R.f32(k), c[:, None], s[:, None]), R.key_group)
    assert np.array_equal(R.f32(cache[2][0, :, :, :4]), scale)
    assert np.array_equal(R.codes(cache[0][0].cpu().numpy(), d, R.key_place), code)


@pytest.mark.parametrize("d", [64, 128])
def test_groups_of_zeros_extremes_and_nonfinite_values(jl, d):
    x = normal(3, 12, 1, d).float()
    x[0] = 0
    x[1, :, : d // 4] = 0                          # a group of zeros among others
    x[2] *= 1e-36                                  # scale below 2^-100: stored as zeros
    x[3] *= 2.0**-95                               # just above
    x[4] = 3.3e38                                  # the largest bf16 magnitudes
    x[5, 0, 3] = float("nan")
    x[6, 0, d - 1] = float("inf")
    x[7, 0, 5] = float("-inf")
    x[8] = torch.arange(d, device="cuda") % 29 - 14.0  # ties: scale 2, odd values halfway between codes
    x[9] = 7.0
    x[10, 0, 1:] = 0
    x = x.to(torch.bfloat16)
    cos, sin = torch.ones((12, d // 2), device="cuda"), torch.zeros((12, d // 2), device="cuda")
    cache = jl.jl_kv_cache_q4_empty(1, 12, 1, d)
    jl.jl_kv_cache_fill_q4(x, x, dev([0, 12], torch.int32), cos, sin, *cache)
    lens = dev([12], torch.int32)
    k, v = jl.jl_kv_cache_read_q4(*cache, lens)
    jl.jl_sync_status()
    with np.errstate(all="ignore"):
        kx = R.rotate_f32(R.f32(x), np.float32(1), np.float32(0))
    for which, y, group, place, at, back in ((0, kx, R.key_group, R.key_place, 0, k),
                                             (1, R.f32(x), R.value_group, R.value_place, 4, v)):
        code, scale = R.quantise(y, group)
        assert np.array_equal(R.codes(cache[which][0].cpu().numpy(), d, place), code)
        assert np.array_equal(R.f32(cache[2][0, :, :, at:at + 4]), scale, equal_nan=True)
        g = np.array([group(d, c) for c in range(d)])
        want = torch.from_numpy((code.astype(np.float32) - 8) * scale[..., g]).to(torch.bfloat16)
        assert np.array_equal(R.f32(back[0]), want.float().numpy(), equal_nan=True)
    assert bool(torch.isnan(v[0, 5, 0, : d // 4]).all()) and not bool(torch.isnan(v[0, 5, 0, d // 4:]).any())


@pytest.mark.parametrize("d,hkv", [(64, 2), (128, 8), (128, 3)])
@pytest.mark.parametrize("page", [0, 32, 40])
def test_read_returns_what_rows_stand_for(jl, d, hkv, page):
    stride, lens, starts = 80, (80, 0, 33, 7), (3, 0, 32, 7)
    cache = random_cache(5, 4, stride, hkv, d)
    want = R.values(*cache)
    out = [torch.full((4, 79, hkv, d), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    args = dict(starts=dev(starts, torch.int32), k_out=out[0], v_out=out[1])
    if page:
        pools = [paged(x, page) for x in cache]
        jl.jl_kv_cache_read_q4_paged(*(x for x, _ in pools), pools[0][1], dev(lens, torch.int32), **args)
    else:
        jl.jl_kv_cache_read_q4(*cache, dev(lens, torch.int32), **args)
    jl.jl_sync_status()
    for got, w in zip(out, want):
        for b in range(4):
            n = lens[b] - starts[b]
            ref = torch.from_numpy(w[b, starts[b]:lens[b]].astype(np.float32)).to(torch.bfloat16).float().numpy()
            assert np.array_equal(R.f32(got[b, :n]), ref)
            assert bool((got[b, n:] == 9.0).all())


@pytest.mark.parametrize("d,hq,hkv", [(64, 8, 2), (128, 32, 8), (128, 3, 3)])
@pytest.mark.parametrize("page", [0, 32, 7])
def test_append_equals_fill_of_one_token(jl, d, hq, hkv, page):
    lens, stride = (1, 64, 33, 128, 97), 128
    B = len(lens)
    q, k, v = normal(1, B, hq, d), normal(2, B, hkv, d), normal(3, B, hkv, d)
    cos, sin = tables(stride, d)
    sl = dev(lens, torch.int32)
    cache = random_cache(6, B, stride, hkv, d)
    ref = [x.clone() for x in cache]
    jl.jl_kv_cache_fill_q4(k, v, dev(range(B + 1), torch.int32), cos, sin, *ref, past_lens=sl - 1)
    if page:
        pools = [paged(x, page) for x in cache]
        qo = jl.jl_decode_append_q4_paged(q, k, v, sl, cos, sin, *(x for x, _ in pools), pools[0][1])
        got = [x[t.long()].flatten(1, 2)[:, :stride] for x, t in pools]
    else:
        qo = jl.jl_decode_append_q4(q, k, v, sl, cos, sin, *cache)
        got = cache
    jl.jl_sync_status()
    for x, y in zip(got, ref):
        assert torch.equal(x, y)  # the one row, and no other
    want = R.rope64(R.f32(q).astype(np.float64), np.array(lens)[:, None] - 1, BASE)
    assert (np.abs(R.f32(qo) - want) <= 2.0**-8 * np.abs(want) + 1e-6).all()


def test_positions_and_pages_outside_are_skipped_and_reported(jl):
    d, hkv = 64, 2
    cos, sin = tables(40, d)
    cache = random_cache(7, 2, 32, hkv, d)
    before = [x.clone() for x in cache]
    k = normal(1, 2, hkv, d)
    jl.jl_kv_cache_fill_q4(k, k, dev([0, 1, 2], torch.int32), cos, sin, *cache, past_lens=dev([32, -1], torch.int32))
    with pytest.raises(jl.JetLongError, match="outside"):
        jl.jl_sync_status()
    jl.jl_decode_append_q4(k, k, k, dev([0, 33], torch.int32), cos, sin, *cache)
    with pytest.raises(jl.JetLongError, match="outside"):
        jl.jl_sync_status()
    jl.jl_kv_cache_fill_q4_paged(k, k, dev([0, 1, 2], torch.int32), cos, sin, *cache, dev([[2], [-1]], torch.int32))
    with pytest.raises(jl.JetLongError, match="outside"):
        jl.jl_sync_status()
    for x, y in zip(cache, before):
        assert torch.equal(x, y)
    out = [torch.full((2, 8, hkv, d), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for lens, starts in (((33, 9), (30, 0)), ((5, 5), (-1, -4))):  # behind the stride, more rows than out has, negative
        jl.jl_kv_cache_read_q4(*cache, dev(lens, torch.int32), starts=dev(starts, torch.int32), k_out=out[0], v_out=out[1])
        with pytest.raises(jl.JetLongError, match="outside"):
            jl.jl_sync_status()
        assert bool((out[0] == 9.0).all()) and bool((out[1] == 9.0).all())
    jl.jl_sync_status()


# --------------------------------------------------------------------- decode --

SHAPES = [(64, 8, 2), (128, 32, 8), (128, 16, 8), (128, 3, 3), (64, 1, 1), (128, 12, 4), (128, 16, 2), (128, 16, 1),
          (64, 40, 8), (128, 10, 2), (64, 48, 12), (128, 60, 12)]


@pytest.mark.parametrize("d,hq,hkv", SHAPES)
@pytest.mark.parametrize("w0,w_pre", [(0, 64), (50, 100), (128, 4096), (33, 37)])
def test_decode_against_the_definition(jl, d, hq, hkv, w0, w_pre):
    lens = (1, 0, 31, 32, 33, 129, 300, 517)
    cache = random_cache(11, len(lens), 520, hkv, d)
    q = normal(12, len(lens), hq, d)
    cos, sin = tables(520, d)
    want = expect(q, cache, lens, w0, w_pre)
    sl = dev(lens, torch.int32)
    out, lse = jl.jl_bifocal_decode_q4(q, *cache, sl, 520, w0, w_pre, cos, sin)
    jl.jl_sync_status()
    close(out, lse, want)
    again, _ = jl.jl_bifocal_decode_q4(q, *cache, sl, 520, w0, w_pre, cos, sin, want_lse=False)
    assert torch.equal(out, again)  # the order of the sums does not change from call to call


@pytest.mark.parametrize("page", [16, 32, 48, 96, 256])
@pytest.mark.parametrize("d,hq,hkv", [(128, 32, 8), (64, 6, 3), (128, 8, 2)])
def test_paged_decode_equals_contiguous(jl, page, d, hq, hkv):
    lens = (513, 1, 96, 0, 255, 256)
    cache = random_cache(13, len(lens), 544, hkv, d)
    q = normal(14, len(lens), hq, d)
    cos, sin = tables(768, d)
    pools = [paged(x, page) for x in cache]
    sl = dev(lens, torch.int32)
    out, lse = jl.jl_bifocal_decode_q4(q, *cache, sl, 520, 40, 128, cos, sin)
    got, glse = jl.jl_bifocal_decode_q4_paged(q, *(x for x, _ in pools), pools[0][1], sl, 520, 40, 128, cos, sin)
    jl.jl_sync_status()
    assert torch.equal(out, got) and torch.equal(lse, glse)
    close(out, lse, expect(q, cache, lens, 40, 128))


@pytest.mark.parametrize("B,L", [(1, 1), (1, 4737), (3, 2000), (70, 40), (300, 9)])
def test_batches_and_lengths_share_the_ctas(jl, B, L):
    """One entry over many CTAs, many entries on one, and every mixture of first, whole and last parts."""
    d, hq, hkv = 128, 8, 2
    rng = np.random.default_rng(B)
    lens = [L] + [int(x) for x in rng.integers(0, L + 1, B - 1)]
    cache = random_cache(15, B, L + 1, hkv, d)
    q = normal(16, B, hq, d)
    cos, sin = tables(L + 1, d)
    want = expect(q, cache, lens, 16, 700)
    for bound in (L, L + 1):
        out, lse = jl.jl_bifocal_decode_q4(q, *cache, dev(lens, torch.int32), bound, 16, 700, cos, sin)
        jl.jl_sync_status()
        close(out, lse, want)


def test_rows_behind_the_length_may_hold_anything(jl):
    d, hq, hkv, lens = 128, 32, 8, (5, 45, 0, 64)
    cache = random_cache(17, 4, 64, hkv, d)
    q = normal(18, 4, hq, d)
    cos, sin = tables(64, d)
    sl = dev(lens, torch.int32)
    clean = jl.jl_bifocal_decode_q4(q, *cache, sl, 64, 8, 20, cos, sin)
    for b, n in enumerate(lens):
        cache[0][b, n:] = 255
        cache[2][b, n:] = float("nan")
    cache[2][0, 5:] = float("inf")
    got = jl.jl_bifocal_decode_q4(q, *cache, sl, 64, 8, 20, cos, sin)
    jl.jl_sync_status()
    assert torch.equal(clean[0], got[0]) and torch.equal(clean[1], got[1])
    assert bool((got[0][2] == 0).all()) and bool(torch.isneginf(got[1][2]).all())


def test_a_nan_scale_inside_reaches_only_its_heads(jl):
    d, hq, hkv = 128, 8, 2
    cache = random_cache(19, 1, 100, hkv, d)
    q = normal(20, 1, hq, d)
    cos, sin = tables(100, d)
    clean = jl.jl_bifocal_decode_q4(q, *cache, dev([100], torch.int32), 100, 10, 40, cos, sin)
    cache[2][0, 50, 1, 2] = float("nan")  # a key scale of KV head 1
    out, lse = jl.jl_bifocal_decode_q4(q, *cache, dev([100], torch.int32), 100, 10, 40, cos, sin)
    assert torch.equal(out[:, :4], clean[0][:, :4]) and torch.equal(lse[:, :4], clean[1][:, :4])
    assert bool(torch.isnan(out[:, 4:]).all()) and bool(torch.isnan(lse[:, 4:]).all())


def test_large_and_small_scales(jl):
    """Scores up to several hundred (one key takes all the weight), and values of 1e-20 and 1e20."""
    d, hq, hkv, L = 128, 4, 1, 200
    cos, sin = tables(L, d)
    sl = dev([L], torch.int32)
    q = normal(21, 1, hq, d)
    for ks, vs in ((60.0, 1.0), (1e-30, 1.0), (1.0, 1e-20), (1.0, 1e20)):
        cache = list(random_cache(22, 1, L, hkv, d))
        s = cache[2].float()
        s[..., :4] *= ks
        s[..., 4:] *= vs
        cache[2] = s.to(torch.bfloat16)
        want = expect(q, cache, [L], 0, L)  # G = 1: scores without a rotation, so exact products of the codes
        out, lse = jl.jl_bifocal_decode_q4(q, *cache, sl, L, 0, L, cos, sin)
        err = np.abs(R.f32(out) - want[0]) / vs
        assert err.max() <= 2e-2 and err.mean() <= 2e-3
        # fp32 sums of 128 products and queries to 2^-22 of their largest: 2^-20 of the scores' size
        assert np.abs(R.f32(lse) - want[1]).max() <= 2.0**-20 * max(1.0, np.abs(want[1]).max()) * 8


def test_softmax_scale_out_of_a_given_buffer_and_other_stream(jl):
    d, hq, hkv, L = 128, 16, 8, 777
    cache = random_cache(23, 1, 800, hkv, d)
    q = normal(24, 1, hq, d)
    cos, sin = tables(800, d)
    sl = dev([L], torch.int32)
    k, v = R.values(*cache)
    want = R.decode(R.f32(q)[0].astype(np.float64), k[0, :L], v[0, :L], 100, 300, BASE, scale=0.02)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = torch.empty_like(q), torch.empty((1, hq), device="cuda")
    ws = torch.empty(jl.jl_bifocal_decode_q4_workspace_size(hq, d), dtype=torch.uint8, device="cuda")
    ws.fill_(255)  # NaN in every float
    s.wait_stream(torch.cuda.current_stream())
    jl.jl_bifocal_decode_q4(q, *cache, sl, 800, 100, 300, cos, sin, softmax_scale=0.02, out=out, lse=lse, workspace=ws, stream=s)
    other, _ = jl.jl_bifocal_decode_q4(q, *cache, sl, 800, 100, 300, cos, sin, softmax_scale=0.02, stream=s.cuda_stream)
    jl.jl_sync_status(s)
    close(out, lse, (want[0][None], want[1][None]))
    assert torch.equal(out, other)


def test_bad_lengths_and_pages_are_reported(jl):
    d, hq, hkv = 64, 4, 2
    cache = random_cache(25, 3, 64, hkv, d)
    q = normal(26, 3, hq, d)
    cos, sin = tables(64, d)
    lens = (40, -3, 50)
    out, lse = jl.jl_bifocal_decode_q4(q, *cache, dev(lens, torch.int32), 45, 8, 16, cos, sin)
    with pytest.raises(jl.JetLongError, match="outside"):
        jl.jl_sync_status()
    assert bool(torch.isnan(out[1:]).all()) and bool(torch.isnan(lse[1:]).all())
    want = expect(q[:1], [x[:1] for x in cache], [40], 8, 16)
    close(out[:1], lse[:1], want)
    pools = [paged(x, 32) for x in cache]
    table = pools[0][1].clone()
    table[0, 1] = 99  # keys 32 .. 39 of entry 0 read as zeros
    out, lse = jl.jl_bifocal_decode_q4_paged(q, *(x for x, _ in pools), table, dev((40, 5, 0), torch.int32), 64, 8, 4096, cos, sin)
    with pytest.raises(jl.JetLongError, match="outside"):
        jl.jl_sync_status()
    cache[2][0, 32:] = 0
    close(out[:2], lse[:2], expect(q[:2], [x[:2] for x in cache], [40, 5], 8, 4096))
    jl.jl_sync_status()


# ------------------------------------------------------------------- together --

def test_a_stream_prefill_append_decode_across_g(jl):
    """A prompt filled in two chunks, tokens appended one by one across a change of G by a captured and
    replayed step, each decode against the definition on the cache as it then stands; then the cache read
    back and continued by a chunked prefill."""
    d, hq, hkv, w0, w_pre, stride = 128, 8, 2, 40, 100, 320
    total = 304
    q, k, v = normal(31, total, hq, d), normal(32, total, hkv, d), normal(33, total, hkv, d)
    cos, sin = tables(stride, d)
    cache = jl.jl_kv_cache_q4_empty(1, stride, hkv, d)
    for lo, hi in ((0, 190), (190, 296)):
        jl.jl_kv_cache_fill_q4(k[lo:hi], v[lo:hi], dev([0, hi - lo], torch.int32), cos, sin, *cache,
                               past_lens=dev([lo], torch.int32))
    sl = dev([297], torch.int32)
    qs, ks, vs = (torch.empty_like(x[:1]) for x in (q, k, v))
    qr, out, lse = torch.empty_like(qs), torch.empty_like(qs), torch.empty((1, hq), device="cuda")
    ws = torch.empty(jl.jl_bifocal_decode_q4_workspace_size(hq, d), dtype=torch.uint8, device="cuda")

    def step():
        jl.jl_decode_append_q4(qs, ks, vs, sl, cos, sin, *cache, q_out=qr)
        jl.jl_bifocal_decode_q4(qr, *cache, sl, stride, w0, w_pre, cos, sin, out=out, lse=lse, workspace=ws)

    def load(n):
        for x, y in ((qs, q), (ks, k), (vs, v)):
            x.copy_(y[n:n + 1])
        sl.fill_(n + 1)

    load(296)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in range(296, total):  # L = 297 .. 304: G goes from 3 to 4 at 301
        load(n)
        graph.replay()
        torch.cuda.synchronize()
        close(out, lse, expect(qr, cache, [n + 1], w0, w_pre))
    jl.jl_sync_status()
    kb, vb = jl.jl_kv_cache_read_q4(*cache, sl)
    # a chunk of four more queries against the cache read back, beside the same call on the reference's cache
    ref = [torch.zeros_like(kb), torch.zeros_like(vb)]
    for x, y in zip(ref, R.values(*(x[:, :total] for x in cache))):
        x[:, :total] = torch.from_numpy(y.astype(np.float32)).to(torch.bfloat16).cuda()
    cu, past = dev([0, 4], torch.int32), dev([total - 4], torch.int32)
    kb[:, total:] = vb[:, total:] = 0
    a, _ = jl.jl_bifocal_prefill_chunk(q[:4], cu, past, 4, total, kb, vb, w0, w_pre, cos, sin)
    b, _ = jl.jl_bifocal_prefill_chunk(q[:4], cu, past, 4, total, *ref, w0, w_pre, cos, sin)
    assert torch.equal(a, b)


def test_two_captured_graphs_share_a_workspace_in_turn(jl):
    d, hq, hkv = 128, 16, 8
    cos, sin = tables(700, d)
    ws = torch.empty(jl.jl_bifocal_decode_q4_workspace_size(hq, d), dtype=torch.uint8, device="cuda")
    runs = []
    for seed, L in ((41, 700), (42, 333)):
        cache, q, sl = random_cache(seed, 1, 700, hkv, d), normal(seed, 1, hq, d), dev([L], torch.int32)
        out = torch.empty_like(q)
        call = lambda q=q, cache=cache, sl=sl, out=out: jl.jl_bifocal_decode_q4(  # noqa: E731
            q, *cache, sl, 700, 64, 200, cos, sin, out=out, want_lse=False, workspace=ws)
        call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        runs.append((g, out, expect(q, cache, [L], 64, 200), (q, cache, sl)))
    for _ in range(3):
        for g, out, want, _ in runs:
            out.zero_()
            g.replay()
        torch.cuda.synchronize()
        for _, out, want, _ in runs:
            close(out, None, want)


@pytest.mark.parametrize("d,hq,hkv", [(128, 16, 4), (128, 32, 8), (64, 8, 8), (128, 4, 1), (128, 16, 2), (128, 20, 2)])
def test_a_long_cache(jl, d, hq, hkv):
    """G = 3 at 70001 keys: many tiles to a CTA, offsets behind 2^31 bits in the codes, lse to fp32's accuracy."""
    L = 70001
    cache = random_cache(43, 1, L, hkv, d)
    q = normal(44, 1, hq, d)
    cos, sin = tables(L, d)
    out, lse = jl.jl_bifocal_decode_q4(q, *cache, dev([L], torch.int32), L, 4096, 32768, cos, sin)
    jl.jl_sync_status()
    want = expect(q, cache, [L], 4096, 32768)
    close(out, lse, want)
    assert np.abs(R.f32(lse) - want[1]).max() <= 1e-4


@pytest.mark.parametrize("d,hq,hkv", SHAPES + [(64, 12, 2), (64, 8, 1), (64, 16, 1), (64, 32, 2), (128, 32, 2), (128, 15, 3)])
def test_remote_scores_are_as_good_as_fp32(jl, d, hq, hkv):
    """A turned component is off by the 44 steps of its cos and sin, 14 * 44 * 2^-24 code steps, and by its
    remainder's three roundings, 3 * 14 * 2^-8 * 2^-12: 7.7e-5 at the most, at a step of 0.4 and independent over
    the channels a score error of 2e-5 (1e-5 in the mean square of evenly spread ones); the lse averages that over
    the keys.  Keys turned in one fp16 number are off by 2^-8 code steps and more, fifty times that."""
    lens = (700, 2048)
    cache = random_cache(71, len(lens), 2048, hkv, d)
    q = normal(72, len(lens), hq, d)
    cos, sin = tables(2048, d)
    _, lse = jl.jl_bifocal_decode_q4(q, *cache, dev(lens, torch.int32), 2048, 0, 500, cos, sin)
    jl.jl_sync_status()
    want = expect(q, cache, lens, 0, 500)
    assert np.abs(R.f32(lse) - want[1]).max() <= 2e-5


def test_rows_past_two_gigabytes(jl):
    """A pool whose code tensors pass 2^31 bytes: the last pages are written, read and attended."""
    d, hq, hkv, page = 128, 16, 8, 256
    pages = (1 << 31) // (page * hkv * d // 2) + 3
    kc, vc, scales = jl.jl_kv_cache_q4_empty(pages, page, hkv, d)
    table = dev([[pages - 1, 0, pages - 2]], torch.int32)
    L = 700
    cos, sin = tables(768, d)
    k, v, q = normal(51, L, hkv, d), normal(52, L, hkv, d), normal(53, 1, hq, d)
    jl.jl_kv_cache_fill_q4_paged(k, v, dev([0, L], torch.int32), cos, sin, kc, vc, scales, table)
    sl = dev([L], torch.int32)
    out, lse = jl.jl_bifocal_decode_q4_paged(q, kc, vc, scales, table, sl, 768, 64, 256, cos, sin)
    kb, _ = jl.jl_kv_cache_read_q4_paged(kc, vc, scales, table, sl, rows=L)
    jl.jl_sync_status()
    flat = jl.jl_kv_cache_q4_empty(1, 768, hkv, d)
    jl.jl_kv_cache_fill_q4(k, v, dev([0, L], torch.int32), cos, sin, *flat)
    kf, _ = jl.jl_kv_cache_read_q4(*flat, sl, rows=L)
    assert torch.equal(kb, kf)
    close(out, lse, expect(q, flat, [L], 64, 256))


def test_wrong_devices_shapes_and_strides_are_refused(jl):
    cache = random_cache(1, 1, 8, 2, 64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        jl.jl_kv_cache_read_q4(*cache, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="shape"):
        jl.jl_kv_cache_read_q4(*cache, dev([8], torch.int32), starts=dev([0, 0], torch.int32))
    with pytest.raises(ValueError, match="contiguous"):
        jl.jl_kv_cache_read_q4(cache[0].flip(1)[:, ::2], cache[1][:, ::2], cache[2][:, ::2], dev([8], torch.int32))
    with pytest.raises(ValueError, match="one entry"):
        jl.jl_kv_cache_read_q4(*cache, dev([8, 8], torch.int32))
