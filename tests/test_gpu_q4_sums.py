"""The sums of the 4-bit decode by themselves: the values' sums over many keys of one warp, where the result is
a small difference, and outputs of long caches relative to their own size."""
import numpy as np
import pytest
import torch

import test_gpu_q4 as Q
from test_gpu_q4 import jl  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def uniform_codes(g, *shape):
    n = lambda: torch.randint(1, 16, shape, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    return n() | n() << 4


def value_rows(v_codes, scales):
    """The fp32 values of rows [..][d/2], [..][8], on the GPU (exact: four bits times eight)."""
    d = 2 * v_codes.shape[-1]
    place = [Q.R.value_place(d, c) for c in range(d)]
    byte = torch.tensor([b for b, _ in place], device="cuda")
    shift = torch.tensor([s for _, s in place], device="cuda", dtype=torch.uint8)
    group = torch.tensor([4 + Q.R.value_group(d, c) for c in range(d)], device="cuda")
    return ((v_codes[..., byte] >> shift) & 15).float().sub_(8).mul_(scales.float()[..., group])


def key_rows(k_codes, scales):
    d = 2 * k_codes.shape[-1]
    place = [Q.R.key_place(d, c) for c in range(d)]
    byte = torch.tensor([b for b, _ in place], device="cuda")
    shift = torch.tensor([s for _, s in place], device="cuda", dtype=torch.uint8)
    group = torch.tensor([Q.R.key_group(d, c) for c in range(d)], device="cuda")
    return ((k_codes[..., byte] >> shift) & 15).float().sub_(8).mul_(scales.float()[..., group])


def rope64(x, pos):
    """R(pos) x, rows x [n][..][d] in 64 bits, pos [n]."""
    h = x.shape[-1] // 2
    ang = pos.double()[:, None] * Q.BASE ** (-2.0 * torch.arange(h, device="cuda", dtype=torch.float64) / (2 * h))
    z = torch.complex(x[..., :h], x[..., h:]) * torch.polar(torch.ones_like(ang), ang).unflatten(0, (-1, *[1] * (x.dim() - 2)))
    return torch.cat([z.real, z.imag], -1)


def expect_gpu(q, cache, L, w0, w_pre):
    """The definition in 64 bits on the GPU: q [hq][d], cache rows [stride][hkv][..] of one entry -> out, lse, and
    what errors are relative to: the sums of the weights times the values' sizes, and by channel the largest weight
    times value scale."""
    k, v = key_rows(cache[0][:L], cache[2][:L]).double(), value_rows(cache[1][:L], cache[2][:L]).double()
    grow, i = max(1, -(-L // w_pre)), L - 1
    edge = max(0, min(L, i - w0 + 1)) if grow > 1 else 0  # keys before it are remote
    j = torch.arange(edge, device="cuda")
    k[:edge] = rope64(k[:edge], j // grow - j)
    near = q.double()
    far = rope64(near[None], torch.tensor([i // grow - i], device="cuda"))[0]
    kv = torch.arange(q.shape[0], device="cuda") // (q.shape[0] // k.shape[1])
    k, v = k.transpose(0, 1)[kv], v.transpose(0, 1)[kv]  # [hq][L][d]
    s = torch.cat([(k[:, :edge] @ far[:, :, None]), (k[:, edge:] @ near[:, :, None])], 1)[..., 0] / q.shape[1] ** 0.5
    w = torch.softmax(s, -1)
    step = cache[2][:L].double()[..., 4:].transpose(0, 1)[kv]  # [hq][L][4]
    most = (w[..., None] * step).amax(1).repeat_interleave(q.shape[1] // 4, 1)
    return (w[:, None] @ v)[:, 0], torch.logsumexp(s, -1), (w[:, None] @ v.abs())[:, 0], most


def excess(out, want):
    """How far a bf16 result is off beyond its own rounding (half a step of the wanted value's binade), as a
    share of the root mean square of its head's wanted values."""
    want = want.double()
    step = torch.exp2(torch.floor(torch.log2(want.abs().clamp(min=2.0**-120))))
    over = (out.double() - want).abs() - 2.0**-8 * step
    return (over / want.square().mean(-1, keepdim=True).sqrt()).max().item()


# (B, L, hq, hkv, d): one entry over all CTAs; one entry a CTA, all of its keys in eight warps, or in one
MANY = [(1, 131072, 32, 8, 128), (148, 65536, 1, 1, 64), (150, 20000, 4, 1, 128), (148, 16384, 16, 1, 128),
        (148, 8192, 8, 8, 64), (149, 9000, 10, 2, 128)]


@pytest.mark.parametrize("B,L,hq,hkv,d", MANY)
def test_values_that_cancel_leave_nothing(jl, B, L, hq, hkv, d):  # noqa: F811
    """Equal weights, keys 2n and 2n + 1 with opposite values, so the result is 0.  While the sums that the kernel
    holds stay below 2^9 weights, an instruction that is off by a last place two bits above fp32's is off by 2^-22
    of that: 2^-13 of a weight for sixteen keys, if always to one side 2^-17 of a value's step.  The weights' sum is
    one of L / 16 equal terms a lane and head at the most, each addition off by half a last place, 2^-24."""
    g = torch.Generator(device="cuda").manual_seed(91)
    vc = uniform_codes(g, B, L // 2, 1, hkv, d // 2).expand(B, L // 2, 2, hkv, d // 2).clone()
    low, high = vc[:, :, 1] & 15, vc[:, :, 1] >> 4
    vc[:, :, 1] = (16 - low) | (16 - high) << 4
    sc = torch.empty(B, L // 2, 1, hkv, 8, device="cuda").uniform_(0.15, 0.31, generator=g).bfloat16()
    sc = sc.expand(B, L // 2, 2, hkv, 8).clone()
    vc, sc, kc = vc.flatten(1, 2), sc.flatten(1, 2), uniform_codes(g, B, L, hkv, d // 2)
    tab = torch.ones(L, d // 2, device="cuda")
    q = torch.zeros(B, hq, d, dtype=torch.bfloat16, device="cuda")
    out, lse = jl.jl_bifocal_decode_q4(q, kc, vc, sc, Q.dev([L] * B, torch.int32), L, 0, L, tab, tab)
    jl.jl_sync_status()
    assert out.float().abs().max().item() <= 0.31 * 2.0**-17
    assert (lse - np.log(L)).abs().max().item() <= 2.0**-20 * np.log(L) + 2.0**-24 * L / 16


@pytest.mark.parametrize("B,L,hq,hkv,d", MANY)
def test_mean_of_many_values(jl, B, L, hq, hkv, d):  # noqa: F811
    """Equal weights: their products with a bf16 scale are exact in fp16, so what is left beside the output's
    rounding is that of the sums, which are of the size of the result: a thousandth of it covers 2^13 roundings of
    2^-23 all to one side."""
    g = torch.Generator(device="cuda").manual_seed(92)
    kc, vc = uniform_codes(g, B, L, hkv, d // 2), uniform_codes(g, B, L, hkv, d // 2)
    sc = torch.empty(B, L, hkv, 8, device="cuda").uniform_(0.15, 0.31, generator=g).bfloat16()
    tab = torch.ones(L, d // 2, device="cuda")
    q = torch.zeros(B, hq, d, dtype=torch.bfloat16, device="cuda")
    out, _ = jl.jl_bifocal_decode_q4(q, kc, vc, sc, Q.dev([L] * B, torch.int32), L, 0, L, tab, tab)
    jl.jl_sync_status()
    for b in (0, B // 2, B - 1):
        want = value_rows(vc[b], sc[b]).double().mean(0).repeat_interleave(hq // hkv, 0)
        assert excess(out[b], want) <= 1e-3


@pytest.mark.parametrize("B,L,hq,hkv,d", [(148, 65536, 1, 1, 64), (150, 20000, 4, 1, 128), (148, 16384, 8, 8, 64),
                                          (148, 16384, 16, 1, 128), (149, 9000, 10, 2, 128)])
def test_many_keys_a_warp_relative_to_their_size(jl, B, L, hq, hkv, d):  # noqa: F811
    """Batches that leave a warp up to 16384 keys, values quantised from a normal distribution.  Weights rounded
    to fp16 as in the test below: six deviations of 2^-11 / sqrt(3).  An instruction for sixteen keys may cut the
    running sum by its last place, 2^-23 of it, to one side: 2^-13 after a warp's 1024 of them."""
    g = torch.Generator(device="cuda").manual_seed(96)
    kc = uniform_codes(g, B, L, hkv, d // 2)
    vc, sc = torch.empty_like(kc), torch.empty(B, L, hkv, 8, dtype=torch.bfloat16, device="cuda")
    tab = torch.ones(L, d // 2, device="cuda")
    for b in range(B):  # the values as the writer quantises them
        v = torch.randn(L, hkv, d, generator=g, device="cuda").bfloat16()
        spare = torch.empty(1, L, hkv, d // 2, dtype=torch.uint8, device="cuda")
        jl.jl_kv_cache_fill_q4(v, v, Q.dev([0, L], torch.int32), tab, tab * 0, spare, vc[b:b + 1], sc[b:b + 1])
    sc[..., :4].uniform_(0.15, 0.31, generator=g)
    q = torch.randn(B, hq, d, generator=g, device="cuda").bfloat16()
    out, lse = jl.jl_bifocal_decode_q4(q, kc, vc, sc, Q.dev([L] * B, torch.int32), L, 0, L, tab, tab)
    jl.jl_sync_status()
    for b in (0, B // 2, B - 1):
        want, want_lse, _, _ = expect_gpu(q[b], (kc[b], vc[b], sc[b]), L, 0, L)
        assert excess(out[b], want) <= 6 * 2.0**-11 / 3**0.5 + 2.0**-13
        assert (lse[b] - want_lse).abs().max().item() <= 2e-5


@pytest.mark.parametrize("d,hq,hkv", [(128, 32, 8), (128, 16, 8), (64, 16, 4), (128, 20, 5), (128, 16, 1), (64, 8, 1)])
@pytest.mark.parametrize("w0,w_pre", [(4096, 32768), (0, 1 << 20)])
def test_long_outputs_relative_to_their_size(jl, d, hq, hkv, w0, w_pre):  # noqa: F811
    """131072 keys.  A weight times a value scale is rounded to fp16, by 2^-11 at the most and independently of the
    others: a root mean square of 2^-11 / sqrt(3) of each term, and as much of the output, whose terms have either
    sign alike.  Six of those deviations cover the 4096 outputs; the scores' and sums' fp32 errors are far below."""
    L = 131072
    cache = Q.random_cache(93, 1, L, hkv, d)
    q = Q.normal(94, 1, hq, d)
    cos, sin = Q.tables(L, d)
    out, lse = jl.jl_bifocal_decode_q4(q, *cache, Q.dev([L], torch.int32), L, w0, w_pre, cos, sin)
    jl.jl_sync_status()
    want, want_lse, _, _ = expect_gpu(q[0], [x[0] for x in cache], L, w0, w_pre)
    assert excess(out[0], want) <= 6 * 2.0**-11 / 3**0.5
    assert (lse[0] - want_lse).abs().max().item() <= 2e-5


def scale_pattern(name, B, L, hkv):
    """Factors [B][L][hkv][4] of the value scales."""
    g = np.random.default_rng(97)
    groups = np.broadcast_to(np.array([1.0, 1e10, 1e-20, 1e30]), (B, L, hkv, 4))
    ramp = 10.0 ** np.linspace(-15, 15, L)[None, :, None, None]
    return {
        "groups": groups,
        "bits": np.broadcast_to(2.0 ** np.array([-97, 0, 50, 110]), (B, L, hkv, 4)),
        "keys": 10.0 ** g.uniform(-20, 20, (B, L, hkv, 1)) * np.ones(4),
        "both": 10.0 ** g.uniform(-20, 20, (B, L, hkv, 4)),
        "growing": ramp * np.ones((B, L, hkv, 4)),
        "falling": 1 / ramp * np.array([1.0, 1e10, 1e-20, 1e20]),
        "zeros first": np.where(np.arange(L)[None, :, None, None] < 500, 0.0, groups),
        "zeros last": np.where(np.arange(L)[None, :, None, None] < 40, groups, 0.0),
        "one group of zeros": groups * np.array([1.0, 0.0, 1.0, 1.0]),
    }[name]


@pytest.mark.parametrize("d,hq,hkv", [(128, 32, 8), (128, 3, 3), (64, 8, 2), (128, 12, 2), (64, 6, 1), (128, 16, 1), (64, 9, 1)])
@pytest.mark.parametrize("pattern", ["groups", "bits", "keys", "both", "growing", "falling", "zeros first", "zeros last",
                                     "one group of zeros"])
def test_value_scales_of_any_size(jl, d, hq, hkv, pattern):  # noqa: F811
    """Each channel against what its own weights and values allow.  A weight times a scale is rounded to fp16, by 2^-11
    of it or, among subnormals, by 2^-25, where the largest of its group was 2^6 at least when the factor was set:
    2^-31 of that for each key, times a code of 7.  The scores are off by some 2e-5 (2^-15) and the fp32 sums by less;
    the output by half a bf16 step."""
    lens = (777, 30)
    cache = list(Q.random_cache(98, 2, 777, hkv, d))
    factor = torch.from_numpy(scale_pattern(pattern, 2, 777, hkv).copy()).cuda()
    cache[2][..., 4:] = (cache[2][..., 4:].double() * factor).bfloat16()
    q = Q.normal(99, 2, hq, d)
    cos, sin = Q.tables(777, d)
    out, lse = jl.jl_bifocal_decode_q4(q, *cache, Q.dev(lens, torch.int32), 777, 50, 300, cos, sin)
    jl.jl_sync_status()
    for b, L in enumerate(lens):
        rows = [x[b] for x in cache]
        want, want_lse, size, most = expect_gpu(q[b], rows, L, 50, 300)
        step = torch.exp2(torch.floor(torch.log2(want.abs().clamp(min=2.0**-126))) - 8)
        assert bool(((out[b].double() - want).abs() <= step + (2.0**-11 + 2.0**-15) * size + 7 * L * 2.0**-31 * most).all())
        assert (lse[b] - want_lse).abs().max().item() <= 2e-5


@pytest.mark.parametrize("d,hq,hkv", [(128, 32, 8), (64, 8, 2), (128, 12, 2), (128, 16, 1)])
def test_a_lone_key_gives_its_values(jl, d, hq, hkv):  # noqa: F811
    """Lengths of one: the weight is 1, so a product with a bf16 scale is exact in fp16, and the output
    is the key's value rounded once, ties included."""
    B = 9
    cache = Q.random_cache(95, B, 4, hkv, d)
    q = Q.normal(96, B, hq, d)
    cos, sin = Q.tables(4, d)
    out, _ = jl.jl_bifocal_decode_q4(q, *cache, Q.dev([1] * B, torch.int32), 4, 2, 3, cos, sin)
    jl.jl_sync_status()
    want = value_rows(cache[1][:, 0], cache[2][:, 0]).bfloat16().repeat_interleave(hq // hkv, 1)
    assert torch.equal(out, want)


@pytest.mark.parametrize("octaves", [0.9, 3.3, 7.7, 30.0])
@pytest.mark.parametrize("d,hq,hkv", [(128, 16, 1), (64, 4, 1), (128, 8, 2)])
def test_scores_that_rise_with_the_keys(jl, d, hq, hkv, octaves):  # noqa: F811
    """Scores that rise by some octaves every 128 keys, value scales that fall as fast, so that every key counts and
    the references move again and again; a batch that leaves each entry to one CTA or two.  Bounds as above, with the
    scores' error on top: fp32 scores, up to 700 in units of ln 2 here, to 2^-22 of themselves."""
    B, L = 150, 128 * max(3, min(40, int(700 / octaves)))
    g = torch.Generator(device="cuda").manual_seed(97)
    kc = torch.full((B, L, hkv, d // 2), 0xff, dtype=torch.uint8, device="cuda")  # 7 in every channel
    vc = uniform_codes(g, B, L, hkv, d // 2)
    level = torch.arange(L, device="cuda") // 128 * octaves  # of the first head, in octaves
    q = torch.rand(B, hq, 1, generator=g, device="cuda").mul_(0.05).add_(0.95).expand(B, hq, d).bfloat16()
    unit = 7 * d**0.5  # the score of a key scale of 1 for a query of ones
    sc = torch.empty(B, L, hkv, 8, device="cuda").uniform_(0.9, 1.1, generator=g)
    sc[..., :4] = (level * np.log(2) / unit)[:, None, None]
    sc[..., 4:] *= torch.exp2(60 - level.clamp(max=150))[:, None, None]
    sc[..., 5] *= 1e-20
    sc = sc.bfloat16()
    tab = torch.ones(L, d // 2, device="cuda")
    out, lse = jl.jl_bifocal_decode_q4(q, kc, vc, sc, Q.dev([L] * B, torch.int32), L, 0, L, tab, tab)
    jl.jl_sync_status()
    for b in (0, 1, B // 2, B - 1):
        want, want_lse, size, most = expect_gpu(q[b], (kc[b], vc[b], sc[b]), L, 0, L)
        step = torch.exp2(torch.floor(torch.log2(want.abs().clamp(min=2.0**-126))) - 8)
        slack = (2.0**-11 + 700 * np.log(2) * 2.0**-22) * size + 7 * L * 2.0**-31 * most
        assert bool(((out[b].double() - want).abs() <= step + slack).all())
        assert bool(((lse[b] - want_lse).abs() <= 2.0**-21 * want_lse.abs() + 1e-5).all())


@pytest.mark.parametrize("d,hq,hkv", [(128, 16, 1), (64, 4, 1), (128, 8, 2)])
def test_a_group_that_grows_while_scores_rise(jl, d, hq, hkv):  # noqa: F811
    """Every 128 keys one group's value scales grow by eight octaves, so that references and factors move each time,
    while scores rise by 0.97 and the other groups' scales fall by as much: their keys count alike to the last, and a
    factor that lost that part of an octave at every move would round them among subnormals."""
    B, tiles = 150, 27
    L = 128 * tiles
    g = torch.Generator(device="cuda").manual_seed(98)
    kc = torch.full((B, L, hkv, d // 2), 0xff, dtype=torch.uint8, device="cuda")  # 7 in every channel
    vc = uniform_codes(g, B, L, hkv, d // 2)
    tile = torch.arange(L, device="cuda") // 128
    q = torch.full((B, hq, d), 0.97 * np.log(2) * 128 / (7 * d**0.5), device="cuda").bfloat16()
    sc = torch.empty(B, L, hkv, 8, device="cuda").uniform_(0.9, 1.1, generator=g)
    sc[..., :4] = (tile / 128)[:, None, None]  # exact in bf16
    sc[..., 4:7] *= torch.exp2(-0.97 * tile)[:, None, None]
    sc[..., 7] *= torch.exp2(-95 + 8.1 * tile)[:, None]
    sc = sc.bfloat16()
    tab = torch.ones(L, d // 2, device="cuda")
    out, _ = jl.jl_bifocal_decode_q4(q, kc, vc, sc, Q.dev([L] * B, torch.int32), L, 0, L, tab, tab)
    jl.jl_sync_status()
    for b in (0, B // 2, B - 1):
        want, _, size, most = expect_gpu(q[b], (kc[b], vc[b], sc[b]), L, 0, L)
        # beside the largest of a group all keys of the last tiles count, so the root mean square of the
        # roundings stands for them: six deviations, as in the tests of long outputs above
        at = slice(0, 3 * d // 4)
        assert excess(out[b][:, at], want[:, at]) <= 6 * 2.0**-11 / 3**0.5
        step = torch.exp2(torch.floor(torch.log2(want.abs().clamp(min=2.0**-126))) - 8)
        assert bool(((out[b].double() - want).abs() <= step + (2.0**-11 + 2.0**-15) * size + 7 * L * 2.0**-31 * most).all())
