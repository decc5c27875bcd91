"""What is measured of the 4-bit KV cache: writing it, reading it back, and decoding against it.

The cache is the framework's base-RoPE KV cache held in 4 bits.  One (position, KV head) row of d channels is

  k_codes  uint8 [d / 2]   key codes, two to a byte
  v_codes  uint8 [d / 2]   value codes, two to a byte
  scales   bf16  [8]       four key scales, then four value scales

and stands for x = scale * (code - 8), code in 1 .. 15.  A key scale is shared by the d/8 rotate-half pairs
(c, c + d/2) of its group, so a rotation does not change the group; a value scale by d/4 neighbouring channels.
The codes are stored in the order in which a warp's matrix instructions take them:

  key pair c: group w = c / (d/8), then r = c % (d/8), t = r / (d/32), e = r % (d/32); the pair's byte is
    16 t + 4 w + e                          for d = 128,
    8 t + 4 (w / 2) + 2 e + w % 2           for d = 64,
    with channel c in the low four bits and channel c + d/2 in the high four;
  value channel c: byte (d/16) (c % 8) + c / 16, in the low four bits where c % 16 < 8, else in the high four.

A group's scale is bf16(max |x| / 7), zero where that is below 2^-100 and NaN where the group holds a NaN or an
infinity; code = clamp(round(x / scale), -7, 7) + 8, halves to even, and 8 where the scale is zero or NaN.  Keys are
rotated in fp32 first.
"""
import math

import torch

own = False

DEV = "cuda"
F32, F64, BF16 = torch.float32, torch.float64, torch.bfloat16


# ---------------------------------------------------------------- the cases --

def listed():
    # Head layouts and lengths: the framework's own decode and prefill workloads (32/8 and 16/8 heads of 128 channels,
    # window 32768, local window 4096, caches of 8K to 128K, packed sequences of 4K to 128K).
    return [
        # one short conversation, one user: the smallest call, all latency
        decode("decode_short", "1000", 16, 8, 128),
        # a batch of small-headed rows of odd lengths, one slot of the batch empty
        decode("decode_d64_ragged", "1,257,4097,0,1023,3333", 8, 2, 64, w0=512, w_pre=8192, theta=1e4),
        # the headline decode's shortest and longest caches (G = 1 and G = 4)
        decode("decode_8k", "8192", 32, 8, 128),
        decode("decode_128k", "131072", 32, 8, 128),
        # a serving batch of ragged lengths, each with its own G, in pages of 128 positions
        decode("decode_paged_ragged", "5420,9973,17041,30011,44444,70001,98305,120712", 16, 8, 128, page=128),
        # one token written to a cache, for one user and for a paged batch
        append("append_one", "8192", 32, 8, 128),
        append("append_paged_batch", ",".join(str(1 + 61 * n) for n in range(64)), 16, 8, 128, page=64),
        # a chunk that continues a conversation, a whole long prompt, packed prompts into pages
        fill("fill_chunk", "777", "1203", 8, 128),
        fill("fill_128k", "131072", "0", 8, 128),
        fill("fill_paged_d64", "5420,33,9973,1,0,17041", "0,7,130,64,5,1", 4, 64, page=128, theta=1e4),
        # a cache taken back to 16 bits: one user's long one, and a ragged batch's tails
        read("read_64k", "65536", "0", 8, 128),
        read("read_ragged", "5420,9973,30,4097", "20,0,30,4000", 2, 128),
    ]


def decode(name, lens, hq, hkv, d, w0=4096, w_pre=32768, theta=1e6, page=0):
    return {"name": name, "op": "decode", "lens": lens, "hq": hq, "hkv": hkv, "d": d, "w0": w0, "w_pre": w_pre, "theta": theta, "page": page}


def append(name, lens, hq, hkv, d, theta=1e6, page=0):
    return {"name": name, "op": "append", "lens": lens, "hq": hq, "hkv": hkv, "d": d, "theta": theta, "page": page}


def fill(name, new, past, hkv, d, theta=1e6, page=0):
    return {"name": name, "op": "fill", "new": new, "past": past, "hkv": hkv, "d": d, "theta": theta, "page": page}


def read(name, lens, starts, hkv, d, page=0):
    return {"name": name, "op": "read", "lens": lens, "starts": starts, "hkv": hkv, "d": d, "page": page}


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["decode", "decode", "append", "fill", "read"])
    d, hkv = rng.choice([128, 128, 64]), rng.choice([1, 2, 3, 4, 5, 8, 8, 12])
    group = rng.choice([1, 2, 3, 4, 4, 5, 8, 16])
    page, theta = rng.choice([0, 0, 32, 64, 128, 256]), rng.choice([1e4, 1e6])
    batch = rng.choice([1, 1, log(1, 16)])
    longest = log(1, min(131072, 8 * 131072 // (batch * hkv)))  # no more tokens x heads than the largest listed case
    lens = [longest] + [rng.randint(0, longest) for _ in range(batch - 1)]
    rng.shuffle(lens)
    text = lambda v: ",".join(map(str, v))  # noqa: E731
    if op == "decode":
        c = decode("", text(lens), hkv * group, hkv, d, rng.choice([0, 128, 1000, 4096]), rng.choice([4096, 8192, 32768]), theta, page)
    elif op == "append":
        c = append("", text([max(1, n) for n in lens]), hkv * group, hkv, d, theta, page)
    elif op == "fill":
        c = fill("", text(lens), text([rng.randint(0, 300) for _ in lens]), hkv, d, theta, page)
    else:
        c = read("", text(lens), text([rng.randint(0, n) // rng.choice([1, 1000]) for n in lens]), hkv, d, page)
    del c["name"]
    return c


def numbers(text):
    return [int(x) for x in text.split(",")]


# --------------------------------------------------------------- the inputs --

def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    hkv, d, op = c["hkv"], c["d"], c["op"]
    normal = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    if op == "fill":
        new, past = numbers(c["new"]), numbers(c["past"])
        lens = [a + b for a, b in zip(new, past)]
    else:
        lens = numbers(c["lens"])
    batch, longest = len(lens), max(1, max(lens))
    s = {"case": c, "lens": ints(lens), "max_len": longest}
    # keys with outlier channels, values without; both of unit variance
    outlier = torch.empty(d, device=DEV).uniform_(0.5, 2.0, generator=gen)

    page = c["page"]
    if page:  # a pool with the entries' pages in a mixed order
        per = -(-longest // page)
        pages = batch * per
        s["block_table"] = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32).view(batch, per)
        outer = (pages, page)
    else:
        stride = longest + 5
        s["block_table"] = None
        outer = (batch, stride)
    shape = (*outer, hkv)
    if op in ("decode", "read"):  # a cache as it stands after its keys and values were written
        k, v = normal(*shape, d).mul_(outlier), normal(*shape, d)
        kq, ks = quantise_keys(k)
        del k
        vq, vs = quantise_values(v)
        del v
        s["k_codes"], s["v_codes"], s["scales"] = kq, vq, torch.cat([ks, vs], -1).contiguous()
    else:
        s["k_codes"] = torch.zeros(*shape, d // 2, dtype=torch.uint8, device=DEV)
        s["v_codes"] = torch.zeros_like(s["k_codes"])
        s["scales"] = torch.zeros(*shape, 8, dtype=BF16, device=DEV)
    if op != "read":
        ang = torch.arange(longest, device=DEV, dtype=F64)[:, None] * frequencies(d, c["theta"])
        s["cos"], s["sin"] = ang.cos().to(F32), ang.sin().to(F32)
    if op in ("decode", "append"):
        s["q"] = normal(batch, c["hq"], d).to(BF16)
    if op == "append":
        s["k"], s["v"] = normal(batch, hkv, d).mul_(outlier).to(BF16), normal(batch, hkv, d).to(BF16)
        s["starts"] = s["lens"] - 1
    if op == "fill":
        total = sum(new)
        s["k"], s["v"] = normal(total, hkv, d).mul_(outlier).to(BF16), normal(total, hkv, d).to(BF16)
        s["cu"] = ints([sum(new[:n]) for n in range(batch + 1)])
        s["starts"] = ints(past)
    if op == "read":
        s["starts"] = ints(numbers(c["starts"]))
    if op == "append":
        s["rows"] = 1
    elif op in ("fill", "read"):
        first = past if op == "fill" else numbers(c["starts"])
        s["rows"] = max(1, max(a - b for a, b in zip(lens, first)))
    if op != "decode":  # where a read leaves its rows; those behind an entry's last stay as they are
        s["k_out"] = torch.zeros(batch, s["rows"], hkv, d, dtype=BF16, device=DEV)
        s["v_out"] = torch.zeros_like(s["k_out"])
    return s


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def frequencies(d, theta):
    return theta ** (-2.0 * torch.arange(d // 2, device=DEV, dtype=F64) / d)


# ----------------------------------------------------------------- one pass --

def run(s):
    if own:
        return run_own(s)
    op = s["case"]["op"]
    if op == "decode":
        return plain_decode(s)
    if op == "append":
        at = (s["lens"] - 1).long()
        entry = torch.arange(at.numel(), device=DEV)
        q_out = rotate(s["q"].float(), s["cos"][at][:, None], s["sin"][at][:, None]).to(BF16)
        plain_write(s, s["k"], s["v"], entry, at)
        return {"q_out": q_out, **plain_read(s)}
    if op == "fill":
        t = torch.arange(s["k"].shape[0], device=DEV)
        entry = torch.searchsorted(s["cu"][1:].long(), t, right=True)
        plain_write(s, s["k"], s["v"], entry, t - s["cu"].long()[entry] + s["starts"].long()[entry])
    return plain_read(s)


def run_own(s):
    from rope_context_extension_sm_b200 import jetlong as jl
    c, table = s["case"], s["block_table"]
    cache = (s["k_codes"], s["v_codes"], s["scales"])
    if c["op"] == "decode":
        if table is None:
            out, lse = jl.jl_bifocal_decode_q4(s["q"], *cache, s["lens"], s["max_len"], c["w0"], c["w_pre"], s["cos"], s["sin"])
        else:
            out, lse = jl.jl_bifocal_decode_q4_paged(s["q"], *cache, table, s["lens"], s["max_len"], c["w0"], c["w_pre"], s["cos"], s["sin"])
        return {"out": out, "lse": lse}
    got = {}
    if c["op"] == "append":
        if table is None:
            got["q_out"] = jl.jl_decode_append_q4(s["q"], s["k"], s["v"], s["lens"], s["cos"], s["sin"], *cache)
        else:
            got["q_out"] = jl.jl_decode_append_q4_paged(s["q"], s["k"], s["v"], s["lens"], s["cos"], s["sin"], *cache, table)
    if c["op"] == "fill":
        if table is None:
            jl.jl_kv_cache_fill_q4(s["k"], s["v"], s["cu"], s["cos"], s["sin"], *cache, past_lens=s["starts"])
        else:
            jl.jl_kv_cache_fill_q4_paged(s["k"], s["v"], s["cu"], s["cos"], s["sin"], *cache, table, past_lens=s["starts"])
    if table is None:
        k, v = jl.jl_kv_cache_read_q4(*cache, s["lens"], starts=s["starts"], k_out=s["k_out"], v_out=s["v_out"])
    else:
        k, v = jl.jl_kv_cache_read_q4_paged(*cache, table, s["lens"], starts=s["starts"], k_out=s["k_out"], v_out=s["v_out"])
    return {**got, "k": k, "v": v}


# ---------------------------------------------------------- the plain forms --

def rotate(x, cos, sin):
    """R(p) x for rows of d channels in the rotate-half pairing; each product and sum is rounded to fp32."""
    a, b = x.chunk(2, -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def key_bytes(d):
    c = torch.arange(d // 2, device=DEV)
    w, r = c // (d // 8), c % (d // 8)
    t, e = r // (d // 32), r % (d // 32)
    return 16 * t + 4 * w + e if d == 128 else 8 * t + 4 * (w // 2) + 2 * e + w % 2


def value_places(d):
    c = torch.arange(d, device=DEV)
    return (d // 16) * (c % 8) + c // 16, 4 * (c % 16 // 8)


def codes_of(x, group):
    """(codes, scales) of rows x [.., d]; `group`: the scale of each channel."""
    d = x.shape[-1]
    order = torch.argsort(group, stable=True)
    top = x[..., order].unflatten(-1, (4, d // 4)).abs().amax(-1)
    scale = (top / 7).to(BF16)
    scale = torch.where(scale.float() < 2.0**-100, 0.0, scale)
    scale = torch.where(top.isfinite(), scale, math.nan)
    wide = scale.float()[..., group]
    code = torch.where(wide > 0, torch.round(x / wide).clamp(-7, 7) + 8, 8.0)
    return code.to(torch.uint8), scale


def quantise_keys(x):
    d = x.shape[-1]
    code, scale = codes_of(x, torch.arange(d, device=DEV) % (d // 2) // (d // 8))
    lo, hi = code.chunk(2, -1)
    at = torch.argsort(key_bytes(d))
    return (lo | hi << 4)[..., at].contiguous(), scale


def quantise_values(x):
    d = x.shape[-1]
    code, scale = codes_of(x, torch.arange(d, device=DEV) // (d // 4))
    byte, shift = value_places(d)
    low, high = torch.argsort(byte + shift * d)[: d // 2], torch.argsort(byte + shift * d)[d // 2 :]
    return (code[..., low] | code[..., high] << 4).contiguous(), scale


def values_of(k_codes, v_codes, scales):
    """The fp32 keys and values that cache rows stand for."""
    d = 2 * k_codes.shape[-1]
    c, scales = torch.arange(d, device=DEV), scales.float()
    byte, shift = value_places(d)
    k = k_codes[..., key_bytes(d)]
    k = torch.cat([k & 15, k >> 4], -1).float().sub_(8).mul_(scales[..., c % (d // 2) // (d // 8)])
    v = (v_codes[..., byte] >> shift & 15).float().sub_(8).mul_(scales[..., 4 + c // (d // 4)])
    return k, v


def rows_of(s, entry, pos):
    """Rows of the flattened cache of positions `pos` of entries `entry`."""
    if s["block_table"] is None:
        return entry * s["k_codes"].shape[1] + pos
    page = s["k_codes"].shape[1]
    return s["block_table"].long()[entry, pos // page] * page + pos % page


def plain_write(s, k, v, entry, pos):
    k = rotate(k.float(), s["cos"][pos][:, None], s["sin"][pos][:, None])
    at = rows_of(s, entry, pos)
    kq, ks = quantise_keys(k)
    vq, vs = quantise_values(v.float())
    s["k_codes"].flatten(0, 1)[at] = kq
    s["v_codes"].flatten(0, 1)[at] = vq
    s["scales"].flatten(0, 1)[at] = torch.cat([ks, vs], -1)


def plain_read(s):
    n = s["lens"] - s["starts"]
    r = torch.arange(s["rows"], device=DEV)
    entry, row = torch.nonzero(r[None] < n[:, None], as_tuple=True)
    at = rows_of(s, entry, row + s["starts"].long()[entry])
    k, v = values_of(*(s[x].flatten(0, 1)[at] for x in ("k_codes", "v_codes", "scales")))
    s["k_out"][entry, row] = k.to(BF16)
    s["v_out"][entry, row] = v.to(BF16)
    return {"k": s["k_out"], "v": s["v_out"]}


def plain_decode(s):
    c, lens = s["case"], s["lens"].long()
    hkv, d, batch = c["hkv"], c["d"], lens.numel()
    pos = torch.arange(s["max_len"], device=DEV)
    there = pos[None] < lens[:, None]
    at = rows_of(s, torch.arange(batch, device=DEV)[:, None].expand(batch, pos.numel()), torch.where(there, pos[None], 0))
    k, v = values_of(*(s[x].flatten(0, 1)[at] for x in ("k_codes", "v_codes", "scales")))
    g = ((lens + c["w_pre"] - 1) // c["w_pre"]).clamp(min=1)
    i = (lens - 1).clamp(min=0)
    remote = (i[:, None] - pos[None] >= c["w0"]) & (g[:, None] > 1) & there
    # the corrections R(f(x) - x): rows x - f(x) of the tables with the sine negated, row 0 for local keys
    n = torch.where(remote, pos[None] - pos[None] // g[:, None], 0)
    a, b = k.chunk(2, -1)
    cos, sin = s["cos"][n][:, :, None], s["sin"][n][:, :, None]
    k = torch.cat([a * cos + b * sin, b * cos - a * sin], -1)
    del a, b, cos, sin
    q = s["q"].float()
    qn = i - i // g
    far = rotate(q, s["cos"][qn][:, None], -s["sin"][qn][:, None])
    near, far = (x.unflatten(1, (hkv, -1)) for x in (q, far))
    k = k.transpose(1, 2)
    score = torch.where(remote[:, None, None], far @ k.mT, near @ k.mT) / math.sqrt(d)
    score = score.masked_fill(~there[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top.isfinite(), top, 0))
    total = p.sum(-1, keepdim=True)
    out = (p @ v.transpose(1, 2)) / torch.where(total > 0, total, 1)
    return {"out": out.flatten(1, 2).to(BF16), "lse": (top + total.log()).flatten(1)}


# ------------------------------------------------------- the bytes and sums --

def work(case):
    c = dict(case)
    hkv, d = c["hkv"], c["d"]
    row, pair = d + 16, 4 * d  # bytes of a 4-bit row (keys, values, scales), and of its keys and values in bf16
    if c["op"] == "decode":
        tokens, batch = sum(numbers(c["lens"])), len(numbers(c["lens"]))
        return {"bytes": tokens * hkv * row + batch * c["hq"] * (4 * d + 4), "flops": 4.0 * d * c["hq"] * tokens}
    if c["op"] == "append":
        batch = len(numbers(c["lens"]))
        return {"bytes": batch * (c["hq"] * 4 * d + 4 * d + hkv * (2 * pair + row)), "flops": batch * (c["hq"] + 2.0 * hkv) * 4 * d}
    if c["op"] == "fill":
        tokens = sum(numbers(c["new"]))
        return {"bytes": tokens * (4 * d + hkv * (2 * pair + row)), "flops": 10.0 * tokens * hkv * d}
    tokens = sum(max(0, a - b) for a, b in zip(numbers(c["lens"]), numbers(c["starts"])))
    return {"bytes": tokens * hkv * (row + pair) + 8, "flops": 4.0 * tokens * hkv * d}


# ------------------------------------------------------ in 64 bits, by hand --

def exact(case, seed):
    s = prepare(case, seed)
    c, d = s["case"], case["d"]
    lens = s["lens"].tolist()
    theta = frequencies(d, c["theta"]) if "theta" in c else None

    def turned(x, angle):  # rows as complex numbers, channel c with channel c + d/2, turned by `angle`
        z = torch.complex(x[..., : d // 2].to(F64), x[..., d // 2 :].to(F64)) * torch.polar(torch.ones_like(angle), angle)
        return torch.cat([z.real, z.imag], -1)

    def line(name, b, lo, hi):  # positions lo .. hi - 1 of entry b
        x = s[name]
        if s["block_table"] is None:
            return x[b, lo:hi]
        return x[s["block_table"][b].long()].flatten(0, 1)[lo:hi]

    nibble = {"k": [None] * d, "v": [None] * d}  # where each channel stands: 2 * byte + (1 for the high four bits)
    for ch in range(d):
        p, high = ch % (d // 2), ch // (d // 2)
        w, r = divmod(p, d // 8)
        t, e = divmod(r, d // 32)
        nibble["k"][ch] = 2 * (16 * t + 4 * w + e if d == 128 else 8 * t + 4 * (w // 2) + 2 * e + w % 2) + high
        nibble["v"][ch] = 2 * (d // 16 * (ch % 8) + ch // 16) + (ch // 8) % 2
    group = {"k": [ch % (d // 2) // (d // 8) for ch in range(d)], "v": [4 + ch // (d // 4) for ch in range(d)]}

    def stands_for(which, b, lo, hi):
        q = line(which + "_codes", b, lo, hi)
        q = torch.stack([q % 16, q // 16], -1).flatten(-2)[..., nibble[which]]
        return (q.to(F64) - 8) * line("scales", b, lo, hi).to(F64)[..., group[which]]

    def held(x, which):  # the values that rows x stand for once they are held in 4 bits
        g = torch.tensor([n % 4 for n in group[which]], device=DEV)
        top = torch.stack([x[..., g == n].abs().amax(-1) for n in range(4)], -1)
        step = (top / 7).to(BF16).to(F64)[..., g]
        return torch.where(step > 0, torch.round(x / step).clamp(-7, 7) * step, 0)

    if c["op"] == "decode":
        outs, lses = [], []
        for b, n in enumerate(lens):
            q = s["q"][b].to(F64)
            if n == 0:
                outs.append(torch.zeros_like(q))
                lses.append(torch.full((c["hq"],), -math.inf, device=DEV, dtype=F64))
                continue
            grow, i = max(1, -(-n // c["w_pre"])), n - 1
            edge = max(0, i - c["w0"] + 1) if grow > 1 else 0  # the first local key
            k, v = stands_for("k", b, 0, n), stands_for("v", b, 0, n)
            j = torch.arange(edge, device=DEV)
            far_q = turned(q, theta * (i // grow - i))
            k[:edge] = turned(k[:edge], ((j // grow - j).to(F64)[:, None] * theta)[:, None])
            kv = torch.arange(c["hq"], device=DEV) // (c["hq"] // c["hkv"])
            score = torch.cat([torch.einsum("hd,jhd->hj", far_q, k[:edge, kv]), torch.einsum("hd,jhd->hj", q, k[edge:, kv])], -1) / math.sqrt(d)
            lses.append(torch.logsumexp(score, -1))
            outs.append(torch.einsum("hj,jhd->hd", torch.softmax(score, -1), v[:, kv]))
        return {"out": torch.stack(outs), "lse": torch.stack(lses)}
    k_out, v_out = torch.zeros_like(s["k_out"], dtype=F64), torch.zeros_like(s["v_out"], dtype=F64)
    got = {}
    if c["op"] == "append":
        at = (s["lens"].to(F64) - 1)[:, None, None] * theta
        got["q_out"] = turned(s["q"], at)
        k_out[:, 0], v_out[:, 0] = held(turned(s["k"], at), "k"), held(s["v"].to(F64), "v")
    elif c["op"] == "fill":
        cu = s["cu"].tolist()
        for b, past in enumerate(s["starts"].tolist()):
            n = cu[b + 1] - cu[b]
            at = (torch.arange(n, device=DEV) + past).to(F64)[:, None, None] * theta
            k_out[b, :n] = held(turned(s["k"][cu[b] : cu[b + 1]], at), "k")
            v_out[b, :n] = held(s["v"][cu[b] : cu[b + 1]].to(F64), "v")
    else:
        for b, (n, first) in enumerate(zip(lens, s["starts"].tolist())):
            k_out[b, : n - first], v_out[b, : n - first] = stands_for("k", b, first, n), stands_for("v", b, first, n)
    return {**got, "k": k_out, "v": v_out}
