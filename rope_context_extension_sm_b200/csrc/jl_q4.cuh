// jl_q4.cuh -- the base-RoPE KV cache held in 4 bits: its layout, its writers and its reader.
//
// The cache of "Jet-Long: Efficient Long-Context Extension with Dynamic Bifocal RoPE"
// (Methodology section 2: base keys R(j) k_j at their exact positions, written once per
// token) at a quarter of its size.  One (position, KV head) row of D channels is D/2 bytes
// of key codes, D/2 bytes of value codes and eight bf16 scales (four for the key, four for
// the value), and stands for x = scale * (code - 8), code in 1 .. 15.
//
// Scale groups.  A key scale belongs to D/8 rotate-half pairs (c, c + D/2): both channels
// of a pair share it, so the decode's correction rotation R(f(j) - j) acts on the codes
// alone and the scale is applied to the scores of its group.  A value scale belongs to D/4
// neighbouring channels.
//
// Order of the codes.  The decode feeds mma.m16n8k16 fragments straight from registers, so
// a row is stored in the order in which lanes take it: lane (g, t) of a quad loads the
// bytes of its own channels with one access and no shuffle.
//   key pair c:  w = c / (D/8), r = c % (D/8), t = r / (D/32), e = r % (D/32);
//                byte 16 t + 4 w + e (D = 128), 8 t + 4 (w / 2) + 2 e + w % 2 (D = 64);
//                channel c in the low four bits, c + D/2 in the high four
//   value channel c:  byte (D/16) (c % 8) + c / 16, low four bits if c % 16 < 8, else high
//
// Rounding.  scale = bf16(max|x| * fp32(1/7)) (bf16 keeps the range of the inputs, and the codes are
// formed with the rounded scale, so its 8 bits cost no accuracy: a largest value past 7 scales is
// off by 7 * 2^-8 of one, less than a code's rounding); code = round-half-even(x / scale) clamped
// to +-7.  A group whose scale would be below 2^-100 is stored as zeros (the residuals below stay
// normal numbers), one that holds a NaN or an infinity gets a NaN scale, so it does not turn
// into finite values.
#pragma once

#include "jl_append.cuh"
#include "jl_device.cuh"

namespace jl {

constexpr int kQ4Scales = 8;  // bf16 scales of a row: 4 key groups, 4 value groups

struct Q4Params {
  const __nv_bfloat16* q;      // append: raw query rows [B][Hq][D]
  const __nv_bfloat16* k;      // raw key rows
  const __nv_bfloat16* v;
  const int32_t* lens;         // fill: cu_seqlens [batch+1]; append: seqlens [B]; read: lens [B]
  const int32_t* past;         // fill: tokens already in each entry; read: first row (NULL = 0)
  const float* cos_tab;
  const float* sin_tab;
  __nv_bfloat16* q_out;        // append: rotated query rows
  __nv_bfloat16* k_out;        // read: [B][out_rows][Hkv][D]
  __nv_bfloat16* v_out;
  uint8_t* k_codes;            // [B][stride][Hkv][D/2], or pages
  uint8_t* v_codes;
  __nv_bfloat16* scales;       // [B][stride][Hkv][8]
  int64_t total_tokens;
  int64_t cache_stride;
  int64_t n_tab_rows;
  int64_t out_rows;
  int32_t batch, Hq, Hkv;
  const int32_t* block_table;
  int32_t page_size, max_pages, num_pages;
};

// Cache row of entry b's position pos, already checked against cache_stride; -1 when the
// page index is outside the pool.
__device__ __forceinline__ int64_t q4_row(const Q4Params& p, int b, int64_t pos) {
  if (p.block_table == nullptr) return static_cast<int64_t>(b) * p.cache_stride + pos;
  const uint32_t x = static_cast<uint32_t>(pos), n = x / p.page_size;  // positions are below 2^31
  const int32_t page = p.block_table[static_cast<int64_t>(b) * p.max_pages + n];
  if (page < 0 || page >= p.num_pages) return -1;
  return static_cast<int64_t>(page) * p.page_size + (x - n * p.page_size);
}

// Rows of the cache, contiguous or paged (debug-bounds checks).
__device__ __forceinline__ int64_t q4_rows(const Q4Params& p) {
  return p.block_table != nullptr ? static_cast<int64_t>(p.num_pages) * p.page_size : p.batch * p.cache_stride;
}

// The scale of a group from the largest |x| of it, given as float bits (so that a NaN or an
// infinity stays the largest).
__device__ __forceinline__ __nv_bfloat16 q4_scale(uint32_t top_bits) {
  if (top_bits >= 0x7f800000u) return __ushort_as_bfloat16(0x7fc0);
  const __nv_bfloat16 s = __float2bfloat16_rn(__fmul_rn(__uint_as_float(top_bits), 1.0f / 7.0f));
  return __bfloat162float(s) < 0x1p-100f ? __ushort_as_bfloat16(0) : s;
}

__device__ __forceinline__ float q4_inverse(__nv_bfloat16 s) {
  const float f = __bfloat162float(s);
  return f > 0.f ? 1.0f / f : 0.f;
}

// A row is handled by four lanes, one for each scale group: lane w of the team holds its
// group's D/8 key pairs and D/4 value channels, so a group's maximum and scale need no
// shuffle and are formed once.  (A warp a row, eight lanes to a group, took 2.6 times as
// long: six shuffles and both scales for every eight values.)  Codes then change places in a
// 4 x 4 transpose of words, and each lane stores or loads one contiguous quarter of a row.

// e[i] of lane w becomes e[w] of lane i, among the four lanes of a team.
__device__ __forceinline__ void q4_transpose(uint32_t (&e)[4], int w) {
  const bool b0 = w & 1, b1 = w & 2;
  uint32_t x = __shfl_xor_sync(0xffffffffu, b0 ? e[0] : e[1], 1), y = __shfl_xor_sync(0xffffffffu, b0 ? e[2] : e[3], 1);
  if (b0) e[0] = x, e[2] = y; else e[1] = x, e[3] = y;
  x = __shfl_xor_sync(0xffffffffu, b1 ? e[0] : e[2], 2), y = __shfl_xor_sync(0xffffffffu, b1 ? e[1] : e[3], 2);
  if (b1) e[0] = x, e[1] = y; else e[2] = x, e[3] = y;
}

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// Codes of two values under a scale (inv = 1 / scale), each in the low four bits of a word.
// The quotient is corrected once by its residual (Markstein 1990: q' = q + (x - q s) / s is
// the correctly rounded x / s when 1 / s is), so halves are real halves; adding 1.5 * 2^23 + 8
// rounds it to the nearest integer, halves to even, plus 8, in the lowest bits.  |x / s| is at
// most 7 (1 + 2^-8), so nothing has to be clamped.  inv = 0 gives 8 for finite values.
__device__ __forceinline__ void q4_codes(uint64_t x, uint64_t inv, uint64_t minus_s, uint32_t& lo, uint32_t& hi) {
  const uint64_t q = f2_mul(x, inv);
  const uint64_t n = f2_add(f2_fma(f2_fma(q, minus_s, x), inv, q), f2_pack(12582920.f, 12582920.f));
  float a, b;
  f2_unpack(n, a, b);
  lo = __float_as_uint(a);
  hi = __float_as_uint(b);
}

// Four bytes from four pairs of codes: byte i holds low[i] and, above it, high[i].
__device__ __forceinline__ uint32_t q4_bytes(const uint32_t (&low)[4], const uint32_t (&high)[4]) {
  const uint32_t a = __byte_perm(__byte_perm(low[0], low[1], 0x0040), __byte_perm(low[2], low[3], 0x0040), 0x5410);
  const uint32_t b = __byte_perm(__byte_perm(high[0], high[1], 0x0040), __byte_perm(high[2], high[3], 0x0040), 0x5410);
  return (a & 0x0f0f0f0fu) | (b << 4 & 0xf0f0f0f0u);
}

// A lane's quarter of a row of codes: four words, or two for D = 64.
template <int D>
__device__ __forceinline__ void q4_store_quarter(uint8_t* row, int w, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  if constexpr (D == 128) *reinterpret_cast<uint4*>(row + 16 * w) = make_uint4(a, b, c, d);
  else *reinterpret_cast<uint2*>(row + 8 * w) = make_uint2(a, b);
}

// One team quantises one (token, head) row, if it has one (all lanes of the warp take part in
// the exchanges): key rotated by table row pos, value as it is.  The rotation rounds every
// product and sum to fp32 (no fused multiply-add), so the codes are the same whatever computes
// them.
template <int D>
__device__ __forceinline__ void q4_write_row(const Q4Params& p, bool live, const __nv_bfloat16* __restrict__ k,
                                             const __nv_bfloat16* __restrict__ v, int64_t pos, int64_t row, int h, int w) {
  constexpr int HALF = D / 2, NP = D / 8;  // key pairs of a lane
  uint32_t ka[NP / 2] = {}, kb[NP / 2] = {}, vv[NP] = {};  // bf16x2 words
  float cs[NP] = {}, sn[NP] = {};
  if (live) {
#pragma unroll
    for (int i = 0; i < NP / 8; ++i) {
      const uint4 a = *reinterpret_cast<const uint4*>(k + w * NP + 8 * i);
      const uint4 b = *reinterpret_cast<const uint4*>(k + HALF + w * NP + 8 * i);
      ka[4 * i] = a.x, ka[4 * i + 1] = a.y, ka[4 * i + 2] = a.z, ka[4 * i + 3] = a.w;
      kb[4 * i] = b.x, kb[4 * i + 1] = b.y, kb[4 * i + 2] = b.z, kb[4 * i + 3] = b.w;
    }
#pragma unroll
    for (int i = 0; i < NP / 4; ++i) {
      const uint4 a = *reinterpret_cast<const uint4*>(v + w * 2 * NP + 8 * i);
      vv[4 * i] = a.x, vv[4 * i + 1] = a.y, vv[4 * i + 2] = a.z, vv[4 * i + 3] = a.w;
      const float4 c = *reinterpret_cast<const float4*>(p.cos_tab + pos * HALF + w * NP + 4 * i);
      const float4 s = *reinterpret_cast<const float4*>(p.sin_tab + pos * HALF + w * NP + 4 * i);
      cs[4 * i] = c.x, cs[4 * i + 1] = c.y, cs[4 * i + 2] = c.z, cs[4 * i + 3] = c.w;
      sn[4 * i] = s.x, sn[4 * i + 1] = s.y, sn[4 * i + 2] = s.z, sn[4 * i + 3] = s.w;
    }
  }
  uint64_t ya[NP / 2], yb[NP / 2];  // two pairs' low channels, and their high ones
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < NP / 2; ++i) {
    // packed products, but scalar sums: a packed sum of packed products was found to be fused
    const uint64_t c = f2_pack(cs[2 * i], cs[2 * i + 1]), z = f2_pack(sn[2 * i], sn[2 * i + 1]);
    const uint64_t a = f2_pack(__uint_as_float(ka[i] << 16), __uint_as_float(ka[i] & 0xffff0000u));
    const uint64_t b = f2_pack(__uint_as_float(kb[i] << 16), __uint_as_float(kb[i] & 0xffff0000u));
    float ac0, ac1, as0, as1, bc0, bc1, bs0, bs1;
    f2_unpack(f2_mul(a, c), ac0, ac1);
    f2_unpack(f2_mul(a, z), as0, as1);
    f2_unpack(f2_mul(b, c), bc0, bc1);
    f2_unpack(f2_mul(b, z), bs0, bs1);
    const float x0 = __fsub_rn(ac0, bs0), x1 = __fsub_rn(ac1, bs1), x2 = __fadd_rn(bc0, as0), x3 = __fadd_rn(bc1, as1);
    ya[i] = f2_pack(x0, x1);
    yb[i] = f2_pack(x2, x3);
    top = max_nan(max_nan(max_nan(fabsf(x0), fabsf(x1)), max_nan(fabsf(x2), fabsf(x3))), top);
  }
  __nv_bfloat162 vtop = __habs2(*reinterpret_cast<__nv_bfloat162*>(&vv[0]));
#pragma unroll
  for (int i = 1; i < NP; ++i) vtop = __hmax2_nan(vtop, __habs2(*reinterpret_cast<__nv_bfloat162*>(&vv[i])));
  const uint32_t kbits = __float_as_uint(top);
  const uint32_t vbits = __float_as_uint(max_nan(__low2float(vtop), __high2float(vtop)));
  const __nv_bfloat16 ks = q4_scale(kbits), vs = q4_scale(vbits);

  uint8_t* const krow = p.k_codes + (row * p.Hkv + h) * HALF;
  uint8_t* const vrow = p.v_codes + (row * p.Hkv + h) * HALF;
  uint32_t e[4];
  {
    const float f = __bfloat162float(ks), inv = q4_inverse(ks);
    const uint64_t inv2 = f2_pack(inv, inv), ms2 = f2_pack(-f, -f);
    uint32_t word[NP / 4];  // four pairs each
#pragma unroll
    for (int i = 0; i < NP / 4; ++i) {
      uint32_t low[4], high[4];
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        q4_codes(ya[2 * i + z], inv2, ms2, low[2 * z], low[2 * z + 1]);
        q4_codes(yb[2 * i + z], inv2, ms2, high[2 * z], high[2 * z + 1]);
      }
      word[i] = kbits >= 0x7f800000u ? 0x88888888u : q4_bytes(low, high);
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) e[t] = D == 128 ? word[t % (NP / 4)] : word[t / 2] >> (16 * (t & 1)) & 0xffffu;
    q4_transpose(e, w);
    if constexpr (D != 128) {
      e[0] = __byte_perm(e[0], e[1], 0x5140);
      e[1] = __byte_perm(e[2], e[3], 0x5140);
    }
    if (live) q4_store_quarter<D>(krow, w, e[0], e[1], e[2], e[3]);
  }
  {
    const float f = __bfloat162float(vs), inv = q4_inverse(vs);
    const uint64_t inv2 = f2_pack(inv, inv), ms2 = f2_pack(-f, -f);
    uint32_t y[NP / 8][2];  // [tile of 16 channels][half]: bytes of rows 4 half .. 4 half + 3
#pragma unroll
    for (int i = 0; i < NP / 8; ++i)
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        uint32_t low[4], high[4];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t a = vv[8 * i + 2 * z + x], b = vv[8 * i + 4 + 2 * z + x];
          q4_codes(f2_pack(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u)), inv2, ms2, low[2 * x], low[2 * x + 1]);
          q4_codes(f2_pack(__uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u)), inv2, ms2, high[2 * x], high[2 * x + 1]);
        }
        y[i][z] = vbits >= 0x7f800000u ? 0x88888888u : q4_bytes(low, high);
      }
#pragma unroll
    for (int x = 0; x < 4; ++x)
      e[x] = D == 128 ? __byte_perm(y[0][x / 2], y[NP / 8 - 1][x / 2], x & 1 ? 0x7362 : 0x5140) : y[0][x / 2] >> (16 * (x & 1)) & 0xffffu;
    q4_transpose(e, w);
    uint32_t a, b, c = 0, d = 0;
    if constexpr (D == 128) {
      a = __byte_perm(e[0], e[1], 0x5410), b = __byte_perm(e[2], e[3], 0x5410);
      c = __byte_perm(e[0], e[1], 0x7632), d = __byte_perm(e[2], e[3], 0x7632);
    } else {
      const uint32_t x = __byte_perm(e[0], e[1], 0x5140), z = __byte_perm(e[2], e[3], 0x5140);
      a = __byte_perm(x, z, 0x5410), b = __byte_perm(x, z, 0x7632);
    }
    if (live) q4_store_quarter<D>(vrow, w, a, b, c, d);
  }
  // scales: even lanes store two of the key's, odd ones two of the value's
  const uint32_t mine = __bfloat16_as_ushort(ks) | static_cast<uint32_t>(__bfloat16_as_ushort(vs)) << 16;
  const uint32_t next = __shfl_xor_sync(0xffffffffu, mine, 1);
  if (live)
    *reinterpret_cast<uint32_t*>(p.scales + (row * p.Hkv + h) * kQ4Scales + (w & 1) * 4 + (w & 2)) =
        w & 1 ? __byte_perm(next, mine, 0x7632) : __byte_perm(mine, next, 0x5410);
}

constexpr int kQ4Teams = 64;  // rows of a block of 256 threads

// row = token * Hkv + h, in 32 bits where it fits (a 64-bit division costs some 100 instructions).
__device__ __forceinline__ int64_t q4_split(int64_t row, int Hkv, int& h) {
  if (row <= 0xffffffffLL) {
    const uint32_t r = static_cast<uint32_t>(row), t = r / static_cast<uint32_t>(Hkv);
    h = static_cast<int>(r - t * Hkv);
    return t;
  }
  h = static_cast<int>(row % Hkv);
  return row / Hkv;
}

// Prompt tokens: token t of sequence b goes to position past[b] + t - cu_seqlens[b].
template <int D>
__global__ void __launch_bounds__(4 * kQ4Teams, 3) jl_kv_fill_q4_kernel(const Q4Params p) {
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kQ4Teams + threadIdx.x / 4;
  const int w = threadIdx.x & 3;
  bool live = row < p.total_tokens * p.Hkv;
  int64_t pos = 0, crow = 0;
  int h = 0;
  if (live) {
    const int64_t t = q4_split(row, p.Hkv, h);
    int lo = 0, hi = p.batch - 1;  // sequence holding token t: last b with cu[b] <= t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.lens[mid] <= t) lo = mid; else hi = mid - 1;
    }
    pos = t - p.lens[lo] + (p.past != nullptr ? p.past[lo] : 0);
    crow = (pos < 0 || pos >= p.cache_stride || pos >= p.n_tab_rows) ? -1 : q4_row(p, lo, pos);
    if (crow < 0) {
      if (w == 0) atomicOr(&g_status, kDevErrBounds);
      live = false;
    }
  }
  JL_CHECK(!live || (row < p.total_tokens * p.Hkv && pos < p.n_tab_rows && crow >= 0 && crow < q4_rows(p) && h >= 0 &&
                     h < p.Hkv));
  q4_write_row<D>(p, live, p.k + row * D, p.v + row * D, pos, crow, h, w);
}

// One decode step: entry b's new token sits at i = seqlens[b] - 1.  The first B * Hq warps
// rotate the queries into q_out, the others' teams quantise and append key and value.
template <int D>
__global__ void __launch_bounds__(4 * kQ4Teams) jl_decode_append_q4_kernel(const Q4Params p) {
  griddep_launch_dependents();  // the decode that follows may launch now; it waits for this grid to finish
  constexpr int HALF = D / 2, PPL = D / 64;
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) / 32, queries = static_cast<int64_t>(p.batch) * p.Hq;
  const int lane = threadIdx.x & 31;
  if (warp < queries) {
    const int64_t i = static_cast<int64_t>(p.lens[warp / p.Hq]) - 1;
    if (i < 0 || i >= p.cache_stride || i >= p.n_tab_rows) {
      if (lane == 0) atomicOr(&g_status, kDevErrBounds);
      return;
    }
    const int64_t o = warp * D;
    JL_CHECK(warp / p.Hq < p.batch && i < p.n_tab_rows);
#pragma unroll
    for (int e = 0; e < PPL; ++e) {
      const int c = lane * PPL + e;
      const float cs = p.cos_tab[i * HALF + c], sn = p.sin_tab[i * HALF + c];
      const float a = __bfloat162float(p.q[o + c]), bb = __bfloat162float(p.q[o + c + HALF]);
      p.q_out[o + c] = __float2bfloat16_rn(a * cs - bb * sn);
      p.q_out[o + c + HALF] = __float2bfloat16_rn(bb * cs + a * sn);
    }
    return;
  }
  const int64_t row = (warp - queries) * 8 + lane / 4;
  const int w = lane & 3;
  bool live = row < static_cast<int64_t>(p.batch) * p.Hkv;
  int64_t i = 0, crow = 0;
  int h = 0;
  if (live) {
    const int b = static_cast<int>(q4_split(row, p.Hkv, h));
    i = static_cast<int64_t>(p.lens[b]) - 1;
    crow = (i < 0 || i >= p.cache_stride || i >= p.n_tab_rows) ? -1 : q4_row(p, b, i);
    if (crow < 0) {
      if (w == 0) atomicOr(&g_status, kDevErrBounds);
      live = false;
    }
  }
  JL_CHECK(!live || (row < static_cast<int64_t>(p.batch) * p.Hkv && i < p.n_tab_rows && crow >= 0 && crow < q4_rows(p) &&
                     h >= 0 && h < p.Hkv));
  q4_write_row<D>(p, live, p.k + row * D, p.v + row * D, i, crow, h, w);
}

// 16-byte chunks 0 and 1 of lane w, which fill one 32-byte sector each two, change places with
// the neighbour lane's so that the two lanes store a whole sector together: the even lane then
// holds chunk 0 of both lanes, the odd one chunk 1.
__device__ __forceinline__ void q4_pair_chunks(uint4& c0, uint4& c1, int w) {
  const bool odd = w & 1;
  uint4 s = odd ? c0 : c1;
  s.x = __shfl_xor_sync(0xffffffffu, s.x, 1), s.y = __shfl_xor_sync(0xffffffffu, s.y, 1);
  s.z = __shfl_xor_sync(0xffffffffu, s.z, 1), s.w = __shfl_xor_sync(0xffffffffu, s.w, 1);
  if (odd) c0 = s; else c1 = s;
}

// The values of bytes i and i + 1 of a word of codes (low or high four bits), as bf16x2.
template <bool HIGH>
__device__ __forceinline__ uint32_t q4_values(uint32_t word, int i, __nv_bfloat162 scale) {
  uint32_t x = __byte_perm(word, 0, i == 0 ? 0x4140 : 0x4342);
  x = (HIGH ? x >> 4 : x) & 0x000f000fu | 0x43004300u;  // 128 + code
  const __nv_bfloat162 y = __hmul2(__hsub2(*reinterpret_cast<__nv_bfloat162*>(&x), __float2bfloat162_rn(136.f)), scale);
  return *reinterpret_cast<const uint32_t*>(&y);
}

// Rows [past[b], lens[b]) of every entry back to bf16: k_out[b][p - past[b]] holds the
// base-RoPE key that position p stands for (one rounding of scale * (code - 8): a product of
// bf16 numbers, rounded once to bf16), v_out the value.  Rows behind the last are not written.
template <int D>
__global__ void __launch_bounds__(4 * kQ4Teams) jl_kv_read_q4_kernel(const Q4Params p) {
  constexpr int HALF = D / 2, NP = D / 8;
  const int b = blockIdx.y, w = threadIdx.x & 3;
  const int64_t first = p.past != nullptr ? p.past[b] : 0, len = p.lens[b];
  if (first < 0 || len > p.cache_stride || len - first > p.out_rows) {
    if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(&g_status, kDevErrBounds);
    return;
  }
  if (static_cast<int64_t>(blockIdx.x) * kQ4Teams >= (len - first) * p.Hkv) return;
  const int64_t in_entry = static_cast<int64_t>(blockIdx.x) * kQ4Teams + threadIdx.x / 4;  // row of this entry
  int h;
  const int64_t pos = first + q4_split(in_entry, p.Hkv, h), row = b * p.out_rows * p.Hkv + in_entry;
  bool live = pos < len;
  int64_t r = 0;
  if (live) {
    const int64_t crow = q4_row(p, b, pos);
    if (crow < 0) {
      if (w == 0) atomicOr(&g_status, kDevErrBounds);
      live = false;
    }
    r = crow * p.Hkv + h;
  }
  JL_CHECK(!live || (r >= 0 && r < q4_rows(p) * p.Hkv && row < static_cast<int64_t>(p.batch) * p.out_rows * p.Hkv &&
                     in_entry < p.out_rows * p.Hkv && pos < p.cache_stride));
  uint4 kw = make_uint4(0u, 0u, 0u, 0u), vw = kw;  // this lane's quarter of the codes
  uint32_t ks = 0, vs = 0;
  if (live) {
    if constexpr (D == 128) {
      kw = *reinterpret_cast<const uint4*>(p.k_codes + r * HALF + 16 * w);
      vw = *reinterpret_cast<const uint4*>(p.v_codes + r * HALF + 16 * w);
    } else {
      const uint2 a = *reinterpret_cast<const uint2*>(p.k_codes + r * HALF + 8 * w);
      const uint2 b = *reinterpret_cast<const uint2*>(p.v_codes + r * HALF + 8 * w);
      kw.x = a.x, kw.y = a.y, vw.x = b.x, vw.y = b.y;
    }
    ks = __bfloat16_as_ushort(p.scales[r * kQ4Scales + w]);
    vs = __bfloat16_as_ushort(p.scales[r * kQ4Scales + 4 + w]);
  }
  const __nv_bfloat162 kscale = __bfloat162bfloat162(__ushort_as_bfloat16(static_cast<unsigned short>(ks)));
  const __nv_bfloat162 vscale = __bfloat162bfloat162(__ushort_as_bfloat16(static_cast<unsigned short>(vs)));
  uint32_t e[4];
  {  // keys: after the transpose, e[t] holds the pairs of this lane's group that come t-th
    if constexpr (D == 128) {
      e[0] = kw.x, e[1] = kw.y, e[2] = kw.z, e[3] = kw.w;
    } else {
      e[0] = __byte_perm(kw.x, 0, 0x4420), e[1] = __byte_perm(kw.x, 0, 0x4431);
      e[2] = __byte_perm(kw.y, 0, 0x4420), e[3] = __byte_perm(kw.y, 0, 0x4431);
    }
    q4_transpose(e, w);
    uint32_t lo[NP / 2], hi[NP / 2];  // bf16x2
#pragma unroll
    for (int i = 0; i < NP / 2; ++i) {
      const uint32_t word = D == 128 ? e[i / 2] : e[i];
      lo[i] = q4_values<false>(word, D == 128 ? i & 1 : 0, kscale);
      hi[i] = q4_values<true>(word, D == 128 ? i & 1 : 0, kscale);
    }
    __nv_bfloat16* out = p.k_out + row * D;
    if constexpr (D == 128) {
      const int pair = (w & 2) * NP + (w & 1) * 8;  // the even lane's group, and this lane's chunk of it
      uint4 c0 = make_uint4(lo[0], lo[1], lo[2], lo[3]), c1 = make_uint4(lo[4 % (NP / 2)], lo[5 % (NP / 2)], lo[6 % (NP / 2)], lo[7 % (NP / 2)]);
      uint4 d0 = make_uint4(hi[0], hi[1], hi[2], hi[3]), d1 = make_uint4(hi[4 % (NP / 2)], hi[5 % (NP / 2)], hi[6 % (NP / 2)], hi[7 % (NP / 2)]);
      q4_pair_chunks(c0, c1, w);
      q4_pair_chunks(d0, d1, w);
      if (live) {
        *reinterpret_cast<uint4*>(out + pair) = c0;
        *reinterpret_cast<uint4*>(out + pair + NP) = c1;
        *reinterpret_cast<uint4*>(out + HALF + pair) = d0;
        *reinterpret_cast<uint4*>(out + HALF + pair + NP) = d1;
      }
    } else if (live) {
      *reinterpret_cast<uint4*>(out + w * NP) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      *reinterpret_cast<uint4*>(out + HALF + w * NP) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    }
  }
  {  // values: e[x] of this lane holds its channel tiles' bytes of rows 2x and 2x + 1
    uint32_t y[2][2];  // [tile][half]: bytes of rows 4 half .. 4 half + 3
    if constexpr (D == 128) {
      e[0] = __byte_perm(vw.x, vw.z, 0x5410), e[1] = __byte_perm(vw.x, vw.z, 0x7632);
      e[2] = __byte_perm(vw.y, vw.w, 0x5410), e[3] = __byte_perm(vw.y, vw.w, 0x7632);
    } else {
      const uint32_t a = __byte_perm(vw.x, vw.y, 0x5140), b = __byte_perm(vw.x, vw.y, 0x7362);
      e[0] = a & 0xffffu, e[1] = a >> 16, e[2] = b & 0xffffu, e[3] = b >> 16;
    }
    q4_transpose(e, w);
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      if constexpr (D == 128) {
        y[0][z] = __byte_perm(e[2 * z], e[2 * z + 1], 0x6420);
        y[1][z] = __byte_perm(e[2 * z], e[2 * z + 1], 0x7531);
      } else {
        y[0][z] = y[1][z] = __byte_perm(e[2 * z], e[2 * z + 1], 0x5410);
      }
    }
    __nv_bfloat16* out = p.v_out + row * D;
#pragma unroll
    for (int i = 0; i < NP / 8; ++i) {  // tile of 16 channels: low bits are its first eight, high bits its last
      uint4 c0 = make_uint4(q4_values<false>(y[i][0], 0, vscale), q4_values<false>(y[i][0], 1, vscale),
                            q4_values<false>(y[i][1], 0, vscale), q4_values<false>(y[i][1], 1, vscale));
      uint4 c1 = make_uint4(q4_values<true>(y[i][0], 0, vscale), q4_values<true>(y[i][0], 1, vscale),
                            q4_values<true>(y[i][1], 0, vscale), q4_values<true>(y[i][1], 1, vscale));
      q4_pair_chunks(c0, c1, w);
      if (live) {
        const int at = (w & 2) * 2 * NP + 16 * i + (w & 1) * 8;
        *reinterpret_cast<uint4*>(out + at) = c0;
        *reinterpret_cast<uint4*>(out + at + 2 * NP) = c1;
      }
    }
  }
}

}  // namespace jl
