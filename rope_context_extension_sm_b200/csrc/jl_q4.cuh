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
// formed with the rounded scale, so its 8 bits cost no accuracy beyond a clamp of 2^-9 of a
// step); code = round-half-even(x / scale) clamped to +-7.  A group whose scale would be
// below 2^-100 is stored as zeros (the residuals below stay normal numbers), one that holds
// a NaN or an infinity gets a NaN scale, so it does not turn into finite values.
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
  const int32_t page = p.block_table[static_cast<int64_t>(b) * p.max_pages + pos / p.page_size];
  if (page < 0 || page >= p.num_pages) return -1;
  return static_cast<int64_t>(page) * p.page_size + pos % p.page_size;
}

__host__ __device__ constexpr int q4_key_byte(int D, int c) {
  const int w = c / (D / 8), r = c % (D / 8), t = r / (D / 32), e = r % (D / 32);
  return D == 128 ? 16 * t + 4 * w + e : 8 * t + 4 * (w / 2) + 2 * e + w % 2;
}

// The scale of a group from the largest |x| of it, given as float bits (so that a NaN or an
// infinity stays the largest).
__device__ __forceinline__ __nv_bfloat16 q4_scale(uint32_t top_bits) {
  if (top_bits >= 0x7f800000u) return __ushort_as_bfloat16(0x7fc0);
  const __nv_bfloat16 s = __float2bfloat16_rn(__fmul_rn(__uint_as_float(top_bits), 1.0f / 7.0f));
  return __bfloat162float(s) < 0x1p-100f ? __ushort_as_bfloat16(0) : s;
}

// Code of x under `scale` (inv = 1 / scale): the quotient is corrected once by its residual
// (Markstein 1990: q' = q + (x - q s) / s is the correctly rounded x / s when 1 / s is), so
// halves are real halves and go to even.  inv = 0 marks a group of zeros or NaN.
__device__ __forceinline__ uint32_t q4_code(float x, float scale, float inv) {
  if (inv == 0.f) return 8u;
  const float q = __fmul_rn(x, inv);
  const float n = rintf(__fmaf_rn(__fmaf_rn(-q, scale, x), inv, q));
  return static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(n, -7.f), 7.f)) + 8);
}

__device__ __forceinline__ float q4_inverse(__nv_bfloat16 s) {
  const float f = __bfloat162float(s);
  return f > 0.f ? 1.0f / f : 0.f;
}

// Largest of `bits` over the eight lanes of a group.
__device__ __forceinline__ uint32_t q4_group_max(uint32_t bits) {
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, o));
  return bits;
}

// One warp quantises one (token, head) row: key rotated by table row pos, value as it is.
// Lane l owns key pairs PPL*l + e and value channels VPL*l + e, so a group is eight lanes
// for both.  The rotation rounds every product and sum to fp32 (no fused multiply-add), so
// the codes are the same whatever computes them.
template <int D>
__device__ __forceinline__ void q4_write_row(const Q4Params& p, const __nv_bfloat16* __restrict__ k,
                                             const __nv_bfloat16* __restrict__ v, int64_t pos, int64_t row, int h,
                                             int lane) {
  constexpr int HALF = D / 2, PPL = D / 64, VPL = D / 32;
  const int64_t r = row * p.Hkv + h;
  float ya[PPL], yb[PPL], x[VPL];
  uint32_t ktop = 0, vtop = 0;
#pragma unroll
  for (int e = 0; e < PPL; ++e) {
    const int c = lane * PPL + e;
    const float cs = p.cos_tab[pos * HALF + c], sn = p.sin_tab[pos * HALF + c];
    const float a = __bfloat162float(k[c]), b = __bfloat162float(k[c + HALF]);
    ya[e] = __fsub_rn(__fmul_rn(a, cs), __fmul_rn(b, sn));
    yb[e] = __fadd_rn(__fmul_rn(b, cs), __fmul_rn(a, sn));
    ktop = max(ktop, max(__float_as_uint(ya[e]) & 0x7fffffffu, __float_as_uint(yb[e]) & 0x7fffffffu));
  }
#pragma unroll
  for (int e = 0; e < VPL; ++e) {
    x[e] = __bfloat162float(v[lane * VPL + e]);
    vtop = max(vtop, __float_as_uint(x[e]) & 0x7fffffffu);
  }
  const __nv_bfloat16 ks = q4_scale(q4_group_max(ktop)), vs = q4_scale(q4_group_max(vtop));
  const float kf = __bfloat162float(ks), ki = q4_inverse(ks), vf = __bfloat162float(vs), vi = q4_inverse(vs);
#pragma unroll
  for (int e = 0; e < PPL; ++e)
    p.k_codes[r * HALF + q4_key_byte(D, lane * PPL + e)] =
        static_cast<uint8_t>(q4_code(ya[e], kf, ki) | q4_code(yb[e], kf, ki) << 4);
  uint32_t code = 0;
#pragma unroll
  for (int e = 0; e < VPL; ++e) code |= q4_code(x[e], vf, vi) << (8 * e);
  const uint32_t other = __shfl_xor_sync(0xffffffffu, code, 8 / VPL);  // the lane 8 channels on, or back
  const bool high = (lane * VPL) & 8;
  const uint32_t both = high ? (other | code << 4) : (code | other << 4);
#pragma unroll
  for (int e = 0; e < VPL / 2; ++e) {
    const int j = high ? VPL / 2 + e : e, c = lane * VPL + j;
    p.v_codes[r * HALF + (D / 16) * (c % 8) + c / 16] = static_cast<uint8_t>(both >> (8 * j));
  }
  if ((lane & 7) == 0) {
    p.scales[r * kQ4Scales + lane / 8] = ks;
    p.scales[r * kQ4Scales + 4 + lane / 8] = vs;
  }
}

// Prompt tokens: token t of sequence b goes to position past[b] + t - cu_seqlens[b].
template <int D>
__global__ void __launch_bounds__(256) jl_kv_fill_q4_kernel(const Q4Params p) {
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) / 32;
  const int lane = threadIdx.x & 31;
  if (row >= p.total_tokens * p.Hkv) return;
  const int64_t t = row / p.Hkv;
  const int h = static_cast<int>(row % p.Hkv);
  int lo = 0, hi = p.batch - 1;  // sequence holding token t: last b with cu[b] <= t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.lens[mid] <= t) lo = mid; else hi = mid - 1;
  }
  const int64_t pos = t - p.lens[lo] + (p.past != nullptr ? p.past[lo] : 0);
  const int64_t crow = (pos < 0 || pos >= p.cache_stride || pos >= p.n_tab_rows) ? -1 : q4_row(p, lo, pos);
  if (crow < 0) {
    if (lane == 0) atomicOr(&g_status, kDevErrBounds);
    return;
  }
  q4_write_row<D>(p, p.k + row * D, p.v + row * D, pos, crow, h, lane);
}

// One decode step: entry b's new token sits at i = seqlens[b] - 1.  Rows 0 .. Hq-1 rotate
// the query into q_out, rows Hq .. Hq+Hkv-1 quantise and append key and value.
template <int D>
__global__ void __launch_bounds__(256) jl_decode_append_q4_kernel(const Q4Params p) {
  griddep_launch_dependents();  // the decode that follows may launch now; it waits for this grid to finish
  constexpr int HALF = D / 2, PPL = D / 64;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) / 32;
  const int lane = threadIdx.x & 31;
  const int per_b = p.Hq + p.Hkv;
  if (row >= static_cast<int64_t>(p.batch) * per_b) return;
  const int b = static_cast<int>(row / per_b), r = static_cast<int>(row % per_b);
  const int64_t i = static_cast<int64_t>(p.lens[b]) - 1;
  if (i < 0 || i >= p.cache_stride || i >= p.n_tab_rows) {
    if (lane == 0) atomicOr(&g_status, kDevErrBounds);
    return;
  }
  if (r < p.Hq) {
    const int64_t o = (static_cast<int64_t>(b) * p.Hq + r) * D;
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
  const int h = r - p.Hq;
  const int64_t src = (static_cast<int64_t>(b) * p.Hkv + h) * D;
  const int64_t crow = q4_row(p, b, i);
  if (crow < 0) {
    if (lane == 0) atomicOr(&g_status, kDevErrBounds);
    return;
  }
  q4_write_row<D>(p, p.k + src, p.v + src, i, crow, h, lane);
}

// Rows [past[b], lens[b]) of every entry back to bf16: k_out[b][p - past[b]] holds the
// base-RoPE key that position p stands for (one rounding of scale * (code - 8), a product
// that fp32 holds exactly), v_out the value.  Rows behind the last one are not written.
template <int D>
__global__ void __launch_bounds__(256) jl_kv_read_q4_kernel(const Q4Params p) {
  constexpr int HALF = D / 2, PPL = D / 64, VPL = D / 32;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) / 32;
  const int lane = threadIdx.x & 31;
  if (row >= static_cast<int64_t>(p.batch) * p.out_rows * p.Hkv) return;
  const int64_t br = row / p.Hkv;
  const int h = static_cast<int>(row % p.Hkv), b = static_cast<int>(br / p.out_rows);
  const int64_t first = p.past != nullptr ? p.past[b] : 0, pos = first + br % p.out_rows;
  if (first < 0 || p.lens[b] > p.cache_stride || p.lens[b] - first > p.out_rows) {
    if (lane == 0) atomicOr(&g_status, kDevErrBounds);
    return;
  }
  if (pos >= p.lens[b]) return;
  const int64_t crow = q4_row(p, b, pos);
  if (crow < 0) {
    if (lane == 0) atomicOr(&g_status, kDevErrBounds);
    return;
  }
  const int64_t r = crow * p.Hkv + h;
  const float ks = __bfloat162float(p.scales[r * kQ4Scales + lane / 8]);
  const float vs = __bfloat162float(p.scales[r * kQ4Scales + 4 + lane / 8]);
#pragma unroll
  for (int e = 0; e < PPL; ++e) {
    const int c = lane * PPL + e;
    const uint32_t w = p.k_codes[r * HALF + q4_key_byte(D, c)];
    p.k_out[row * D + c] = __float2bfloat16_rn(ks * (static_cast<int>(w & 15u) - 8));
    p.k_out[row * D + c + HALF] = __float2bfloat16_rn(ks * (static_cast<int>(w >> 4) - 8));
  }
#pragma unroll
  for (int e = 0; e < VPL; ++e) {
    const int c = lane * VPL + e;
    const uint32_t w = p.v_codes[r * HALF + (D / 16) * (c % 8) + c / 16] >> (c % 16 / 8 * 4);
    p.v_out[row * D + c] = __float2bfloat16_rn(vs * (static_cast<int>(w & 15u) - 8));
  }
}

}  // namespace jl
