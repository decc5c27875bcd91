// jl_decode_q4.cuh -- bifocal decode against the 4-bit base-RoPE cache of jl_q4.cuh.
//
// Method: "Jet-Long: Efficient Long-Context Extension with Dynamic Bifocal RoPE",
// Methodology section 2, on-the-fly correction rotation, as in jl_decode.cuh: local keys
// score q~ . k~_j, remote keys (R(f(i) - i) q~) . (R(f(j) - j) k~_j), with k~_j and v_j the
// rows the codes and scales stand for.
//
// Work split.  The keys of all entries and heads are one list of tiles, in the order
// (head block, entry, tile), cut into equal ranges, one per CTA.  A CTA walks its range
// segment by segment (a segment is the part of one entry and head block inside the range),
// so a batch of any lengths loads every SM alike, and the split follows the lengths on the
// device, not max_seqlen.  A segment that covers its whole entry writes the result; the
// others leave a partial (m, l, o) that jl_decode_q4_combine_kernel joins.  Only the first
// and the last segment of a range can be partial, so two slots per CTA are enough.
#pragma once

#include "jl_device.cuh"
#include "jl_q4.cuh"

namespace jl {

struct DecodeQ4Params {
  const __nv_bfloat16* q;      // [B][Hq][D], rotated by R(i)
  const uint8_t* k_codes;
  const uint8_t* v_codes;
  const __nv_bfloat16* scales;
  const int32_t* seqlens;
  const float* cos_tab;
  const float* sin_tab;
  float* ws;                   // o [n_cta][2][heads][D], then (m, l) [n_cta][2][heads][2]
  __nv_bfloat16* out;
  float* lse;
  int64_t cache_stride;
  int64_t n_tab_rows;
  const int32_t* block_table;
  int32_t page_size, max_pages, num_pages;
  int32_t B, Hq, Hkv, group;
  int32_t w0, w_pre, max_seqlen;
  int32_t n_cta;
  int32_t heads_per_block;     // KV heads of a head block
  int32_t tile;                // keys of a tile
  float scale_log2;
};

// Tiles of an entry of length L (0 for an empty one, or for a length outside the contract,
// which the combine reports).
__device__ __forceinline__ int q4_tiles(const DecodeQ4Params& p, int L) {
  return L < 1 || L > p.max_seqlen ? 0 : (L + p.tile - 1) / p.tile;
}

// Tiles of all entries, and of the entries before b, by one warp.
__device__ __forceinline__ int2 q4_tiles_before(const DecodeQ4Params& p, int b, int lane) {
  int all = 0, before = 0;
  for (int e = lane; e < p.B; e += 32) {
    const int t = q4_tiles(p, p.seqlens[e]);
    all += t;
    before += e < b ? t : 0;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    all += __shfl_xor_sync(0xffffffffu, all, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  return make_int2(all, before);
}

// CTAs that get a range (every one of at least a tile), the first tile of CTA c's range, and
// the CTA that holds tile x.
__device__ __forceinline__ int q4_ctas(const DecodeQ4Params& p, int64_t total) {
  return static_cast<int>(min(static_cast<int64_t>(p.n_cta), total));
}
__device__ __forceinline__ int64_t q4_range_begin(int64_t total, int n_cta, int c) { return total * c / n_cta; }
__device__ __forceinline__ int q4_cta_of(int64_t total, int n_cta, int64_t x) {
  return static_cast<int>(((x + 1) * n_cta - 1) / total);
}

// Where a range starts: entry and tile inside it.
struct Q4Start {
  int hb, b, tile;
  int64_t begin, end;  // the range in the list of all tiles
};

__device__ __forceinline__ Q4Start q4_range(const DecodeQ4Params& p, int lane) {
  Q4Start s{0, 0, 0, 0, 0};
  const int all = q4_tiles_before(p, 0, lane).x;
  const int64_t total = static_cast<int64_t>(all) * (p.Hkv / p.heads_per_block);
  const int n_cta = q4_ctas(p, total);
  if (static_cast<int>(blockIdx.x) >= n_cta) return s;
  s.begin = q4_range_begin(total, n_cta, blockIdx.x);
  s.end = q4_range_begin(total, n_cta, blockIdx.x + 1);
  s.hb = static_cast<int>(s.begin / all);
  int left = static_cast<int>(s.begin % all);
  for (int e0 = 0; e0 < p.B; e0 += 32) {
    const int e = e0 + lane;
    const int t = e < p.B ? q4_tiles(p, p.seqlens[e]) : 0;
    int sum = t;  // inclusive prefix over the lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += up;
    }
    const unsigned here = __ballot_sync(0xffffffffu, sum > left);
    if (here) {
      const int src = __ffs(here) - 1;
      s.b = e0 + src;
      s.tile = left - __shfl_sync(0xffffffffu, sum - t, src);
      return s;
    }
    left -= __shfl_sync(0xffffffffu, sum, 31);
  }
  return s;
}

// Cache row of entry b's position j; -1 for a page outside the pool.
__device__ __forceinline__ int64_t q4_row(const DecodeQ4Params& p, int b, int j) {
  if (p.block_table == nullptr) return static_cast<int64_t>(b) * p.cache_stride + j;
  const int32_t page = p.block_table[static_cast<int64_t>(b) * p.max_pages + j / p.page_size];
  if (page < 0 || page >= p.num_pages) return -1;
  return static_cast<int64_t>(page) * p.page_size + j % p.page_size;
}

constexpr int kDecodeQ4Threads = 256;
constexpr int kDecodeQ4MaxGroup = 16;

// A CTA takes one KV head; its eight warps take keys in turn, a lane owns D/64 key pairs and
// D/32 value channels.
template <int D>
__global__ void __launch_bounds__(kDecodeQ4Threads) jl_decode_q4_kernel(const DecodeQ4Params p) {
  constexpr int HALF = D / 2, PPL = D / 64, VPL = D / 32, NW = kDecodeQ4Threads / 32, G = kDecodeQ4MaxGroup;
  __shared__ float qs[2][G][D];  // queries in log2 units: local, remote
  __shared__ float red_m[NW][G], red_l[NW][G], red_o[NW][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_wait();
  griddep_launch_dependents();
  const Q4Start s = q4_range(p, lane);
  int64_t cur = s.begin;
  int hb = s.hb, b = s.b, t0 = s.tile;
  while (cur < s.end) {
    const int L = p.seqlens[b], tiles = q4_tiles(p, L);
    const int t1 = static_cast<int>(min(static_cast<int64_t>(tiles), t0 + (s.end - cur)));
    if (t1 > t0) {
      const int i = L - 1, grow = max(1, (L + p.w_pre - 1) / p.w_pre);
      const int jb = grow > 1 ? i - p.w0 : -1;  // remote keys are j <= jb
      const int nq = i - i / grow;
      __syncthreads();
      for (int x = threadIdx.x; x < p.group * HALF; x += kDecodeQ4Threads) {
        const int g = x / HALF, c = x % HALF;
        const __nv_bfloat16* qp = p.q + (static_cast<int64_t>(b) * p.Hq + hb * p.group + g) * D;
        const float lo = __bfloat162float(qp[c]) * p.scale_log2, hi = __bfloat162float(qp[c + HALF]) * p.scale_log2;
        const float cs = p.cos_tab[static_cast<int64_t>(nq) * HALF + c];
        const float sn = p.sin_tab[static_cast<int64_t>(nq) * HALF + c];
        qs[0][g][c] = lo;
        qs[0][g][c + HALF] = hi;
        qs[1][g][c] = lo * cs + hi * sn;
        qs[1][g][c + HALF] = hi * cs - lo * sn;
      }
      __syncthreads();
      float m[G], l[G], o[G][VPL];
#pragma unroll
      for (int g = 0; g < G; ++g) {
        m[g] = -INFINITY;
        l[g] = 0.f;
#pragma unroll
        for (int e = 0; e < VPL; ++e) o[g][e] = 0.f;
      }
      const int j1 = min(L, t1 * p.tile);
      for (int j = t0 * p.tile + warp; j < j1; j += NW) {
        const int64_t row = q4_row(p, b, j);
        if (row < 0) {
          if (lane == 0) atomicOr(&g_status, kDevErrBounds);
          continue;
        }
        const int64_t r = row * p.Hkv + hb;
        const float ks = __bfloat162float(p.scales[r * kQ4Scales + lane / 8]);
        const float vs = __bfloat162float(p.scales[r * kQ4Scales + 4 + lane / 8]);
        const int remote = j <= jb ? 1 : 0;
        const int64_t n = remote ? j - j / grow : 0;
        float klo[PPL], khi[PPL], v[VPL];
#pragma unroll
        for (int e = 0; e < PPL; ++e) {
          const int c = lane * PPL + e;
          const uint32_t w = p.k_codes[r * HALF + q4_key_byte(D, c)];
          const float a = ks * (static_cast<int>(w & 15u) - 8), bb = ks * (static_cast<int>(w >> 4) - 8);
          const float cs = remote ? p.cos_tab[n * HALF + c] : 1.f, sn = remote ? p.sin_tab[n * HALF + c] : 0.f;
          klo[e] = a * cs + bb * sn;
          khi[e] = bb * cs - a * sn;
        }
#pragma unroll
        for (int e = 0; e < VPL; ++e) {
          const int c = lane * VPL + e;
          const uint32_t w = p.v_codes[r * HALF + (D / 16) * (c % 8) + c / 16] >> (c % 16 / 8 * 4);
          v[e] = vs * (static_cast<int>(w & 15u) - 8);
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
          if (g >= p.group) break;
          float acc = 0.f;
#pragma unroll
          for (int e = 0; e < PPL; ++e) {
            acc = fmaf(qs[remote][g][lane * PPL + e], klo[e], acc);
            acc = fmaf(qs[remote][g][HALF + lane * PPL + e], khi[e], acc);
          }
#pragma unroll
          for (int x = 16; x; x >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, x);
          const float mn = fmaxf(m[g], acc);
          const float alpha = m[g] == -INFINITY ? 0.f : ex2_approx(m[g] - mn);
          const float pr = ex2_approx(acc - mn);
          m[g] = mn;
          l[g] = fmaf(l[g], alpha, pr);
#pragma unroll
          for (int e = 0; e < VPL; ++e) o[g][e] = fmaf(o[g][e], alpha, pr * v[e]);
        }
      }
      // join the warps, head by head
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if (g >= p.group) break;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < VPL; ++e) red_o[warp][lane * VPL + e] = o[g][e];
        if (lane == 0) {
          red_m[warp][g] = m[g];
          red_l[warp][g] = l[g];
        }
        __syncthreads();
        float mx = -INFINITY, lsum = 0.f;
        for (int w = 0; w < NW; ++w) mx = fmaxf(mx, red_m[w][g]);
        for (int w = 0; w < NW; ++w) lsum += red_m[w][g] == -INFINITY ? 0.f : red_l[w][g] * ex2_approx(red_m[w][g] - mx);
        const int qh = hb * p.group + g;
        const bool whole = t0 == 0 && t1 == tiles;
        const int64_t slot = (static_cast<int64_t>(blockIdx.x) * 2 + (cur == s.begin ? 0 : 1)) * p.group + g;
        float* ml = p.ws + static_cast<int64_t>(p.n_cta) * 2 * p.group * D;
        for (int c = threadIdx.x; c < D; c += kDecodeQ4Threads) {
          float acc = 0.f;
          for (int w = 0; w < NW; ++w)
            acc += red_m[w][g] == -INFINITY ? 0.f : red_o[w][c] * ex2_approx(red_m[w][g] - mx);
          if (whole) {
            p.out[(static_cast<int64_t>(b) * p.Hq + qh) * D + c] = __float2bfloat16_rn(acc / lsum);
            if (c == 0 && p.lse != nullptr)
              p.lse[static_cast<int64_t>(b) * p.Hq + qh] = (mx + log2f(lsum)) * 0.69314718055994531f;
          } else {
            p.ws[slot * D + c] = acc;
            if (c == 0) {
              ml[slot * 2] = mx;
              ml[slot * 2 + 1] = lsum;
            }
          }
        }
      }
    }
    cur += t1 - t0;
    t0 = 0;
    if (++b == p.B) {
      b = 0;
      ++hb;
    }
  }
}

constexpr int kCombineQ4Threads = 128;

// Joins the partials of one (entry, query head), which lie in the ranges of CTAs c0 .. c1;
// writes zeros and -inf for an empty entry, NaN for a length outside the contract (reported
// by jl_sync_status) or a kernel that gave up.
template <int D>
__global__ void __launch_bounds__(kCombineQ4Threads) jl_decode_q4_combine_kernel(const DecodeQ4Params p) {
  const int qh = blockIdx.x, b = blockIdx.y, lane = threadIdx.x & 31;
  griddep_launch_dependents();
  griddep_wait();
  const int hpb = p.heads_per_block * p.group, hb = qh / hpb;
  const int L = p.seqlens[b], t = q4_tiles(p, L);
  const int2 n = q4_tiles_before(p, b, lane);
  const bool wrong = L < 0 || L > p.max_seqlen;
  const bool bad = wrong || status_failed();
  const int64_t at = static_cast<int64_t>(b) * p.Hq + qh;
  if (bad || t == 0) {
    if (wrong && threadIdx.x == 0 && qh == 0) atomicOr(&g_status, kDevErrBounds);
    const float x = bad ? __int_as_float(0x7fc00000) : 0.f;
    for (int c = threadIdx.x; c < D; c += kCombineQ4Threads) p.out[at * D + c] = __float2bfloat16_rn(x);
    if (threadIdx.x == 0 && p.lse != nullptr) p.lse[at] = bad ? x : -INFINITY;
    return;
  }
  const int64_t total = static_cast<int64_t>(n.x) * (p.Hkv / p.heads_per_block);
  const int64_t first = static_cast<int64_t>(hb) * n.x + n.y;
  const int n_cta = q4_ctas(p, total);
  const int c0 = q4_cta_of(total, n_cta, first), c1 = q4_cta_of(total, n_cta, first + t - 1);
  if (c0 == c1) return;  // the decode wrote the result
  const int s0 = q4_range_begin(total, n_cta, c0) == first ? 0 : 1;
  const float* ml = p.ws + static_cast<int64_t>(p.n_cta) * 2 * hpb * D;
  float mx = -INFINITY, l = 0.f;
  for (int c = c0; c <= c1; ++c) mx = fmaxf(mx, ml[((c * 2LL + (c == c0 ? s0 : 0)) * hpb + qh % hpb) * 2]);
  for (int ch = threadIdx.x; ch < D; ch += kCombineQ4Threads) {
    float acc = 0.f;
    l = 0.f;
    for (int c = c0; c <= c1; ++c) {
      const int64_t slot = (c * 2LL + (c == c0 ? s0 : 0)) * hpb + qh % hpb;
      const float w = ml[slot * 2] == -INFINITY ? 0.f : ex2_approx(ml[slot * 2] - mx);
      acc = fmaf(p.ws[slot * D + ch], w, acc);
      l = fmaf(ml[slot * 2 + 1], w, l);
    }
    p.out[at * D + ch] = __float2bfloat16_rn(acc / l);
  }
  if (threadIdx.x == 0 && p.lse != nullptr) p.lse[at] = (mx + log2f(l)) * 0.69314718055994531f;
}

}  // namespace jl
