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

#include <cuda_fp16.h>

#include <type_traits>

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

// ------------------------------------------------------------- the decode kernel --
//
// Shape.  12 warps a CTA: eight take keys (below), four prepare what they need.  A tile is
// `tile` keys of all KV heads of a head block; it arrives by TMA as [head][32 keys][row]
// boxes of key codes, value codes and scales, in a ring of stages.
//
// Matrix instructions: mma.m16n8k16 with the keys on M for the scores and the channels on M
// for the values.  A lane expands the codes of its own fragment in registers: four to six
// instructions make a register of two operands that the matrix instruction reads at once.
// tcgen05 would need the expanded tile in shared memory: 2 bytes a code written and 2 read
// beside the code's own half, 37 us of shared-memory time for 128K keys of eight heads,
// where the codes take 23 us to arrive; expanded in registers they cost none.
//
// Scores.  The codes less 8 are small integers, exact in fp16.  The query of each head is
// scaled by a power of two to a largest channel in [8, 16) and split into two fp16 numbers,
// columns 2h and 2h + 1 of B, which carry 22 of its bits (bf16 queries are exact, rotated
// ones off by 2^-22).  Local keys therefore score exactly up to the fp32 sums.  A remote
// key's pairs are first turned by R(f(j) - j) in fp16: cos and sin to 2^-12, one product
// and one sum rounded to 11 bits, so a score is off by some 1e-4 of its size, more exact
// than the bf16 keys of the 16-bit cache.  The group scales are applied to the fp32 sums of
// their group, between the matrix instructions.
//
// Weights are multiplied by the value scales of their key in fp32 and rounded to fp16 (2^-11
// of each).  So that the products fit fp16 whatever the scales, the softmax's reference M is
// not the largest score but follows the largest score + log2(largest scale of the key): M
// keeps weight * scale = 2^(score - M) * scale at or below 2^14, where it was 2^10 when M last
// moved, and products down to 2^-34 of the largest still count.  Numerator and denominator
// share M, so it drops out.  Sums and outputs are held in fp32.
//
// The rotations' cos and sin are the same for all heads, so four warps make them once a tile
// for the whole head block: from the table's row of the tile's first key by steps of one
// position in fp32 (at most 32 steps), stored as fp16 in the order of the fragments.

constexpr int kDecodeQ4Ctas = 148;  // one per SM
constexpr int kDecodeQ4KeyWarps = 8, kDecodeQ4TabWarps = 4;
constexpr int kDecodeQ4Threads = 32 * (kDecodeQ4KeyWarps + kDecodeQ4TabWarps);
constexpr int kDecodeQ4MaxStages = 6;
// Registers a thread: 168 at launch; the key warps rise to 216, the others drop to 72.
constexpr int kDecodeQ4Regs = 168, kDecodeQ4KeyRegs = 216, kDecodeQ4TabRegs = 72;
static_assert(kDecodeQ4KeyWarps * kDecodeQ4KeyRegs + kDecodeQ4TabWarps * kDecodeQ4TabRegs <=
                  (kDecodeQ4KeyWarps + kDecodeQ4TabWarps) * kDecodeQ4Regs,
              "the split has to fit the launch's registers, or setmaxnreg waits for good");

// Shared memory: a region for the query fragments, reused to join the key warps, then the
// stages.  A stage: key codes, value codes, scales, cos/sin rows.
struct DecodeQ4Layout {
  int region, codes, scales, table, stage, stages, total;
};

// NQ: score tiles of four query heads; HPB: KV heads of a block; HPW: of a key warp.
__host__ __device__ constexpr DecodeQ4Layout decode_q4_layout(int D, int NQ, int HPW, int HPB, int tile) {
  DecodeQ4Layout l{};
  const int frags = 2 * HPB * NQ * (D / 32) * 512, join = kDecodeQ4KeyWarps * HPW * NQ * 4 * D * 4;
  l.region = frags > join ? frags : join;
  l.codes = tile * HPB * D / 2;
  l.scales = tile * HPB * 16;
  l.table = tile * D * 2;
  l.stage = 2 * l.codes + l.scales + l.table;
  l.stages = (220 * 1024 - l.region) / l.stage;
  if (l.stages > kDecodeQ4MaxStages) l.stages = kDecodeQ4MaxStages;
  l.total = l.region + l.stages * l.stage + 1024;
  return l;
}

struct DecodeQ4Shared {
  uint64_t full[kDecodeQ4MaxStages];   // codes and scales have arrived
  uint64_t turned[kDecodeQ4MaxStages]; // cos/sin rows are written
  uint64_t empty[kDecodeQ4MaxStages];
  float mul[32];                       // log2 units per unit of score, by query head of the block
  float red_m[kDecodeQ4KeyWarps][16], red_l[kDecodeQ4KeyWarps][16];
  Q4Start start;
  int abort;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void key_warps_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kDecodeQ4KeyWarps) : "memory");
}

__device__ __forceinline__ uint32_t h2_bits(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }
__device__ __forceinline__ __half2 bits_h2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
__device__ __forceinline__ uint32_t select_or(uint32_t x, uint32_t mask, uint32_t set) {
  uint32_t y;  // (x & mask) | set
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(y) : "r"(x), "r"(mask), "r"(set));
  return y;
}

// Codes of the low (HIGH = false) or high four bits of bytes 0 and 2 of w, less 8, as two
// fp16.  1024 + n and 1024 + 16 n are fp16 numbers with n in their lowest mantissa bits.
template <bool HIGH>
__device__ __forceinline__ __half2 codes_f16(uint32_t w) {
  if constexpr (HIGH)
    return __hfma2(bits_h2(select_or(w, 0x00f000f0u, 0x64006400u)), __float2half2_rn(0.0625f), __float2half2_rn(-72.f));
  else
    return __hsub2(bits_h2(select_or(w, 0x000f000fu, 0x64006400u)), __float2half2_rn(1032.f));
}

// Row r of a block's sixteen keys holds key q4_key_of(r): neighbouring rows are keys of
// opposite parity, and rows 0, 2, 4, 6 (and 1, 3, 5, 7) fall on different banks in the
// swizzled code boxes, so both the key and the value loads are free of bank conflicts.
__device__ __forceinline__ int q4_key_of(int r) { return r ^ ((r >> 1) & 1); }

// Shared-memory offset of byte x of key `key`'s codes in a [keys][D/2] box (64-byte swizzle
// for D = 128, none for D = 64).
template <int D>
__device__ __forceinline__ int q4_code_at(int key, int x) {
  return D == 128 ? key * 64 + (x ^ (((key >> 1) & 3) << 4)) : key * 32 + x;
}

// Offset of 16-byte chunk (word w, lane t) of cos/sin row r.
template <int D>
__device__ __forceinline__ int q4_turn_at(int r, int w, int t) {
  return r * 2 * D + ((w * 64 + t * 16) ^ ((r & 1) << 6));  // neighbouring rows on different banks
}

// floor(x / G) for x < G + 128: G < 128 by a 16-bit reciprocal (x < 256, exact since
// x * G < 2^16), a larger G by one comparison.
struct SmallDiv {
  int g, magic;
  __device__ __forceinline__ explicit SmallDiv(int G) : g(G), magic(G < 128 ? (65536 + G - 1) / G : 0) {}
  __device__ __forceinline__ int operator()(int x) const { return magic ? (x * magic) >> 16 : (x >= g ? 1 : 0); }
};

template <int D, int NQ, int HPW>
__global__ void __launch_bounds__(kDecodeQ4Threads, 1)
    jl_decode_q4_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                        const __grid_constant__ CUtensorMap ts, const DecodeQ4Params p) {
  constexpr int HALF = D / 2;
  constexpr int KW = D / 32;    // 32-bit words of a lane's key codes (and fragments of four registers)
  constexpr int VW = D / 64;    // of its value codes
  constexpr int MT = D / 16;    // output tiles of 16 channels
  constexpr int NP = (NQ + 1) / 2;  // value tiles of eight columns
  constexpr bool kQueryRegs = NQ * HPW <= 2;
  extern __shared__ uint8_t raw_smem[];
  __shared__ DecodeQ4Shared sh;
  uint8_t* smem = raw_smem + ((1024u - (smem_u32(raw_smem) & 1023u)) & 1023u);
  const int HPB = p.heads_per_block, T = p.tile;
  const DecodeQ4Layout lay = decode_q4_layout(D, NQ, HPW, HPB, T);
  uint8_t* const stages = smem + lay.region;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &sh.abort;

  if (threadIdx.x == 0) {
    for (int s = 0; s < lay.stages; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.turned[s], kDecodeQ4TabWarps);
      mbar_init(&sh.empty[s], kDecodeQ4KeyWarps);
    }
    sh.abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
    tma_prefetch_desc(&ts);
  }
  griddep_wait();  // the cache, the lengths and the query may come from the previous kernel
  griddep_launch_dependents();
  if (warp == 0) {
    Q4Start s = q4_range(p, lane);
    if (__any_sync(0xffffffffu, status_failed())) s.end = s.begin;
    if (lane == 0) sh.start = s;
  }
  __syncthreads();
  const Q4Start st = sh.start;
  int64_t cur = st.begin;
  int hb = st.hb, b = st.b, t0 = st.tile;
  int stage = 0;
  uint32_t phase = 0;

  if (warp >= kDecodeQ4KeyWarps) {
    // ------------------------------------------------ loads and cos/sin rows --
    setmaxnreg_dec<kDecodeQ4TabRegs>();
    const int tw = warp - kDecodeQ4KeyWarps;
    const int per = T / kDecodeQ4TabWarps;  // rows of this warp
    // lane -> the two pairs of one packed register: word w, fragment lane t, register half e
    const bool has = D == 128 || lane < 16;
    const int w = D == 128 ? lane / 8 : (lane & 15) / 8, t = D == 128 ? (lane / 2) & 3 : lane & 3;
    const int e = D == 128 ? lane & 1 : (lane >> 2) & 1;
    const int c0 = D == 128 ? 16 * w + 4 * t + e : 8 * (2 * w + e) + 2 * t, c1 = D == 128 ? c0 + 2 : c0 + 1;
    float step_c[2] = {1.f, 1.f}, step_s[2] = {0.f, 0.f};
    if (p.n_tab_rows > 1) {
      step_c[0] = p.cos_tab[HALF + c0], step_s[0] = p.sin_tab[HALF + c0];
      step_c[1] = p.cos_tab[HALF + c1], step_s[1] = p.sin_tab[HALF + c1];
    }
    int issued = 0;
    bool ok = true;
    while (cur < st.end && ok) {
      const int L = p.seqlens[b], tiles = q4_tiles(p, L);
      const int t1 = static_cast<int>(min(static_cast<int64_t>(tiles), t0 + (st.end - cur)));
      const int grow = max(1, (L + p.w_pre - 1) / p.w_pre);
      const int jb = grow > 1 ? L - 1 - p.w0 : -1;  // remote keys are j <= jb
      int quot = (t0 * T) / grow, rem = (t0 * T) % grow;
      const int dq = T / grow, dr = T % grow;
      for (int tile = t0; tile < t1; ++tile) {
        const int j0 = tile * T;
        const bool remote = j0 <= jb;
        float ac[2], as[2];
        if (remote) {
          const int64_t row = min(static_cast<int64_t>(j0 - quot + tw * per), p.n_tab_rows - 1) * HALF;
          JL_CHECK(row >= 0 && quot == j0 / grow && j0 - quot < p.n_tab_rows);
          ac[0] = p.cos_tab[row + c0], as[0] = p.sin_tab[row + c0];
          ac[1] = p.cos_tab[row + c1], as[1] = p.sin_tab[row + c1];
        }
        if (!warp_wait(&sh.empty[stage], phase ^ 1, abort)) {
          ok = false;
          break;
        }
        uint8_t* base = stages + stage * lay.stage;
        if (tw == 0 && lane == 0) {
          mbar_arrive_expect_tx(&sh.full[stage], 2 * lay.codes + lay.scales);
          for (int x = 0; x < T / 32; ++x) {
            int row = static_cast<int>(b * p.cache_stride + j0 + 32 * x);
            if (p.block_table != nullptr) {
              // pages behind the length need no entry: their keys are never used
              const int j = j0 + 32 * x;
              const int page = j < L ? p.block_table[static_cast<int64_t>(b) * p.max_pages + j / p.page_size] : 0;
              const bool there = page >= 0 && page < p.num_pages;
              if (!there) atomicOr(&g_status, kDevErrBounds);
              row = (there ? page : p.num_pages) * p.page_size + (there ? j % p.page_size : 0);  // outside reads zeros
            }
            tma_load_3d(base + x * HPB * 32 * HALF, &tk, &sh.full[stage], 0, row, hb * HPB);
            tma_load_3d(base + lay.codes + x * HPB * 32 * HALF, &tv, &sh.full[stage], 0, row, hb * HPB);
            tma_load_3d(base + 2 * lay.codes + x * HPB * 512, &ts, &sh.full[stage], 0, row, hb * HPB);
          }
        }
        ++issued;
        if (remote && has) {
          uint8_t* tab = base + 2 * lay.codes + lay.scales;
#pragma unroll 4
          for (int r = tw * per; r < (tw + 1) * per; ++r) {
            uint8_t* at = tab + q4_turn_at<D>(r, w, t) + 4 * e;
            *reinterpret_cast<__half2*>(at) = __floats2half2_rn(ac[0], ac[1]);
            *reinterpret_cast<__half2*>(at + 8) = __floats2half2_rn(as[0], as[1]);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float nc = ac[x] * step_c[x] - as[x] * step_s[x];
              as[x] = as[x] * step_c[x] + ac[x] * step_s[x];
              ac[x] = nc;
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.turned[stage]);
        quot += dq;
        rem += dr;
        if (rem >= grow) {
          rem -= grow;
          ++quot;
        }
        if (++stage == lay.stages) {
          stage = 0;
          phase ^= 1;
        }
      }
      cur += t1 - t0;
      t0 = 0;
      if (++b == p.B) {
        b = 0;
        ++hb;
      }
    }
    if (!ok && tw == 0 && lane == 0) {
      // gave up: the copies in flight land before the block leaves its shared memory
      for (int x = max(0, issued - lay.stages); x < issued; ++x)
        mbar_wait_bounded(&sh.full[x % lay.stages], (x / lay.stages) & 1);
    }
    return;
  }

  // ------------------------------------------------------------------ the keys --
  setmaxnreg_inc<kDecodeQ4KeyRegs>();
  const int g = lane >> 2, t = lane & 3;
  const int wph = kDecodeQ4KeyWarps * HPW / HPB;  // warps that share a head, each its own blocks of keys
  const int wsub = warp % wph, h0 = warp / wph * HPW;  // this warp's first KV head in the block
  const int keyA = q4_key_of(g);                       // its rows' keys in a block: keyA, keyA + 8
  const int key0 = q4_key_of(2 * t), key1 = q4_key_of(2 * t + 1);  // and its value rows' keys
  uint4* const frags = reinterpret_cast<uint4*>(smem);  // [2][HPB][NQ][KW][32]
  float* const join = reinterpret_cast<float*>(smem);   // [warps][HPW][4 NQ][D]
  bool ok = true;

  while (cur < st.end) {
    const int L = p.seqlens[b], tiles = q4_tiles(p, L);
    const int t1 = static_cast<int>(min(static_cast<int64_t>(tiles), t0 + (st.end - cur)));
    if (t1 > t0) {
      const int i = L - 1, grow = max(1, (L + p.w_pre - 1) / p.w_pre);
      const int jb = grow > 1 ? i - p.w0 : -1;

      // Query fragments, a head of the block at a time: local and remote variant, each split
      // into two fp16 columns.
      {
        const int nq = i - i / grow;
        const bool has = D == 128 || lane < 16;
        const int w = D == 128 ? lane / 8 : (lane & 15) / 8, ft = D == 128 ? (lane / 2) & 3 : lane & 3;
        const int e = D == 128 ? lane & 1 : (lane >> 2) & 1;
        const int c0 = D == 128 ? 16 * w + 4 * ft + e : 8 * (2 * w + e) + 2 * ft, c1 = D == 128 ? c0 + 2 : c0 + 1;
        float cs[2], sn[2];
        cs[0] = p.cos_tab[static_cast<int64_t>(nq) * HALF + c0], cs[1] = p.cos_tab[static_cast<int64_t>(nq) * HALF + c1];
        sn[0] = p.sin_tab[static_cast<int64_t>(nq) * HALF + c0], sn[1] = p.sin_tab[static_cast<int64_t>(nq) * HALF + c1];
        for (int x = warp; x < HPB * 4 * NQ; x += kDecodeQ4KeyWarps) {
          const int h = x / (4 * NQ), qh = x % (4 * NQ);  // KV head of the block, query head of its group
          float lo[2] = {0.f, 0.f}, hi[2] = {0.f, 0.f};
          if (qh < p.group && has) {
            const __nv_bfloat16* qp = p.q + (static_cast<int64_t>(b) * p.Hq + (hb * HPB + h) * p.group + qh) * D;
            lo[0] = __bfloat162float(qp[c0]), lo[1] = __bfloat162float(qp[c1]);
            hi[0] = __bfloat162float(qp[c0 + HALF]), hi[1] = __bfloat162float(qp[c1 + HALF]);
          }
          float top = fmaxf(fmaxf(fabsf(lo[0]), fabsf(lo[1])), fmaxf(fabsf(hi[0]), fabsf(hi[1])));
#pragma unroll
          for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          // 2^up brings the largest channel into [8, 16); up in [-120, 120] keeps both factors normal
          const int up = min(120, max(-120, 130 - static_cast<int>(__float_as_uint(top) >> 23)));
          const float f = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
          if (lane == 0) sh.mul[x] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
          if (has) {
#pragma unroll
            for (int var = 0; var < 2; ++var) {
              float y[4];  // channels c0, c1, c0 + D/2, c1 + D/2
#pragma unroll
              for (int n = 0; n < 2; ++n) {
                y[n] = (var ? lo[n] * cs[n] + hi[n] * sn[n] : lo[n]) * f;
                y[2 + n] = (var ? hi[n] * cs[n] - lo[n] * sn[n] : hi[n]) * f;
              }
              uint32_t* at = reinterpret_cast<uint32_t*>(frags + (((var * HPB + h) * NQ + qh / 4) * KW + w) * 32);
              const int col = 2 * (qh & 3);
#pragma unroll
              for (int n = 0; n < 2; ++n) {
                const __half2 big = __floats2half2_rn(y[2 * n], y[2 * n + 1]);
                const float2 bf = __half22float2(big);
                const __half2 small = __floats2half2_rn(y[2 * n] - bf.x, y[2 * n + 1] - bf.y);
                const int reg = D == 128 ? 2 * n + e : 2 * e + n;
                at[(col * 4 + ft) * 4 + reg] = h2_bits(big);
                at[((col + 1) * 4 + ft) * 4 + reg] = h2_bits(small);
              }
            }
          }
        }
      }
      key_warps_sync();

      float o[HPW][NP][MT][4], m[HPW][NQ], l[HPW][NQ], mul[HPW][NQ];
      uint4 qf[kQueryRegs ? HPW * NQ * KW : 1];
      int have = -1;  // the variant that qf holds
#pragma unroll
      for (int h = 0; h < HPW; ++h) {
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          m[h][n] = -INFINITY;
          l[h][n] = 0.f;
          mul[h][n] = sh.mul[(h0 + h) * 4 * NQ + 4 * n + t];
        }
#pragma unroll
        for (int n = 0; n < NP; ++n)
#pragma unroll
          for (int x = 0; x < MT; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) o[h][n][x][y] = 0.f;
      }
      const SmallDiv div(grow);
      int rem = (t0 * T) % grow;
      const int dr = T % grow;

      for (int tile = t0; tile < t1; ++tile) {
        const int j0 = tile * T;
        if (ok) ok = warp_wait(&sh.full[stage], phase, abort) && warp_wait(&sh.turned[stage], phase, abort);
        const uint8_t* base = stages + stage * lay.stage;
        const uint8_t* tab = base + 2 * lay.codes + lay.scales;
        for (int blk = wsub; blk < T / 16 && ok; blk += wph) {
          const int jblk = j0 + blk * 16;
          if (jblk >= L) break;
          const int x0 = (blk >> 1) * HPB * 32, first = (blk & 1) * 16;  // box, and the block's first key in it
          const bool any_far = jblk <= jb, all_far = jblk + 15 <= jb || L - 1 <= jb, tail = jblk + 16 > L;
          float s[HPW][NQ][2];  // scores of rows g and g + 8, head 4 n + t

          uint32_t kc[HPW][2][KW];
          float ks[HPW][2][4], vs[HPW][2][4];
#pragma unroll
          for (int h = 0; h < HPW; ++h)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const int key = first + keyA + 8 * r;
              const uint8_t* at = base + (x0 + (h0 + h) * 32) * HALF + q4_code_at<D>(key, t * KW * 4);
              if constexpr (D == 128) {
                const uint4 v = *reinterpret_cast<const uint4*>(at);
                kc[h][r][0] = v.x, kc[h][r][1] = v.y, kc[h][r][2] = v.z, kc[h][r][3] = v.w;
              } else {
                const uint2 v = *reinterpret_cast<const uint2*>(at);
                kc[h][r][0] = v.x, kc[h][r][1] = v.y;
              }
              uint4 sc = *reinterpret_cast<const uint4*>(base + 2 * lay.codes + (x0 + (h0 + h) * 32 + key) * 16);
              if (tail && jblk + keyA + 8 * r >= L) sc = make_uint4(0u, 0u, 0u, 0u);  // weight 0 times a NaN scale is NaN
              ks[h][r][0] = __uint_as_float(sc.x << 16), ks[h][r][1] = __uint_as_float(sc.x & 0xffff0000u);
              ks[h][r][2] = __uint_as_float(sc.y << 16), ks[h][r][3] = __uint_as_float(sc.y & 0xffff0000u);
              vs[h][r][0] = __uint_as_float(sc.z << 16), vs[h][r][1] = __uint_as_float(sc.z & 0xffff0000u);
              vs[h][r][2] = __uint_as_float(sc.w << 16), vs[h][r][3] = __uint_as_float(sc.w & 0xffff0000u);
            }
          const int d0 = blk * 16 + keyA;  // row of the tile's cos/sin rows: d - floor((rem + d) / G)
          const int rowA = d0 - div(rem + d0), rowB = d0 + 8 - div(rem + d0 + 8);
          JL_CHECK(rowA >= 0 && rowB < T && rem < grow && rem == j0 % grow);

          // Scores of this block under one variant of the query (and, far, of the keys).
          auto scores = [&](auto far_tag, float (&dst)[HPW][NQ][2]) {
            constexpr bool FAR = decltype(far_tag)::value;
            if constexpr (kQueryRegs) {
              if (have != FAR) {
                have = FAR;
#pragma unroll
                for (int h = 0; h < HPW; ++h)
#pragma unroll
                  for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int w = 0; w < KW; ++w)
                      qf[(h * NQ + n) * KW + w] = frags[(((FAR * HPB + h0 + h) * NQ + n) * KW + w) * 32 + lane];
              }
            }
#pragma unroll
            for (int h = 0; h < HPW; ++h)
#pragma unroll
              for (int n = 0; n < NQ; ++n) dst[h][n][0] = dst[h][n][1] = 0.f;
#pragma unroll
            for (int w = 0; w < KW; ++w) {
              uint4 turn[2];
              if constexpr (FAR) {
                turn[0] = *reinterpret_cast<const uint4*>(tab + q4_turn_at<D>(rowA, w, t));
                turn[1] = *reinterpret_cast<const uint4*>(tab + q4_turn_at<D>(rowB, w, t));
              }
#pragma unroll
              for (int h = 0; h < HPW; ++h) {
                uint32_t lo[2][2], hi[2][2];  // [row][register half]
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    const uint32_t word = e ? kc[h][r][w] >> 8 : kc[h][r][w];
                    __half2 a = codes_f16<false>(word), bb = codes_f16<true>(word);
                    if constexpr (FAR) {  // R(-n)
                      const __half2 c = bits_h2(e ? turn[r].y : turn[r].x), sn = bits_h2(e ? turn[r].w : turn[r].z);
                      const __half2 na = __hfma2(a, c, __hmul2(bb, sn));
                      bb = __hfma2(bb, c, __hneg2(__hmul2(a, sn)));
                      a = na;
                    }
                    lo[r][e] = h2_bits(a);
                    hi[r][e] = h2_bits(bb);
                  }
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                  const uint4 q = kQueryRegs ? qf[kQueryRegs ? (h * NQ + n) * KW + w : 0]
                                             : frags[(((FAR * HPB + h0 + h) * NQ + n) * KW + w) * 32 + lane];
                  if constexpr (D == 128) {  // a word is one group: two steps, low channels then high
                    float c[4] = {0.f, 0.f, 0.f, 0.f};
                    mma_f16(c, {lo[0][0], lo[1][0], lo[0][1], lo[1][1]}, q.x, q.y);
                    mma_f16(c, {hi[0][0], hi[1][0], hi[0][1], hi[1][1]}, q.z, q.w);
                    dst[h][n][0] = fmaf(ks[h][0][w], c[0] + c[1], dst[h][n][0]);
                    dst[h][n][1] = fmaf(ks[h][1][w], c[2] + c[3], dst[h][n][1]);
                  } else {  // two groups, a step each
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                      float c[4] = {0.f, 0.f, 0.f, 0.f};
                      mma_f16(c, {lo[0][e], lo[1][e], hi[0][e], hi[1][e]}, e ? q.z : q.x, e ? q.w : q.y);
                      dst[h][n][0] = fmaf(ks[h][0][2 * w + e], c[0] + c[1], dst[h][n][0]);
                      dst[h][n][1] = fmaf(ks[h][1][2 * w + e], c[2] + c[3], dst[h][n][1]);
                    }
                  }
                }
              }
            }
          };
          if (!any_far) {
            scores(std::false_type{}, s);
          } else if (all_far) {
            scores(std::true_type{}, s);
          } else {  // the block that straddles the window edge
            float near[HPW][NQ][2];
            scores(std::true_type{}, s);
            scores(std::false_type{}, near);
#pragma unroll
            for (int h = 0; h < HPW; ++h)
#pragma unroll
              for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) s[h][n][r] = jblk + keyA + 8 * r <= jb ? s[h][n][r] : near[h][n][r];
          }

          // Weights and their products with the value scales.  M moves only when a product
          // passes 2^14 (in the first block: by anything), so most blocks rescale nothing.
          float wt[HPW][NQ][2];
          bool over = false;
#pragma unroll
          for (int h = 0; h < HPW; ++h)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float top = fmaxf(fmax3(vs[h][r][0], vs[h][r][1], vs[h][r][2]), fmaxf(vs[h][r][3], 0x1p-90f));
#pragma unroll
              for (int n = 0; n < NQ; ++n) {
                s[h][n][r] *= mul[h][n];
                if (tail && jblk + keyA + 8 * r >= L) s[h][n][r] = -INFINITY;
                wt[h][n][r] = ex2_approx(s[h][n][r] - m[h][n]);
                over |= wt[h][n][r] * top > 0x1p14f;
              }
            }
          if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int h = 0; h < HPW; ++h) {
              float f[NQ];
#pragma unroll
              for (int n = 0; n < NQ; ++n) {
                float top = m[h][n] + 10.f;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                  const float big = fmaxf(fmax3(vs[h][r][0], vs[h][r][1], vs[h][r][2]), fmaxf(vs[h][r][3], 0x1p-90f));
                  top = fmaxf(top, s[h][n][r] + log2f(big));
                }
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                const float now = top - 10.f;
                f[n] = m[h][n] == -INFINITY ? 0.f : ex2_approx(m[h][n] - now);
                m[h][n] = now;
                l[h][n] *= f[n];
                wt[h][n][0] = ex2_approx(s[h][n][0] - now);
                wt[h][n][1] = ex2_approx(s[h][n][1] - now);
              }
#pragma unroll
              for (int n = 0; n < NP; ++n)
#pragma unroll
                for (int x = 0; x < MT; ++x)
#pragma unroll
                  for (int y = 0; y < 4; ++y) o[h][n][x][y] *= f[NQ == 1 ? 0 : 2 * n + (y & 1)];
            }
          }

          // Values.  Column 2t of the weights is head t of score tile 2n, column 2t + 1 of
          // tile 2n + 1; with one score tile both are head t, the even columns under the
          // scales of the even groups and the odd ones under those of the odd groups.
#pragma unroll
          for (int h = 0; h < HPW; ++h) {
            constexpr int kF = NQ == 1 ? 2 : 4;  // scaled fragments: pairs of groups, or groups
            uint32_t pf[NP][kF][2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
#pragma unroll
              for (int n = 0; n < NQ; ++n) l[h][n] += wt[h][n][r];
#pragma unroll
              for (int n = 0; n < NP; ++n)
#pragma unroll
                for (int f = 0; f < kF; ++f) {
                  const float a = wt[h][NQ == 1 ? 0 : 2 * n][r] * vs[h][r][NQ == 1 ? 2 * f : f];
                  const float bb = wt[h][NQ == 1 ? 0 : 2 * n + 1][r] * vs[h][r][NQ == 1 ? 2 * f + 1 : f];
                  pf[n][f][r] = transpose_8x8(h2_bits(__floats2half2_rn(a, bb)));
                }
            }
            const uint8_t* vrow = base + lay.codes + (x0 + (h0 + h) * 32) * HALF;
            uint32_t vc[4][VW];  // value codes of keys key0, key1, key0 + 8, key1 + 8
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const uint8_t* at = vrow + q4_code_at<D>(first + (r & 1 ? key1 : key0) + 8 * (r >> 1), g * MT);
              if constexpr (D == 128) {
                const uint2 v = *reinterpret_cast<const uint2*>(at);
                vc[r][0] = v.x, vc[r][1] = v.y;
              } else {
                vc[r][0] = *reinterpret_cast<const uint32_t*>(at);
              }
            }
#pragma unroll
            for (int w = 0; w < VW; ++w)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const uint32_t pick = y ? 0x7632u : 0x5410u;
                const uint32_t a = __byte_perm(vc[0][w], vc[1][w], pick), bb = __byte_perm(vc[2][w], vc[3][w], pick);
#pragma unroll
                for (int z = 0; z < 2; ++z) {  // channel tile x: byte 2y + z of word w
                  const int x = 4 * w + 2 * y + z, grp = x * 4 / MT;
                  const uint32_t az = a >> (8 * z), bz = bb >> (8 * z);
                  const uint32_t frag[4] = {h2_bits(codes_f16<false>(az)), h2_bits(codes_f16<true>(az)),
                                            h2_bits(codes_f16<false>(bz)), h2_bits(codes_f16<true>(bz))};
#pragma unroll
                  for (int n = 0; n < NP; ++n) {
                    const int f = NQ == 1 ? grp / 2 : grp;
                    mma_f16(o[h][n][x], frag, pf[n][f % kF][0], pf[n][f % kF][1]);
                  }
                }
              }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[stage]);
        rem += dr;
        if (rem >= grow) rem -= grow;
        if (++stage == lay.stages) {
          stage = 0;
          phase ^= 1;
        }
      }

      // Join the warps that share a head, and write the result or the partial.
#pragma unroll
      for (int h = 0; h < HPW; ++h)
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) l[h][n] += __shfl_xor_sync(0xffffffffu, l[h][n], x);
      key_warps_sync();  // every warp is done with the query fragments
#pragma unroll
      for (int h = 0; h < HPW; ++h)
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          if (g == 0) {
            sh.red_m[warp][(h * NQ + n) * 4 + t] = m[h][n];
            sh.red_l[warp][(h * NQ + n) * 4 + t] = l[h][n];
          }
          float* row = join + ((warp * HPW + h) * 4 * NQ + 4 * n + t) * D + g;
#pragma unroll
          for (int x = 0; x < MT; ++x) {
            const int y = NQ == 1 ? (x * 4 / MT) & 1 : n & 1;  // the column that holds this head under this group's scales
            row[16 * x] = o[h][n / 2][x][y];
            row[16 * x + 8] = o[h][n / 2][x][2 + y];
          }
        }
      key_warps_sync();
      const bool whole = t0 == 0 && t1 == tiles;
      const int hpb = HPB * p.group;
      const int64_t slot0 = (static_cast<int64_t>(blockIdx.x) * 2 + (cur == st.begin ? 0 : 1)) * hpb;
      float* ml = p.ws + static_cast<int64_t>(p.n_cta) * 2 * hpb * D;
      for (int x = threadIdx.x; x < hpb * (D / 4); x += 32 * kDecodeQ4KeyWarps) {
        const int q = x / (D / 4), c = x % (D / 4) * 4;  // query head of the block, its channels c .. c + 3
        const int kv = q / p.group, in = kv % HPW * 4 * NQ + q % p.group, w0 = kv / HPW * wph;
        float mx = -INFINITY;
        for (int w = 0; w < wph; ++w) mx = fmaxf(mx, sh.red_m[w0 + w][in]);
        float lsum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < wph; ++w) {
          const float mw = sh.red_m[w0 + w][in];
          if (mw == -INFINITY) {
            lsum += sh.red_l[w0 + w][in];  // 0, or the NaN of scores that are all NaN
            continue;
          }
          const float f = ex2_approx(mw - mx);
          const float4 v = *reinterpret_cast<const float4*>(join + ((w0 + w) * HPW * 4 * NQ + in) * D + c);
          lsum = fmaf(sh.red_l[w0 + w][in], f, lsum);
          acc.x = fmaf(v.x, f, acc.x), acc.y = fmaf(v.y, f, acc.y);
          acc.z = fmaf(v.z, f, acc.z), acc.w = fmaf(v.w, f, acc.w);
        }
        if (whole) {
          const int64_t at = static_cast<int64_t>(b) * p.Hq + hb * hpb + q;
          const float inv = 1.f / lsum;
          *reinterpret_cast<uint2*>(p.out + at * D + c) =
              make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
          if (c == 0 && p.lse != nullptr) p.lse[at] = (mx + log2f(lsum)) * 0.69314718055994531f;
        } else {
          *reinterpret_cast<float4*>(p.ws + (slot0 + q) * D + c) = acc;
          if (c == 0) *reinterpret_cast<float2*>(ml + (slot0 + q) * 2) = make_float2(mx, lsum);
        }
      }
      key_warps_sync();  // the region is free for the next segment's query
    }
    cur += t1 - t0;
    t0 = 0;
    if (++b == p.B) {
      b = 0;
      ++hb;
    }
  }
}

constexpr int kCombineQ4Threads = 256;

// Joins the partials of one (entry, query head), which lie in the ranges of CTAs c0 .. c1;
// writes zeros and -inf for an empty entry, NaN for a length outside the contract (reported
// by jl_sync_status) or a kernel that gave up.  Every thread asks for all it needs before it
// waits for any of it: thread c for the maximum and sum of partial c0 + c, lane by lane the
// channels of every eighth partial.  One round trip for up to 148 partials.
template <int D>
__global__ void __launch_bounds__(kCombineQ4Threads) jl_decode_q4_combine_kernel(const DecodeQ4Params p) {
  constexpr int NW = kCombineQ4Threads / 32, CPL = D / 32, PER = (kDecodeQ4Ctas + NW - 1) / NW;
  static_assert(kDecodeQ4Ctas <= kCombineQ4Threads, "a thread for each partial");
  __shared__ float weight[kCombineQ4Threads], red[2][NW], sum[NW][D];
  const int qh = blockIdx.x, b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_launch_dependents();
  griddep_wait();
  const int hpb = p.heads_per_block * p.group, hb = qh / hpb;
  const int L = p.seqlens[b], t = q4_tiles(p, L);
  const int2 n = q4_tiles_before(p, b, lane);
  const bool wrong = L < 0 || L > p.max_seqlen;
  const bool bad = wrong || status_failed();
  const int64_t at = static_cast<int64_t>(b) * p.Hq + qh;
  if (__syncthreads_or(bad) || t == 0) {
    if (wrong && threadIdx.x == 0 && qh == 0) atomicOr(&g_status, kDevErrBounds);
    const bool nan = bad || t != 0;
    const float x = nan ? __int_as_float(0x7fc00000) : 0.f;
    for (int c = threadIdx.x; c < D; c += kCombineQ4Threads) p.out[at * D + c] = __float2bfloat16_rn(x);
    if (threadIdx.x == 0 && p.lse != nullptr) p.lse[at] = nan ? x : -INFINITY;
    return;
  }
  const int64_t total = static_cast<int64_t>(n.x) * (p.Hkv / p.heads_per_block);
  const int64_t first = static_cast<int64_t>(hb) * n.x + n.y;
  const int n_cta = q4_ctas(p, total);
  const int c0 = q4_cta_of(total, n_cta, first), c1 = q4_cta_of(total, n_cta, first + t - 1);
  if (c0 == c1) return;  // the decode wrote the result
  const int s0 = q4_range_begin(total, n_cta, c0) == first ? 0 : 1;
  const int count = c1 - c0 + 1;
  auto slot = [&](int c) { return ((c0 + c) * 2LL + (c == 0 ? s0 : 0)) * hpb + qh % hpb; };
  const float* ml = p.ws + static_cast<int64_t>(p.n_cta) * 2 * hpb * D;
  float2 own = make_float2(-INFINITY, 0.f);
  if (threadIdx.x < count) own = *reinterpret_cast<const float2*>(ml + slot(threadIdx.x) * 2);
  float o[PER][CPL];
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    const int c = warp + u * NW;
#pragma unroll
    for (int e = 0; e < CPL; ++e) o[u][e] = 0.f;
    if (c < count) {
      const float* row = p.ws + slot(c) * D + lane * CPL;
      if constexpr (CPL == 4) {
        const float4 x = *reinterpret_cast<const float4*>(row);
        o[u][0] = x.x, o[u][1] = x.y, o[u][2] = x.z, o[u][3] = x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(row);
        o[u][0] = x.x, o[u][1] = x.y;
      }
    }
  }
  float mx = own.x;
#pragma unroll
  for (int x = 16; x; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
  if (lane == 0) red[0][warp] = mx;
  __syncthreads();
  mx = red[0][0];
#pragma unroll
  for (int w = 1; w < NW; ++w) mx = fmaxf(mx, red[0][w]);
  const float f = own.x == -INFINITY ? 1.f : ex2_approx(own.x - mx);  // -inf: the sum is 0, or the NaN of NaN scores
  weight[threadIdx.x] = f;
  float l = own.y * f;
#pragma unroll
  for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
  if (lane == 0) red[1][warp] = l;
  __syncthreads();
  float acc[CPL];
#pragma unroll
  for (int e = 0; e < CPL; ++e) acc[e] = 0.f;
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    if (warp + u * NW >= count) break;
    const float w = weight[warp + u * NW];
#pragma unroll
    for (int e = 0; e < CPL; ++e) acc[e] = fmaf(o[u][e], w, acc[e]);
  }
#pragma unroll
  for (int e = 0; e < CPL; ++e) sum[warp][lane * CPL + e] = acc[e];
  __syncthreads();
  l = 0.f;
#pragma unroll
  for (int w = 0; w < NW; ++w) l += red[1][w];
  if (threadIdx.x < D) {
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) x += sum[w][threadIdx.x];
    p.out[at * D + threadIdx.x] = __float2bfloat16_rn(x / l);
  }
  if (threadIdx.x == 0 && p.lse != nullptr) p.lse[at] = (mx + log2f(l)) * 0.69314718055994531f;
}

}  // namespace jl
