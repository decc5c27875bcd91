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
  float* ws;                   // o [heads of a block][2][n_cta][D], then (m, l) [heads][2][n_cta][2]
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
  int32_t tile, tile_log2;     // keys of a tile, a power of two
  float scale_log2;
};

// G of a length L >= 1.
__device__ __forceinline__ int q4_group(const DecodeQ4Params& p, int L) { return (L - 1) / p.w_pre + 1; }

// Tiles of an entry of length L (0 for an empty one, or for a length outside the contract,
// which the combine reports).
__device__ __forceinline__ int q4_tiles(const DecodeQ4Params& p, int L) {
  return L < 1 || L > p.max_seqlen ? 0 : ((L - 1) >> p.tile_log2) + 1;
}

// Tiles of all entries, and of the entries before b, by one warp; `first` is the tiles of
// entry `lane`.
__device__ __forceinline__ int2 q4_tiles_before(const DecodeQ4Params& p, int b, int lane, int& first) {
  first = lane < p.B ? q4_tiles(p, p.seqlens[lane]) : 0;
  int all = first, before = lane < b ? first : 0;
  for (int e = lane + 32; e < p.B; e += 32) {
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

// Tiles of a CTA's range: CTA c has tiles [c per, (c + 1) per) of the list.
__device__ __forceinline__ int q4_per_cta(const DecodeQ4Params& p, int total) {
  return (static_cast<unsigned>(total) + p.n_cta - 1) / static_cast<unsigned>(p.n_cta);
}

// Where a range starts: entry and tile inside it.
struct Q4Start {
  int hb, b, tile, len;  // head block, entry and its length, tile of the entry
  int begin, end;  // the range in the list of all tiles (the host keeps their number below 2^31)
};

// The place of tile `at` of the list, by one warp; `all`: the tiles of a head block, `t`: those of
// entry `lane`.
__device__ __forceinline__ void q4_place(const DecodeQ4Params& p, int lane, int at, int all, int t, Q4Start& s) {
  s.hb = at / all;
  int left = at % all;
  for (int e0 = 0; e0 < p.B; e0 += 32) {
    const int e = e0 + lane, len = e < p.B ? p.seqlens[e] : 0;
    if (e0 > 0) t = q4_tiles(p, len);
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
      s.len = __shfl_sync(0xffffffffu, len, src);
      return;
    }
    left -= __shfl_sync(0xffffffffu, sum, 31);
  }
}

__device__ __forceinline__ Q4Start q4_range(const DecodeQ4Params& p, int lane) {
  Q4Start s{};
  int t;
  const int all = q4_tiles_before(p, 0, lane, t).x;
  const int total = all * (p.Hkv / p.heads_per_block);
  const int per = q4_per_cta(p, total);
  s.begin = min(static_cast<int64_t>(total), static_cast<int64_t>(per) * blockIdx.x);
  s.end = s.begin + min(per, total - s.begin);
  if (s.begin < s.end) q4_place(p, lane, s.begin, all, t, s);
  return s;
}

// ------------------------------------------------------------- the decode kernel --
//
// What bounds it.  A row of 128 channels is 144 bytes: 128K keys of eight heads are 151 MB,
// 23.0 us at the measured 6.56 TB/s.  Beside that stand, for 16 keys of one head (8192 of
// those a head at 128K), 540 warp instructions in all to expand, weigh and sum 4096 codes and
// to rotate the keys, of which the ALU and the fp16 pipe take two cycles each.  Measured
// (graph-replayed, 32/8 heads of 128, cold caches): 64.1 us at 128K keys (G = 4), 2.4 TB/s,
// of which 55 us are per key and 9 for the start, the first loads and the join; without
// rotation (G = 1) 30 us are per key.  8K keys take 11.2 us.  With the instructions of the
// keys and values left out, the loads alone stream 128K keys in 21 us.  So the arithmetic
// bounds it, although no pipe is full: issue slots are 46 % used, the FMA pipe 43 %, the
// tensor pipe 16 %, DRAM 28 %.  Two warps a scheduler wait for their own results, for one
// another's pipes, and (0.5 of a warp at every issue) for instructions to be fetched.
//
// Shape.  Eight warps of a CTA take keys; one loads; three make the rotations' factors.  A
// tile is `tile` keys of all KV heads of a head block: U sixteens of keys of one head for
// each key warp.  It arrives by TMA as boxes of sixteen keys, in a ring of stages.  Two warps
// a scheduler with more sixteens a tile beat four of U = 1 with half the registers (51 against
// 61 us at 128K, when the rotation had one rounding to fp16): what a warp does once a tile
// costs as much as a third of its sixteen keys.  The values of one sixteen stand beside the
// scores of the next, independent of them and on other pipes: 4 % less than with the scores
// of all sixteens side by side, which keeps them apart.
//
// Matrix instructions: mma.m16n8k16 with the keys on M for the scores and the channels on M
// for the values.  A lane expands the codes of its own fragments in registers.  tcgen05 would
// need the expanded tile in shared memory: 2 bytes a code written and 2 read beside the code's
// own half, 37 us of shared-memory time for 128K keys of eight heads, where the codes take 23
// us to arrive; expanded in registers they cost none.
//
// Scores.  The codes less 8 are small integers, exact in fp16.  The query of each head is
// scaled by a power of two to a largest channel in [8, 16) and split into two fp16 numbers,
// columns 2h and 2h + 1 of B, which carry 22 of its bits (bf16 queries are exact, rotated
// ones off by 2^-22).  Local keys therefore score exactly up to the fp32 sums.  A remote
// key's pairs are first turned by R(f(j) - j).  cos and sin are split into a multiple of 2^-7
// and a remainder of at most 2^-8: the codes turned by the first are whole multiples of 2^-7
// below 2^4, exact in fp16, and turned by the second they are so small that their rounding to
// 11 bits is some 2^-19 of a code.  Both go through the matrix instruction against the same
// query.  A turned channel is off by 7.7e-5 of a code at the most, most of that from the fp32
// steps of cos and sin below (one key's score of tens: 3e-5 measured, 1/40 of that bound's
// sum over the channels); over many keys it averages out, and the lse is as good as with fp32
// scores.  With cos, sin and the turned key rounded to fp16 once, scores were off by 3e-4 of a
// key's part and the lse by 1.4e-6 of itself (5e-8 now, the fp32 sums'); the remainders cost
// 15 us of 61.5 at 128K keys when they came.  The group scales are applied to the fp32 sums of
// their group, between the matrix instructions.
//
// Weights are multiplied by the value scales of their key in fp32 and rounded to fp16 (2^-11 of
// each), three bits more than the bf16 of the cached values' scales and of the output: the output
// is off by 2.0e-4 of its size from it at every length, beside 1.67e-3 of its own rounding.  A second
// fp16 number for the rest would double the values' matrix instructions.  So that the products fit
// fp16 whatever the scales, each head and value group has a factor of its own, a power of two
// that keeps weight * scale * factor at or below 2^15, where it was 2^6 to 2^7 when it last
// moved: products down to 2^-20 of the group's largest keep 11 bits, and down to 2^-31 still
// count.  The softmax's reference M is the largest score when it last moved, or less than an
// octave above, and moves before a weight passes 2^8; a first key that has all the weight has
// a weight of 1 and gives its values exactly, ties of their rounding included.  The factors
// are taken off the sums at the end.  Sums and outputs are held in fp32.
//
// The rotations' cos and sin are the same for all heads, so three warps make them once a tile
// for the whole head block: from the table's row of a run's first key by steps of one position
// in fp32, split as above and stored as fp16 in the order of the fragments.

constexpr int kDecodeQ4Ctas = 148;  // one per SM
constexpr int kDecodeQ4KeyWarps = 8, kDecodeQ4TurnWarps = 3, kDecodeQ4OtherWarps = 1 + kDecodeQ4TurnWarps;  // one loads
constexpr int kDecodeQ4Threads = 32 * (kDecodeQ4KeyWarps + kDecodeQ4OtherWarps);
constexpr int kDecodeQ4MaxStages = 6;

// Test build of the time-outs: one of every CTA's cos/sin warps gives up at its tile of this number.
#ifdef JL_Q4_GIVE_UP
constexpr int kDecodeQ4GiveUp = JL_Q4_GIVE_UP;
#else
constexpr int kDecodeQ4GiveUp = -1;
#endif

// Registers a thread: 168 at launch; the key warps rise to 216, the others drop to 72.
constexpr int kDecodeQ4Regs = 168, kDecodeQ4KeyRegs = 216, kDecodeQ4OtherRegs = 72;
static_assert(kDecodeQ4KeyWarps * kDecodeQ4KeyRegs + kDecodeQ4OtherWarps * kDecodeQ4OtherRegs <=
                  (kDecodeQ4KeyWarps + kDecodeQ4OtherWarps) * kDecodeQ4Regs,
              "the split has to fit the launch's registers, or setmaxnreg waits for good");

// Shared memory: a region for the query fragments, reused to join the key warps, then the
// stages.  A stage: key codes, value codes, scales, cos/sin rows, the rows' remainders.
struct DecodeQ4Layout {
  int region, codes, scales, table, stage, stages, total;
};

// NQ: score tiles of four query heads; HPB: KV heads of a block.
__host__ __device__ constexpr DecodeQ4Layout decode_q4_layout(int D, int NQ, int HPB, int tile) {
  DecodeQ4Layout l{};
  const int frags = 2 * HPB * NQ * (D / 32) * 512, join = kDecodeQ4KeyWarps * NQ * 4 * (D + 8) * 4;
  l.region = ((frags > join ? frags : join) + 1023) / 1024 * 1024;
  l.codes = tile * HPB * D / 2;
  l.scales = tile * HPB * 16;
  l.table = 2 * tile * D * 2;
  l.stage = 2 * l.codes + l.scales + l.table;
  l.stages = (220 * 1024 - l.region) / l.stage;
  if (l.stages > kDecodeQ4MaxStages) l.stages = kDecodeQ4MaxStages;
  l.total = l.region + l.stages * l.stage + 1024;
  return l;
}

struct DecodeQ4Shared {
  uint64_t full[kDecodeQ4MaxStages];   // codes and scales have arrived, cos/sin rows are written
  uint64_t empty[kDecodeQ4MaxStages];  // all key warps are done with the stage; one that gave up frees none
  float mul[32];                       // log2 units per unit of score, by query head of the block
  float red_m[kDecodeQ4KeyWarps][16], red_l[kDecodeQ4KeyWarps][16];
  Q4Start start;
  int abort;
  int issued;  // tiles that the load warp asked for, once it will ask for no more; -1 before
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same with a zero accumulator.
__device__ __forceinline__ void mma_f16_zero(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
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
__device__ __forceinline__ uint32_t h2_of(uint64_t x) {
  float a, b;
  f2_unpack(x, a, b);
  return h2_bits(__floats2half2_rn(a, b));
}
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

// A pair of channels (two keys' or two pairs' of them) turned back by the angle of cos c and sin s.
__device__ __forceinline__ void turn_pair(__half2 a, __half2 b, uint32_t c, uint32_t s, uint32_t& x, uint32_t& y) {
  x = h2_bits(__hfma2(a, bits_h2(c), __hmul2(b, bits_h2(s))));
  y = h2_bits(__hfma2(b, bits_h2(c), __hneg2(__hmul2(a, bits_h2(s)))));
}

// The same for the value codes, the high four bits' in units of 1/16 (taken off at the end).
// The 8 goes off the operands although codes of 0 .. 15, as fp16 subnormals, would need no
// arithmetic and 8 times the sum of the weights could be taken off the sums (1 us less at 128K
// keys): the matrix instruction cuts every product and the sum towards zero, two bits and none
// below the last place of its largest operand.  Signed products are cut to either side, and the
// running sum is no larger than the result; sums of positive ones are all cut one way, by more
// the longer they grow.  The result was off by 4e-4 of itself at 886 keys a warp and by 7e-3 at
// 8192, where signed ones are off by what the weights' rounding gives at every length.
template <bool HIGH>
__device__ __forceinline__ uint32_t value_codes_f16(uint32_t w) {
  const uint32_t x = HIGH ? select_or(w, 0x00f000f0u, 0x64006400u) : select_or(w, 0x000f000fu, 0x64006400u);
  return h2_bits(__hsub2(bits_h2(x), __float2half2_rn(HIGH ? 1152.f : 1032.f)));
}

__device__ __forceinline__ void prefetch_l2(const void* x) { asm volatile("prefetch.global.L2 [%0];" ::"l"(x)); }

// Shared-memory loads by 32-bit address, in order with the barrier waits around them.
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ float bf16_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Row r of a warp's sixteen keys holds key q4_key_of(r).  Neighbouring rows differ in parity
// and in bit 2, rows 0, 2, 4, 6 (and 1, 3, 5, 7) in bits 1 and 2, so that the key, value,
// scale and cos/sin loads are all free of bank conflicts in the swizzled boxes.
__device__ __forceinline__ int q4_key_of(int r) { return r ^ ((r & 1) << 2); }

// A box holds sixteen keys in rows of neighbouring heads, 128 bytes where the block has that
// many, with the swizzle of that row length.  Bytes of a row of codes, and the offset of byte x
// of key `key`'s row of `width` bytes.
__host__ __device__ constexpr int q4_code_row(int D, int HPB) { return HPB * D / 2 < 128 ? HPB * D / 2 : 128; }
__device__ __forceinline__ int q4_at(int width, int key, int x) {
  const int turn = width == 128 ? key & 7 : width == 64 ? (key >> 1) & 3 : width == 32 ? (key >> 2) & 1 : 0;
  return key * width + (x ^ (turn << 4));
}

// Offset of 16-byte chunk (word w, lane t) of a key's cos/sin row.
template <int D>
__device__ __forceinline__ int q4_turn_at(int key, int w, int t) {
  return key * 2 * D + ((w * 64 + t * 16) ^ ((key & 1) << 6));  // neighbouring rows on different banks
}

// NQ: score tiles (of four query heads); U: sixteens of keys of a key warp in a tile.
template <int D, int NQ, int U>
__global__ void __launch_bounds__(kDecodeQ4Threads, 1)
    jl_decode_q4_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                        const __grid_constant__ CUtensorMap ts, const DecodeQ4Params p) {
  constexpr int HALF = D / 2;
  constexpr int KW = D / 32;    // 32-bit words of a lane's key codes (and fragments of four registers)
  constexpr int VW = D / 64;    // of its value codes
  constexpr int MT = D / 16;    // output tiles of 16 channels
  constexpr int NP = (NQ + 1) / 2;  // value tiles of eight columns
  constexpr int kF = NQ == 1 ? 2 : 4;  // weight fragments: pairs of scale groups, or groups
  constexpr bool kQueryRegs = NQ <= 2;  // query fragments stay in registers
  extern __shared__ uint8_t raw_smem[];
  __shared__ DecodeQ4Shared sh;
  uint8_t* smem = raw_smem + ((1024u - (smem_u32(raw_smem) & 1023u)) & 1023u);
  const int HPB = p.heads_per_block, T = p.tile;
  const DecodeQ4Layout lay = decode_q4_layout(D, NQ, HPB, T);
  uint8_t* const stages = smem + lay.region;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &sh.abort;

  if (threadIdx.x == 0) {
    for (int s = 0; s < lay.stages; ++s) {
      mbar_init(&sh.full[s], kDecodeQ4OtherWarps);
      mbar_init(&sh.empty[s], kDecodeQ4KeyWarps);
    }
    sh.abort = 0;
    sh.issued = -1;
    fence_mbar_init();
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
    tma_prefetch_desc(&ts);
  }
  griddep_wait();  // the cache, the lengths and the query may come from the previous kernel
  griddep_launch_dependents();
  if (warp == 0) {
    const bool failed = status_failed();
    Q4Start s = q4_range(p, lane);
    if (__any_sync(0xffffffffu, failed)) s.end = s.begin;
    if (lane == 0) sh.start = s;
  } else if (warp == 1) {
    // The first queries are asked for before the loads of the tiles, behind which they would
    // queue for some microseconds; a small batch has no others.
    const int64_t bytes = min(static_cast<int64_t>(p.B) * p.Hq * D * 2, static_cast<int64_t>(16384));
    for (int x = lane * 128; x < bytes; x += 32 * 128) prefetch_l2(reinterpret_cast<const char*>(p.q) + x);
  }
  __syncthreads();
  const Q4Start st = sh.start;
  int cur = st.begin;
  int hb = st.hb, b = st.b, t0 = st.tile, L = st.len;
  int stage = 0;
  uint32_t phase = 0;

  if (warp >= kDecodeQ4KeyWarps) {
    setmaxnreg_dec<kDecodeQ4OtherRegs>();
    bool ok = true;
    if (warp == kDecodeQ4KeyWarps) {
      // ---------------------------------------------------------------- loads --
      const int boxes = T / 16, rows = HPB * HALF / q4_code_row(D, HPB);  // of a tile; of codes, a key
      int issued = 0;
      while (cur < st.end && ok) {
        const int tiles = q4_tiles(p, L);
        const int t1 = min(tiles, t0 + (st.end - cur));
        int row = 0;  // lane x: the cache row of box x of the 32 asked for last
        for (int tile = t0; tile < t1; ++tile) {
          const int at = (tile - t0) * boxes % 32;
          if (at == 0) {
            const int j = tile * T + 16 * lane;
            row = static_cast<int>(b * p.cache_stride + j);
            if (p.block_table != nullptr) {
              // pages behind the length need no entry: their keys are never used
              const int page = j < L ? p.block_table[static_cast<int64_t>(b) * p.max_pages + j / p.page_size] : 0;
              const bool there = page >= 0 && page < p.num_pages;
              if (!there) atomicOr(&g_status, kDevErrBounds);
              row = (there ? page : p.num_pages) * p.page_size + (there ? j % p.page_size : 0);  // outside reads zeros
            }
            JL_CHECK(j >= L || p.block_table != nullptr ||
                     (j < p.cache_stride && row >= 0 && row < static_cast<int64_t>(p.B) * p.cache_stride));
            JL_CHECK(j >= L || p.block_table == nullptr || (j < p.max_pages * static_cast<int64_t>(p.page_size) && row >= 0 &&
                                                            row <= static_cast<int64_t>(p.num_pages) * p.page_size));
            JL_CHECK(b >= 0 && b < p.B && (hb + 1) * HPB <= p.Hkv);
          }
          if (!warp_wait(&sh.empty[stage], phase ^ 1, abort)) {
            ok = false;
            break;
          }
          uint8_t* base = stages + stage * lay.stage;
          if (lane == 0) mbar_arrive_expect_tx(&sh.full[stage], 2 * lay.codes + lay.scales);
          __syncwarp();
          if (lane >= at && lane < at + boxes) {
            const int x = lane - at;
            tma_load_3d(base + x * HPB * 16 * HALF, &tk, &sh.full[stage], 0, row, hb * rows);
            tma_load_3d(base + lay.codes + x * HPB * 16 * HALF, &tv, &sh.full[stage], 0, row, hb * rows);
            tma_load_3d(base + 2 * lay.codes + x * HPB * 256, &ts, &sh.full[stage], 0, row, hb);
          }
          ++issued;
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
        if (cur < st.end) L = p.seqlens[b];
      }
      // Drain: never leave the block with a copy still landing in its shared memory.  A stage is
      // loaded again only after all key warps saw its last load, so these tiles' copies are the only
      // ones in flight; `full` completes for each, as a cos/sin warp that gives up arrives for it too.
      if (lane == 0) {
        *static_cast<volatile int*>(&sh.issued) = issued;
        for (int x = max(0, issued - lay.stages); x < issued; ++x)
          mbar_wait_bounded(&sh.full[x % lay.stages], (x / lay.stages) & 1);
      }
      return;
    }
    // ------------------------------------------------------------ cos/sin rows --
    // Each warp makes a third of a tile's rows (half a warp a sixth, of 64 channels): from the
    // tables' row of its first key (row j - floor(j / G)), asked for a tile ahead, by one
    // position's step after the other in fp32 (at most 44 steps: an error of some 2^-18).
    // Eight keys at a time, each from a row of its own asked for eight keys ahead, took 27 us
    // for 128K keys, the rows' latency; one warp for all of a tile's rows took 43.
    const int tw = warp - kDecodeQ4KeyWarps - 1;
    // lane -> the two pairs of one packed register: word w, fragment lane t, register half e
    const int w = D == 128 ? lane / 8 : (lane & 15) / 8, t = (lane / 2) & 3, e = lane & 1;
    const int c0 = D == 128 ? 16 * w + 4 * t + e : 8 * (2 * w + e) + 2 * t, c1 = D == 128 ? c0 + 2 : c0 + 1;
    // one position's step of both pairs, packed; with a table of one row nothing is remote
    const int64_t one = p.n_tab_rows > 1 ? HALF : 0;
    const uint64_t step_c = f2_pack(p.cos_tab[one + c0], p.cos_tab[one + c1]);
    const uint64_t step_s = f2_pack(p.sin_tab[one + c0], p.sin_tab[one + c1]);
    const uint64_t step_n = f2_pack(-p.sin_tab[one + c0], -p.sin_tab[one + c1]);
    constexpr int kRuns = kDecodeQ4TurnWarps * 128 / D;  // runs of rows: half a warp does one of 64 channels
    const int run = D == 128 ? tw : 2 * tw + lane / 16;
    const int row0 = T / 4 * run / kRuns * 4, row1 = T / 4 * (run + 1) / kRuns * 4;
    const int rest = lay.table / 2;  // the remainders' rows, behind the others
    const uint64_t grid = f2_pack(98304.f, 98304.f);  // 1.5 * 2^16: a sum with it ends at 2^-7
    int made = 0;  // tiles that this warp arrived for, where it gave up
    while (cur < st.end && ok) {
      const int tiles = q4_tiles(p, L);
      const int t1 = min(tiles, t0 + (st.end - cur));
      const int grow = q4_group(p, L);
      const int jb = grow > 1 ? L - 1 - p.w0 : -1;  // remote keys are j <= jb
      const int far_tiles = jb < 0 ? 0 : min(t1, jb / T + 1);
      float2 next_c = make_float2(1.f, 1.f), next_s = make_float2(0.f, 0.f);
      int next_left = grow;
      auto ask = [&](int j) {
        const int quot = j / grow;
        next_left = grow - (j - quot * grow);  // keys until f steps; that key keeps the angle of the one before it
        const int64_t row = min(static_cast<int64_t>(j - quot), p.n_tab_rows - 1) * HALF;  // behind the length: none
        JL_CHECK(j >= 0 && quot >= 0 && quot <= j && (j >= L || j - quot < p.n_tab_rows));
        next_c = make_float2(p.cos_tab[row + c0], p.cos_tab[row + c1]);
        next_s = make_float2(p.sin_tab[row + c0], p.sin_tab[row + c1]);
      };
      if (t0 < far_tiles) ask(t0 * T + row0);
      for (int tile = t0; tile < t1; ++tile) {
        if (!warp_wait(&sh.empty[stage], phase ^ 1, abort) ||
            (kDecodeQ4GiveUp >= 0 && tw == 0 && cur - st.begin + tile - t0 == kDecodeQ4GiveUp)) {
          ok = false;
          made = cur - st.begin + tile - t0;
          break;
        }
        if (tile < far_tiles) {
          uint64_t ac = f2_pack(next_c.x, next_c.y), as = f2_pack(next_s.x, next_s.y);
          int left = next_left;
          if (tile + 1 < far_tiles) ask((tile + 1) * T + row0);
          // even and odd rows from two places, so that the offsets in the loop are constants
          uint8_t* const rows = stages + stage * lay.stage + 2 * lay.codes + lay.scales + row0 * 2 * D;
          uint8_t* even = rows + q4_turn_at<D>(0, w, t) + 8 * e;
          uint8_t* odd = rows + q4_turn_at<D>(1, w, t) + 8 * e - 2 * D;
          for (int r = row0; r < row1; r += 4) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint8_t* at = (x & 1 ? odd : even) + x * 2 * D;
              const uint64_t gc = f2_sub(f2_add(ac, grid), grid), gs = f2_sub(f2_add(as, grid), grid);
              *reinterpret_cast<uint2*>(at) = make_uint2(h2_of(gc), h2_of(gs));
              *reinterpret_cast<uint2*>(at + rest) = make_uint2(h2_of(f2_sub(ac, gc)), h2_of(f2_sub(as, gs)));
              // no branch, so that the next rows' steps fill the waits of this one's
              const uint64_t nc = f2_fma(ac, step_c, f2_mul(as, step_n)), ns = f2_fma(as, step_c, f2_mul(ac, step_s));
              const bool stay = --left == 0;
              ac = stay ? ac : nc;
              as = stay ? as : ns;
              left = stay ? grow : left;
            }
            even += 8 * D;
            odd += 8 * D;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.full[stage]);
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
      if (cur < st.end) L = p.seqlens[b];
    }
    if (!ok && lane == 0) {
      // Gave up: tiles that were asked for complete `full` all the same, for the load warp's drain.
      // That warp's waits end, its own limit or the abort flag being seen, within one limit.
      *abort = 1;
      atomicOr(&g_status, kDevErrTimeout);
      const volatile int* issued = &sh.issued;
      const long long since = clock64();
      while (*issued < 0 && clock64() - since < 2 * JL_WAIT_LIMIT_CYCLES) {
      }
      for (int x = made; x < *issued; ++x) mbar_arrive(&sh.full[x % lay.stages]);
    }
    return;
  }

  // ------------------------------------------------------------------ the keys --
  setmaxnreg_inc<kDecodeQ4KeyRegs>();
  const int g = lane >> 2, t = lane & 3;
  const int wph = kDecodeQ4KeyWarps / HPB;                          // warps that share a head
  const int wsub = warp % wph, head = warp / wph;      // this warp's place among them, its KV head in the block
  const int keyA = q4_key_of(g);                       // its score rows' keys of a sixteen: keyA, keyA + 8
  const int key0 = q4_key_of(2 * t), key1 = q4_key_of(2 * t + 1);  // its value fragments': these and 8 on
  const int width = q4_code_row(D, HPB), in_row = width / HALF;    // a row of codes and its heads
  const uint32_t eight = 8 * width, next_codes = HPB * 16 * HALF, next_scales = HPB * 256;  // eight keys, a box on
  // offsets in a stage
  const int box = wsub * U * HPB * 16 * HALF + head / in_row * 16 * width, x0 = head % in_row * HALF;
  const uint32_t at_key = box + q4_at(width, keyA, x0 + t * KW * 4);
  const uint32_t at_val0 = lay.codes + box + q4_at(width, key0, x0 + g * MT);
  const uint32_t at_val1 = lay.codes + box + q4_at(width, key1, x0 + g * MT);
  const uint32_t at_scale = 2 * lay.codes + wsub * U * HPB * 256 + q4_at(HPB * 16, keyA, head * 16);
  const uint32_t at_turn0 = 2 * lay.codes + lay.scales + q4_turn_at<D>(wsub * 16 * U + keyA, 0, t);  // words 0, 2
  const uint32_t at_turn1 = 2 * lay.codes + lay.scales + q4_turn_at<D>(wsub * 16 * U + keyA, 1, t);  // words 1, 3
  const uint32_t stages_at = smem_u32(stages);
  const uint32_t frags_at = smem_u32(smem) + head * NQ * KW * 512 + lane * 16;  // [2][HPB][NQ][KW][32] uint4
  const uint32_t far_frags = HPB * NQ * KW * 512;
  float* const join = reinterpret_cast<float*>(smem);  // [warps][4 NQ][D + 8]: the four heads of a tile on different banks
  bool ok = true;

  while (cur < st.end) {
    const int tiles = q4_tiles(p, L);
    const int t1 = min(tiles, t0 + (st.end - cur));
    if (t1 > t0) {
      const int i = L - 1, grow = q4_group(p, L);
      const int jb = grow > 1 ? i - p.w0 : -1;

      // Query fragments: this warp's query heads of the block, local and remote variant, each
      // split into two fp16 columns.  All loads come first.
      {
        constexpr int kRows = 32 / kDecodeQ4KeyWarps;  // HPB * NQ <= 8
        const int nq = i - i / grow;
        JL_CHECK(nq >= 0 && nq < p.n_tab_rows && b < p.B && (hb + 1) * HPB * p.group <= p.Hq);
        const bool has = D == 128 || lane < 16;
        const int w = D == 128 ? lane / 8 : (lane & 15) / 8, ft = D == 128 ? (lane / 2) & 3 : lane & 3;
        const int e = D == 128 ? lane & 1 : (lane >> 2) & 1;
        const int c0 = D == 128 ? 16 * w + 4 * ft + e : 8 * (2 * w + e) + 2 * ft, c1 = D == 128 ? c0 + 2 : c0 + 1;
        float y[kRows][4];  // channels c0, c1, c0 + D/2, c1 + D/2
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          const int x = warp + u * kDecodeQ4KeyWarps, h = x / (4 * NQ), qh = x % (4 * NQ);  // KV head, query head of its group
#pragma unroll
          for (int n = 0; n < 4; ++n) y[u][n] = 0.f;
          if (h < HPB && qh < p.group && has) {
            const __nv_bfloat16* qp = p.q + (static_cast<int64_t>(b) * p.Hq + (hb * HPB + h) * p.group + qh) * D;
            y[u][0] = __bfloat162float(qp[c0]), y[u][1] = __bfloat162float(qp[c1]);
            y[u][2] = __bfloat162float(qp[c0 + HALF]), y[u][3] = __bfloat162float(qp[c1 + HALF]);
          }
        }
        float cs[2], sn[2];
        cs[0] = p.cos_tab[static_cast<int64_t>(nq) * HALF + c0], cs[1] = p.cos_tab[static_cast<int64_t>(nq) * HALF + c1];
        sn[0] = p.sin_tab[static_cast<int64_t>(nq) * HALF + c0], sn[1] = p.sin_tab[static_cast<int64_t>(nq) * HALF + c1];
        float top[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u)
          top[u] = fmaxf(fmaxf(fabsf(y[u][0]), fabsf(y[u][1])), fmaxf(fabsf(y[u][2]), fabsf(y[u][3])));
#pragma unroll
        for (int o = 16; o; o >>= 1)
#pragma unroll
          for (int u = 0; u < kRows; ++u) top[u] = fmaxf(top[u], __shfl_xor_sync(0xffffffffu, top[u], o));
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          const int x = warp + u * kDecodeQ4KeyWarps, h = x / (4 * NQ), qh = x % (4 * NQ);
          // 2^up brings the largest channel into [8, 16); up in [-120, 120] keeps both factors normal
          const int up = min(120, max(-120, 130 - static_cast<int>(__float_as_uint(top[u]) >> 23)));
          const float f = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
          if (lane == 0 && h < HPB) sh.mul[x] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
          if (has && h < HPB) {
#pragma unroll
            for (int var = 0; var < 2; ++var) {
              uint32_t* at = reinterpret_cast<uint32_t*>(smem) + (((var * HPB + h) * NQ + qh / 4) * KW + w) * 128;
              const int col = 2 * (qh & 3);
#pragma unroll
              for (int n = 0; n < 2; ++n) {  // low channels, high channels
                float v[2];
#pragma unroll
                for (int z = 0; z < 2; ++z)
                  v[z] = (var == 0 ? y[u][2 * n + z] : n == 0 ? y[u][z] * cs[z] + y[u][2 + z] * sn[z]
                                                              : y[u][2 + z] * cs[z] - y[u][z] * sn[z]) * f;
                const __half2 big = __floats2half2_rn(v[0], v[1]);
                const float2 bf = __half22float2(big);
                const __half2 small = __floats2half2_rn(v[0] - bf.x, v[1] - bf.y);
                const int reg = D == 128 ? 2 * n + e : 2 * e + n;
                at[(col * 4 + ft) * 4 + reg] = h2_bits(big);
                at[((col + 1) * 4 + ft) * 4 + reg] = h2_bits(small);
              }
            }
          }
        }
      }
      key_warps_sync();

      float o[NP][MT][4], m[NQ], l[NQ], mul[NQ];
      // Factors of the value groups (two fp32 each), powers of two from 2^-119 to 2^119, and the
      // largest of this lane's heads.
      uint64_t fac[NQ][2], fac_max[2] = {f2_pack(0x1p119f, 0x1p119f), f2_pack(0x1p119f, 0x1p119f)};
      uint4 qf[kQueryRegs ? NQ * KW : 1];
      int have = -1;  // the variant that qf holds
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        m[n] = -INFINITY;
        l[n] = 0.f;
#pragma unroll
        for (int f = 0; f < 2; ++f) fac[n][f] = f2_pack(0x1p119f, 0x1p119f);
        mul[n] = sh.mul[head * 4 * NQ + 4 * n + t];
      }
#pragma unroll
      for (int n = 0; n < NP; ++n)
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
          for (int x = 0; x < MT; ++x) o[n][x][y] = 0.f;

      uint32_t base = 0;         // the stage's address
      int j = 0;                 // first key of the sixteen at hand
      uint32_t pf[NP][kF][2];    // weight fragments of the sixteen before it

      // Scores of sixteen keys under one variant of the query (and, far, of the keys); rows g and
      // g + 8, head 4 n + t.
      auto scores = [&](auto far_tag, int u, float (&dst)[NQ][2]) {
        constexpr bool FAR = decltype(far_tag)::value;
        const uint32_t fa = frags_at + (FAR ? far_frags : 0u);
        if constexpr (kQueryRegs) {
          if (have != FAR) {
            have = FAR;
#pragma unroll
            for (int x = 0; x < NQ * KW; ++x) qf[x] = lds128(fa + x * 512);
          }
        }
        uint32_t kc[2][KW];
        uint2 ks[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t at = base + at_key + u * next_codes + r * eight;
          if constexpr (D == 128) {
            const uint4 v = lds128(at);
            kc[r][0] = v.x, kc[r][1] = v.y, kc[r][2] = v.z, kc[r][3] = v.w;
          } else {
            const uint2 v = lds64(at);
            kc[r][0] = v.x, kc[r][1] = v.y;
          }
          ks[r] = lds64(base + at_scale + u * next_scales + r * 128 * HPB);
        }
        const uint32_t turn0 = base + at_turn0 + u * 32 * D, turn1 = base + at_turn1 + u * 32 * D;
#pragma unroll
        for (int n = 0; n < NQ; ++n) dst[n][0] = dst[n][1] = 0.f;
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          uint32_t lo[2][2], hi[2][2];    // [row][register half]
          uint32_t rlo[2][2], rhi[2][2];  // far: what the remainders of cos and sin add
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            uint4 turn, rest;
            if constexpr (FAR) {
              const uint32_t at = (w & 1 ? turn1 : turn0) + (w >> 1) * 128 + r * 16 * D;
              turn = lds128(at);
              rest = lds128(at + lay.table / 2);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t word = e ? kc[r][w] >> 8 : kc[r][w];
              const __half2 a = codes_f16<false>(word), bb = codes_f16<true>(word);
              if constexpr (FAR) {  // R(-n)
                turn_pair(a, bb, e ? turn.z : turn.x, e ? turn.w : turn.y, lo[r][e], hi[r][e]);
                turn_pair(a, bb, e ? rest.z : rest.x, e ? rest.w : rest.y, rlo[r][e], rhi[r][e]);
              } else {
                lo[r][e] = h2_bits(a);
                hi[r][e] = h2_bits(bb);
              }
            }
          }
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            uint4 q;
            if constexpr (kQueryRegs) q = qf[n * KW + w];
            else q = lds128(fa + (n * KW + w) * 512);
            if constexpr (D == 128) {  // a word is one group: two steps, low channels then high
              float c[4];
              mma_f16_zero(c, {lo[0][0], lo[1][0], lo[0][1], lo[1][1]}, q.x, q.y);
              mma_f16(c, {hi[0][0], hi[1][0], hi[0][1], hi[1][1]}, q.z, q.w);
              if constexpr (FAR) {
                mma_f16(c, {rlo[0][0], rlo[1][0], rlo[0][1], rlo[1][1]}, q.x, q.y);
                mma_f16(c, {rhi[0][0], rhi[1][0], rhi[0][1], rhi[1][1]}, q.z, q.w);
              }
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const uint32_t sc = w < 2 ? ks[r].x : ks[r].y;
                dst[n][r] = fmaf(w & 1 ? bf16_high(sc) : bf16_low(sc), c[2 * r] + c[2 * r + 1], dst[n][r]);
              }
            } else {  // two groups, a step each
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float c[4];
                mma_f16_zero(c, {lo[0][e], lo[1][e], hi[0][e], hi[1][e]}, e ? q.z : q.x, e ? q.w : q.y);
                if constexpr (FAR)
                  mma_f16(c, {rlo[0][e], rlo[1][e], rhi[0][e], rhi[1][e]}, e ? q.z : q.x, e ? q.w : q.y);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                  const uint32_t sc = w == 0 ? ks[r].x : ks[r].y;
                  dst[n][r] = fmaf(e ? bf16_high(sc) : bf16_low(sc), c[2 * r] + c[2 * r + 1], dst[n][r]);
                }
              }
            }
          }
        }
      };

      // Weights of sixteen keys and their products with the value scales.  M and the factors move
      // when a weight passes 2^8 or a product 2^15 (in the first keys: by anything), then those of
      // all heads, each with eight octaves to spare: with only the ones that had to, or four
      // octaves, they moved so often that groups of five and more heads took 10 to 20 % longer.
      auto weights = [&](int u, float (&s)[NQ][2], auto tail_tag) {
        constexpr bool TAIL = decltype(tail_tag)::value;
        uint2 vs[2];
        uint64_t vf[2][2];  // two fp32 each
        float wt[NQ][2];
        bool over = false;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          vs[r] = lds64(base + at_scale + u * next_scales + r * 128 * HPB + 8);
          if (TAIL && j + keyA + 8 * r >= L) {  // behind the length: weight 0, and no NaN scale that it could meet
            vs[r] = make_uint2(0u, 0u);
#pragma unroll
            for (int n = 0; n < NQ; ++n) s[n][r] = -INFINITY;
          }
          vf[r][0] = f2_pack(bf16_low(vs[r].x), bf16_high(vs[r].x));
          vf[r][1] = f2_pack(bf16_low(vs[r].y), bf16_high(vs[r].y));
          // what a weight is multiplied by at the most, known before the scores are
          float x[4];
          f2_unpack(f2_mul(vf[r][0], fac_max[0]), x[0], x[1]);
          f2_unpack(f2_mul(vf[r][1], fac_max[1]), x[2], x[3]);
          const float top = fmax3(fmax3(x[0], x[1], x[2]), x[3], 0x1p7f);
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            wt[n][r] = ex2_approx(__fmul_rn(s[n][r], mul[n]) - m[n]);  // 1 where the score is M
            over |= wt[n][r] * top > 0x1p15f;
          }
        }
        if (__any_sync(0xffffffffu, over)) {
          float by[NQ][4], most[4] = {};
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            float top[5];  // of the scores and the groups' scales, and of the scores
            top[4] = fmaxf(__fmul_rn(s[n][0], mul[n]), __fmul_rn(s[n][1], mul[n]));
#pragma unroll
            for (int f = 0; f < 4; ++f) {
              float v[2], w[2];
              f2_unpack(vf[0][f / 2], v[0], v[1]);
              f2_unpack(vf[1][f / 2], w[0], w[1]);
              top[f] = fmaxf(fmaf(s[n][0], mul[n], __log2f(v[f & 1])), fmaf(s[n][1], mul[n], __log2f(w[f & 1])));
            }
#pragma unroll
            for (int x = 4; x < 32; x <<= 1)
#pragma unroll
              for (int f = 0; f < 5; ++f) top[f] = fmaxf(top[f], __shfl_xor_sync(0xffffffffu, top[f], x));
            // M rises by whole octaves, so that the factors can follow exactly; where little of what
            // was before is left (and at first) to the score itself
            const float rise = top[4] - m[n];
            const float now = rise > 24.f ? top[4] : m[n] + ceilf(fmaxf(rise, 0.f));
            const bool first = m[n] == -INFINITY;
            l[n] *= first ? 0.f : ex2_approx(m[n] - now);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float fc[2];
              f2_unpack(fac[n][h], fc[0], fc[1]);
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                const int f = 2 * h + z;
                // log2 of the weight * scale, before M, whose product is 1: as it was, and from now on
                const float was = first ? -INFINITY : m[n] - (static_cast<int>(__float_as_uint(fc[z]) >> 23) - 127);
                const float to = fmaxf(was, top[f] - 7.f);
                const float up = floorf(fminf(119.f, fmaxf(-119.f, now - to)) + 0.0625f);  // M's own rounding
                by[n][f] = first ? 0.f : ex2_approx(was - now + up);
                fc[z] = __uint_as_float(static_cast<uint32_t>(127 + static_cast<int>(up)) << 23);
                most[f] = fmaxf(most[f], fc[z]);
              }
              fac[n][h] = f2_pack(fc[0], fc[1]);
            }
            m[n] = now;
#pragma unroll
            for (int r = 0; r < 2; ++r) wt[n][r] = ex2_approx(__fmul_rn(s[n][r], mul[n]) - now);
          }
          fac_max[0] = f2_pack(most[0], most[1]);
          fac_max[1] = f2_pack(most[2], most[3]);
#pragma unroll
          for (int n = 0; n < NP; ++n)
#pragma unroll
            for (int x = 0; x < MT; ++x)
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const int z = y & 1, f = x * 4 / MT;
                if constexpr (NQ == 1) o[n][x][y] *= by[0][(f & 2) + z];
                else o[n][x][y] *= by[2 * n + z][f];
              }
        }
        // Column 2t of the weights is head t of score tile 2n, column 2t + 1 of tile 2n + 1; with
        // one score tile both are head t, the even columns under the scales of the even groups
        // and the odd ones under those of the odd groups.
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float x[NQ][4];
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            l[n] += wt[n][r];
            const uint64_t w2 = f2_pack(wt[n][r], wt[n][r]);
#pragma unroll
            for (int h = 0; h < 2; ++h)  // the factor first: 2^8 * 2^119 at the most, so that is finite
              f2_unpack(f2_mul(f2_mul(w2, fac[n][h]), vf[r][h]), x[n][2 * h], x[n][2 * h + 1]);
          }
#pragma unroll
          for (int n = 0; n < NP; ++n)
#pragma unroll
            for (int f = 0; f < kF; ++f) {
              if constexpr (NQ == 1) pf[n][f][r] = transpose_8x8(h2_bits(__floats2half2_rn(x[0][2 * f], x[0][2 * f + 1])));
              else pf[n][f][r] = transpose_8x8(h2_bits(__floats2half2_rn(x[2 * n][f], x[2 * n + 1][f])));
            }
        }
      };

      auto values = [&](int u) {
        uint32_t vc[4][VW];  // value codes of keys key0, key1, key0 + 8, key1 + 8
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t at = base + (r & 1 ? at_val1 : at_val0) + u * next_codes + (r >> 1) * eight;
          if constexpr (D == 128) {
            const uint2 v = lds64(at);
            vc[r][0] = v.x, vc[r][1] = v.y;
          } else {
            vc[r][0] = lds32(at);
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
              const int x = 4 * w + 2 * y + z, f = NQ == 1 ? x * 2 / MT : x * 4 / MT;
              const uint32_t az = a >> (8 * z), bz = bb >> (8 * z);
              const uint32_t frag[4] = {value_codes_f16<false>(az), value_codes_f16<true>(az), value_codes_f16<false>(bz),
                                        value_codes_f16<true>(bz)};
#pragma unroll
              for (int n = 0; n < NP; ++n) mma_f16(o[n][x], frag, pf[n][f][0], pf[n][f][1]);
            }
          }
      };

      // A tile that is all local or all remote: the values of one sixteen beside the scores of the
      // next, whose instructions keep different pipes busy.
      auto whole_tile = [&](auto far_tag) {
#pragma unroll
        for (int u = 0; u <= U; ++u) {
          float s[NQ][2];
          if (u < U) scores(far_tag, u, s);
          if (u > 0) values(u - 1);
          if (u < U) weights(u, s, std::false_type{});
        }
      };

      for (int tile = t0; tile < t1; ++tile) {
        j = tile * T + wsub * 16 * U;
        if (ok) ok = warp_wait(&sh.full[stage], phase, abort);
        base = stages_at + stage * lay.stage;
        JL_CHECK(tile < tiles && j >= 0 && L <= p.max_seqlen && head < HPB && hb * HPB + head < p.Hkv);
        if (!ok) {
        } else if (j + 16 * U <= L && j > jb) {
          whole_tile(std::false_type{});
        } else if (j + 16 * U <= L && j + 16 * U - 1 <= jb) {
          whole_tile(std::true_type{});
        } else {  // the window's edge or the entry's end
#pragma unroll 1
          for (int u = 0; u < U && j < L; ++u, j += 16) {
            float s[NQ][2] = {}, near[NQ][2];
            if (j <= jb) scores(std::true_type{}, u, s);
            if (j + 15 > jb) {
              scores(std::false_type{}, u, near);
#pragma unroll
              for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) s[n][r] = j + keyA + 8 * r <= jb ? s[n][r] : near[n][r];
            }
            weights(u, s, std::true_type{});
            values(u);
          }
        }
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(&sh.empty[stage]);
        if (++stage == lay.stages) {
          stage = 0;
          phase ^= 1;
        }
      }

      // Join the warps that share a head, and write the result or the partial.
      float unit[NQ][4];  // of the groups' sums
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          f2_unpack(fac[n][h], unit[n][2 * h], unit[n][2 * h + 1]);
          unit[n][2 * h] = 1.f / unit[n][2 * h];
          unit[n][2 * h + 1] = 1.f / unit[n][2 * h + 1];
        }
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[n] += __shfl_xor_sync(0xffffffffu, l[n], x);
      const bool whole = t0 == 0 && t1 == tiles;
      const int hpb = HPB * p.group;
      const int slot0 = (cur == st.begin ? 0 : p.n_cta) + blockIdx.x;  // query head q's partial: slot0 + 2 q n_cta
      float* ml = p.ws + static_cast<int64_t>(p.n_cta) * 2 * hpb * D;
      // two partials a CTA and head of a block, the first or the last segment of its range
      JL_CHECK(whole || (slot0 + 2 * (hpb - 1) * p.n_cta < 2 * hpb * p.n_cta && hpb <= p.Hq &&
                         (cur == st.begin || cur + t1 - t0 == st.end)));
      if (wph == 1) {  // this warp has all of its head: straight from its registers
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          if (4 * n + t >= p.group) continue;
          const int q = head * p.group + 4 * n + t;
          const int64_t at = static_cast<int64_t>(b) * p.Hq + hb * hpb + q;
          const int slot = slot0 + 2 * q * p.n_cta;
          const float inv = 1.f / l[n];
#pragma unroll
          for (int x = 0; x < MT; ++x) {
            const int f = x * 4 / MT, y = NQ == 1 ? f & 1 : n & 1;
            const float lo = o[n / 2][x][y] * unit[n][f], hi = o[n / 2][x][2 + y] * (0.0625f * unit[n][f]);
            if (whole) {
              p.out[at * D + 16 * x + g] = __float2bfloat16_rn(lo * inv);
              p.out[at * D + 16 * x + 8 + g] = __float2bfloat16_rn(hi * inv);
            } else {
              p.ws[static_cast<int64_t>(slot) * D + 16 * x + g] = lo;
              p.ws[static_cast<int64_t>(slot) * D + 16 * x + 8 + g] = hi;
            }
          }
          if (g == 0) {
            if (!whole) *reinterpret_cast<float2*>(ml + slot * 2) = make_float2(m[n], l[n]);
            else if (p.lse != nullptr) p.lse[at] = (m[n] + log2f(l[n])) * 0.69314718055994531f;
          }
        }
      } else {
      key_warps_sync();  // every warp is done with the query fragments
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        if (g == 0) {
          sh.red_m[warp][4 * n + t] = m[n];
          sh.red_l[warp][4 * n + t] = l[n];
        }
        float* row = join + (warp * 4 * NQ + 4 * n + t) * (D + 8) + g;
#pragma unroll
        for (int x = 0; x < MT; ++x) {
          const int f = x * 4 / MT, y = NQ == 1 ? f & 1 : n & 1;  // the column that holds this head under this group's scales
          row[16 * x] = o[n / 2][x][y] * unit[n][f];
          row[16 * x + 8] = o[n / 2][x][2 + y] * (0.0625f * unit[n][f]);
        }
      }
      key_warps_sync();
      for (int x = threadIdx.x; x < hpb * (D / 4); x += 32 * kDecodeQ4KeyWarps) {
        const int q = x / (D / 4), c = x % (D / 4) * 4;  // query head of the block, its channels c .. c + 3
        const int in = q % p.group, w0 = q / p.group * wph;
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
          const float4 v = *reinterpret_cast<const float4*>(join + ((w0 + w) * 4 * NQ + in) * (D + 8) + c);
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
          const int slot = slot0 + 2 * q * p.n_cta;
          *reinterpret_cast<float4*>(p.ws + static_cast<int64_t>(slot) * D + c) = acc;
          if (c == 0) *reinterpret_cast<float2*>(ml + slot * 2) = make_float2(mx, lsum);
        }
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
    if (cur < st.end) L = p.seqlens[b];
  }
}

constexpr int kCombineQ4Threads = 256;

// Joins the partials of one (entry, query head), which lie in the ranges of CTAs c0 .. c1;
// writes zeros and -inf for an empty entry, NaN for a length outside the contract (reported
// by jl_sync_status) or a kernel that gave up.  SPLIT blocks share a head, each a part of its
// channels: with few heads to join, one block a head left 32 SMs to fetch 77 KB each (3.2 us
// against 0.9).  Every warp asks at once for the maxima and sums of all partials, which it
// needs for its weights, and for its channels of the first ones: one round trip and one
// barrier for up to 148 partials.
//
// RANGES false: blockIdx.y is an entry, blockIdx.z its head block; every warp adds up the tiles of
// the entries before it.  Of a large batch that is quadratic, and only the entries that two ranges
// share, one for each CTA at the most, have something to join.  RANGES true: blockIdx.y is the
// CTA in whose range such an entry begins, found by one warp; the entries that have no keys are
// shared out over the same blocks.
template <int D, int SPLIT, bool RANGES>
__global__ void __launch_bounds__(kCombineQ4Threads) jl_decode_q4_combine_kernel(const DecodeQ4Params p) {
  constexpr int NW = kCombineQ4Threads / 32, CH = D / SPLIT, LANES = CH / 4;  // a float4 a lane
  constexpr int ROWS = kCombineQ4Threads / LANES, PER = 5;                    // partials at a time, and rounds in flight
  constexpr int OWN = (kDecodeQ4Ctas + 31) / 32;
  __shared__ float weight[NW][32 * OWN];
  __shared__ __align__(16) float sum[NW][CH];
  const int hpb = p.heads_per_block * p.group, q = blockIdx.x / SPLIT;  // head of its block
  const int ch = blockIdx.x % SPLIT * CH + threadIdx.x % LANES * 4, row = threadIdx.x / LANES;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_launch_dependents();
  // The decode lets this kernel start only after it waited for everything before it, so the
  // lengths are there; its own partials and the status word are there after the wait.
  int b, hb, c0, s0, count;  // the entry and its head block, its first CTA and that one's slot, its CTAs
  bool wrong = false, none = false;
  if constexpr (!RANGES) {
    b = blockIdx.y;
    hb = blockIdx.z;
    const int L = p.seqlens[b], t = q4_tiles(p, L);
    int unused;
    const int2 n = q4_tiles_before(p, b, lane, unused);
    const unsigned per = max(1, q4_per_cta(p, n.x * (p.Hkv / p.heads_per_block))), first = hb * n.x + n.y;
    c0 = first / per;
    const int c1 = t ? (first + t - 1) / per : c0;
    s0 = c0 * per == first ? 0 : 1;
    count = c1 > c0 ? c1 - c0 + 1 : 0;  // 0: the decode wrote the result, or there is none
    wrong = L < 0 || L > p.max_seqlen;
    none = t == 0;
  } else {
    __shared__ int found[5];
    if (warp == 0) {
      Q4Start s{};
      int t, joined = 0, slot0 = 0;
      const int all = q4_tiles_before(p, 0, lane, t).x, total = all * (p.Hkv / p.heads_per_block);
      const int64_t per = q4_per_cta(p, total), begin = per * blockIdx.y, next = begin + per;
      if (next < total) {
        q4_place(p, lane, static_cast<int>(next), all, t, s);
        const int64_t first = next - s.tile;  // of the entry that has the next range's first tile
        if (s.tile > 0 && first >= begin) {
          joined = static_cast<int>((first + q4_tiles(p, s.len) - 1) / per) - static_cast<int>(blockIdx.y) + 1;
          slot0 = first == begin ? 0 : 1;
        }
      }
      if (lane == 0) found[0] = s.b, found[1] = s.hb, found[2] = blockIdx.y, found[3] = slot0, found[4] = joined;
    }
    __syncthreads();
    b = found[0], hb = found[1], c0 = found[2], s0 = found[3], count = found[4];
  }
  // the partials of a head lie side by side: by CTA, first those of segments that begin a range
  auto slot = [&](int c) { return (2 * q + (c == 0 ? s0 : 0)) * p.n_cta + c0 + c; };
  const float* ml = p.ws + static_cast<int64_t>(p.n_cta) * 2 * hpb * D;
  JL_CHECK(count == 0 || (c0 >= 0 && c0 + count <= p.n_cta && count <= 32 * OWN && b < p.B && (hb + 1) * hpb <= p.Hq));
  JL_CHECK(count == 0 || slot(count - 1) < 2 * hpb * p.n_cta);
  // zeros and -inf, or NaN, for head q of head block `of` of entry e
  auto write_none = [&](int e, int of, bool nan, bool report) {
    const float x = nan ? __int_as_float(0x7fc00000) : 0.f;
    const int64_t to = static_cast<int64_t>(e) * p.Hq + of * hpb + q;
    if (row == 0) *reinterpret_cast<uint2*>(p.out + to * D + ch) = make_uint2(pack_bf16x2(x, x), pack_bf16x2(x, x));
    if (threadIdx.x == 0 && blockIdx.x % SPLIT == 0) {
      if (p.lse != nullptr) p.lse[to] = nan ? x : -INFINITY;
      if (report && q == 0) atomicOr(&g_status, kDevErrBounds);
    }
  };
  griddep_wait();
  bool failed = false;
  if constexpr (RANGES) {
    failed = status_failed();
    for (int e = blockIdx.y; e < p.B; e += gridDim.y) {
      const int L = p.seqlens[e];
      const bool outside = L < 0 || L > p.max_seqlen;
      if (failed || outside || L == 0)
        for (int of = 0; of < p.Hkv / p.heads_per_block; ++of) write_none(e, of, failed || outside, outside);
    }
    if (failed) return;
  }
  float2 own[OWN];  // maxima and sums, lane + 32 x
#pragma unroll
  for (int x = 0; x < OWN; ++x)
    own[x] = lane + 32 * x < count ? *reinterpret_cast<const float2*>(ml + slot(lane + 32 * x) * 2)
                                   : make_float2(-INFINITY, 0.f);
  float4 o[PER];
  auto ask = [&](int c) {
#pragma unroll
    for (int u = 0; u < PER; ++u)
      if (c + u * ROWS < count) o[u] = *reinterpret_cast<const float4*>(p.ws + static_cast<int64_t>(slot(c + u * ROWS)) * D + ch);
  };
  ask(row);
  const int64_t at = static_cast<int64_t>(b) * p.Hq + hb * hpb + q;
  if constexpr (!RANGES) {
    failed = status_failed();  // after the loads above are asked for: 0.7 us less
    if (failed || none) {  // the same for all threads: nothing sets the status word meanwhile but this
      write_none(b, hb, failed || wrong, wrong);
      return;
    }
  }
  if (count == 0) return;
  float mx = own[0].x;
#pragma unroll
  for (int x = 1; x < OWN; ++x) mx = fmaxf(mx, own[x].x);
#pragma unroll
  for (int x = 16; x; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
  float l = 0.f;
#pragma unroll
  for (int x = 0; x < OWN; ++x) {
    if (32 * x >= count) break;
    const float f = own[x].x == -INFINITY ? 1.f : ex2_approx(own[x].x - mx);  // -inf: l is 0, or the NaN of NaN scores
    weight[warp][lane + 32 * x] = f;
    l = fmaf(own[x].y, f, l);
  }
#pragma unroll
  for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
  __syncwarp();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = row; c < count; c += PER * ROWS) {
    if (c != row) ask(c);
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      if (c + u * ROWS >= count) break;
      const float w = weight[warp][c + u * ROWS];
      acc.x = fmaf(o[u].x, w, acc.x), acc.y = fmaf(o[u].y, w, acc.y);
      acc.z = fmaf(o[u].z, w, acc.z), acc.w = fmaf(o[u].w, w, acc.w);
    }
  }
#pragma unroll
  for (int x = LANES; x < 32; x <<= 1) {  // the warp's rows
    acc.x += __shfl_xor_sync(0xffffffffu, acc.x, x), acc.y += __shfl_xor_sync(0xffffffffu, acc.y, x);
    acc.z += __shfl_xor_sync(0xffffffffu, acc.z, x), acc.w += __shfl_xor_sync(0xffffffffu, acc.w, x);
  }
  if (lane < LANES) *reinterpret_cast<float4*>(&sum[warp][lane * 4]) = acc;
  __syncthreads();
  if (threadIdx.x < CH) {
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) x += sum[w][threadIdx.x];
    p.out[at * D + blockIdx.x % SPLIT * CH + threadIdx.x] = __float2bfloat16_rn(x / l);
  }
  if (threadIdx.x == 0 && blockIdx.x % SPLIT == 0 && p.lse != nullptr)
    p.lse[at] = (mx + log2f(l)) * 0.69314718055994531f;
}

}  // namespace jl
