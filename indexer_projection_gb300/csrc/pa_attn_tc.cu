// The attention of pre_attn_attention_ext on tcgen05, for items of several rows
// (use_attn_tc) that are dealt in slices or a CTA each (pa_attn.cuh; small
// calls go to clusters of pa_attn_kernel): the (row, head)s of an item are the 128
// rows of S = Q K^T and of O = P V (f16 operands, f32 in tensor memory), so a
// block's codes are converted to f16 once for all of them, and a softmax
// thread has one (row, head) to itself.  (pa_attn_kernel converts them again
// for each row.)
//
// Warps: two groups of four do the softmax, a (row, head) a thread, of the
// even and the odd entries of the ring, each with an O of its own; four
// convert keys (and lay out the queries), four values; one thread issues the
// MMAs, one resolves the blocks, one asks for them.  S(n) is issued ahead of
// O += P V of entry n - 1, so one group's exponentials run beside the tensor
// core's work for the other.  P replaces S in tensor memory, as the A operand
// of the second product.
//
// What bounds it (FP8, 128 items of 7 rows x 16 heads and 18 blocks, 62 us, 1.2
// TB/s): instructions and their fetch.  A block takes 10900 warp instructions,
// some 6400 of them the softmax's (1600 a warp, of 32 (row, head)s x 128 keys),
// at about 0.57 a clock and scheduler: 2.4 us (NVFP4 1.5).  In front are 5 us to the
// first keys and some 6 to the first products, behind 6 to the last store.
// Longer code is slower even where it has fewer instructions to run (the roles'
// loops share the schedulers' instruction caches): turns of 64 keys 64.5,
// the NVFP4 conversions unrolled 120 for 114 (64 x 7 rows on every block); turns
// of 16 keys pay their latencies more often (68).  Right and no faster, too: one
// pass over the scores with the references looked at turn by turn (65 when this
// took 65); 16 softmax warps of 16 (row, head)s, a quarter of the keys a lane
// (74: 30% more instructions); 16 converting warps (77: no registers left for
// them); all eight converters on keys, then on values (70).
//
// Arithmetic as in pa_attn.cu (references, lift, unit of the products), the
// state of a (row, head) in one thread's registers: no exchange but at the
// segment's end, where the two groups' parts are added up.
//
// Order.  A segment (an item's part of a slice) is its blocks' entries of the
// ring, then one without a block for each softmax group; it may have no block at
// all (a request without keys).  A wait names a phase of an mbarrier by its
// parity alone, so whoever completes a phase first waits for evidence that all
// readers are past the one before: the products' thread for `meet` of the
// segment before, the queries' and the values' warps for item_seen.  (The 62 us,
// and 30 for one long request's rows in slices, are the same with and without.)
//
// Keys that a row does not see have no weight, but the tile of values is all
// rows': keys that no row sees are written as zeros, and where not every row
// sees every key, a NaN value is written as zero and the rows that see it are
// noted for its dim: they get NaN there.
#include <atomic>
#include <cstdint>

#include "../../include/pre_attn.h"
#include "pa_attn.cuh"
#include "pa_attn_tc.h"
#include "pa_tc.cuh"

namespace pa {

constexpr int kTcThreads = 640;  // 8 softmax, 8 converting, 4 other warps
constexpr int kTcSoftRegs = 136, kTcConvRegs = 72, kTcCtlRegs = 64;  // a thread, after the split
constexpr int kTcTile = 128 * 256;  // bytes of an f16 tile of 128 x 128
constexpr int kTcKeys = 32;         // keys a softmax thread takes at a time (tc_ld32)
// When the references move: that of the products (NVFP4: the weights) once one
// is above 2^15; FP8's weights stay in f32, and theirs when they leave that.
constexpr float kTcMost = 15.f;
template <int FMT>
constexpr float kTcSlack = FMT == 0 ? 40.f : kTcMost - kAtLift;
// FP8: while a block's V scales are within 2^kTcSpread of each other, the
// largest weight x V scale is taken from the largest score and the smallest
// scale; it is then no more than that, and less than 2^kTcMost with the lift.
constexpr float kTcSpread = kTcMost - kAtLift - 2.f;

template <int FMT>
struct TcShared : AttnRing<kAtMaxRows, kTcMaxWidth> {
  uint64_t k_full, k_empty;        // the tile of keys; entries without a block go through too
  uint64_t v_full, v_empty;        // that of values
  uint64_t s_full[2], p_full[2], pv_done[2];  // by the softmax group
  uint64_t item_full, item_seen;   // an item's queries and what goes with them; every softmax warp has waited for them
  uint64_t meet, seg_done;         // the groups' sums are there; a segment's O has been read
  uint64_t never, drain;
  uint32_t tmem;
  int first[2];                    // by the segment's parity: the first row's position
  int nan_any[4];                  // by the segment, modulo 4 (written and cleared by the value warps):
  uint32_t nan_rows[4][kHeadDim];  // rows that see a NaN value in a dim, of keys not all see
  float row_scale[2][128];
  float4 sums[2][128];             // a group's m, l, factor of o, and whether it had a block
  // FP8, of entry n at n % 4: K and V scales, log2 |V scale| (-inf where the codes are all zero), the largest and smallest of those
  __align__(16) float scales[FMT == 0 ? 4 : 1][3][128];
  __align__(16) float most_of[FMT == 0 ? 4 : 1][4], least_of[FMT == 0 ? 4 : 1][4];
};

template <int FMT>
struct TcSmem {  // Q, K and V tiles, the stages, the rest
  static constexpr int kRest = 3 * kTcTile + (int)sizeof(TcShared<FMT>) + 1024;
  static constexpr int kFit = (kAtSmem - kRest) / AttnStage<FMT>::kBytes;
  static constexpr int kStages = kFit < 5 ? kFit : 5;
  static constexpr int kBytes = kRest + kStages * AttnStage<FMT>::kBytes;
};

// The f16 tiles are rows of 128 bytes (64 elements) with the 128-byte swizzle,
// two such halves of 16 KB: 16-byte piece c (of 16) of row r.
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
  return (uint32_t)((c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}
// MN-major operand: rows are elements of K, 8 of them 1024 bytes on (SBO), the
// next 64 elements of N 16 KB on (LBO).
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(16384 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// 16 elements of K on, in a descriptor's 16-byte units: along the 128-byte
// rows and into the other half (K-major), 16 rows (MN-major).
__device__ __forceinline__ uint32_t step_k(int k) { return (uint32_t)((k & 3) * 2 + (k >> 2) * 1024); }
__device__ __forceinline__ uint32_t step_mn(int k) { return (uint32_t)(k * 128); }
// kind::f16, f16 operands, f32 accumulator; tb: B MN-major.
__device__ __forceinline__ uint32_t idesc_f16(int m, int n, int tb) {
  return (1u << 4) | ((uint32_t)tb << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{.reg .pred p; setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// A from tensor memory (K-major, 2 f16 a 32-bit column, row i in lane i).
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{.reg .pred p; setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;}" ::"r"(d),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tc_st(uint32_t taddr, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]), "f"(v[10]),
      "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// ------------------------------------------------------------- converters
// One 16-byte piece of E4M3 codes as 16 f16 values.
__device__ __forceinline__ void e4m3x16_f16(uint4 w, uint4 &lo, uint4 &hi) {
  const uint2 a = e4m3x4_f16(w.x), b = e4m3x4_f16(w.y), c = e4m3x4_f16(w.z), d = e4m3x4_f16(w.w);
  lo = make_uint4(a.x, a.y, b.x, b.y);
  hi = make_uint4(c.x, c.y, d.x, d.y);
}
// E2M1 codes of 32 dims of a token and their two scales as the tile's pieces
// 4 t .. 4 t + 3 of row tok.
__device__ __forceinline__ void e2m1x32_tile(uint4 w, uint32_t sf2, uint8_t *tile, int tok, int t) {
  const uint32_t fh = e4m3x4_f16(sf2).x;
  const uint32_t f[2] = {__byte_perm(fh, fh, 0x1010), __byte_perm(fh, fh, 0x3232)};
  const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int y = 0; y < 4; ++y) {
    uint32_t h[4];
    e2m1x8_f16(ww[y], h);
    *reinterpret_cast<uint4 *>(tile + tile_at(tok, 4 * t + y)) =
        make_uint4(mul_f16x2(h[0], f[y >> 1]), mul_f16x2(h[1], f[y >> 1]), mul_f16x2(h[2], f[y >> 1]),
                   mul_f16x2(h[3], f[y >> 1]));
  }
}
// The keys of a block, by 128 threads: a token each.
template <int FMT>
__device__ __forceinline__ void convert_k(const uint8_t *st, uint8_t *tile, int pt, int tok) {
  if constexpr (FMT == 0) {
#pragma unroll 2
    for (int c = 0; c < 8; ++c) {
      uint4 lo, hi;
      e4m3x16_f16(*reinterpret_cast<const uint4 *>(st + (tok >> 4) * 2048 + c * 256 + (tok & 15) * 16), lo, hi);
      *reinterpret_cast<uint4 *>(tile + tile_at(tok, 2 * c)) = lo;
      *reinterpret_cast<uint4 *>(tile + tile_at(tok, 2 * c + 1)) = hi;
    }
  } else {
    const int in = tok & (pt - 1);
    const uint8_t *base = st + (tok - in) * 144;
    const uint2 sf = *reinterpret_cast<const uint2 *>(base + pt * 64 + in * 8);
#pragma unroll 1  // (short code, see above)
    for (int k = 0; k < 4; ++k) {
      const int t = (k + tok) & 3;  // (neighbours' reads 64 bytes apart then meet in a bank two at a time)
      e2m1x32_tile(*reinterpret_cast<const uint4 *>(base + in * 64 + 16 * t), (t < 2 ? sf.x : sf.y) >> (16 * (t & 1)) & 0xffffu,
                   tile, tok, t);
    }
  }
}

// The rows of an item that see a key: of `rows` (those that attend its block),
// row i at position first + i.
__device__ __noinline__ uint32_t rows_that_see(const CacheAttnParams &a, int key, int first, uint32_t rows) {
  uint32_t m = 0;
  for (int i = 0; i < kAtMaxRows; ++i)
    if (key <= first + i && (a.window == 0 || key > first + i - a.window || key < a.sinks)) m |= 1u << i;
  return m & rows;
}
// Of the 16 keys from key0 on, those that one of the rows sees, a bit each
// (within a window the rows that attend a block follow one another).
__device__ __forceinline__ uint32_t keys_seen(const CacheAttnParams &a, int key0, int first, uint32_t rows) {
  if (rows == 0) return 0;
  const int upto = first + 31 - __clz(rows) - key0;
  uint32_t m = upto >= 15 ? 0xffffu : upto < 0 ? 0u : (2u << upto) - 1u;
  if (a.window) {
    const int out = first + __ffs(rows) - 1 - a.window - key0 + 1, sunk = a.sinks - key0;
    m &= ~(out >= 16 ? 0xffffu : out <= 0 ? 0u : (1u << out) - 1u) | (sunk >= 16 ? 0xffffu : sunk <= 0 ? 0u : (1u << sunk) - 1u);
  }
  return m;
}
// The values of a block, by 128 threads: FP8 a dim each, NVFP4 a token each.
// all: every row of the item sees every key.
template <int FMT>
__device__ __forceinline__ void convert_v(const CacheAttnParams &a, const uint8_t *st, uint8_t *tile, int pt, int ct, int key0,
                                          int first, uint32_t rows, bool all, uint32_t (&nan_rows)[kHeadDim], int *nan_any) {
  auto note = [&](int d, uint32_t who) {
    if (who) atomicOr(&nan_rows[d], who), *nan_any = 1;
  };
  if constexpr (FMT == 0) {
    const int d = ct;
#pragma unroll 2
    for (int pg = 0; pg < 8; ++pg) {
      uint4 w = *reinterpret_cast<const uint4 *>(st + AttnStage<0>::kV + pg * 2048 + d * 16);
      uint32_t x[4] = {w.x, w.y, w.z, w.w};
      if (!all) {
        const uint32_t seen = keys_seen(a, key0 + 16 * pg, first, rows);
        uint32_t any = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          x[q] &= ((((seen >> (4 * q)) & 15u) * 0x00204081u) & 0x01010101u) * 255u;  // a byte a key
          any |= (x[q] & 0x7f7f7f7fu) + 0x01010101u;                                 // bit 7 of a byte: its code is NaN
        }
        if (any & 0x80808080u) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (((x[e >> 2] >> (8 * (e & 3))) & 0x7fu) == 0x7fu) {
              x[e >> 2] &= ~(0xffu << (8 * (e & 3)));
              note(d, rows_that_see(a, key0 + 16 * pg + e, first, rows));
            }
        }
        w = make_uint4(x[0], x[1], x[2], x[3]);
      }
      uint4 lo, hi;
      e4m3x16_f16(w, lo, hi);
      *reinterpret_cast<uint4 *>(tile + tile_at(d, 2 * pg)) = lo;
      *reinterpret_cast<uint4 *>(tile + tile_at(d, 2 * pg + 1)) = hi;
    }
  } else {
    const int tok = ct, in = tok & (pt - 1);
    const uint8_t *base = st + (tok - in) * 144 + pt * 72;
    const bool seen = all || (keys_seen(a, key0 + (tok & ~15), first, rows) >> (tok & 15)) & 1u;
    // the scales of four tokens are eight words, a token a byte of each
    const uint4 s0 = *reinterpret_cast<const uint4 *>(base + pt * 64 + (in >> 2) * 32), s1 = *reinterpret_cast<const uint4 *>(base + pt * 64 + (in >> 2) * 32 + 16);
    const uint32_t by = (in & 3) | ((in & 3) + 4) << 4;
    const uint32_t sf4[4] = {__byte_perm(s0.x, s0.y, by), __byte_perm(s0.z, s0.w, by), __byte_perm(s1.x, s1.y, by), __byte_perm(s1.z, s1.w, by)};
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
      const int t = (k + tok) & 3;
      uint4 w = *reinterpret_cast<const uint4 *>(base + in * 64 + 16 * t);
      uint32_t sf2 = (t & 2 ? (t & 1 ? sf4[3] : sf4[2]) : (t & 1 ? sf4[1] : sf4[0])) & 0xffffu;
      if (!all) {
        if (!seen) w = make_uint4(0, 0, 0, 0), sf2 = 0;
#pragma unroll
        for (int g = 0; g < 2; ++g)
          if (((sf2 >> (8 * g)) & 0x7fu) == 0x7fu) {
            sf2 &= ~(0xffu << (8 * g));
            const uint32_t who = rows_that_see(a, key0 + tok, first, rows);
            for (int d = 32 * t + 16 * g; d < 32 * t + 16 * g + 16; ++d) note(d, who);
          }
      }
      e2m1x32_tile(w, sf2, tile, tok, t);
    }
  }
}

__device__ __forceinline__ int whole_of(float x) { return (int)fminf(fmaxf(x, -1e6f), 1e6f); }

// What a softmax thread knows of its (row, head).
struct TcRow {
  float m, l;  // the softmax's reference, the sum of the weights, lifted
  int gref;    // FP8: the reference of the products (weight x V scale), an exponent
  bool begun;  // o has a block
};
// Of keys k0 .. + 31, those that a row at p sees.
__device__ __forceinline__ uint32_t keys_of_row(const CacheAttnParams &a, bool sees, int p, int k0) {
  if (!sees) return 0u;
  const int upto = p - k0;
  uint32_t s = upto >= 31 ? 0xffffffffu : upto < 0 ? 0u : (2u << upto) - 1u;
  if (a.window) {
    const int out = p - a.window - k0 + 1, sunk = a.sinks - k0;
    s &= ~(out >= 32 ? 0xffffffffu : out <= 0 ? 0u : (1u << out) - 1u) | (sunk >= 32 ? 0xffffffffu : sunk <= 0 ? 0u : (1u << sunk) - 1u);
  }
  return s;
}
// The references up to the largest score `top` (FP8: a whole number) and the
// largest weight x V scale of the block, of every (row, head) of the warp when
// one's have been outgrown, so that this comes two or three times a segment; o
// and l follow.  lv: FP8, the block's largest and smallest log2 |V scale|.
template <int FMT>
__device__ __noinline__ TcRow move_references(const CacheAttnParams &a, TcRow r, float top, float2 lv, float sc, const float *scales,
                                             uint32_t s_col, uint32_t o_col, bool cut, bool sees, int p, int key0) {
  const float was = r.m;
  if (r.m == -INFINITY || (FMT == 0 ? top > r.m + kTcSlack<FMT> : top > r.m)) r.m = FMT == 0 ? ceilf(top) : top;
  float al = 1.f;  // what o is multiplied by
  if (was != r.m && was != -INFINITY) {
    const float f = ex2_approx(was - r.m);
    r.l *= f;
    if constexpr (FMT == 1) al = f;
  }
  if constexpr (FMT == 0) {
    float most[2] = {-INFINITY, -INFINITY};
    // (the keys one by one: 3400 clocks, of some 60000 that a group's nine blocks take)
    const bool near = lv.x - lv.y <= kTcSpread;
    if (near) most[0] = top + lv.y;
#pragma unroll 1
    for (int c = near ? 8 : 0; c < 8; ++c) {  // (of keys that the row sees: the rest are not looked at)
      float y[16];
      tc_ld16(s_col + 16 * c, y);
      const uint32_t mask = cut ? keys_of_row(a, sees, p, key0 + 16 * c) : 0xffffu;
      tc_wait_ld();
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        const float4 k4 = *reinterpret_cast<const float4 *>(scales + 16 * c + e), v4 = *reinterpret_cast<const float4 *>(scales + 256 + 16 * c + e);
        const float k[4] = {k4.x, k4.y, k4.z, k4.w}, v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
        for (int q = 0; q < 4; ++q)
          most[q & 1] = fmaxf(most[q & 1], (mask >> (e + q)) & 1u ? fmaf(y[e + q], sc * k[q], v[q]) : -INFINITY);
      }
    }
    const float big = fmaxf(most[0], most[1]);
    const int mi = whole_of(r.m);
    int to = r.begun ? r.gref : mi - kAtUnit;  // none known: the largest unit
    if (big > (float)to) to = whole_of(floorf(big));
    to = max(min(to, mi + 126), mi - kAtUnit);  // the unit is a normal number
    if (r.begun && to != r.gref) al = r.gref - to < -126 ? 0.f : pow2i(min(r.gref - to, 127));
    r.gref = to;
  }
  if (r.begun && __any_sync(0xffffffffu, al != 1.f)) {
#pragma unroll 1
    for (int c = 0; c < 8; ++c) {
      float o[16];
      tc_ld16(o_col + 16 * c, o);
      tc_wait_ld();
#pragma unroll
      for (int e = 0; e < 16; ++e) o[e] *= al;
      tc_st(o_col + 16 * c, o);
    }
    tc_wait_st();
  }
  return r;
}

template <int FMT>
__global__ void __launch_bounds__(kTcThreads, 1) pa_attn_tc_kernel(const __grid_constant__ AttnMaps maps,
                                                                   const __grid_constant__ CacheAttnParams a) {
  using St = AttnStage<FMT>;
  using Sm = TcSmem<FMT>;
  static_assert(Sm::kBytes <= kAtSmem && Sm::kStages >= 3, "shared memory of a CTA");
  constexpr int kStages = Sm::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *q_tile = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t *k_tile = q_tile + kTcTile, *v_tile = k_tile + kTcTile, *ring = v_tile + kTcTile;
  TcShared<FMT> &sh = *reinterpret_cast<TcShared<FMT> *>(ring + kStages * St::kBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == 16 && (FMT == 0 ? lane < 4 : lane == 0 && a.bs <= 128))
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.m[lane])) : "memory");
  if (warp == 17) attn_prefetch(a, a.mode);
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 8);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sh.batch_full[s], 1);
      mbar_init(&sh.batch_empty[s], 1);
      mbar_init(&sh.s_full[s], 1);
      mbar_init(&sh.p_full[s], 4);
      mbar_init(&sh.pv_done[s], 1);
    }
    for (int s = 0; s < 4; ++s) sh.nan_any[s] = 0;
    mbar_init(&sh.k_full, 4);
    mbar_init(&sh.k_empty, 1);
    mbar_init(&sh.v_full, 4);
    mbar_init(&sh.v_empty, 1);
    mbar_init(&sh.item_full, 8);
    mbar_init(&sh.item_seen, 8);
    mbar_init(&sh.meet, 8);
    mbar_init(&sh.seg_done, 8);
    mbar_init(&sh.never, 1);
    mbar_init(&sh.drain, 1);
    fence_mbar_init();
  }
  if (tid < 4 * kHeadDim) (&sh.nan_rows[0][0])[tid] = 0;
  pdl_wait();  // queries, caches and lists come from the previous kernels
  pdl_trigger();
  const AttnSlice sl = attn_slice<8, true>(a, sh, a.mode);
  if (sl.none) return;
  if (warp == 19) tc_alloc(&sh.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  constexpr uint32_t kOCol = 256;  // S of the groups: columns 0 and 128; O: 256 and 384
  const int pt = min(a.bs, 128);

  if (warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTcCtlRegs));
    if (warp == 16 && lane == 0) attn_copies<FMT, kStages, 2, false>(a, maps, sh, sl, ring, nullptr);
    if (warp == 17) attn_resolve<FMT, true>(a, sh, sl, a.mode);
    if (warp == 18 && lane == 0) {
      // ------------------------------------------------------------ the MMAs
      const uint64_t kd = sdesc_sw128(smem_u32(k_tile)), qd = sdesc_sw128(smem_u32(q_tile));
      // V: rows are dims (FP8: pages hold a dim's keys together) or keys (NVFP4)
      const uint64_t vd = FMT == 0 ? sdesc_sw128(smem_u32(v_tile)) : sdesc_mn(smem_u32(v_tile));
      const uint32_t ids = idesc_f16(128, 128, 0), idp = idesc_f16(128, 128, FMT == 0 ? 0 : 1);
      bool ok = true;
      uint32_t n = 0, nb = 0, seg = 0;      // entries, blocks whose PV is issued, segments
      uint32_t had[2] = {0, 0}, pc[2] = {0, 0};  // by group: S issued, PV issued
      int v0, v1, v;
      for (int it = sl.first; ok && sl.segment(a, sh, it, v0, v1, v); ++it, ++seg) {
        bool begun[2] = {false, false}, pending = false, any = false;
        // every softmax warp has taken the last entries of the segment before: a
        // phase of s_full does not pass one by (within a segment S of the group's
        // next entry waits for P of its last)
        if (seg > 0 && !(ok = mbar_wait(&sh.meet, (seg - 1) & 1, a.status, a.lim))) break;
        for (int ends = 0; ok && ends < 2; ++n) {
          const int g = n & 1;
          if (!(ok = mbar_wait(&sh.k_full, n & 1, a.status, a.lim))) break;
          const bool end = sh.info[n % kAtInfo].x < 0;
          if (!end) {
            // P of the group's block before is in S's place until its product is done
            if (had[g] > 0 && !(ok = mbar_wait(&sh.pv_done[g], (had[g] - 1) & 1, a.status, a.lim))) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 8; ++k) mma_f16_ss(tmem + g * 128, qd + step_k(k), kd + step_k(k), ids, k > 0);
            tc_commit(&sh.s_full[g]);
            tc_commit(&sh.k_empty);
            ++had[g];
          }
          if (pending) {
            const int h = g ^ 1;
            if (!(ok = mbar_wait(&sh.p_full[h], pc[h] & 1, a.status, a.lim) && mbar_wait(&sh.v_full, nb & 1, a.status, a.lim))) break;
            // the segment before is out of O
            if (!any && seg > 0 && !(ok = mbar_wait(&sh.seg_done, (seg - 1) & 1, a.status, a.lim))) break;
            any = true;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mma_f16_ts(tmem + kOCol + h * 128, tmem + h * 128 + 8 * k, vd + (FMT == 0 ? step_k(k) : step_mn(k)), idp,
                         begun[h] || k > 0);
            begun[h] = true;
            tc_commit(&sh.pv_done[h]);
            tc_commit(&sh.v_empty);
            ++pc[h], ++nb;
          }
          pending = !end;
          if (end) {
            tc_commit(&sh.s_full[g]);  // behind every product of the segment
            mbar_arrive(&sh.k_empty);
            ++ends;
          }
        }
      }
      // what was issued completes before the tensor memory is freed
      tc_commit(&sh.drain);
      mbar_wait(&sh.drain, 0, a.status, a.lim);
    }
  } else if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTcConvRegs));
    // ---------------------------------------------------------- converters
    const int ct = tid & 127;
    uint32_t j = 0, seg = 0;  // entries, segments
    bool ok = true;
    auto all_got = [&](bool got) { return ok = __all_sync(0xffffffffu, got) != 0; };
    int v0, v1, v;
    if (warp < 12) {
      // keys and queries: (row, head) ct / 2 and, in a second turn, 64 + ct / 2; 64 dims a thread
      AttnItem nx;
      auto lay_out = [&](uint32_t sg) {
#pragma unroll 1
        for (int turn = 0; turn < 2; ++turn) {
          const int at = 64 * turn + (ct >> 1), d0 = 64 * (ct & 1);
          const bool have = at < nx.rows * a.group;
          const int row = have ? at / a.group : 0, head = have ? at - row * a.group : 0;
          const int64_t off = ((int64_t)nx.r * a.q_len + nx.row0 + row) * a.q_stride + (int64_t)(nx.h * a.group + head) * kHeadDim + d0;
          const uint4 *src = reinterpret_cast<const uint4 *>(a.q + (a.q_is_fp8 ? off : 2 * off));
          uint4 qr[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) qr[k] = have && (k < 4 || !a.q_is_fp8) ? __ldg(src + k) : make_uint4(0, 0, 0, 0);
          auto values = [&](int k, float (&x)[8]) {  // dims d0 + 8 k .. + 7
            if (a.q_is_fp8) {
              const uint4 w = qr[k >> 1];
              const uint2 h0 = e4m3x4_f16(k & 1 ? w.z : w.x), h1 = e4m3x4_f16(k & 1 ? w.w : w.y);
              const uint32_t h[4] = {h0.x, h0.y, h1.x, h1.y};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[e]));
                x[2 * e] = f.x, x[2 * e + 1] = f.y;
              }
            } else {
              const uint32_t h[4] = {qr[k].x, qr[k].y, qr[k].z, qr[k].w};
#pragma unroll
              for (int e = 0; e < 4; ++e) x[2 * e] = bf16_to_f32(h[e] & 0xffffu), x[2 * e + 1] = bf16_to_f32(h[e] >> 16);
            }
          };
          float top = 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float x[8];
            values(k, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[e]));
          }
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          const int ex = max(exponent_of(top), -110) - 14;
          const float down = pow2i(-ex);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float x[8];
            values(k, x);
            *reinterpret_cast<uint4 *>(q_tile + tile_at(at, (d0 >> 3) + k)) =
                make_uint4(f16x2_bits(x[0] * down, x[1] * down), f16x2_bits(x[2] * down, x[3] * down),
                           f16x2_bits(x[4] * down, x[5] * down), f16x2_bits(x[6] * down, x[7] * down));
          }
          if ((ct & 1) == 0) sh.row_scale[sg & 1][at] = a.score_scale * pow2i(ex);
        }
        if (ct == 0) sh.first[sg & 1] = nx.first;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.item_full);
      };
      auto look_up = [&](int it) {
        bool bad = false;
        nx = attn_item(a, it, &bad);
      };
      if (sl.segment(a, sh, sl.first, v0, v1, v)) {
        look_up(sl.first);
        lay_out(0);
      }
      for (int it = sl.first; ok && sl.segment(a, sh, it, v0, v1, v); ++it, ++seg) {
        int w0, w1, w;
        const bool next = sl.segment(a, sh, it + 1, w0, w1, w);
        if (next) {
          look_up(it + 1);
          if (ct < nx.rows * a.group) {  // into L2
            const int row = ct / a.group;
            const int64_t off = ((int64_t)nx.r * a.q_len + nx.row0 + row) * a.q_stride + (int64_t)(nx.h * a.group + ct - row * a.group) * kHeadDim;
            prefetch_l2(a.q + (a.q_is_fp8 ? off : 2 * off));
            if (!a.q_is_fp8) prefetch_l2(a.q + 2 * off + 128);
          }
        }
        for (int ends = 0; ends < 2; ++j) {
          const int s = j % kStages;
          if (!all_got(mbar_wait(&sh.full[s], (j / kStages) & 1, a.status, a.lim) &&
                       mbar_wait(&sh.k_empty, (j & 1) ^ 1, a.status, a.lim)))
            break;
          const bool more = sh.info[j % kAtInfo].x >= 0;
          if (more) {
            const uint8_t *st = ring + s * St::kBytes;
            convert_k<FMT>(st, k_tile, pt, ct);
            if constexpr (FMT == 0) {
              // the ors of the codes of the warp's tokens: eight dims x 16 tokens a load
              uint32_t some[2] = {0, 0};
              const uint8_t *codes = st + St::kV + (ct >> 5) * 4096 + 4 * lane;
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                some[0] |= *reinterpret_cast<const uint32_t *>(codes + 128 * k);
                some[1] |= *reinterpret_cast<const uint32_t *>(codes + 2048 + 128 * k);
              }
#pragma unroll
              for (int o = 4; o < 32; o <<= 1)
                some[0] |= __shfl_xor_sync(0xffffffffu, some[0], o), some[1] |= __shfl_xor_sync(0xffffffffu, some[1], o);
              const uint32_t lo = __shfl_sync(0xffffffffu, some[0], (lane >> 2) & 3), hi = __shfl_sync(0xffffffffu, some[1], (lane >> 2) & 3);
              const float kz = *reinterpret_cast<const float *>(st + St::kKs + 4 * ct), vz = *reinterpret_cast<const float *>(st + St::kVs + 4 * ct);
              // a row of zeros counts for nothing, whatever its scale: it does not
              // set the products' unit, in which its weight x scale could leave f16
              const bool zero = (((lane < 16 ? lo : hi) >> (8 * (lane & 3))) & 0x7fu) == 0u && fabsf(vz) < INFINITY;
              sh.scales[j & 3][0][ct] = kz;
              sh.scales[j & 3][1][ct] = zero ? 0.f : vz;
              const float lv = zero ? -INFINITY : lg2_approx(fabsf(vz));
              sh.scales[j & 3][2][ct] = lv;
              float most = lv, least = lv;
#pragma unroll
              for (int o = 16; o > 0; o >>= 1) {
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
                least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
              }
              if (lane == 0) sh.most_of[j & 3][warp & 3] = most, sh.least_of[j & 3][warp & 3] = least;
            }
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sh.k_full);
            mbar_arrive(&sh.empty[s]);
          }
          if (!more && ends++ == 0 && next) {
            // (the last S of this segment is done: its queries may be replaced; the
            // softmax warps are behind the segment before and its item_full)
            if (!all_got(mbar_wait(&sh.item_seen, seg & 1, a.status, a.lim))) break;
            lay_out(seg + 1);
          }
        }
      }
    } else {
      // values
      uint32_t nv = 0;  // blocks
      for (int it = sl.first; ok && sl.segment(a, sh, it, v0, v1, v); ++it, ++seg) {
        // The next segment's notes are cleared when the softmax is in the segment
        // before, so past that which had their place, and before it comes to this
        // one: nothing is noted for the next segment until it has
        if (seg > 0 && !all_got(mbar_wait(&sh.item_seen, (seg - 1) & 1, a.status, a.lim))) break;
        sh.nan_rows[(seg + 1) & 3][ct] = 0;
        if (ct == 0) sh.nan_any[(seg + 1) & 3] = 0;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.item_full);
        bool bad = false;
        const AttnItem x = attn_item(a, it, &bad);
        const uint32_t every = (1u << x.rows) - 1u;
        for (int ends = 0; ends < 2; ++j) {
          const int s = j % kStages;
          if (!all_got(mbar_wait(&sh.full[s], (j / kStages) & 1, a.status, a.lim))) break;
          const int2 info = sh.info[j % kAtInfo];
          if (info.x >= 0) {
            if (!all_got(mbar_wait(&sh.v_empty, (nv & 1) ^ 1, a.status, a.lim))) break;
            const int key0 = info.x * 128, p1 = x.first + x.rows - 1;
            const bool all = (uint32_t)info.y == every && key0 + 127 <= x.first &&
                             (a.window == 0 || key0 > p1 - a.window || key0 + 127 < a.sinks);
            convert_v<FMT>(a, ring + s * St::kBytes, v_tile, pt, ct, key0, x.first, (uint32_t)info.y, all, sh.nan_rows[seg & 3],
                           &sh.nan_any[seg & 3]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.v_full);
            ++nv;
          } else {
            ++ends;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.empty[s]);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTcSoftRegs));
    // ------------------------------------------------------------- softmax
    const int g = warp >> 2, at = tid & 127;  // the group, the (row, head)
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t s_col = lanes + g * 128, o_col = lanes + kOCol + g * 128;
    uint32_t n = g, ns = 0, seg = 0;  // the group's next entry, its number among the group's, segments
    bool ok = true;
    auto wait = [&](uint64_t *b, uint32_t parity) {
      return ok = __all_sync(0xffffffffu, mbar_wait(b, parity, a.status, a.lim)) != 0;
    };
    int v0, v1, v;
    for (int it = sl.first; ok && sl.segment(a, sh, it, v0, v1, v); ++it, ++seg) {
      if (!wait(&sh.item_full, seg & 1)) break;
      if (lane == 0) mbar_arrive(&sh.item_seen);
      const AttnItem x = attn_place(a, it);
      const int first = sh.first[seg & 1];
      const bool have = at < x.rows * a.group;
      const bool idle = !__any_sync(0xffffffffu, have);  // the warp has no (row, head)
      const int row = have ? at / a.group : 0, head = at - row * a.group, p = first + row;
      const float sc = have ? sh.row_scale[seg & 1][at] : 0.f;
      const int low = p - a.window;
      TcRow st = {-INFINITY, 0.f, 0, false};
      while (true) {
        if (!wait(&sh.s_full[g], ns & 1)) break;
        if (a.test_timeout && !wait(&sh.never, 0)) break;
        tc_fence_after();
        const int2 info = sh.info[n % kAtInfo];
        const uint32_t entry = n;
        n += 2, ++ns;
        if (info.x < 0) break;
        if (!idle) {
          const int key0 = info.x * 128;
          const bool sees = have && ((info.y >> row) & 1);
          // some of the block's keys are out of the row's sight
          const bool cut = __any_sync(0xffffffffu, have && (!sees || key0 + 127 > p || (a.window && key0 <= low && key0 + 127 >= a.sinks)));
          const float *ks = sh.scales[FMT == 0 ? entry & 3 : 0][0];
          // Twice over the block's scores, kTcKeys a turn: their largest (the
          // references move once it has outgrown them), then the weights, in one
          // short loop
          float tops[2] = {-INFINITY, -INFINITY}, off = 0.f, unit = 1.f;
          f32x2 s2[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
          const f32x2 sc2 = pack2(sc, sc);
          constexpr int kTurns = 128 / kTcKeys;
          float next[kTcKeys];
          tc_ld32(s_col, next);
#pragma unroll 1
          for (int i = 0; i < 2 * kTurns; ++i) {
            const int c = i & (kTurns - 1);
            f32x2 y[kTcKeys / 2];
            const f32x2 off2 = pack2(off, off);
            uint32_t mask = 0xffffffffu;
            bool masked = cut;
            if constexpr (FMT == 0)  // (NVFP4: the look for turns without a mask cost more than it saved, 62.9 us for 61.5)
              if (__builtin_expect(cut, 0)) {
                mask = keys_of_row(a, sees, p, key0 + kTcKeys * c);
                masked = __any_sync(0xffffffffu, have && mask != 0xffffffffu);
              }
            tc_wait_ld();
#pragma unroll
            for (int e = 0; e < kTcKeys / 2; e += 2) {
              f32x2 f0 = sc2, f1 = sc2;
              if constexpr (FMT == 0) {
                const float4 k4 = *reinterpret_cast<const float4 *>(ks + kTcKeys * c + 2 * e);
                f0 = mul2(sc2, pack2(k4.x, k4.y)), f1 = mul2(sc2, pack2(k4.z, k4.w));
              }
              y[e] = fma2(pack2(next[2 * e], next[2 * e + 1]), f0, off2), y[e + 1] = fma2(pack2(next[2 * e + 2], next[2 * e + 3]), f1, off2);
            }
            tc_ld32(s_col + kTcKeys * ((i + 1) & (kTurns - 1)), next);
            if (__builtin_expect(masked, 0)) {
              if constexpr (FMT == 1) mask = keys_of_row(a, sees, p, key0 + kTcKeys * c);
#pragma unroll
              for (int e = 0; e < kTcKeys / 2; ++e) {
                const float2 z = unpack2(y[e]);
                y[e] = pack2((mask >> (2 * e)) & 1u ? z.x : -INFINITY, (mask >> (2 * e)) & 2u ? z.y : -INFINITY);
              }
            }
            if (i < kTurns) {
#pragma unroll
              for (int e = 0; e < kTcKeys / 2; ++e) {
                const float2 z = unpack2(y[e]);
                tops[e & 1] = max3(tops[e & 1], z.x, z.y);
              }
              if (i == kTurns - 1) {
                const float top = fmaxf(tops[0], tops[1]);
                float2 lv = make_float2(0.f, 0.f);  // the largest and the smallest log2 |V scale|
                if constexpr (FMT == 0) {
                  const float4 z = *reinterpret_cast<const float4 *>(sh.most_of[entry & 3]), y4 = *reinterpret_cast<const float4 *>(sh.least_of[entry & 3]);
                  lv = make_float2(max3(fmaxf(z.x, z.y), z.z, z.w), fminf(fminf(y4.x, y4.y), fminf(y4.z, y4.w)));
                }
                const bool moves = top > st.m + kTcSlack<FMT> || st.m == -INFINITY ||
                                   (FMT == 0 && (!st.begun || top + lv.x > (float)st.gref + (kTcMost - kAtLift)));
                if (__builtin_expect(__any_sync(0xffffffffu, have && moves), 0)) {
                  tc_wait_ld();
                  st = move_references<FMT>(a, st, top, lv, sc, ks, s_col, o_col, cut, sees, p, key0);
                  tc_ld32(s_col, next);
                }
                off = st.m == -INFINITY ? 0.f : kAtLift - st.m;
                if constexpr (FMT == 0) unit = st.m == -INFINITY ? 0.f : pow2i(whole_of(st.m) - st.gref);
              }
              continue;
            }
            float pk[kTcKeys / 2];  // P, two keys each; in the place of S that has been read
            const f32x2 u2 = pack2(unit, unit);
#pragma unroll
            for (int e = 0; e < kTcKeys / 2; e += 2) {
              const float2 z0 = unpack2(y[e]), z1 = unpack2(y[e + 1]);
              f32x2 w0 = pack2(ex2_approx(z0.x), ex2_approx(z0.y)), w1 = pack2(ex2_approx(z1.x), ex2_approx(z1.y));
              s2[(e >> 1) & 1] = add2(s2[(e >> 1) & 1], add2(w0, w1));
              if constexpr (FMT == 0) {
                const float4 v4 = *reinterpret_cast<const float4 *>(ks + 128 + kTcKeys * c + 2 * e);
                w0 = mul2(mul2(w0, pack2(v4.x, v4.y)), u2), w1 = mul2(mul2(w1, pack2(v4.z, v4.w)), u2);
              }
              const float2 r0 = unpack2(w0), r1 = unpack2(w1);
              pk[e] = __uint_as_float(f16x2_bits(r0.x, r0.y)), pk[e + 1] = __uint_as_float(f16x2_bits(r1.x, r1.y));
            }
            if (FMT == 0 && __builtin_expect(masked, 0)) {  // whatever the scale of a key that is not seen
#pragma unroll
              for (int e = 0; e < kTcKeys / 2; ++e)
                pk[e] = __uint_as_float(__float_as_uint(pk[e]) & (((mask >> (2 * e)) & 1u ? 0xffffu : 0u) | ((mask >> (2 * e)) & 2u ? 0xffff0000u : 0u)));
            }
            tc_st(s_col + kTcKeys / 2 * c, pk);
          }
          tc_wait_ld();
          const float2 su = unpack2(add2(s2[0], s2[1]));
          const float sum = su.x + su.y;
          st.l += sum;
          if (a.wpart && sees) {
            const int64_t mi = (int64_t)x.r * a.q_len + x.row0 + row;
            a.wpart[(((mi * a.n_kv + x.h) * a.bt_width + info.x) << a.lg_heads) + head] = st.m + lg2_approx(sum);
          }
          tc_wait_st();
          st.begun = true;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[g]);
      }
      if (!ok) break;
      // ------------------------------------------------ the segment's result
      float up = 1.f;
      if constexpr (FMT == 0) {
        // o leaves its unit, with l near 2^-kAtSumDown (as in pa_attn_kernel)
        const int eu = st.m == -INFINITY ? 0 : whole_of(st.m) - st.gref;
        const int el = st.l > 0.f && st.l < INFINITY ? min(exponent_of(st.l) + kAtSumDown, 126 - eu) : 0;
        up = pow2i(max(-eu - el, -126));
        st.m += (float)el;
        st.l *= pow2i(-el);
      }
      sh.sums[g][at] = make_float4(st.m, st.l, up, st.begun ? 1.f : 0.f);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.meet);
      if (!wait(&sh.meet, seg & 1)) break;
      const bool whole = v0 == 0 && v1 == v;
      float *pp = nullptr;
      if (!whole) {
        pp = a.part + (int64_t)(2 * sl.cta + (v0 > 0 ? 0 : 1)) * kAtPartFloats;
        if (v0 == 0 && tid == 0) {
          const int last = sh.offs[it + 1] - 1;
          a.shares[it] = make_int2(sl.cta, (int)((((int64_t)last + 1) * sl.ctas - 1) / sl.total));
        }
      } else if (sl.sliced && tid == 0) {
        a.shares[it] = make_int2(0, 0);
      }
      if (!idle) {
        const float4 z0 = sh.sums[0][at], z1 = sh.sums[1][at];
        const float top = fmaxf(z0.w != 0.f ? z0.x : -INFINITY, z1.w != 0.f ? z1.x : -INFINITY);
        const float f0 = z0.w == 0.f ? 0.f : z0.x == top ? 1.f : ex2_approx(z0.x - top);
        const float f1 = z1.w == 0.f ? 0.f : z1.x == top ? 1.f : ex2_approx(z1.x - top);
        const float all = f0 * z0.y + f1 * z1.y;
        const float inv = whole ? (all == 0.f ? 0.f : a.out_scale / all) : 1.f;
        // (a factor that is 0 takes what a group without a block has in o with it)
        const float u0 = f0 * z0.z, u1 = f1 * z1.z;
        const int64_t mi = (int64_t)x.r * a.q_len + x.row0 + row;
        const bool nans = sh.nan_any[seg & 3] != 0;
        const bool both0 = __any_sync(0xffffffffu, z0.w != 0.f), both1 = __any_sync(0xffffffffu, z1.w != 0.f);
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {  // 32 dims of this group's half
          const int d0 = 64 * g + 32 * c;
          float o[32], y[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = 0.f;
          if (both0) {
            tc_ld32(lanes + kOCol + d0, o);
            tc_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = u0 * o[e];
          }
          if (both1) {
            tc_ld32(lanes + kOCol + 128 + d0, o);
            tc_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = fmaf(u1, o[e], y[e]);
          }
          if (nans)
            for (int e = 0; e < 32; ++e)
              if ((sh.nan_rows[seg & 3][d0 + e] >> row) & 1u)
#pragma unroll
                for (int q = 0; q < 32; ++q)
                  if (q == e) y[q] = __int_as_float(0x7fc00000);
          if (!have) continue;
          if (whole) {
            __nv_bfloat16 *dst = a.out + mi * a.out_stride + (int64_t)(x.h * a.group + head) * kHeadDim + d0;
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              *reinterpret_cast<uint4 *>(dst + e) =
                  make_uint4(bf16x2_bits(y[e] * inv, y[e + 1] * inv), bf16x2_bits(y[e + 2] * inv, y[e + 3] * inv),
                             bf16x2_bits(y[e + 4] * inv, y[e + 5] * inv), bf16x2_bits(y[e + 6] * inv, y[e + 7] * inv));
          } else {
            float *dst = pp + (row * 16 + head) * kHeadDim + d0;
#pragma unroll
            for (int e = 0; e < 32; e += 4) *reinterpret_cast<float4 *>(dst + e) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
          }
        }
        if (have && !whole && g == 0)
          *reinterpret_cast<float2 *>(pp + kAtMaxRows * 16 * kHeadDim + (row * 16 + head) * 2) = make_float2(top, all);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.seg_done);
      if (!wait(&sh.seg_done, seg & 1)) break;
    }
  }
  __syncwarp();
  __syncthreads();  // every wait has an end
  if (warp == 19) tc_dealloc(tmem, 512);
}

template <int FMT>
static cudaError_t launch_tc(const AttnMaps &maps, const CacheAttnParams &a, int grid, bool pdl, cudaStream_t stream) {
  constexpr int smem = TcSmem<FMT>::kBytes;
  const void *kern = reinterpret_cast<const void *>(pa_attn_tc_kernel<FMT>);
  cudaError_t e = ensure_smem_attr(kern, smem);
  if (e != cudaSuccess) return e;
  static std::atomic<int> launch_regs;  // holds the registers it splits
  int regs = launch_regs.load(std::memory_order_relaxed);
  if (regs == 0) {
    cudaFuncAttributes at;
    if ((e = cudaFuncGetAttributes(&at, kern)) != cudaSuccess) return e;
    launch_regs.store(regs = at.numRegs, std::memory_order_relaxed);
  }
  if (regs * kTcThreads < 256 * kTcSoftRegs + 256 * kTcConvRegs + 128 * kTcCtlRegs) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = smem;
  return cudaLaunchKernelEx(&cfg, pa_attn_tc_kernel<FMT>, maps, a);
}

cudaError_t launch_attn_tc(int fmt, const AttnMaps &maps, const CacheAttnParams &a, int grid, bool pdl, cudaStream_t stream) {
  return fmt == 0 ? launch_tc<0>(maps, a, grid, pdl, stream) : launch_tc<1>(maps, a, grid, pdl, stream);
}

}  // namespace pa
