// Attention over the paged KV caches for items of several query rows, on
// tcgen05: the keys are the rows of S = K Q^T (128 keys x 16 heads of each of
// the item's rows) and the dims those of O = V^T P, so every product has M =
// 128 and N = 16 rows, whatever the number of rows, and a key block is read
// from shared memory once for all of them.  (pa_attn.cu's mma.sync kernel
// converts the codes of a block again for each row: about 1900 (FP8) and 2800
// (NVFP4) warp instructions a (row, block), which bounds it; here a block is
// converted once and a (row, block) takes about 400.)
//
// Warps: eight convert a block's codes to f16 tiles (E4M3 codes and E2M1 code
// x E4M3 scale are f16 values) and lay out the queries; one thread issues the
// MMAs; two groups of four do the softmax, a key a thread, the even and the
// odd rows; one resolves the blocks, one thread asks for them.  S has two
// buffers in tensor memory, O stays there; the weights P go through shared
// memory.  S of the next block is issued before O of the last, so the tensor
// core and the converters run while the exponentials do.
//
// Arithmetic as in pa_attn.cu, except that the 16 heads of a row share one
// power-of-two scale of the queries (a value is exact down to 2^-29 of the
// row's largest, and off by at most 2^-40 of it below).  The reference m of a
// (row, head) follows its maximum once that is 2^4 above it; all keys' threads
// of the group agree on that with a barrier that ors a predicate, and o in
// tensor memory and the sums are then scaled.
//
// Keys that a row does not see (after its position, or of a block it does not
// attend) have no weight, but the tile of values is all rows': keys after the
// item's last row are written as zeros, and where not every row sees every
// key, a NaN value is written as zero and the rows that see it noted for its
// dim: they get NaN there.
#include <cstdint>

#include "../../include/pre_attn.h"
#include "pa_attn.cuh"
#include "pa_attn_tc.h"
#include "pa_tc.cuh"

namespace pa {

constexpr int kTcThreads = 640;  // 8 softmax, 8 converting, 4 other warps
constexpr int kTcSoftRegs = 112, kTcConvRegs = 88, kTcCtlRegs = 80;  // a thread, after the split
constexpr int kTcTile = 128 * 256;  // bytes of an f16 tile of 128 x 128

template <int FMT>
struct TcShared : AttnRing<kAtMaxRows, kTcMaxWidth> {
  uint64_t k_full, k_empty;        // the f16 tile of keys; entries without a block go through too
  uint64_t v_full[2], v_empty[2];  // that of values, by halves of 64 keys
  uint64_t v_end;                  // the V warps have passed a segment's end
  uint64_t s_full[2], s_empty[2];             // S in tensor memory
  uint64_t p_full, pv_done;                   // P written; O += V^T P done
  uint64_t seg_done;                          // a segment's result is out
  uint64_t never, drain;
  uint32_t tmem;
  int dead;                    // a softmax warp's wait ran out
  int first[2];                // by the segment's parity: the first row's position
  float row_scale[2][kAtMaxRows];
  uint32_t nan_rows[2][2][kHeadDim];  // for each softmax group: rows that see a NaN value in a dim, of keys not all see
  float off[kAtMaxRows][16];   // lift - m of (row, head)
  float m[kAtMaxRows][16];
  float warp_max[2][4][20];    // by group and warp: a row's maxima, and the largest V scale
  float warp_sum[2][4][16];
  float scales[FMT == 0 ? 4 : 1][2][128];  // FP8: K and V scales of entry n at n % 4
};

template <int FMT>
struct TcSmem {  // K, V, P and Q tiles, the stages, the rest
  static constexpr int kRest = 4 * kTcTile + (int)sizeof(TcShared<FMT>) + 1024;
  static constexpr int kFit = (kAtSmem - kRest) / AttnStage<FMT>::kBytes;
  static constexpr int kStages = kFit < 4 ? kFit : 4;
  static constexpr int kBytes = kRest + kStages * AttnStage<FMT>::kBytes;
};

// The f16 tiles are rows of 128 bytes (64 elements) with the 128-byte swizzle,
// two such halves of 16 KB: 16-byte piece c (of 16) of row r.  (Tiles of plain
// 8 x 16-byte core matrices took the MMAs about four times as long.)
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
  return (uint32_t)((c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}
// MN-major operand: rows are elements of K, 8 of them 1024 bytes on (SBO), the
// next 64 elements of M or N 16 KB on (LBO).
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(16384 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// 16 elements of K on, in a descriptor's 16-byte units: along the 128-byte
// rows and into the other half (K-major), 16 rows (MN-major).
__device__ __forceinline__ uint32_t step_k(int k) { return (uint32_t)((k & 3) * 2 + (k >> 2) * 1024); }
__device__ __forceinline__ uint32_t step_mn(int k) { return (uint32_t)(k * 128); }
// kind::f16, f16 operands, f32 accumulator; ta, tb: A, B MN-major.
__device__ __forceinline__ uint32_t idesc_f16(int m, int n, int ta, int tb) {
  return (1u << 4) | ((uint32_t)ta << 15) | ((uint32_t)tb << 16) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(m >> 4) << 24);
}
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{.reg .pred p; setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t taddr, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])),
      "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])),
      "r"(__float_as_uint(v[8])), "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
      "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])), "r"(__float_as_uint(v[15]))
      : "memory");
}
// Whether the predicate holds for any of the barrier's 128 threads.
__device__ __forceinline__ bool bar_any(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{.reg .pred p, q; setp.ne.b32 p, %1, 0; barrier.cta.red.or.pred q, %2, 128, p; selp.u32 %0, 1, 0, q;}"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(id)
      : "memory");
  return r != 0;
}
// The largest of a warp's values (NaN above all).
__device__ __forceinline__ float warp_max(float x) {
  const int u = __float_as_int(x);
  const int o = __reduce_max_sync(0xffffffffu, u < 0 ? u ^ 0x7fffffff : u);
  return __int_as_float(o < 0 ? o ^ 0x7fffffff : o);
}

// ------------------------------------------------------------- converters
// One 16-byte piece of E4M3 codes as 16 f16 values.
__device__ __forceinline__ void e4m3x16_f16(uint4 w, uint4 &lo, uint4 &hi) {
  const uint2 a = e4m3x4_f16(w.x), b = e4m3x4_f16(w.y), c = e4m3x4_f16(w.z), d = e4m3x4_f16(w.w);
  lo = make_uint4(a.x, a.y, b.x, b.y);
  hi = make_uint4(c.x, c.y, d.x, d.y);
}
// Bytes e >= n of a piece cleared.
__device__ __forceinline__ uint4 keep_bytes(uint4 w, int n) {
  uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int left = n - 4 * k;
    x[k] &= left >= 4 ? 0xffffffffu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
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
#pragma unroll
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
#pragma unroll
    for (int t = 0; t < 4; ++t)
      e2m1x32_tile(*reinterpret_cast<const uint4 *>(base + in * 64 + 16 * t), (t < 2 ? sf.x : sf.y) >> (16 * (t & 1)) & 0xffffu,
                   tile, tok, t);
  }
}

// Of the block's keys, row i of `rows` (those that attend the block) sees
// those up to first + i, no row one after last; all: every row of the item
// sees every key.
__device__ __forceinline__ uint32_t rows_that_see(int key, int first, uint32_t rows) {
  return key <= first ? rows : rows & ~((1u << min(key - first, 31)) - 1u);
}
__device__ __forceinline__ void note_nan(uint32_t (&nan_rows)[2][kHeadDim], int d, uint32_t rows) {
  atomicOr(&nan_rows[0][d], rows);
  atomicOr(&nan_rows[1][d], rows);
}
// Half (64 keys) of a block's values, by 128 threads: FP8 a dim each, NVFP4 two
// of the four 32-dim parts of a token each.
template <int FMT>
__device__ __forceinline__ void convert_v(const uint8_t *st, uint8_t *tile, int pt, int ct, int half, int first, int last,
                                          uint32_t rows, bool all, uint32_t (&nan_rows)[2][kHeadDim]) {
  if constexpr (FMT == 0) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int pg = 4 * half + k, d = ct;
      uint4 w = *reinterpret_cast<const uint4 *>(st + AttnStage<0>::kV + pg * 2048 + d * 16);
      if (!all) {
        if (last < 127) w = keep_bytes(w, last + 1 - 16 * pg);
        uint32_t x[4] = {w.x, w.y, w.z, w.w}, any = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) any |= (x[q] & 0x7f7f7f7fu) + 0x01010101u;  // bit 7 of a byte: its code is NaN
        if (any & 0x80808080u) {
          for (int e = 0; e < 16; ++e)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if ((e >> 2) == q && ((x[q] >> (8 * (e & 3))) & 0x7fu) == 0x7fu) {
                x[q] &= ~(0xffu << (8 * (e & 3)));
                note_nan(nan_rows, d, rows_that_see(16 * pg + e, first, rows));
              }
          w = make_uint4(x[0], x[1], x[2], x[3]);
        }
      }
      uint4 lo, hi;
      e4m3x16_f16(w, lo, hi);
      *reinterpret_cast<uint4 *>(tile + tile_at(d, 2 * pg)) = lo;
      *reinterpret_cast<uint4 *>(tile + tile_at(d, 2 * pg + 1)) = hi;
    }
  } else {
    const int tok = 64 * half + (ct & 63), in = tok & (pt - 1);
    const uint8_t *base = st + (tok - in) * 144 + pt * 72;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int t = 2 * (ct >> 6) + k;
      uint4 w = *reinterpret_cast<const uint4 *>(base + in * 64 + 16 * t);
      const uint8_t *sf = base + pt * 64 + (in >> 2) * 32 + 8 * t + (in & 3);
      uint32_t sf2 = (uint32_t)sf[0] | ((uint32_t)sf[4] << 8);
      if (!all) {
        if (tok > last) w = make_uint4(0, 0, 0, 0), sf2 = 0;
#pragma unroll
        for (int g = 0; g < 2; ++g)
          if (((sf2 >> (8 * g)) & 0x7fu) == 0x7fu) {
            sf2 &= ~(0xffu << (8 * g));
            for (int d = 32 * t + 16 * g; d < 32 * t + 16 * g + 16; ++d) note_nan(nan_rows, d, rows_that_see(tok, first, rows));
          }
      }
      e2m1x32_tile(w, sf2, tile, tok, t);
    }
  }
}

template <int FMT>
__global__ void __launch_bounds__(kTcThreads, 1) pa_attn_tc_kernel(const __grid_constant__ AttnMaps maps,
                                                                   const __grid_constant__ CacheAttnParams a) {
  using St = AttnStage<FMT>;
  using Sm = TcSmem<FMT>;
  static_assert(Sm::kBytes <= kAtSmem && Sm::kStages >= 2, "shared memory of a CTA");
  constexpr int kStages = Sm::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *k_tile = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t *v_tile = k_tile + kTcTile, *p_tile = v_tile + kTcTile, *q_tile = p_tile + kTcTile, *ring = q_tile + kTcTile;
  TcShared<FMT> &sh = *reinterpret_cast<TcShared<FMT> *>(ring + kStages * St::kBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_trigger();
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 8);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sh.batch_full[s], 1);
      mbar_init(&sh.batch_empty[s], 1);
      mbar_init(&sh.s_full[s], 1);
      mbar_init(&sh.s_empty[s], 8);
    }
    mbar_init(&sh.k_full, 4);
    mbar_init(&sh.k_empty, 1);
    for (int h = 0; h < 2; ++h) {
      mbar_init(&sh.v_full[h], 4);
      mbar_init(&sh.v_empty[h], 1);
    }
    mbar_init(&sh.v_end, 4);
    mbar_init(&sh.p_full, 8);
    mbar_init(&sh.pv_done, 1);
    mbar_init(&sh.seg_done, 8);
    mbar_init(&sh.never, 1);
    mbar_init(&sh.drain, 1);
    sh.dead = 0;
    fence_mbar_init();
  }
  if (tid < 4 * kHeadDim) (&sh.nan_rows[0][0][0])[tid] = 0;
  const AttnSlice sl = attn_slice<8>(a, sh, a.mode);
  if (sl.none) return;
  if (warp == 19) tc_alloc(&sh.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  // S: columns 0 and 128; O, 16 columns a row; each key's thread's sums of the weights, as many
  constexpr uint32_t kOCol = 256, kLCol = 384;
  const int pt = min(a.bs, 128);

  if (warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTcCtlRegs));
    if (warp == 16 && lane == 0) attn_copies<FMT, kStages, false>(a, maps, sh, sl, ring, nullptr);
    if (warp == 17) attn_resolve<FMT>(a, sh, sl, a.mode);
    if (warp == 18 && lane == 0) {
      // ------------------------------------------------------------ the MMAs
      // K and Q: rows are keys, (row, head)s.  V: rows are dims (FP8: pages hold
      // a dim's keys together) or keys (NVFP4).  P: rows are keys
      const uint64_t kd = sdesc_sw128(smem_u32(k_tile)), qd = sdesc_sw128(smem_u32(q_tile)), pd = sdesc_mn(smem_u32(p_tile));
      const uint64_t vd = FMT == 0 ? sdesc_sw128(smem_u32(v_tile)) : sdesc_mn(smem_u32(v_tile));
      bool ok = true;
      uint32_t n = 0, np = 0, ends = 0;  // entries, blocks whose PV is issued, segments ended
      int v0, v1, v;
      for (int it = sl.first; ok && sl.segment(a, sh, it, v0, v1, v); ++it) {
        const int rows = attn_place(a, it).rows;
        const uint32_t ids = idesc_f16(128, 16 * rows, 0, 0), idp = idesc_f16(128, 16 * rows, FMT == 0 ? 0 : 1, 1);
        // S of entry n and O of the block before it, whichever can go first; O
        // by halves of 64 keys
        bool pending = false, begun = false, more = true;
        while (ok && more) {
          bool s_out = false;
          int halves = pending ? 0 : 2;
          const uint64_t t0 = globaltimer();
          while (!s_out || halves < 2) {
            bool moved = false;
            if (halves < 2 && mbar_try_wait(smem_u32(&sh.v_full[halves]), np & 1) &&
                (halves == 1 || mbar_try_wait(smem_u32(&sh.p_full), np & 1))) {
              tc_fence_after();
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int kk = 4 * halves + k;
                mma_f16_ss(tmem + kOCol, vd + (FMT == 0 ? step_k(kk) : step_mn(kk)), pd + step_mn(kk), idp,
                           (begun || k > 0) ? 1u : 0u);
              }
              begun = true;
              if (halves == 1) tc_commit(&sh.pv_done);
              tc_commit(&sh.v_empty[halves]);
              ++halves;
              moved = true;
            }
            if (!s_out && mbar_try_wait(smem_u32(&sh.k_full), n & 1) &&
                mbar_try_wait(smem_u32(&sh.s_empty[n & 1]), ((n >> 1) & 1) ^ 1)) {
              more = sh.info[n % kAtInfo].x >= 0;
              if (more) {
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < 8; ++k) mma_f16_ss(tmem + (n & 1) * 128, kd + step_k(k), qd + step_k(k), ids, k > 0);
                tc_commit(&sh.s_full[n & 1]);
                tc_commit(&sh.k_empty);
              }
              s_out = true;
              moved = true;
            }
            if (!moved && globaltimer() - t0 > a.lim) {
              set_status(a.status, kDevWaitTimeout);
              ok = false;
              break;
            }
          }
          if (!ok) break;
          if (pending) ++np;
          pending = more;
          if (!more) {  // the end of the segment: the softmax groups read O
            if (!(ok = mbar_wait(&sh.v_end, ends & 1, a.status, a.lim))) break;
            ++ends;
            tc_commit(&sh.s_full[n & 1]);
            tc_commit(&sh.k_empty);
          }
          ++n;
        }
      }
      if (!ok) {  // the MMAs issued complete before the tensor memory is freed
        tc_commit(&sh.drain);
        mbar_wait(&sh.drain, 0, a.status, a.lim);
      }
    }
  } else if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTcConvRegs));
    // ---------------------------------------------------------- converters
    const int ct = tid & 127, cw = warp & 3;
    uint32_t j = 0, seg = 0;  // entries, segments
    bool ok = true;
    auto all_got = [&](bool got) { return ok = __all_sync(0xffffffffu, got) != 0; };
    int v0, v1, v;
    if (warp < 12) {
      // keys and queries.  A (row, head)'s 64 dims a thread, two threads each:
      // rows cw and cw + 4, the first asked for a segment ahead
      uint4 qr[8];
      AttnItem nx;
      const int qhead = lane >> 1, qd0 = 64 * (lane & 1);
      auto ask = [&](int row) {
        const bool have = row < nx.rows && qhead < a.group;
        const int64_t at = ((int64_t)nx.r * a.q_len + nx.row0 + row) * a.q_stride + (int64_t)(nx.h * a.group + qhead) * kHeadDim + qd0;
        const uint4 *src = reinterpret_cast<const uint4 *>(a.q + (a.q_is_fp8 ? at : 2 * at));
#pragma unroll
        for (int k = 0; k < 8; ++k) qr[k] = have && (k < 4 || !a.q_is_fp8) ? __ldg(src + k) : make_uint4(0, 0, 0, 0);
      };
      auto look_up = [&](int it) {
        bool bad = false;
        nx = attn_item(a, it, &bad);
        ask(cw);
        if (cw + 4 < nx.rows && qhead < a.group)
          prefetch_l2(a.q + (((int64_t)nx.r * a.q_len + nx.row0 + cw + 4) * a.q_stride +
                             (int64_t)(nx.h * a.group + qhead) * kHeadDim + qd0) * (a.q_is_fp8 ? 1 : 2));
      };
      // f16 values into the tile: a (row, head) a row of it
      auto lay_out_row = [&](int row, uint32_t sg) {
        float top = 0.f;
        auto values = [&](int k, float (&x)[8]) {  // dims qd0 + 8 k .. + 7
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
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float x[8];
          values(k, x);
#pragma unroll
          for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[e]));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int ex = max(exponent_of(top), -110) - 14;
        const float down = pow2i(-ex);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float x[8];
          values(k, x);
          *reinterpret_cast<uint4 *>(q_tile + tile_at(row * 16 + qhead, (qd0 >> 3) + k)) =
              make_uint4(f16x2_bits(x[0] * down, x[1] * down), f16x2_bits(x[2] * down, x[3] * down),
                         f16x2_bits(x[4] * down, x[5] * down), f16x2_bits(x[6] * down, x[7] * down));
        }
        if (lane == 0) sh.row_scale[sg & 1][row] = a.score_scale * pow2i(ex);
      };
      auto lay_out = [&](uint32_t sg) {
#pragma unroll 1
        for (int row = cw; row < nx.rows; row += 4) {
          if (row >= 4) ask(row);
          lay_out_row(row, sg);
        }
        if (ct == 0) sh.first[sg & 1] = nx.first;
      };
      if (sl.segment(a, sh, sl.first, v0, v1, v)) {
        look_up(sl.first);
        lay_out(0);
      }
      for (int it = sl.first; ok && sl.segment(a, sh, it, v0, v1, v); ++it, ++seg) {
        int w0, w1, w;
        const bool next = sl.segment(a, sh, it + 1, w0, w1, w);
        if (next) look_up(it + 1);
        for (bool more = true; more; ++j) {
          const int s = j % kStages;
          if (!all_got(mbar_wait(&sh.full[s], (j / kStages) & 1, a.status, a.lim) &&
                       mbar_wait(&sh.k_empty, (j & 1) ^ 1, a.status, a.lim)))
            break;
          more = sh.info[j % kAtInfo].x >= 0;
          if (more) {
            const uint8_t *st = ring + s * St::kBytes;
            convert_k<FMT>(st, k_tile, pt, ct);
            if constexpr (FMT == 0) {
              sh.scales[j & 3][0][ct] = *reinterpret_cast<const float *>(st + St::kKs + 4 * ct);
              sh.scales[j & 3][1][ct] = *reinterpret_cast<const float *>(st + St::kVs + 4 * ct);
            }
          } else if (next) {
            // the segment before this one is out: its scales may be replaced
            if (seg > 0 && !all_got(mbar_wait(&sh.seg_done, (seg - 1) & 1, a.status, a.lim))) break;
            lay_out(seg + 1);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sh.k_full);
            mbar_arrive(&sh.empty[s]);
          }
        }
      }
    } else {
      // values
      uint32_t nv = 0;  // blocks
      for (int it = sl.first; ok && sl.segment(a, sh, it, v0, v1, v); ++it, ++seg) {
        bool bad = false;
        const AttnItem x = attn_item(a, it, &bad);
        const int every = (1 << x.rows) - 1;
        for (bool more = true; more; ++j) {
          const int s = j % kStages;
          if (!all_got(mbar_wait(&sh.full[s], (j / kStages) & 1, a.status, a.lim))) break;
          const int2 info = sh.info[j % kAtInfo];
          more = info.x >= 0;
          if (more) {
            const int first = x.first - info.x * 128;
            for (int half = 0; ok && half < 2; ++half) {
              if (!all_got(mbar_wait(&sh.v_empty[half], (nv & 1) ^ 1, a.status, a.lim))) break;
              convert_v<FMT>(ring + s * St::kBytes, v_tile, pt, ct, half, first, first + x.rows - 1, (uint32_t)info.y,
                             info.y == every && first >= 127, sh.nan_rows[seg & 1]);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(&sh.v_full[half]);
            }
            if (!ok) break;
            ++nv;
          } else if (seg > 0 && !all_got(mbar_wait(&sh.seg_done, (seg - 1) & 1, a.status, a.lim))) {
            break;
          }
          __syncwarp();
          if (lane == 0) {
            if (!more) mbar_arrive(&sh.v_end);
            mbar_arrive(&sh.empty[s]);
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTcSoftRegs));
    // ------------------------------------------------------------- softmax
    const int grp = warp >> 2, gw = warp & 3, key = 32 * gw + lane, bar = 1 + grp;
    const uint32_t lanes = tmem + ((uint32_t)(32 * gw) << 16);
    uint32_t n = 0, np = 0, seg = 0;  // entries, blocks, segments
    bool dead = false, live = true;
    auto wait = [&](uint64_t *b, uint32_t parity) {  // after the first that runs out, none waits
      if (!dead) dead = !__all_sync(0xffffffffu, mbar_wait(b, parity, a.status, a.lim));
    };
    int v0, v1, v;
    for (int it = sl.first; live && sl.segment(a, sh, it, v0, v1, v); ++it, ++seg) {
      const AttnItem x = attn_place(a, it);
      {
        float zero[16];
#pragma unroll
        for (int h = 0; h < 16; ++h) zero[h] = 0.f;
        for (int row = grp; row < x.rows; row += 2) tc_st16(lanes + kLCol + 16 * row, zero);
        tc_wait_st();
      }
      if ((tid & 127) < 64) {
        const int row = 2 * ((tid & 127) >> 4) + grp;
        sh.off[row][tid & 15] = 1e30f;  // any score is above the limit: the first sets m
        sh.m[row][tid & 15] = -INFINITY;
      }
      if (bar_any(bar, dead)) break;
      int ev = -126;
      float vlimit = pow2i(-125), unit = pow2i(126);
      while (true) {
        wait(&sh.s_full[n & 1], (n >> 1) & 1);
        if (a.test_timeout) wait(&sh.never, 0);
        tc_fence_after();
        if (bar_any(bar, dead)) {  // (also: all of the group see the entry before it can be reused)
          live = false;
          break;
        }
        const int2 info = sh.info[n % kAtInfo];
        if (info.x < 0) break;
        const int first = sh.first[seg & 1];
        const int kj = info.x * 128 + key;
        float ks = 1.f, vs = 1.f;
        if constexpr (FMT == 0) ks = sh.scales[n & 3][0][key], vs = sh.scales[n & 3][1][key];
        bool waited = false;
#pragma unroll 1
        for (int row = grp; row < x.rows; row += 2) {
          uint4 *p0 = reinterpret_cast<uint4 *>(p_tile + tile_at(key, 2 * row)), *p1 = reinterpret_cast<uint4 *>(p_tile + tile_at(key, 2 * row + 1));
          if (!((info.y >> row) & 1)) {  // the row does not attend the block
            if (!waited) wait(&sh.pv_done, (np & 1) ^ 1), waited = true;
            *p0 = *p1 = make_uint4(0, 0, 0, 0);
            continue;
          }
          float s[16], y[16], l[16];
          tc_ld16(lanes + (n & 1) * 128 + 16 * row, s);
          tc_ld16(lanes + kLCol + 16 * row, l);
          const bool seen = kj <= first + row;
          const float kk = ks * sh.row_scale[seg & 1][row];
          tc_wait_ld();
          auto scores = [&]() {
            float top = -INFINITY;
            const float4 *of = reinterpret_cast<const float4 *>(sh.off[row]);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float4 o4 = of[q];
              y[4 * q] = seen ? fmaf(s[4 * q], kk, o4.x) : -INFINITY;
              y[4 * q + 1] = seen ? fmaf(s[4 * q + 1], kk, o4.y) : -INFINITY;
              y[4 * q + 2] = seen ? fmaf(s[4 * q + 2], kk, o4.z) : -INFINITY;
              y[4 * q + 3] = seen ? fmaf(s[4 * q + 3], kk, o4.w) : -INFINITY;
              top = fmaxf(top, fmaxf(fmaxf(y[4 * q], y[4 * q + 1]), fmaxf(y[4 * q + 2], y[4 * q + 3])));
            }
            return top;
          };
          const float top = scores();
          const float va = FMT == 0 && seen ? fabsf(vs) : 0.f;
          if (bar_any(bar, top > kAtLift + kAtSlack || (FMT == 0 && va > vlimit))) {
            // m of the row's heads (and the V unit) move: the new maxima over
            // all keys of the block, then o and the sums are scaled
            if (!waited) wait(&sh.pv_done, (np & 1) ^ 1), waited = true;
            tc_fence_after();
#pragma unroll
            for (int h = 0; h < 16; ++h) {
              const float t = warp_max(seen ? s[h] * kk : -INFINITY);
              if (lane == h) sh.warp_max[grp][gw][h] = t;
            }
            if constexpr (FMT == 0) {
              const float t = warp_max(va);
              if (lane == 16) sh.warp_max[grp][gw][16] = t;
            }
            dead |= bar_any(bar, dead);
            float f = 1.f;
            if constexpr (FMT == 0) {
              float t = 0.f;
#pragma unroll
              for (int w = 0; w < 4; ++w) t = fmaxf(t, sh.warp_max[grp][w][16]);
              const int e2 = max(ev, min(exponent_of(t), 126));
              f = e2 - ev > 125 ? 0.f : pow2i(ev - e2);
              ev = e2;
              vlimit = pow2i(ev + 1), unit = pow2i(-ev);
            }
            float o[16];
            if (f != 1.f) {  // the group's other rows
#pragma unroll 1
              for (int r2 = grp; r2 < x.rows; r2 += 2) {
                if (r2 == row) continue;
                tc_ld16(lanes + kOCol + 16 * r2, o);
                tc_wait_ld();
#pragma unroll
                for (int h = 0; h < 16; ++h) o[h] *= f;
                tc_st16(lanes + kOCol + 16 * r2, o);
              }
            }
            tc_ld16(lanes + kOCol + 16 * row, o);
            tc_wait_ld();
            float nm = -INFINITY;
#pragma unroll
            for (int h = 0; h < 16; ++h) {
              const float was = sh.m[row][h];
              float t = was;
#pragma unroll
              for (int w = 0; w < 4; ++w) t = fmaxf(t, sh.warp_max[grp][w][h]);
              const float al = t == was ? 1.f : ex2_approx(was - t);
              l[h] *= al;
              o[h] *= al * f;
              if ((tid & 127) == h) nm = t;
            }
            tc_st16(lanes + kOCol + 16 * row, o);
            tc_wait_st();
            tc_fence_before();
            dead |= bar_any(bar, dead);  // everyone has read the old m
            if ((tid & 127) < 16) {
              sh.m[row][tid & 15] = nm;
              sh.off[row][tid & 15] = nm == -INFINITY ? 1e30f : kAtLift - nm;
            }
            dead |= bar_any(bar, dead);
            scores();
          }
          if (!waited) wait(&sh.pv_done, (np & 1) ^ 1), waited = true;
          float wu = 1.f;
          if constexpr (FMT == 0) wu = seen ? vs * unit : 0.f;
          uint32_t w[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const float e0 = ex2_approx(y[2 * q]), e1 = ex2_approx(y[2 * q + 1]);
            l[2 * q] += e0, l[2 * q + 1] += e1;
            w[q] = f16x2_bits(FMT == 0 ? e0 * wu : e0, FMT == 0 ? e1 * wu : e1);
          }
          *p0 = make_uint4(w[0], w[1], w[2], w[3]);
          *p1 = make_uint4(w[4], w[5], w[6], w[7]);
          tc_st16(lanes + kLCol + 16 * row, l);
        }
        tc_wait_st();
        if (!waited) wait(&sh.pv_done, (np & 1) ^ 1);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sh.s_empty[n & 1]);
          mbar_arrive(&sh.p_full);
        }
        ++n, ++np;
      }
      if (!live) break;
      // ------------------------------------------------ the segment's result
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
      const float up = FMT == 0 ? pow2i(ev) : 1.f;
      const uint32_t nan_rows = sh.nan_rows[seg & 1][grp][key];  // this thread's dim is `key`
      sh.nan_rows[seg & 1][grp][key] = 0;
#pragma unroll 1
      for (int row = grp; row < x.rows; row += 2) {
        float l[16];
        tc_ld16(lanes + kLCol + 16 * row, l);
        tc_wait_ld();
#pragma unroll
        for (int h = 0; h < 16; ++h) {
          float t = l[h];
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
          if (lane == h) sh.warp_sum[grp][gw][h] = t;
        }
        dead |= bar_any(bar, dead);
        float o[16];
        tc_ld16(lanes + kOCol + 16 * row, o);
        tc_wait_ld();
        const int64_t m = (int64_t)x.r * a.q_len + x.row0 + row;
        const bool lost = (nan_rows >> row) & 1u;
#pragma unroll
        for (int h = 0; h < 16; ++h) {
          const float sum = ((sh.warp_sum[grp][0][h] + sh.warp_sum[grp][1][h]) + sh.warp_sum[grp][2][h]) + sh.warp_sum[grp][3][h];
          const float val = lost ? NAN : sum == 0.f ? 0.f : o[h] * up;  // (o holds nothing where no key came)
          if (h < a.group) {
            if (whole) {
              a.out[m * a.out_stride + (int64_t)(x.h * a.group + h) * kHeadDim + key] =
                  __float2bfloat16_rn(sum == 0.f ? 0.f : val * (a.out_scale / sum));
            } else {
              pp[(row * 16 + h) * kHeadDim + key] = val;
              if ((tid & 127) == h)
                *reinterpret_cast<float2 *>(pp + kAtMaxRows * 16 * kHeadDim + (row * 16 + h) * 2) = make_float2(sh.m[row][h], sum);
            }
          }
        }
        dead |= bar_any(bar, dead);  // warp_sum is free
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sh.s_empty[n & 1]);
        mbar_arrive(&sh.seg_done);
      }
      ++n;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 19) {
    tc_fence_after();
    tc_dealloc(tmem, 512);
  }
}

template <int FMT>
static cudaError_t launch_tc(const AttnMaps &maps, const CacheAttnParams &a, int grid, bool pdl, cudaStream_t stream) {
  auto kern = pa_attn_tc_kernel<FMT>;
  constexpr int smem = TcSmem<FMT>::kBytes;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(kern), smem);
  if (e != cudaSuccess) return e;
  static int regs = 0;
  if (regs == 0) {
    cudaFuncAttributes at;
    e = cudaFuncGetAttributes(&at, reinterpret_cast<const void *>(kern));
    if (e != cudaSuccess) return e;
    regs = at.numRegs;
  }
  if (regs * 5 < 2 * kTcSoftRegs + 2 * kTcConvRegs + kTcCtlRegs) return cudaErrorInvalidConfiguration;
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
  return cudaLaunchKernelEx(&cfg, kern, maps, a);
}

cudaError_t launch_attn_tc(int fmt, const AttnMaps &maps, const CacheAttnParams &a, int grid, bool pdl, cudaStream_t stream) {
  return fmt == 0 ? launch_tc<0>(maps, a, grid, pdl, stream) : launch_tc<1>(maps, a, grid, pdl, stream);
}

}  // namespace pa
