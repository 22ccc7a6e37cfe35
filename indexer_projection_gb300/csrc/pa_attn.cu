// Attention over the step's paged KV caches (pre_attn_attention): query rows
// r * q_len + i at positions p = seq_lens[r] - q_len + i against the keys
// j <= p of their blocks (a list per row and KV head, or all), FP8 pages
// ("vllm.models.minimax_m3.amd.mono.kernels.pre_attn", head tasks) or NVFP4
// pages ("vllm.models.minimax_m3.nvidia.ops.qkv_index_fused_epilogue",
// _nvfp4_cache_views):
//   out = sum_j exp2(s_j - m) v_j / sum_j exp2(s_j - m),
//   s_j = q . k_j * sm_scale * log2(e)
// with the running reference m of an online softmax.
//
// Work.  An item is (request, up to 8 of its rows, KV head): the rows share
// the key blocks, so a block is read from memory once for all rows that
// attend it.  A persistent grid (a CTA an SM) walks the list of all items'
// blocks in even contiguous slices; an item that several CTAs share leaves
// partial sums in the workspace and pa_attn_join_kernel adds them up.  A
// producer warp keeps a ring of 128-key blocks in flight with bulk copies;
// a query row's (up to 16) heads are the 16 rows of mma.sync m16n8k16, and
// the eight compute warps are dealt to the item's rows: WPR = 8, 4, 2 or 1
// warps a row, each with its part of the keys.
//
// Arithmetic.  E4M3 codes and E2M1 code x E4M3 scale are f16 values, so keys
// and values are converted exactly in registers and multiplied on the f16
// tensor path with f32 sums.  A query head row is scaled by a power of two to
// a maximum in [2^14, 2^15) first, so its bf16 values are f16 values too
// unless they are 2^-29 of that maximum or less.  The per-token K scale
// multiplies the score, the per-token V scale the weight.  A weight rounds to
// f16 (2^-12 relative) for the second product: it is 2^9 exp2(s - m) times
// the V scale over a power of two near the largest V scale so far, so it
// stays in f16's normal range for keys whose weight is up to 2^-23 of the
// largest.  The sum of the weights is taken in f32 before that rounding.
#include <cmath>
#include <cstdint>

#include <cuda_fp16.h>

#include "../../include/pre_attn.h"
#include "pa_device.cuh"
#include "pa_f16.cuh"
#include "pa_launch.h"
#include "pa_tma.h"

namespace pa {

constexpr int kAtWarps = 8;                        // compute warps
constexpr int kAtThreads = 32 * (kAtWarps + 4);    // and the producer's warpgroup (one warp of it works)
// Registers a thread after the split (setmaxnreg): the compute warps hold o,
// the queries and the codes of 32 keys.  Their sum must not exceed what the
// CTA was launched with, which launch_attn checks.
constexpr int kAtComputeRegs = 200, kAtProducerRegs = 96;
constexpr int kAtMaxRows = 8;                      // query rows an item
constexpr int kAtMaxItems = 2048;                  // items the sliced grid lists in shared memory
constexpr int kAtMaxWidth = 16384;                 // block-table width
constexpr int kAtMaxTopk = 256;
constexpr float kAtLift = 9.0f;   // weights are 2^9 exp2(s - m)
constexpr float kAtSlack = 4.0f;  // m follows the maximum once that is 2^4 above it
constexpr int kAtPartFloats = kAtMaxRows * 16 * (kHeadDim + 2);  // o, then (m, l), of one partial

struct AttnParams {
  const uint8_t *q;
  int q_is_fp8;
  int64_t q_stride;
  const uint8_t *k_cache, *v_cache;  // FP8
  const float *k_scale, *v_scale;
  int64_t num_pages16;
  int kps;
  const uint8_t *kv_cache;           // NVFP4
  int64_t kv_pages, kv_page_bytes;
  int bs;
  const int32_t *block_table, *seq_lens, *blocks, *counts;
  int topk;                          // 0: every block
  int R, q_len, bt_width, n_kv, group;
  int lg_kv, lg_groups;              // log2 of n_kv and of the items a (request, KV head) has
  int rows_per;                      // rows an item (the last of a request may have fewer)
  int items, sliced;
  float score_scale, out_scale;
  __nv_bfloat16 *out;
  int64_t out_stride;
  float *part;                       // [2 * grid][kAtPartFloats]
  int2 *shares;                      // [items] first and last CTA of an item
  uint32_t *status;
  uint64_t lim;
  int test_timeout;
};

// Tensor maps of a block's copies: FP8 K pages, V pages, K scales, V scales;
// NVFP4 a KV head's K and V slots (pages of up to 128 tokens).
struct AttnMaps {
  CUtensorMap m[4];
};

template <int FMT>
struct AttnStage;
template <>
struct AttnStage<0> {  // K and V pages as they are (8 of 2048 bytes each), then the scales of 128 tokens
  static constexpr int kV = 16384, kKs = 32768, kVs = 33280, kBytes = 33792;
  static constexpr int stages(bool joined) { return joined ? 4 : 5; }
};
template <>
struct AttnStage<1> {  // pieces of pt = min(block_size, 128) tokens: K codes (64 bytes a token), K scales (8), V codes,
                       // V scales, as the page holds them
  static constexpr int kBytes = 18432;
  static constexpr int stages(bool joined) { return joined ? 7 : 10; }
};

struct AttnShared {
  uint64_t full[10], empty[10];
  uint64_t fin;     // the compute warps, twice an item
  uint64_t never;   // testing: nothing arrives on it
  int2 info[10];    // block (-1: the end of an item), rows that attend it
  int scan[kAtWarps];
  float2 ml[kAtWarps][16];
  int offs[kAtMaxItems + 8];
  uint16_t list[kAtMaxRows * kAtMaxTopk];
  uint32_t bits[kAtMaxRows][kAtMaxWidth / 32];
};

template <int FMT, int WPR>
constexpr int attn_smem() {
  return AttnStage<FMT>::stages(WPR > 1) * AttnStage<FMT>::kBytes + (WPR > 1 ? kAtWarps * 16 * kHeadDim * 4 : 0) +
         (int)sizeof(AttnShared) + 128;
}
static_assert(attn_smem<0, 8>() <= 232448 && attn_smem<0, 1>() <= 232448 && attn_smem<1, 8>() <= 232448 &&
                  attn_smem<1, 1>() <= 232448,
              "a CTA has 227 KB of shared memory");

// An item's request, KV head and rows; its request is without keys when
// seq < 1, seq < q_len or its blocks exceed the table.
struct AttnItem {
  int r, h, row0, rows, seq, first;  // first: position of row row0
  __device__ int blocks_upto(int rows_) const { return seq > 0 ? (first + rows_ - 1) / 128 + 1 : 0; }
};
__device__ __forceinline__ AttnItem attn_item(const AttnParams &a, int it, bool *bad) {
  AttnItem x;
  x.h = it & (a.n_kv - 1);
  const int rg = it >> a.lg_kv;
  x.r = rg >> a.lg_groups;
  x.row0 = (rg - (x.r << a.lg_groups)) * a.rows_per;
  x.rows = min(a.rows_per, a.q_len - x.row0);
  x.seq = __ldg(a.seq_lens + x.r);
  if (x.seq > 0 && (x.seq < a.q_len || (x.seq - 1) / 128 + 1 > a.bt_width)) {
    *bad = true;
    x.seq = 0;
  }
  if (x.seq < 0) x.seq = 0;
  x.first = x.seq - a.q_len + x.row0;
  return x;
}
// The share of the grid's work that an item stands for (at least one unit):
// its blocks, or the length of its rows' lists (whose union the producer
// scales to it).
__device__ __forceinline__ int attn_units(const AttnParams &a, int it, bool *bad) {
  const AttnItem x = attn_item(a, it, bad);
  if (x.seq == 0) return 1;
  if (a.topk == 0) return x.blocks_upto(x.rows);
  int n = 0;
  const int32_t *c = a.counts + ((int64_t)x.r * a.q_len + x.row0) * a.n_kv + x.h;
#pragma unroll
  for (int i = 0; i < kAtMaxRows; ++i)
    if (i < x.rows) n += min(max(__ldg(c + i * a.n_kv), 0), a.topk);
  return max(n, 1);
}

// The CTA's slice as segments: item it, units v0 .. v1 of its v.
struct AttnSlice {
  int lo, hi, total, cta, ctas;
};

__device__ __forceinline__ void tma_pages(uint32_t dst, const CUtensorMap *map, int row, int page, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(page), "r"(smem_u32(bar))
      : "memory");
}

template <int FMT, int WPR>
__global__ void __launch_bounds__(kAtThreads, 1) pa_attn_kernel(const __grid_constant__ AttnMaps maps,
                                                                const __grid_constant__ AttnParams a) {
  using St = AttnStage<FMT>;
  constexpr int kStages = St::stages(WPR > 1);
  // a warp takes 32 keys at least: with eight warps a row, two groups of four
  // take alternate blocks
  constexpr int kParts = WPR > 4 ? 4 : WPR, kGroups = WPR / kParts, kKeys = 128 / kParts;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = smem_raw + ((128 - (smem_u32(smem_raw) & 127)) & 127);
  float *joint = reinterpret_cast<float *>(ring + kStages * St::kBytes);  // [warp][16 heads][128], WPR > 1
  AttnShared &sh = *reinterpret_cast<AttnShared *>(ring + kStages * St::kBytes +
                                                   (WPR > 1 ? kAtWarps * 16 * kHeadDim * 4 : 0));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  pdl_wait();  // queries, caches and lists come from the previous kernels
  pdl_trigger();
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], kAtWarps);
    }
    mbar_init(&sh.fin, kAtWarps);
    mbar_init(&sh.never, 1);
    fence_mbar_init();
  }
  AttnSlice sl;
  sl.cta = blockIdx.x;
  int first_item = blockIdx.x;
  if (a.sliced) {
    // the running sums of the items' units, 256 items a round
    int before = 0;
    bool bad = false;
    for (int i0 = 0; i0 < a.items; i0 += 32 * kAtWarps) {
      const int it = i0 + tid;
      const int n = warp < kAtWarps && it < a.items ? attn_units(a, it, &bad) : 0;
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (warp < kAtWarps && lane == 31) sh.scan[warp] = incl;
      __syncthreads();
      int round = 0, mine = before + incl - n;
#pragma unroll
      for (int w = 0; w < kAtWarps; ++w) {
        const int v = sh.scan[w];
        if (w < warp) mine += v;
        round += v;
      }
      if (warp < kAtWarps) sh.offs[it] = mine;
      before += round;
      __syncthreads();
    }
    if (tid == 0) sh.offs[a.items] = before;
    if (blockIdx.x == 0 && bad) set_status(a.status, kDevSlotRange);
    __syncthreads();
    sl.total = sh.offs[a.items];
    sl.ctas = min((int)gridDim.x, sl.total);
    if (sl.cta >= sl.ctas) return;
    sl.lo = (int)((int64_t)sl.total * sl.cta / sl.ctas);
    sl.hi = (int)((int64_t)sl.total * (sl.cta + 1) / sl.ctas);
    first_item = 0;
    for (int step = kAtMaxItems / 2; step > 0; step >>= 1)
      if (first_item + step < a.items && sh.offs[first_item + step] <= sl.lo) first_item += step;
  } else {
    sl.total = sl.ctas = 0;
    sl.lo = 0;
    sl.hi = 1;
    __syncthreads();
  }
  // segment k of the slice: its item's units v0 .. v1 of v
  auto segment = [&](int it, int &v0, int &v1, int &v) {
    if (!a.sliced) {
      v0 = 0;
      v1 = v = 1;
      return it == first_item;
    }
    if (it >= a.items || sh.offs[it] >= sl.hi) return false;
    v0 = max(sl.lo, sh.offs[it]) - sh.offs[it];
    v1 = min(sl.hi, sh.offs[it + 1]) - sh.offs[it];
    v = sh.offs[it + 1] - sh.offs[it];
    return true;
  };

  if (warp >= kAtWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kAtProducerRegs));
    if (warp > kAtWarps) return;
    // -------------------------------------------------------------- producer
    int j = 0;
    bool ok = true;
    auto acquire = [&]() {  // stage j % kStages is free (lane 0's answer for the warp)
      bool got = true;
      if (lane == 0) got = mbar_wait(&sh.empty[j % kStages], ((uint32_t)(j / kStages) & 1) ^ 1, a.status, a.lim);
      return __shfl_sync(0xffffffffu, got, 0) != 0;
    };
    int v0, v1, v;
    for (int it = first_item; ok && segment(it, v0, v1, v); ++it) {
      bool bad = false;
      const AttnItem x = attn_item(a, it, &bad);
      if (!a.sliced && bad && lane == 0) set_status(a.status, kDevSlotRange);
      const int nb = x.blocks_upto(x.rows);
      int u0 = 0, u1 = 0;  // the segment's blocks (of the union list, or of the request)
      if (a.topk == 0) {
        u0 = (int)((int64_t)nb * v0 / v);
        u1 = (int)((int64_t)nb * v1 / v);
      } else if (nb > 0) {
        // the rows' lists as bit sets over the request's blocks, then the
        // union's blocks u0 .. u1 in ascending order
        const int words = (nb + 31) / 32;
        __syncwarp();
        for (int i = 0; i < x.rows; ++i)
          for (int w = lane; w < words; w += 32) sh.bits[i][w] = 0;
        const int64_t at = ((int64_t)x.r * a.q_len + x.row0) * a.n_kv + x.h;
        int count[kAtMaxRows];
#pragma unroll
        for (int i = 0; i < kAtMaxRows; ++i) count[i] = i < x.rows ? __ldg(a.counts + at + i * a.n_kv) : 0;
        bool out_of_range = false;
        for (int e0 = 0; e0 < a.topk; e0 += 32) {
          int b[kAtMaxRows];
          const bool in = e0 + lane < a.topk;
#pragma unroll
          for (int i = 0; i < kAtMaxRows; ++i)
            b[i] = in && i < x.rows ? __ldg(a.blocks + (at + i * a.n_kv) * a.topk + e0 + lane) : 0;
          __syncwarp();
#pragma unroll
          for (int i = 0; i < kAtMaxRows; ++i)
            if (in && e0 + lane < count[i]) {
              if (b[i] < 0 || b[i] > (x.first + i) / 128) out_of_range = true;
              else atomicOr(&sh.bits[i][b[i] >> 5], 1u << (b[i] & 31));
            }
        }
        if (__any_sync(0xffffffffu, out_of_range) && lane == 0) set_status(a.status, kDevSlotRange);
        __syncwarp();
        int total = 0;
        for (int w = lane; w < words; w += 32) {
          uint32_t u = 0;
          for (int i = 0; i < x.rows; ++i) u |= sh.bits[i][w];
          total += __popc(u);
        }
        total = __reduce_add_sync(0xffffffffu, total);
        u0 = (int)((int64_t)total * v0 / v);
        u1 = (int)((int64_t)total * v1 / v);
        int before = 0;
        for (int w0 = 0; w0 < words; w0 += 32) {
          uint32_t u = 0;
          if (w0 + lane < words)
            for (int i = 0; i < x.rows; ++i) u |= sh.bits[i][w0 + lane];
          int incl = __popc(u);
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
          }
          int at = before + incl - __popc(u);
          before += __shfl_sync(0xffffffffu, incl, 31);
          for (; u; u &= u - 1, ++at)
            if (at >= u0 && at < u1) sh.list[at - u0] = (uint16_t)(32 * (w0 + lane) + __ffs(u) - 1);
        }
        __syncwarp();
      }
      for (int base = u0; ok && base < u1; base += 32) {
        // 32 blocks at a time, one a lane: their ids and the rows they serve
        int b = -1, rows = 0;
        int64_t blk = -1;
        if (base + lane < u1) {
          b = a.topk ? sh.list[base + lane - u0] : base + lane;
          for (int i = 0; i < x.rows; ++i)
            if (a.topk ? (sh.bits[i][b >> 5] >> (b & 31)) & 1u : b <= (x.first + i) / 128) rows |= 1 << i;
          blk = __ldg(a.block_table + (int64_t)x.r * a.bt_width + b);
          const bool in = FMT == 0 ? blk >= 0 && blk * a.kps + 8 <= a.num_pages16
                                   : blk >= 0 && (blk + 1) * 128 <= a.kv_pages * a.bs;
          if (!in) {
            blk = -1;
            set_status(a.status, kDevSlotRange);
          }
        }
        const int m = min(32, u1 - base);
        for (int k = 0; k < m; ++k) {
          const int64_t id = __shfl_sync(0xffffffffu, blk, k);
          const int bk = __shfl_sync(0xffffffffu, b, k), rk = __shfl_sync(0xffffffffu, rows, k);
          if (id < 0) continue;
          if (!(ok = acquire())) break;
          const int s = j % kStages;
          uint64_t *bar = &sh.full[s];
          uint8_t *st = ring + s * St::kBytes;
          if (lane == 0) {
            sh.info[s] = make_int2(bk, rk);
            mbar_expect_tx(bar, St::kBytes);
          }
          __syncwarp();
          if constexpr (FMT == 0) {  // the block's 8 pages of the head: K, V, their scales
            if (lane < 4) {
              const int off = lane == 0 ? 0 : lane == 1 ? St::kV : lane == 2 ? St::kKs : St::kVs;
              tma_pages(smem_u32(st + off), &maps.m[lane], x.h, (int)(id * a.kps), bar);
            }
          } else if (a.bs <= 128) {  // the head's K and V slots of 128 / bs pages
            if (lane == 0)
              tma_pages(smem_u32(st), &maps.m[0], 2 * x.h * max(a.bs >> 4, 1), (int)(id * (128 / a.bs)), bar);
          } else if (lane < 4) {  // 128 tokens within a page: K codes, K scales, V codes, V scales
            const int v2 = lane >> 1, sf = lane & 1;
            const int64_t page = id * 128 / a.bs;
            const int t0 = (int)(id * 128 - page * a.bs);
            const uint8_t *base8 = a.kv_cache + page * a.kv_page_bytes + (int64_t)(2 * x.h + v2) * a.bs * 72;
            bulk_g2s(st + v2 * 9216 + sf * 8192, base8 + (sf ? a.bs * 64 + t0 * 8 : t0 * 64), sf ? 1024 : 8192, bar);
          }
          ++j;
        }
      }
      if (ok && (ok = acquire())) {  // the end of the segment
        if (lane == 0) {
          sh.info[j % kStages] = make_int2(-1, 0);
          mbar_arrive(&sh.full[j % kStages]);
        }
        ++j;
      }
      __syncwarp();
    }
    // the copies issued land before the CTA exits
    if (lane == 0)
      for (int k = j - 1; k >= 0 && k >= j - kStages; --k)
        mbar_wait(&sh.full[k % kStages], (uint32_t)(k / kStages) & 1, a.status, a.lim);
    return;
  }

  // ----------------------------------------------------------------- compute
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kAtComputeRegs));
  const int row = warp / WPR, part = warp % WPR;
  const int key0 = part % kParts * kKeys;
  const int pt = min(a.bs, 128);  // NVFP4: tokens a piece of a stage
  int j = 0;
  uint32_t fin_phase = 0;
  auto fin_sync = [&]() {  // all compute warps; bounded
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.fin);
    const bool got = mbar_wait(&sh.fin, fin_phase, a.status, a.lim);
    fin_phase ^= 1;
    return __all_sync(0xffffffffu, got) != 0;
  };
  int v0, v1, v;
  for (int it = first_item; segment(it, v0, v1, v); ++it) {
    bool bad = false;
    const AttnItem x = attn_item(a, it, &bad);
    const bool live = row < x.rows && x.seq > 0;
    const int p = x.first + row;
    // the row's queries as A fragments: heads g and g + 8, k-step ks holding
    // dims dim0(ks) .. + 3 of this thread (an order of the dims that the key
    // fragments follow: 16 ks + 4 t for FP8 pages, 32 t + 4 ks for NVFP4)
    uint32_t qf[8][4];
    float sc[2];  // score = product * sc (* the key's scale)
    {
      float qv[2][32];
      const int64_t m = (int64_t)x.r * a.q_len + x.row0 + row;
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int head = g + 8 * hh;
        const bool have = live && head < a.group;
        const int64_t at = m * a.q_stride + (int64_t)(x.h * a.group + head) * kHeadDim;
        float top = 0.f;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          const int d = FMT == 0 ? 16 * ks + 4 * t : 32 * t + 4 * ks;
          if (a.q_is_fp8) {
            const uint32_t w = have ? __ldg(reinterpret_cast<const uint32_t *>(a.q + at + d)) : 0u;
            const uint2 h2 = e4m3x4_f16(w);
            const float2 f0 = __half22float2(*reinterpret_cast<const __half2 *>(&h2.x));
            const float2 f1 = __half22float2(*reinterpret_cast<const __half2 *>(&h2.y));
            qv[hh][4 * ks] = f0.x, qv[hh][4 * ks + 1] = f0.y, qv[hh][4 * ks + 2] = f1.x, qv[hh][4 * ks + 3] = f1.y;
          } else {
            const uint2 w = have ? __ldg(reinterpret_cast<const uint2 *>(a.q + 2 * (at + d))) : make_uint2(0u, 0u);
            qv[hh][4 * ks] = bf16_to_f32(w.x & 0xffffu), qv[hh][4 * ks + 1] = bf16_to_f32(w.x >> 16);
            qv[hh][4 * ks + 2] = bf16_to_f32(w.y & 0xffffu), qv[hh][4 * ks + 3] = bf16_to_f32(w.y >> 16);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(qv[hh][4 * ks + e]));
        }
        const int ex = max(exponent_of(quad_max(top)), -110) - 14;
        sc[hh] = a.score_scale * pow2i(ex);
        const float down = pow2i(-ex);
#pragma unroll
        for (int e = 0; e < 32; ++e) qv[hh][e] *= down;
      }
#pragma unroll
      for (int ks = 0; ks < 8; ++ks)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          qf[ks][hh] = f16x2_bits(qv[hh][4 * ks], qv[hh][4 * ks + 1]);
          qf[ks][2 + hh] = f16x2_bits(qv[hh][4 * ks + 2], qv[hh][4 * ks + 3]);
        }
    }
    float o[16][4];  // n8 tile n: FP8 dims 8 n + 2 t + e, NVFP4 dims 16 (2 t + e) + n; heads g (0, 1) and g + 8 (2, 3)
#pragma unroll
    for (int n = 0; n < 16; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
    float mref[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    int ev = -126;  // FP8: o is in units of 2^ev, V scales up to 2^(ev + 1) = vlimit
    float vlimit = pow2i(-125);
    while (true) {
      const int s = j % kStages;
      bool got = mbar_wait(&sh.full[s], (uint32_t)(j / kStages) & 1, a.status, a.lim);
      if (got && a.test_timeout) got = mbar_wait(&sh.never, 0, a.status, a.lim);
      if (!__all_sync(0xffffffffu, got)) return;  // the warp gives up; the others' waits are bounded too
      const int2 info = sh.info[s];
      ++j;
      if (info.x >= 0 && ((info.y >> row) & 1) && (kGroups == 1 || (j & (kGroups - 1)) == part / kParts)) {
        const uint8_t *st = ring + s * St::kBytes;
        const bool cut = info.x * 128 + 127 > p;  // keys after the row's position
#pragma unroll 1
        for (int k0 = key0; k0 < key0 + kKeys; k0 += 32) {
          // scores of 32 keys: this thread's are keys k0 + 16 y + 4 t + (e + rot) % 4, y = 0, 1, e = 0 .. 3
          float c[4][4];
#pragma unroll
          for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) c[nt][e] = 0.f;
          float sv[2][8];     // [head g, g + 8][4 y + e]
          uint32_t vraw[32];  // the value codes of those keys, read before the softmax needs its results
          uint32_t vsf[2];
          if constexpr (FMT == 0) {
            // a page is [8 chunks of 16 dims][16 tokens][16 bytes].  Column n
            // of tile nt is key 4 (n / 2) + 2 (nt ^ n / 4) + n % 2: the eight
            // rows of each 8x8 tile then sit in distinct banks
            const int n = lane & 7, nt = (lane >> 3) & 1;
            const int tok = 4 * (n >> 1) + 2 * (nt ^ (n >> 2)) + (n & 1);
            const uint32_t at = smem_u32(st) + (k0 >> 4) * 2048 + (lane >> 4) * 256 + tok * 16;
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) {
              uint32_t w[2][4];
              ldsm_x4(at + cc * 512, w[0]);
              ldsm_x4(at + 2048 + cc * 512, w[1]);
#pragma unroll
              for (int z = 0; z < 2; ++z)
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                  for (int u = 0; u < 2; ++u) {
                    const uint2 k2 = e4m3x4_f16(w[y][2 * z + u]);
                    mma_f16(c[2 * y + u], qf[2 * cc + z], k2.x, k2.y);
                  }
            }
            // a page of values is [128 dims][16 tokens]
            const uint32_t vat = smem_u32(st) + St::kV + (k0 >> 4) * 2048 + lane * 16;
#pragma unroll
            for (int q4 = 0; q4 < 8; ++q4) {
              uint32_t w[4];
              ldsm_x4(vat + q4 * 512, w);
#pragma unroll
              for (int y = 0; y < 4; ++y) vraw[4 * q4 + y] = w[y];
            }
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
              for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const float lo = c[2 * y][2 * hh + e], hi = c[2 * y + 1][2 * hh + e];
                  sv[hh][4 * y + e] = t < 2 ? lo : hi;
                  sv[hh][4 * y + 2 + e] = t < 2 ? hi : lo;
                }
          } else {
            // a token is 64 bytes of codes; thread t takes the 16 of dims
            // 32 t .. + 31 (two scale groups).  Column n of tile nt is key
            // 4 (n / 2) + (2 nt + n % 2 + n / 2) % 4: with that rotation the
            // value reads below meet in a bank two at a time, not four
            uint32_t f0[4], f1[4];
            uint4 kw[4];
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
              const int quad = k0 + 16 * (nt >> 1) + 4 * (g >> 1), in = quad & (pt - 1);
              const int tok = in + ((2 * (nt & 1) + (g & 1) + (g >> 1)) & 3);
              const uint8_t *kp = st + (quad - in) * 144;
              kw[nt] = *reinterpret_cast<const uint4 *>(kp + tok * 64 + 16 * t);
              const uint32_t fh = e4m3x4_f16(*reinterpret_cast<const uint16_t *>(kp + pt * 64 + tok * 8 + 2 * t)).x;
              f0[nt] = __byte_perm(fh, fh, 0x1010), f1[nt] = __byte_perm(fh, fh, 0x3232);
            }
#pragma unroll
            for (int y = 0; y < 4; ++y)
#pragma unroll
              for (int nt = 0; nt < 4; ++nt) {
                uint32_t h[4];
                e2m1x8_f16(y == 0 ? kw[nt].x : y == 1 ? kw[nt].y : y == 2 ? kw[nt].z : kw[nt].w, h);
                const uint32_t f = y < 2 ? f0[nt] : f1[nt];
                mma_f16(c[nt], qf[2 * y], mul_f16x2(h[0], f), mul_f16x2(h[1], f));
                mma_f16(c[nt], qf[2 * y + 1], mul_f16x2(h[2], f), mul_f16x2(h[3], f));
              }
            // values: thread g takes dims 16 g .. + 15 (one scale group) of its tokens
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int quad = k0 + 16 * y + 4 * t, in = quad & (pt - 1);
              const uint8_t *vp = st + (quad - in) * 144 + pt * 72;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint2 w2 = *reinterpret_cast<const uint2 *>(vp + (in + ((e + t) & 3)) * 64 + 8 * g);
                vraw[16 * y + 2 * e] = w2.x, vraw[16 * y + 2 * e + 1] = w2.y;
              }
              const uint32_t f4 = *reinterpret_cast<const uint32_t *>(vp + pt * 64 + in * 8 + 4 * g);
              vsf[y] = __funnelshift_r(f4, f4, 8 * t);
            }
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
              for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  sv[hh][4 * y + e] = c[2 * y][2 * hh + e], sv[hh][4 * y + 2 + e] = c[2 * y + 1][2 * hh + e];
          }
          // scale, mask
          float vs[8];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            float ks[4] = {1.f, 1.f, 1.f, 1.f};
            if constexpr (FMT == 0) {
              const float4 k4 = *reinterpret_cast<const float4 *>(st + St::kKs + (k0 + 16 * y + 4 * t) * 4);
              const float4 v4 = *reinterpret_cast<const float4 *>(st + St::kVs + (k0 + 16 * y + 4 * t) * 4);
              ks[0] = k4.x, ks[1] = k4.y, ks[2] = k4.z, ks[3] = k4.w;
              vs[4 * y] = v4.x, vs[4 * y + 1] = v4.y, vs[4 * y + 2] = v4.z, vs[4 * y + 3] = v4.w;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              sv[0][4 * y + e] *= FMT == 0 ? ks[e] * sc[0] : sc[0];
              sv[1][4 * y + e] *= FMT == 0 ? ks[e] * sc[1] : sc[1];
            }
          }
          if (cut) {  // keys after the row's position: no score, no value (whatever the cache holds there)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int left = p - info.x * 128 - k0 - 16 * y - 4 * t;  // the last of the four keys that counts
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if ((FMT == 0 ? e : (e + t) & 3) > left) {
                  sv[0][4 * y + e] = sv[1][4 * y + e] = -INFINITY;
                  if constexpr (FMT == 0) {
                    vs[4 * y + e] = 0.f;
#pragma unroll
                    for (int n = 0; n < 16; ++n) vraw[16 * y + n] &= ~(0xffu << (8 * e));
                  } else {
                    vraw[16 * y + 2 * e] = vraw[16 * y + 2 * e + 1] = 0u;
                    vsf[y] &= ~(0xffu << (8 * e));
                  }
                }
            }
          }
          // the reference m (and the V unit) move only when a score (a V
          // scale) has outgrown them
          float top[2], vtop = 0.f;
#pragma unroll
          for (int hh = 0; hh < 2; ++hh)
            top[hh] = fmaxf(fmaxf(fmaxf(sv[hh][0], sv[hh][1]), fmaxf(sv[hh][2], sv[hh][3])),
                            fmaxf(fmaxf(sv[hh][4], sv[hh][5]), fmaxf(sv[hh][6], sv[hh][7])));
          bool grow = top[0] > mref[0] + kAtSlack || top[1] > mref[1] + kAtSlack;
          if constexpr (FMT == 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e) vtop = fmaxf(vtop, fabsf(vs[e]));
            grow |= vtop > vlimit;
          }
          if (__any_sync(0xffffffffu, grow)) {
            float f = 1.f;
            if constexpr (FMT == 0) {
              const int e2 = max(ev, min(exponent_of(quad_max(vtop)), 126));
              f = e2 - ev > 125 ? 0.f : pow2i(ev - e2);  // nothing summed yet where it is 0
              ev = e2;
              vlimit = pow2i(ev + 1);
            }
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const float nm = fmaxf(mref[hh], quad_max(top[hh]));
              const float al = nm == mref[hh] ? 1.f : ex2_approx(mref[hh] - nm);
              mref[hh] = nm;
              l[hh] *= al;
#pragma unroll
              for (int n = 0; n < 16; ++n) o[n][2 * hh] *= al * f, o[n][2 * hh + 1] *= al * f;
            }
          }
          uint32_t pa[2][4];
          {
            float unit = 1.f;
            if constexpr (FMT == 0) unit = pow2i(-ev);
            float w[2][8];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const float base = mref[hh] == -INFINITY ? 0.f : mref[hh] - kAtLift;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float x2 = ex2_approx(sv[hh][e] - base);
                l[hh] += x2;
                w[hh][e] = FMT == 0 ? x2 * (vs[e] * unit) : x2;
              }
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              pa[y][0] = f16x2_bits(w[0][4 * y], w[0][4 * y + 1]);
              pa[y][1] = f16x2_bits(w[1][4 * y], w[1][4 * y + 1]);
              pa[y][2] = f16x2_bits(w[0][4 * y + 2], w[0][4 * y + 3]);
              pa[y][3] = f16x2_bits(w[1][4 * y + 2], w[1][4 * y + 3]);
            }
          }
          // o += weights . values
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            if constexpr (FMT == 0) {
#pragma unroll
              for (int n = 0; n < 16; ++n) {
                const uint2 v2 = e4m3x4_f16(vraw[16 * y + n]);
                mma_f16(o[n], pa[y], v2.x, v2.y);
              }
            } else {
              // nibbles of two tokens are paired before the conversion
              const uint2 f = e4m3x4_f16(vsf[y]);
              const uint32_t *w = vraw + 16 * y;
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                constexpr uint32_t kLow = 0x0f0f0f0fu;
                uint32_t e01[4], d01[4], e23[4], d23[4];  // even, odd dims of tokens 0, 1 and 2, 3
                e2m1x8_f16((w[z] & kLow) | ((w[2 + z] & kLow) << 4), e01);
                e2m1x8_f16(((w[z] >> 4) & kLow) | (w[2 + z] & ~kLow), d01);
                e2m1x8_f16((w[4 + z] & kLow) | ((w[6 + z] & kLow) << 4), e23);
                e2m1x8_f16(((w[4 + z] >> 4) & kLow) | (w[6 + z] & ~kLow), d23);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                  mma_f16(o[8 * z + 2 * b], pa[y], mul_f16x2(e01[b], f.x), mul_f16x2(e23[b], f.y));
                  mma_f16(o[8 * z + 2 * b + 1], pa[y], mul_f16x2(d01[b], f.x), mul_f16x2(d23[b], f.y));
                }
              }
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[s]);
      if (info.x < 0) break;
    }

    // -------------------------------------------------- the segment's result
    l[0] = quad_sum(l[0]);
    l[1] = quad_sum(l[1]);
    if constexpr (FMT == 0) {
      const float up = pow2i(ev);
#pragma unroll
      for (int n = 0; n < 16; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][e] *= up;
    }
    const bool whole = v0 == 0 && v1 == v;
    float *pp = nullptr;  // the segment's partial result: [row][head][128], then (m, l)
    if (!whole) {
      const bool head_seg = v0 > 0;  // the item began in an earlier CTA
      pp = a.part + (int64_t)(2 * sl.cta + (head_seg ? 0 : 1)) * kAtPartFloats;
      if (!head_seg && tid == 0) {
        const int last = sh.offs[it + 1] - 1;
        a.shares[it] = make_int2(sl.cta, (int)((((int64_t)last + 1) * sl.ctas - 1) / sl.total));
      }
    } else if (a.sliced && tid == 0) {
      a.shares[it] = make_int2(0, 0);
    }
    const int64_t m = (int64_t)x.r * a.q_len + x.row0 + row;
    if constexpr (WPR == 1) {
      if (row < x.rows) {
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const int head = g + 8 * hh;
          if (head >= a.group) continue;
          if (whole) {
            const float inv = l[hh] == 0.f ? 0.f : a.out_scale / l[hh];
            __nv_bfloat16 *dst = a.out + m * a.out_stride + (int64_t)(x.h * a.group + head) * kHeadDim;
            if constexpr (FMT == 0) {
#pragma unroll
              for (int n = 0; n < 16; ++n)
                *reinterpret_cast<uint32_t *>(dst + 8 * n + 2 * t) = bf16x2_bits(o[n][2 * hh] * inv, o[n][2 * hh + 1] * inv);
            } else {
#pragma unroll
              for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int n = 0; n < 16; n += 8) {
                  auto two = [&](int k) { return bf16x2_bits(o[k][2 * hh + e] * inv, o[k + 1][2 * hh + e] * inv); };
                  *reinterpret_cast<uint4 *>(dst + 16 * (2 * t + e) + n) = make_uint4(two(n), two(n + 2), two(n + 4), two(n + 6));
                }
            }
          } else {
            float *dst = pp + (row * 16 + head) * kHeadDim;
            if constexpr (FMT == 0) {
#pragma unroll
              for (int n = 0; n < 16; ++n)
                *reinterpret_cast<float2 *>(dst + 8 * n + 2 * t) = make_float2(o[n][2 * hh], o[n][2 * hh + 1]);
            } else {
#pragma unroll
              for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int n = 0; n < 16; n += 4)
                  *reinterpret_cast<float4 *>(dst + 16 * (2 * t + e) + n) =
                      make_float4(o[n][2 * hh + e], o[n + 1][2 * hh + e], o[n + 2][2 * hh + e], o[n + 3][2 * hh + e]);
            }
            if (t == 0)
              *reinterpret_cast<float2 *>(pp + kAtMaxRows * 16 * kHeadDim + (row * 16 + head) * 2) =
                  make_float2(mref[hh], l[hh]);
          }
        }
      }
    } else {
      // the row's warps meet in shared memory: [warp][head][128], pairs of
      // dims moved within the row so that a store's lanes hit distinct banks
      auto place = [](int head, int d) {
        return head * kHeadDim + (d ^ ((head & 3) << 3) ^ (FMT == 0 ? 0 : 2 * (d >> 5)));
      };
      float *mine = joint + warp * 16 * kHeadDim;
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int head = g + 8 * hh;
        if constexpr (FMT == 0) {
#pragma unroll
          for (int n = 0; n < 16; ++n)
            *reinterpret_cast<float2 *>(mine + place(head, 8 * n + 2 * t)) = make_float2(o[n][2 * hh], o[n][2 * hh + 1]);
        } else {
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int n = 0; n < 16; n += 2)
              *reinterpret_cast<float2 *>(mine + place(head, 16 * (2 * t + e) + n)) =
                  make_float2(o[n][2 * hh + e], o[n + 1][2 * hh + e]);
        }
        if (t == 0) sh.ml[warp][head] = make_float2(mref[hh], l[hh]);
      }
      if (!fin_sync()) return;
      if (row < x.rows) {
        for (int head = part; head < a.group; head += WPR) {
          float top = -INFINITY, sum = 0.f;
#pragma unroll
          for (int w = 0; w < WPR; ++w) top = fmaxf(top, sh.ml[row * WPR + w][head].x);
          float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};  // dims 2 lane, 64 + 2 lane
#pragma unroll
          for (int w = 0; w < WPR; ++w) {
            const float2 ml = sh.ml[row * WPR + w][head];
            const float f = ml.x == top ? 1.f : ex2_approx(ml.x - top);
            sum += f * ml.y;
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const float2 y = *reinterpret_cast<const float2 *>(joint + (row * WPR + w) * 16 * kHeadDim +
                                                                 place(head, 64 * z + 2 * lane));
              if (f != 0.f) acc[z].x += f * y.x, acc[z].y += f * y.y;
            }
          }
          const float inv = sum == 0.f ? 0.f : a.out_scale / sum;
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            if (whole)
              *reinterpret_cast<uint32_t *>(a.out + m * a.out_stride + (int64_t)(x.h * a.group + head) * kHeadDim + 64 * z +
                                            2 * lane) = bf16x2_bits(acc[z].x * inv, acc[z].y * inv);
            else
              *reinterpret_cast<float2 *>(pp + (row * 16 + head) * kHeadDim + 64 * z + 2 * lane) = acc[z];
          }
          if (!whole && lane == 0)
            *reinterpret_cast<float2 *>(pp + kAtMaxRows * 16 * kHeadDim + (row * 16 + head) * 2) = make_float2(top, sum);
        }
      }
      if (!fin_sync()) return;  // `joint` is free for the next item
    }
  }
}

// Join the partial results of items that several CTAs share, in CTA order:
// W warps a (item, row, head), each every W-th partial, 16 of them in flight
// a lane (four dims); the W sums meet in shared memory.  The first CTA's
// partial is its slot 1 (the item starts there), the others' their slot 0.
constexpr int kJoinWarps = 8;
template <int W>
__global__ void __launch_bounds__(32 * kJoinWarps) pa_attn_join_kernel(const __grid_constant__ AttnParams a, int grid) {
  __shared__ float4 acc_s[kJoinWarps][32];
  __shared__ float2 ml_s[kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int it = blockIdx.x / a.rows_per, row = blockIdx.x % a.rows_per;
  const int head = blockIdx.y * (kJoinWarps / W) + warp / W;
  const int h = it & (a.n_kv - 1), rg = it >> a.lg_kv, r = rg >> a.lg_groups;
  const int row0 = (rg - (r << a.lg_groups)) * a.rows_per;
  pdl_wait();
  const int2 s = a.shares[it];
  const int c0 = max(s.x, 0), c1 = min(s.y, grid - 1);
  if (c1 <= c0 || row0 + row >= a.q_len) return;  // the same for the whole CTA
  const bool have = head < a.group;
  const float *base = a.part + (int64_t)2 * c0 * kAtPartFloats + (row * 16 + (have ? head : 0)) * kHeadDim + 4 * lane;
  const float *mls = a.part + (int64_t)2 * c0 * kAtPartFloats + kAtMaxRows * 16 * kHeadDim + (row * 16 + (have ? head : 0)) * 2;
  float top = -INFINITY, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kIn = 16;
  const int n = c1 - c0 + 1;
  for (int k0 = warp % W; k0 < n; k0 += W * kIn) {
    float4 y[kIn];
    float2 ml[kIn];
    float t2 = top;
#pragma unroll
    for (int k = 0; k < kIn; ++k) {
      const int c = k0 + k * W;
      const int64_t off = (int64_t)(2 * c + (c == 0 ? 1 : 0)) * kAtPartFloats;
      ml[k] = c < n ? *reinterpret_cast<const float2 *>(mls + off) : make_float2(-INFINITY, 0.f);
      y[k] = c < n ? *reinterpret_cast<const float4 *>(base + off) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int k = 0; k < kIn; ++k) t2 = fmaxf(t2, ml[k].x);
    const float f0 = top == t2 ? 1.f : ex2_approx(top - t2);
    top = t2;
    sum *= f0, acc.x *= f0, acc.y *= f0, acc.z *= f0, acc.w *= f0;
#pragma unroll
    for (int k = 0; k < kIn; ++k) {
      const float f = ml[k].x == top ? 1.f : ex2_approx(ml[k].x - top);
      sum += f * ml[k].y;
      if (f != 0.f) acc.x += f * y[k].x, acc.y += f * y[k].y, acc.z += f * y[k].z, acc.w += f * y[k].w;
    }
  }
  if constexpr (W > 1) {
    acc_s[warp][lane] = acc;
    if (lane == 0) ml_s[warp] = make_float2(top, sum);
    __syncthreads();
    if (warp % W) return;
    float t2 = -INFINITY;
#pragma unroll
    for (int w = 0; w < W; ++w) t2 = fmaxf(t2, ml_s[warp + w].x);
    sum = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float2 ml = ml_s[warp + w];
      const float4 y = acc_s[warp + w][lane];
      const float f = ml.x == t2 ? 1.f : ex2_approx(ml.x - t2);
      sum += f * ml.y;
      if (f != 0.f) acc.x += f * y.x, acc.y += f * y.y, acc.z += f * y.z, acc.w += f * y.w;
    }
  }
  if (!have) return;
  const float inv = sum == 0.f ? 0.f : a.out_scale / sum;
  const int64_t m = (int64_t)r * a.q_len + row0 + row;
  *reinterpret_cast<uint2 *>(a.out + m * a.out_stride + (int64_t)(h * a.group + head) * kHeadDim + 4 * lane) =
      make_uint2(bf16x2_bits(acc.x * inv, acc.y * inv), bf16x2_bits(acc.z * inv, acc.w * inv));
}

static bool attn_maps(AttnMaps *maps, const AttnParams &a, int fmt) {
  if (fmt == 0) {
    const uint64_t kv = (uint64_t)a.n_kv, pages = (uint64_t)a.num_pages16;
    return map_page_rows(&maps->m[0], a.k_cache, 2048, kv, kv * 2048, pages, 1, 8) &&
           map_page_rows(&maps->m[1], a.v_cache, 2048, kv, kv * 2048, pages, 1, 8) &&
           map_page_rows(&maps->m[2], a.k_scale, 64, kv, kv * 64, pages, 1, 8) &&
           map_page_rows(&maps->m[3], a.v_scale, 64, kv, kv * 64, pages, 1, 8);
  }
  if (a.bs > 128) return true;
  const uint32_t row = 72u * (a.bs < 16 ? a.bs : 16), per = a.bs < 16 ? 1 : a.bs / 16;  // rows of a slot
  return map_page_rows(&maps->m[0], a.kv_cache, row, (uint64_t)2 * a.n_kv * per, (uint64_t)a.kv_page_bytes,
                       (uint64_t)a.kv_pages, 2 * per, 128u / a.bs);
}

template <int FMT>
static cudaError_t launch_attn(const AttnParams &a, int sms, bool pdl, cudaStream_t stream) {
  AttnMaps maps;
  if (!attn_maps(&maps, a, FMT)) return cudaErrorInvalidValue;
  using Kern = void (*)(const AttnMaps, const AttnParams);
  Kern kern = pa_attn_kernel<FMT, 1>;
  int smem = attn_smem<FMT, 1>();
  if (a.rows_per == 1) kern = pa_attn_kernel<FMT, 8>, smem = attn_smem<FMT, 8>();
  else if (a.rows_per == 2) kern = pa_attn_kernel<FMT, 4>, smem = attn_smem<FMT, 4>();
  else if (a.rows_per <= 4) kern = pa_attn_kernel<FMT, 2>, smem = attn_smem<FMT, 2>();
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(kern), smem);
  if (e != cudaSuccess) return e;
  static int regs[4] = {0, 0, 0, 0};  // of the four kernels at launch
  int &held = regs[a.rows_per == 1 ? 0 : a.rows_per == 2 ? 1 : a.rows_per <= 4 ? 2 : 3];
  if (held == 0) {
    cudaFuncAttributes at;
    e = cudaFuncGetAttributes(&at, reinterpret_cast<const void *>(kern));
    if (e != cudaSuccess) return e;
    held = at.numRegs;
  }
  if (held * kAtThreads < 32 * kAtWarps * kAtComputeRegs + (kAtThreads - 32 * kAtWarps) * kAtProducerRegs)
    return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  cfg.gridDim = dim3(a.sliced ? sms : a.items);
  cfg.blockDim = dim3(kAtThreads);
  cfg.dynamicSmemBytes = smem;
  e = cudaLaunchKernelEx(&cfg, kern, maps, a);
  if (e != cudaSuccess || !a.sliced || a.test_timeout) return e;
  // few items: many partials each, a CTA a head; else a warp a head
  const bool many = a.items * 8 <= sms;
  cfg.gridDim = dim3(a.items * a.rows_per, many ? a.group : (a.group + kJoinWarps - 1) / kJoinWarps);
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, many ? pa_attn_join_kernel<kJoinWarps> : pa_attn_join_kernel<1>, a, sms);
}

}  // namespace pa

extern "C" size_t pre_attn_attention_workspace_bytes(int R, int q_len, int n_kv_heads, int num_sms) {
  if (R < 0 || R > 65535 || q_len < 1 || q_len > 16 || num_sms < 1 || num_sms > 4096) return 0;
  if (n_kv_heads != 1 && n_kv_heads != 2 && n_kv_heads != 4) return 0;
  return (size_t)2 * num_sms * pa::kAtPartFloats * sizeof(float) + pa::kAtMaxItems * sizeof(int2);
}

extern "C" int pre_attn_attention(const pa_attention_args *in, void *stream) {
  if (!in) return PA_ERR_NULL;
  const pa_attention_args &x = *in;
  auto aligned = [](const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
  if (!x.caches || !x.block_table || !x.seq_lens || !x.out || !x.status) return PA_ERR_NULL;
  if (!x.q == !x.q_fp8) return PA_ERR_CONFIG;
  if (x.cache_format != PA_CACHE_FP8 && x.cache_format != PA_CACHE_NVFP4) return PA_ERR_CONFIG;
  if (x.n_kv_heads != 1 && x.n_kv_heads != 2 && x.n_kv_heads != 4) return PA_ERR_CONFIG;
  if (x.n_q_heads < 1 || x.n_q_heads % x.n_kv_heads || x.n_q_heads / x.n_kv_heads > 16) return PA_ERR_CONFIG;
  if (x.flags & ~(uint32_t)(PA_FLAG_NO_PDL | PA_FLAG_TEST_WAIT_TIMEOUT)) return PA_ERR_CONFIG;
  if (!(x.sm_scale > 0.0f) || !std::isfinite(x.sm_scale)) return PA_ERR_CONFIG;
  if (x.q_fp8 && (!(x.q_fp8_scale > 0.0f) || !std::isfinite(x.q_fp8_scale))) return PA_ERR_CONFIG;
  if (x.R < 0 || x.R > 65535 || x.q_len < 1 || x.q_len > 16 || x.bt_width < 1 || x.bt_width > pa::kAtMaxWidth)
    return PA_ERR_SHAPE;
  if (x.q_stride < (int64_t)x.n_q_heads * 128 || x.out_stride < (int64_t)x.n_q_heads * 128) return PA_ERR_SHAPE;
  if (x.blocks) {
    if (!x.counts) return PA_ERR_NULL;
    if (x.topk < 1 || x.topk > pa::kAtMaxTopk) return PA_ERR_SHAPE;
  }
  const pa_caches &c = *x.caches;
  const bool fp8 = x.cache_format == PA_CACHE_FP8;
  int kps = x.kv_page_stride;
  if (fp8) {
    if (!c.k_cache || !c.v_cache || !c.k_scale || !c.v_scale) return PA_ERR_NULL;
    if (x.block_size != 16 || (kps != 0 && kps < 8) || c.num_pages16 < 1 || c.num_pages16 > INT32_MAX)
      return PA_ERR_CONFIG;
    if (!aligned(c.k_cache, 16) || !aligned(c.v_cache, 16) || !aligned(c.k_scale, 16) || !aligned(c.v_scale, 16))
      return PA_ERR_ALIGN;
    if (kps == 0) kps = 8;
  } else {
    if (!c.kv_cache) return PA_ERR_NULL;
    const int bs = x.block_size;
    if (bs < 4 || bs % 4 || bs > 1024 || c.kv_pages < 1 || c.kv_pages > INT32_MAX) return PA_ERR_CONFIG;
    if (128 % bs && bs % 128) return PA_ERR_UNSUPPORTED;
    if (c.kv_page_bytes < (int64_t)2 * x.n_kv_heads * bs * 72) return PA_ERR_CONFIG;
    if (!(c.k_global_scale > 0.0f) || !(c.v_global_scale > 0.0f)) return PA_ERR_CONFIG;
    if (c.kv_page_bytes % 32 || !aligned(c.kv_cache, 32)) return PA_ERR_ALIGN;
  }
  if ((x.q && !aligned(x.q, 16)) || (x.q_fp8 && !aligned(x.q_fp8, 16)) || x.q_stride % 16 || !aligned(x.out, 16) ||
      x.out_stride % 8 || !aligned(x.block_table, 4) || !aligned(x.seq_lens, 4) || !aligned(x.blocks, 4) ||
      !aligned(x.counts, 4) || !aligned(x.status, 4))
    return PA_ERR_ALIGN;
  if (x.R == 0) return PA_OK;
  const int64_t M = (int64_t)x.R * x.q_len;
  {
    const uintptr_t q0 = reinterpret_cast<uintptr_t>(x.q ? x.q : x.q_fp8), o0 = reinterpret_cast<uintptr_t>(x.out);
    const uintptr_t q1 = q0 + (uintptr_t)(M * x.q_stride) * (x.q ? 2 : 1), o1 = o0 + (uintptr_t)(M * x.out_stride) * 2;
    if (q0 < o1 && o0 < q1) return PA_ERR_ALIAS;
  }
  const int sms = pa::current_device_sms();
  if (sms < 1) return pa::record_cuda_error(cudaGetLastError());
  if (!x.workspace || x.workspace_bytes < pre_attn_attention_workspace_bytes(x.R, x.q_len, x.n_kv_heads, sms))
    return PA_ERR_WORKSPACE;
  if (!aligned(x.workspace, 256)) return PA_ERR_ALIGN;
  pa::AttnParams a = {};
  a.q = static_cast<const uint8_t *>(x.q ? x.q : x.q_fp8);
  a.q_is_fp8 = x.q ? 0 : 1;
  a.q_stride = x.q_stride;
  a.k_cache = static_cast<const uint8_t *>(c.k_cache);
  a.v_cache = static_cast<const uint8_t *>(c.v_cache);
  a.k_scale = c.k_scale;
  a.v_scale = c.v_scale;
  a.num_pages16 = c.num_pages16;
  a.kps = kps;
  a.kv_cache = static_cast<const uint8_t *>(c.kv_cache);
  a.kv_pages = c.kv_pages;
  a.kv_page_bytes = c.kv_page_bytes;
  a.bs = x.block_size;
  a.block_table = x.block_table;
  a.seq_lens = x.seq_lens;
  a.blocks = x.blocks;
  a.counts = x.counts;
  a.topk = x.blocks ? x.topk : 0;
  a.R = x.R;
  a.q_len = x.q_len;
  a.bt_width = x.bt_width;
  a.n_kv = x.n_kv_heads;
  a.group = x.n_q_heads / x.n_kv_heads;
  a.lg_kv = x.n_kv_heads == 4 ? 2 : x.n_kv_heads - 1;
  a.lg_groups = x.q_len > pa::kAtMaxRows ? 1 : 0;
  a.rows_per = (x.q_len + a.lg_groups) >> a.lg_groups;
  a.items = x.R * x.n_kv_heads << a.lg_groups;
  a.sliced = a.items <= pa::kAtMaxItems;
  a.score_scale = (float)((double)x.sm_scale * 1.4426950408889634 * (x.q ? 1.0 : (double)x.q_fp8_scale) *
                          (fp8 ? 1.0 : (double)c.k_global_scale));
  a.out_scale = fp8 ? 1.0f : c.v_global_scale;
  a.out = static_cast<__nv_bfloat16 *>(x.out);
  a.out_stride = x.out_stride;
  a.part = static_cast<float *>(x.workspace);
  a.shares = reinterpret_cast<int2 *>(a.part + (size_t)2 * sms * pa::kAtPartFloats);
  a.status = x.status;
  a.test_timeout = (x.flags & PA_FLAG_TEST_WAIT_TIMEOUT) ? 1 : 0;
  a.lim = a.test_timeout ? pa::kTestWaitNs : pa::kWaitNs;
  const bool pdl = !(x.flags & PA_FLAG_NO_PDL);
  const cudaError_t e = fp8 ? pa::launch_attn<0>(a, sms, pdl, (cudaStream_t)stream)
                            : pa::launch_attn<1>(a, sms, pdl, (cudaStream_t)stream);
  return e == cudaSuccess ? PA_OK : pa::record_cuda_error(e);
}
