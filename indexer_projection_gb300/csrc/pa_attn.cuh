// The producing side of pre_attn_attention: the kernels' parameters, the items
// and the CTAs' shares of them (a cluster of CTAs an item, slices of all
// items' blocks, or a CTA an item), and the ring of 128-key blocks with the
// warps that fill it.
//
// Work.  An item is (request, up to 8 of its rows, KV head): the rows share
// the key blocks, so a block is read from memory once for all rows that
// attend it.  In a CTA one warp works out which blocks come next, one thread
// keeps a ring of them in flight with tensor-map copies (a copy a 2 KB page
// and scale row took about 110 clocks each, more than the data), the others
// compute.
#pragma once

#include <cuda_fp16.h>

#include "pa_device.cuh"
#include "pa_f16.cuh"
#include "pa_launch.h"
#include "pa_tma.h"

namespace pa {

constexpr int kAtWarps = 8;                        // compute warps
constexpr int kAtMaxRows = 8;                      // query rows an item
constexpr int kAtMaxItems = 2048;                  // items the sliced grid lists in shared memory
constexpr int kAtMaxWidth = 16384;                 // block-table width
constexpr int kAtMaxTopk = 256;
constexpr float kAtLift = 9.0f;   // weights are 2^9 exp2(s - m)
constexpr float kAtSlack = 4.0f;  // NVFP4: m follows the maximum once that is 2^4 above it
constexpr float kAtMostSum = 65536.f;  // FP8: .. once a lane's weights of a step sum to more
// FP8: a part's sum of weights, as it leaves its warp, is about 2^-16: up to
// 8 warps, 8 CTAs of a cluster or 152 slices (each a warp or eight) then sum to less than one
constexpr int kAtSumDown = 16;
constexpr int kAtUnit = 100;      // FP8: the unit of the products before any is known is 2^100
constexpr int kAtMaxSplit = 8;    // CTAs a cluster
// (blocks a CTA) x (rows) of a cluster at most; twice that where clusters take a third of the SMs or more
constexpr int kAtClusterWork = 12;
constexpr int kAtPartFloats = kAtMaxRows * 16 * (kHeadDim + 2);  // o, then (m, l), of one partial

// How the items meet the CTAs: a CTA an item; even slices of all items'
// blocks over a persistent grid, with partial results joined by a second
// kernel; or a cluster of CTAs an item, joined through distributed shared
// memory (small calls: no scan of the items, no second kernel).
enum { kAtWhole = 0, kAtSliced = 1, kAtCluster = 2 };

struct CacheAttnParams {
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
  int items, mode;                   // kAtWhole, kAtSliced, kAtCluster
  int split;                         // kAtCluster: CTAs an item
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
};
template <>
struct AttnStage<1> {  // pieces of pt = min(block_size, 128) tokens: K codes (64 bytes a token), K scales (8), V codes,
                       // V scales, as the page holds them
  static constexpr int kBytes = 18432;
};
constexpr int kAtMaxStages = 10;
constexpr int kAtInfo = 16;  // more entries than lie between the copies and the last reader

// 32 blocks of a segment, resolved ahead of their copies.
struct AttnBatch {
  int blk[32];   // ids in the cache (-1: none)
  int2 info[32]; // block of the request, rows that attend it
  int n, seq, first_pos;
  int first, last;  // of the segment
};

// What the producing warps and the readers of a ring of blocks share.
template <int ROWS>  // rows of an item at most
struct AttnRing {
  uint64_t full[kAtMaxStages], empty[kAtMaxStages];
  uint64_t batch_full[2], batch_empty[2];
  uint64_t q_full, q_empty;  // an item's queries; read into registers at once
  int2 info[kAtInfo];        // entry j's block (-1: the end of a segment), rows that attend it, at j % kAtInfo
  int2 q_item;               // first row's position, keys
  int scan[kAtWarps];
  AttnBatch batch[2];
  int offs[kAtMaxItems + 8];
  uint16_t list[ROWS * kAtMaxTopk];
  uint32_t bits[ROWS][kAtMaxWidth / 32];
};

constexpr int kAtSmem = 232448;  // 227 KB a CTA

// An item's request, KV head and rows; its request is without keys when
// seq < 1, seq < q_len or its blocks exceed the table.
struct AttnItem {
  int r, h, row0, rows, seq, first;  // first: position of row row0
  __device__ int blocks_upto(int rows_) const { return seq > 0 ? (first + rows_ - 1) / 128 + 1 : 0; }
};
// its place, without the request's keys
__device__ __forceinline__ AttnItem attn_place(const CacheAttnParams &a, int it) {
  AttnItem x;
  x.h = it & (a.n_kv - 1);
  const int rg = it >> a.lg_kv;
  x.r = rg >> a.lg_groups;
  x.row0 = (rg - (x.r << a.lg_groups)) * a.rows_per;
  x.rows = min(a.rows_per, a.q_len - x.row0);
  x.seq = x.first = 0;
  return x;
}
__device__ __forceinline__ AttnItem attn_item(const CacheAttnParams &a, int it, bool *bad) {
  AttnItem x = attn_place(a, it);
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
__device__ __forceinline__ int attn_units(const CacheAttnParams &a, int it, bool *bad) {
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


__device__ __forceinline__ void tma_pages(uint32_t dst, const CUtensorMap *map, int row, int page, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(page), "r"(smem_u32(bar))
      : "memory");
}

// The CTA's share of the work: of units lo .. hi of the total in the sliced
// mode, of part lo of `total` parts of one item otherwise.
struct AttnSlice {
  int lo, hi, total, cta, ctas, first;
  bool sliced, none;  // none: nothing for this CTA
  // whether item `it` has a segment here: its units (or parts) v0 .. v1 of v
  template <class S>
  __device__ bool segment(const CacheAttnParams &a, const S &sh, int it, int &v0, int &v1, int &v) const {
    if (!sliced) {
      v0 = lo, v1 = hi, v = total;
      return it == first;
    }
    if (it >= a.items || sh.offs[it] >= hi) return false;
    v0 = max(lo, sh.offs[it]) - sh.offs[it];
    v1 = min(hi, sh.offs[it + 1]) - sh.offs[it];
    v = sh.offs[it + 1] - sh.offs[it];
    return true;
  }
};

// Every thread of the CTA calls it (WARPS: warps that share the scan); it
// ends behind a barrier of the CTA.
template <int WARPS, class S>
__device__ __forceinline__ AttnSlice attn_slice(const CacheAttnParams &a, S &sh, int mode) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  AttnSlice sl;
  sl.cta = sl.first = blockIdx.x;
  sl.sliced = mode == kAtSliced;
  sl.none = false;
  if (mode == kAtSliced) {
    // the running sums of the items' units, 256 items a round
    int before = 0;
    bool bad = false;
    for (int i0 = 0; i0 < a.items; i0 += 32 * WARPS) {
      const int it = i0 + tid;
      const int n = warp < WARPS && it < a.items ? attn_units(a, it, &bad) : 0;
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (warp < WARPS && lane == 31) sh.scan[warp] = incl;
      __syncthreads();
      int round = 0, mine = before + incl - n;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const int v = sh.scan[w];
        if (w < warp) mine += v;
        round += v;
      }
      if (warp < WARPS) sh.offs[it] = mine;
      before += round;
      __syncthreads();
    }
    if (tid == 0) sh.offs[a.items] = before;
    if (blockIdx.x == 0 && bad) set_status(a.status, kDevSlotRange);
    __syncthreads();
    sl.total = sh.offs[a.items];
    sl.ctas = min((int)gridDim.x, sl.total);
    sl.none = sl.cta >= sl.ctas;
    sl.lo = (int)((int64_t)sl.total * sl.cta / sl.ctas);
    sl.hi = (int)((int64_t)sl.total * (sl.cta + 1) / sl.ctas);
    sl.first = 0;
    for (int step = kAtMaxItems / 2; step > 0; step >>= 1)
      if (sl.first + step < a.items && sh.offs[sl.first + step] <= sl.lo) sl.first += step;
  } else {
    sl.total = mode == kAtCluster ? a.split : 1;
    sl.ctas = 0;
    sl.lo = mode == kAtCluster ? (int)cta_rank() : 0;
    sl.hi = sl.lo + 1;
    if (mode == kAtCluster) sl.first = blockIdx.x / a.split;
    __syncthreads();
  }
  return sl;
}

// One warp, before the wait on the previous kernels: into L2 what the CTA's
// first loads will find there (lengths, lists, the block table, queries, each
// a latency of the chain in front of the first block).  No value is used, so
// it does not matter that those kernels may still write them.
__device__ __forceinline__ void attn_prefetch(const CacheAttnParams &a, int mode) {
  const int lane = threadIdx.x & 31;
  auto line = [](const void *p, int64_t bytes, int64_t k) {  // 128-byte line k of a span
    if (128 * k < bytes) prefetch_l2(static_cast<const uint8_t *>(p) + 128 * k);
  };
  if (mode == kAtSliced) {  // every CTA a share of the whole
    const int64_t k = (int64_t)blockIdx.x * 32 + lane, M = (int64_t)a.R * a.q_len;
    line(a.seq_lens, (int64_t)a.R * 4, k);
    line(a.block_table, (int64_t)a.R * a.bt_width * 4, k);
    if (a.topk) {
      line(a.counts, M * a.n_kv * 4, k);
      line(a.blocks, M * a.n_kv * a.topk * 4, k);
    }
    return;
  }
  const int it = mode == kAtCluster ? blockIdx.x / a.split : blockIdx.x;
  const AttnItem x = attn_place(a, it);
  const int64_t m = (int64_t)x.r * a.q_len + x.row0;
  if (lane == 0) prefetch_l2(a.seq_lens + x.r);
  line(a.block_table + (int64_t)x.r * a.bt_width, (int64_t)a.bt_width * 4, lane);
  if (a.topk) {
    line(a.counts + m * a.n_kv, (int64_t)x.rows * a.n_kv * 4, lane);
    line(a.blocks + m * a.n_kv * a.topk, (int64_t)x.rows * a.n_kv * a.topk * 4, lane);
  }
  const int es = a.q_is_fp8 ? 1 : 2;
  for (int i = 0; i < x.rows; ++i)
    line(a.q + ((m + i) * a.q_stride + x.h * a.group * kHeadDim) * es, a.group * kHeadDim * es, lane);
}

// One warp: what is to be copied, a batch of up to 32 blocks ahead of the
// copies, so that the latency of the lists and the block table (behind the
// copies already asked for) is hidden.
template <int FMT, class S>
__device__ __forceinline__ void attn_resolve(const CacheAttnParams &a, S &sh, const AttnSlice &sl, int mode) {
  const int lane = threadIdx.x & 31;
  bool ok = true;
  int nbt = 0;
  int v0, v1, v;
  for (int it = sl.first; ok && sl.segment(a, sh, it, v0, v1, v); ++it) {
    bool bad = false;
    int b1 = -1, count1 = 0;  // a single row's short list, an entry a lane: asked for together with the length
    if (a.topk > 0 && a.topk <= 32 && a.rows_per == 1) {
      const AttnItem y = attn_place(a, it);
      const int64_t at = ((int64_t)y.r * a.q_len + y.row0) * a.n_kv + y.h;
      count1 = __ldg(a.counts + at);
      if (lane < a.topk) b1 = __ldg(a.blocks + at * a.topk + lane);
    }
    const AttnItem x = attn_item(a, it, &bad);
    if (mode != kAtSliced && bad && lane == 0) set_status(a.status, kDevSlotRange);
    const int nb = x.blocks_upto(x.rows);
    int u0 = 0, u1 = 0;  // the segment's blocks (of the union list, or of the request)
    if (a.topk == 0) {
      u0 = (int)((int64_t)nb * v0 / v);
      u1 = (int)((int64_t)nb * v1 / v);
    } else if (a.rows_per == 1 && a.topk <= 32) {
      // one short list: its distinct blocks in list order
      if (nb > 0) {
        int b = b1;
        const bool given = lane < min(count1, a.topk);
        const bool fits = given && b >= 0 && b < nb;
        if (__any_sync(0xffffffffu, given && !fits) && lane == 0) set_status(a.status, kDevSlotRange);
        if (!fits) b = -1 - lane;
        const uint32_t same = __match_any_sync(0xffffffffu, b);
        const uint32_t kept = __ballot_sync(0xffffffffu, fits && (same & ((1u << lane) - 1u)) == 0);
        const int total = __popc(kept), pos = __popc(kept & ((1u << lane) - 1u));
        u0 = total * v0 / v;
        u1 = total * v1 / v;
        __syncwarp();
        if (((kept >> lane) & 1u) && pos >= u0 && pos < u1) {
          sh.list[pos - u0] = (uint16_t)b;
          sh.bits[0][b >> 5] = 0xffffffffu;  // (the batches ask it for the rows)
        }
        __syncwarp();
      }
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
    for (int base = u0; ok && (base < u1 || base == u0); base += 32) {
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
      if (lane == 0) ok = mbar_wait(&sh.batch_empty[nbt & 1], ((uint32_t)(nbt >> 1) & 1) ^ 1, a.status, a.lim);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      AttnBatch &bt = sh.batch[nbt & 1];
      bt.blk[lane] = blk < 0 ? -1 : (int)blk;
      bt.info[lane] = make_int2(b, rows);
      if (lane == 0) {
        bt.n = min(32, u1 - base);
        bt.first_pos = x.first, bt.seq = x.seq;
        bt.first = base == u0, bt.last = base + 32 >= u1;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.batch_full[nbt & 1]);
      ++nbt;
    }
  }
}

// One thread: an item's queries when its first batch comes, then a stage a
// block; kGroups groups of readers take the entries in turn, and each segment
// ends with an entry without a block for each of them.
template <int FMT, int kStages, int kGroups, class S>
__device__ __forceinline__ void attn_copies(const CacheAttnParams &a, const AttnMaps &maps, S &sh, const AttnSlice &sl,
                                            uint8_t *ring, uint8_t *q_smem) {
  using St = AttnStage<FMT>;
  int j = 0, nq = 0;  // stages filled, items begun
  bool ok = true;
  auto acquire = [&]() {
    return mbar_wait(&sh.empty[j % kStages], ((uint32_t)(j / kStages) & 1) ^ 1, a.status, a.lim);
  };
  int v0, v1, v, it = sl.first;
  for (int nbt = 0; ok && sl.segment(a, sh, it, v0, v1, v); ++nbt) {
    const AttnBatch &bt = sh.batch[nbt & 1];
    if (!(ok = mbar_wait(&sh.batch_full[nbt & 1], (uint32_t)(nbt >> 1) & 1, a.status, a.lim))) break;
    const AttnItem x = attn_place(a, it);
    if (bt.first) {
      if (!(ok = mbar_wait(&sh.q_empty, (uint32_t)(nq & 1) ^ 1, a.status, a.lim))) break;
      sh.q_item = make_int2(bt.first_pos, bt.seq);
      const int es = a.q_is_fp8 ? 1 : 2, bytes = a.group * kHeadDim * es;
      const uint8_t *src = a.q + (((int64_t)x.r * a.q_len + x.row0) * a.q_stride + x.h * a.group * kHeadDim) * es;
      mbar_expect_tx(&sh.q_full, x.rows * bytes);
      for (int i = 0; i < x.rows; ++i, src += a.q_stride * es) bulk_g2s(q_smem + i * bytes, src, bytes, &sh.q_full);
      ++nq;
    }
    for (int k = 0; k < bt.n; ++k) {
      const int64_t id = bt.blk[k];
      if (id < 0) continue;
      if (!(ok = acquire())) break;
      const int s = j % kStages;
      uint64_t *bar = &sh.full[s];
      uint8_t *st = ring + s * St::kBytes;
      sh.info[j % kAtInfo] = bt.info[k];
      mbar_expect_tx(bar, St::kBytes);
      if constexpr (FMT == 0) {  // the block's 8 pages of the head: K, V, their scales
        const int page = (int)(id * a.kps);
        tma_pages(smem_u32(st), &maps.m[0], x.h, page, bar);
        tma_pages(smem_u32(st + St::kKs), &maps.m[2], x.h, page, bar);
        tma_pages(smem_u32(st + St::kV), &maps.m[1], x.h, page, bar);
        tma_pages(smem_u32(st + St::kVs), &maps.m[3], x.h, page, bar);
      } else if (a.bs <= 128) {  // the head's K and V slots of 128 / bs pages
        tma_pages(smem_u32(st), &maps.m[0], 2 * x.h * max(a.bs >> 4, 1), (int)(id * (128 / a.bs)), bar);
      } else {  // 128 tokens within a page: K codes, K scales, V codes, V scales
        const int64_t page = id * 128 / a.bs;
        const int t0 = (int)(id * 128 - page * a.bs);
        const uint8_t *slot = a.kv_cache + page * a.kv_page_bytes + (int64_t)(2 * x.h) * a.bs * 72;
        for (int v2 = 0; v2 < 2; ++v2, slot += a.bs * 72) {
          bulk_g2s(st + v2 * 9216, slot + t0 * 64, 8192, bar);
          bulk_g2s(st + v2 * 9216 + 8192, slot + a.bs * 64 + t0 * 8, 1024, bar);
        }
      }
      ++j;
    }
    if (!ok) break;
    if (bt.last) {
      for (int k = 0; k < kGroups && ok; ++k) {  // an entry for each group of readers
        if (!(ok = acquire())) break;
        sh.info[j % kAtInfo] = make_int2(-1, 0);
        mbar_arrive(&sh.full[j % kStages]);
        ++j;
      }
      if (!ok) break;
      ++it;
    }
    mbar_arrive(&sh.batch_empty[nbt & 1]);
  }
  // the copies issued land before the CTA exits
  for (int k = j - 1; k >= 0 && k >= j - kStages; --k)
    mbar_wait(&sh.full[k % kStages], (uint32_t)(k / kStages) & 1, a.status, a.lim);
  if (nq > 0) mbar_wait(&sh.q_full, (uint32_t)(nq - 1) & 1, a.status, a.lim);
}

}  // namespace pa
