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
// warps a row, each with 1 / WPR of a block's keys.
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

namespace pa {

constexpr int kAtWarps = 8;                        // compute warps
constexpr int kAtThreads = 32 * (kAtWarps + 1);    // and the producer
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
  int row_groups, rows_per;          // items of a (request, KV head), rows an item
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

template <int FMT>
struct AttnStage;
template <>
struct AttnStage<0> {  // K and V pages as they are (8 of 2048 bytes each), then the scales of 128 tokens
  static constexpr int kV = 16384, kKs = 32768, kVs = 33280, kBytes = 33792;
  static constexpr int stages(bool joined) { return joined ? 4 : 5; }
};
template <>
struct AttnStage<1> {  // 128 x 64 bytes of K, of V, then 128 x 8 scale bytes of K (linear), of V (4-token groups)
  static constexpr int kV = 8192, kKs = 16384, kVs = 17408, kBytes = 18432;
  static constexpr int stages(bool joined) { return joined ? 7 : 10; }
};

struct AttnShared {
  uint64_t full[10], empty[10];
  uint64_t fin;     // the compute warps, twice an item
  uint64_t never;   // testing: nothing arrives on it
  int2 info[10];    // block (-1: the end of an item), rows that attend it
  int scan[kAtWarps];
  float2 ml[kAtWarps][16];
  int offs[kAtMaxItems + 1];
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
  x.h = it % a.n_kv;
  const int rg = it / a.n_kv;
  x.r = rg / a.row_groups;
  x.row0 = (rg - x.r * a.row_groups) * a.rows_per;
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
  for (int i = 0; i < x.rows; ++i)
    n += min(max(__ldg(a.counts + ((int64_t)x.r * a.q_len + x.row0 + i) * a.n_kv + x.h), 0), a.topk);
  return max(n, 1);
}

// The CTA's slice as segments: item it, units v0 .. v1 of its v.
struct AttnSlice {
  int lo, hi, total, cta, ctas;
};

template <int FMT, int WPR>
__global__ void __launch_bounds__(kAtThreads, 1) pa_attn_kernel(const __grid_constant__ AttnParams a) {
  using St = AttnStage<FMT>;
  constexpr int kStages = St::stages(WPR > 1);
  constexpr int kKeys = 128 / WPR;  // keys of a block a warp takes
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
    // units of every item, then their running sums: 8 items a thread
    constexpr int kPer = kAtMaxItems / (32 * kAtWarps);
    int n[kPer], sum = 0;
    bool bad = false;
    if (warp < kAtWarps) {
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int it = tid * kPer + k;
        n[k] = it < a.items ? attn_units(a, it, &bad) : 0;
        sum += n[k];
      }
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (warp < kAtWarps && lane == 31) sh.scan[warp] = incl;
    if (blockIdx.x == 0 && bad) set_status(a.status, kDevSlotRange);
    __syncthreads();
    if (warp < kAtWarps) {
      int run = incl - sum;
      for (int w = 0; w < warp; ++w) run += sh.scan[w];
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        sh.offs[tid * kPer + k] = run;
        run += n[k];
      }
      if (tid == 32 * kAtWarps - 1) sh.offs[kAtMaxItems] = run;
    }
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

  if (warp == kAtWarps) {
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
        for (int k = lane; k < x.rows * words; k += 32) sh.bits[k / words][k % words] = 0;
        __syncwarp();
        bool out_of_range = false;
        for (int k = lane; k < x.rows * a.topk; k += 32) {
          const int i = k / a.topk, e = k - i * a.topk;
          const int64_t at = ((int64_t)x.r * a.q_len + x.row0 + i) * a.n_kv + x.h;
          if (e >= __ldg(a.counts + at)) continue;
          const int b = __ldg(a.blocks + at * a.topk + e);
          if (b < 0 || b > (x.first + i) / 128) out_of_range = true;
          else atomicOr(&sh.bits[i][b >> 5], 1u << (b & 31));
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
          if (FMT == 0) {  // 8 pages x (K, V, K scales, V scales), one copy a lane
            const int pg = lane & 7, kind = lane >> 3;
            const int64_t page = (id * a.kps + pg) * a.n_kv + x.h;
            if (kind < 2)
              bulk_g2s(st + kind * St::kV + pg * 2048, (kind ? a.v_cache : a.k_cache) + page * 2048, 2048, bar);
            else
              bulk_g2s(st + (kind == 3 ? St::kVs : St::kKs) + pg * 64, (kind == 3 ? a.v_scale : a.k_scale) + page * 16,
                       64, bar);
          } else {  // pieces of min(bs, 128) tokens x (K codes, K scales, V codes, V scales)
            const int pt = min(a.bs, 128), pieces = 128 / pt;
            for (int c = lane; c < 4 * pieces; c += 32) {
              const int piece = c >> 2, v2 = (c >> 1) & 1, sf = c & 1;
              const int64_t slot = id * 128 + piece * pt, page = slot / a.bs;
              const int t0 = (int)(slot - page * a.bs);
              const uint8_t *base8 = a.kv_cache + page * a.kv_page_bytes + (int64_t)(2 * x.h + v2) * a.bs * 72;
              if (sf)
                bulk_g2s(st + (v2 ? St::kVs : St::kKs) + piece * pt * 8, base8 + a.bs * 64 + t0 * 8, pt * 8, bar);
              else
                bulk_g2s(st + (v2 ? St::kV : 0) + piece * pt * 64, base8 + t0 * 64, pt * 64, bar);
            }
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
  const int row = warp / WPR, part = warp % WPR;
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
    int ev = -126;  // FP8: o is in units of 2^ev
    while (true) {
      const int s = j % kStages;
      bool got = mbar_wait(&sh.full[s], (uint32_t)(j / kStages) & 1, a.status, a.lim);
      if (got && a.test_timeout) got = mbar_wait(&sh.never, 0, a.status, a.lim);
      if (!__all_sync(0xffffffffu, got)) return;  // the warp gives up; the others' waits are bounded too
      const int2 info = sh.info[s];
      ++j;
      if (info.x >= 0 && ((info.y >> row) & 1)) {
        const uint8_t *st = ring + s * St::kBytes;
        const bool cut = info.x * 128 + 127 > p;  // keys after the row's position
#pragma unroll 1
        for (int k0 = part * kKeys; k0 < (part + 1) * kKeys; k0 += 16) {
          // scores of 16 keys: this thread's are keys k0 + 4 t .. + 3
          float c[2][4];
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) c[nt][e] = 0.f;
          float sv[2][4];  // [head g, g + 8][key]
          if constexpr (FMT == 0) {
            // a page is [8 chunks of 16 dims][16 tokens][16 bytes].  Column n
            // of tile nt is key 4 (n / 2) + 2 (nt ^ n / 4) + n % 2: the eight
            // rows of each 8x8 tile then sit in distinct banks
            const int n = lane & 7, nt = (lane >> 3) & 1;
            const int tok = 4 * (n >> 1) + 2 * (nt ^ (n >> 2)) + (n & 1);
            const uint32_t at = smem_u32(st) + (k0 >> 4) * 2048 + (lane >> 4) * 256 + tok * 16;
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) {
              uint32_t w[4];
              ldsm_x4(at + cc * 512, w);
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const uint2 k2 = e4m3x4_f16(w[y]);
                mma_f16(c[y & 1], qf[2 * cc + (y >> 1)], k2.x, k2.y);
              }
            }
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                sv[hh][e] = t < 2 ? c[0][2 * hh + e] : c[1][2 * hh + e];
                sv[hh][2 + e] = t < 2 ? c[1][2 * hh + e] : c[0][2 * hh + e];
              }
          } else {
            // a token is 64 bytes of codes; thread t takes the 16 of dims
            // 32 t .. + 31 (two scale groups).  Column n of tile nt is key
            // 4 (n / 2) + 2 nt + n % 2
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
              const int tok = k0 + 4 * (g >> 1) + 2 * nt + (g & 1);
              const uint4 w4 = *reinterpret_cast<const uint4 *>(st + tok * 64 + 16 * t);
              const uint32_t sf2 = *reinterpret_cast<const uint16_t *>(st + St::kKs + tok * 8 + 2 * t);
              const uint32_t fh = e4m3x4_f16(sf2).x;
              const uint32_t f0 = __byte_perm(fh, fh, 0x1010), f1 = __byte_perm(fh, fh, 0x3232);
              const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                uint32_t h[4];
                e2m1x8_f16(w[y], h);
                const uint32_t f = y < 2 ? f0 : f1;
                mma_f16(c[nt], qf[2 * y], mul_f16x2(h[0], f), mul_f16x2(h[1], f));
                mma_f16(c[nt], qf[2 * y + 1], mul_f16x2(h[2], f), mul_f16x2(h[3], f));
              }
            }
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
#pragma unroll
              for (int e = 0; e < 2; ++e) sv[hh][e] = c[0][2 * hh + e], sv[hh][2 + e] = c[1][2 * hh + e];
          }
          // scale, mask
          float vs[4];
          if constexpr (FMT == 0) {
            const float4 k4 = *reinterpret_cast<const float4 *>(st + St::kKs + (k0 + 4 * t) * 4);
            const float4 v4 = *reinterpret_cast<const float4 *>(st + St::kVs + (k0 + 4 * t) * 4);
            const float ks[4] = {k4.x, k4.y, k4.z, k4.w};
            vs[0] = v4.x, vs[1] = v4.y, vs[2] = v4.z, vs[3] = v4.w;
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
#pragma unroll
              for (int e = 0; e < 4; ++e) sv[hh][e] *= ks[e] * sc[hh];
          } else {
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
#pragma unroll
              for (int e = 0; e < 4; ++e) sv[hh][e] *= sc[hh];
          }
          int left = 4;  // of this thread's four keys, those up to the row's position
          if (cut) {
            left = min(max(p - info.x * 128 - k0 - 4 * t + 1, 0), 4);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (e >= left) {
                sv[0][e] = sv[1][e] = -INFINITY;
                if constexpr (FMT == 0) vs[e] = 0.f;
              }
          }
          // the reference m (and the V unit) move only when a score (a V
          // scale) has outgrown them
          const float top0 = fmaxf(fmaxf(sv[0][0], sv[0][1]), fmaxf(sv[0][2], sv[0][3]));
          const float top1 = fmaxf(fmaxf(sv[1][0], sv[1][1]), fmaxf(sv[1][2], sv[1][3]));
          bool grow = top0 > mref[0] + kAtSlack || top1 > mref[1] + kAtSlack;
          float vtop = 0.f;
          if constexpr (FMT == 0) {
            vtop = fmaxf(fmaxf(fabsf(vs[0]), fabsf(vs[1])), fmaxf(fabsf(vs[2]), fabsf(vs[3])));
            grow |= vtop > pow2i(min(ev + 1, 127));
          }
          if (__any_sync(0xffffffffu, grow)) {
            float f = 1.f;
            if constexpr (FMT == 0) {
              const int e2 = max(ev, min(exponent_of(quad_max(vtop)), 126));
              f = e2 - ev > 125 ? 0.f : pow2i(ev - e2);  // nothing summed yet where it is 0
              ev = e2;
            }
            const float nm[2] = {fmaxf(mref[0], quad_max(top0)), fmaxf(mref[1], quad_max(top1))};
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const float al = nm[hh] == mref[hh] ? 1.f : ex2_approx(mref[hh] - nm[hh]);
              mref[hh] = nm[hh];
              l[hh] *= al;
#pragma unroll
              for (int n = 0; n < 16; ++n) o[n][2 * hh] *= al * f, o[n][2 * hh + 1] *= al * f;
            }
          }
          uint32_t pa[4];
          {
            float unit = 1.f;
            if constexpr (FMT == 0) unit = pow2i(-ev);
            float w[2][4];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const float base = mref[hh] == -INFINITY ? 0.f : mref[hh] - kAtLift;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float y = ex2_approx(sv[hh][e] - base);
                l[hh] += y;
                w[hh][e] = FMT == 0 ? y * (vs[e] * unit) : y;
              }
            }
            pa[0] = f16x2_bits(w[0][0], w[0][1]);
            pa[1] = f16x2_bits(w[1][0], w[1][1]);
            pa[2] = f16x2_bits(w[0][2], w[0][3]);
            pa[3] = f16x2_bits(w[1][2], w[1][3]);
          }
          // o += weights . values (keys 4 t, 4 t + 1 | 4 t + 2, 4 t + 3 are this thread's k rows)
          if constexpr (FMT == 0) {
            // a page is [128 dims][16 tokens]: tile n's rows are dims 8 n ..
            const uint32_t keep = left >= 4 ? 0xffffffffu : (1u << (8 * left)) - 1u;
            const uint32_t at = smem_u32(st) + St::kV + (k0 >> 4) * 2048 + lane * 16;
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4) {
              uint32_t w[4];
              ldsm_x4(at + q4 * 512, w);
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const uint2 v2 = e4m3x4_f16(cut ? w[y] & keep : w[y]);
                mma_f16(o[4 * q4 + y], pa, v2.x, v2.y);
              }
            }
          } else {
            // thread g takes dims 16 g .. + 15 (one scale group) of its four
            // tokens; nibbles of two tokens are paired before the conversion
            uint32_t w[4][2];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint2 w2 = *reinterpret_cast<const uint2 *>(st + St::kV + (k0 + 4 * t + e) * 64 + 8 * g);
              w[e][0] = w2.x, w[e][1] = w2.y;
            }
            uint32_t sf4 = *reinterpret_cast<const uint32_t *>(st + St::kVs + (k0 + 4 * t) * 8 + 4 * g);
            if (cut) {
              sf4 &= left >= 4 ? 0xffffffffu : (1u << (8 * left)) - 1u;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (e >= left) w[e][0] = w[e][1] = 0u;
            }
            const uint2 f = e4m3x4_f16(sf4);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              constexpr uint32_t kLow = 0x0f0f0f0fu;
              uint32_t e01[4], d01[4], e23[4], d23[4];  // even, odd dims of tokens 0, 1 and 2, 3
              e2m1x8_f16((w[0][y] & kLow) | ((w[1][y] & kLow) << 4), e01);
              e2m1x8_f16(((w[0][y] >> 4) & kLow) | (w[1][y] & ~kLow), d01);
              e2m1x8_f16((w[2][y] & kLow) | ((w[3][y] & kLow) << 4), e23);
              e2m1x8_f16(((w[2][y] >> 4) & kLow) | (w[3][y] & ~kLow), d23);
#pragma unroll
              for (int b = 0; b < 4; ++b) {
                mma_f16(o[8 * y + 2 * b], pa, mul_f16x2(e01[b], f.x), mul_f16x2(e23[b], f.y));
                mma_f16(o[8 * y + 2 * b + 1], pa, mul_f16x2(d01[b], f.x), mul_f16x2(d23[b], f.y));
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
                for (int n = 0; n < 16; n += 2)
                  *reinterpret_cast<uint32_t *>(dst + 16 * (2 * t + e) + n) =
                      bf16x2_bits(o[n][2 * hh + e] * inv, o[n + 1][2 * hh + e] * inv);
            }
          } else {
            float *dst = pp + (row * 16 + head) * kHeadDim;
#pragma unroll
            for (int n = 0; n < 16; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                dst[FMT == 0 ? 8 * n + 2 * t + e : 16 * (2 * t + e) + n] = o[n][2 * hh + e];
            if (t == 0)
              *reinterpret_cast<float2 *>(pp + kAtMaxRows * 16 * kHeadDim + (row * 16 + head) * 2) =
                  make_float2(mref[hh], l[hh]);
          }
        }
      }
    } else {
      // the row's warps meet in shared memory
      float *mine = joint + warp * 16 * kHeadDim;
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int head = g + 8 * hh;
#pragma unroll
        for (int n = 0; n < 16; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            mine[head * kHeadDim + (FMT == 0 ? 8 * n + 2 * t + e : 16 * (2 * t + e) + n)] = o[n][2 * hh + e];
        if (t == 0) sh.ml[warp][head] = make_float2(mref[hh], l[hh]);
      }
      if (!fin_sync()) return;
      if (row < x.rows) {
        for (int head = part; head < a.group; head += WPR) {
          float top = -INFINITY;
#pragma unroll
          for (int w = 0; w < WPR; ++w) top = fmaxf(top, sh.ml[row * WPR + w][head].x);
          float sum = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < WPR; ++w) {
            const float2 ml = sh.ml[row * WPR + w][head];
            const float f = ml.x == -INFINITY && ml.y == 0.f ? 0.f : ml.x == top ? 1.f : ex2_approx(ml.x - top);
            const float4 y =
                *reinterpret_cast<const float4 *>(joint + ((row * WPR + w) * 16 + head) * kHeadDim + 4 * lane);
            sum += f * ml.y;
            if (f != 0.f) acc.x += f * y.x, acc.y += f * y.y, acc.z += f * y.z, acc.w += f * y.w;
          }
          if (whole) {
            const float inv = sum == 0.f ? 0.f : a.out_scale / sum;
            *reinterpret_cast<uint2 *>(a.out + m * a.out_stride + (int64_t)(x.h * a.group + head) * kHeadDim + 4 * lane) =
                make_uint2(bf16x2_bits(acc.x * inv, acc.y * inv), bf16x2_bits(acc.z * inv, acc.w * inv));
          } else {
            *reinterpret_cast<float4 *>(pp + (row * 16 + head) * kHeadDim + 4 * lane) = acc;
            if (lane == 0)
              *reinterpret_cast<float2 *>(pp + kAtMaxRows * 16 * kHeadDim + (row * 16 + head) * 2) =
                  make_float2(top, sum);
          }
        }
      }
      if (!fin_sync()) return;  // `joint` is free for the next item
    }
  }
}

// Join the partial results of items that several CTAs share, in CTA order:
// a warp an (item, row, head), a lane four dims.  The first CTA's partial is
// its slot 1 (the item starts there), the others' their slot 0.
__global__ void __launch_bounds__(128) pa_attn_join_kernel(const __grid_constant__ AttnParams a, int grid) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int it = blockIdx.x / a.rows_per, row = blockIdx.x % a.rows_per, head = 4 * blockIdx.y + warp;
  pdl_wait();
  if (head >= a.group) return;
  const int2 s = a.shares[it];
  const int c0 = max(s.x, 0), c1 = min(s.y, grid - 1);
  if (c1 <= c0) return;
  const int rg = it / a.n_kv, h = it % a.n_kv, r = rg / a.row_groups, row0 = (rg - r * a.row_groups) * a.rows_per;
  if (row0 + row >= a.q_len) return;
  auto part = [&](int c) { return a.part + (int64_t)(2 * c + (c == c0 ? 1 : 0)) * kAtPartFloats; };
  const int at = row * 16 + head;
  float top = -INFINITY;
  for (int c = c0 + lane; c <= c1; c += 32) top = fmaxf(top, part(c)[kAtMaxRows * 16 * kHeadDim + 2 * at]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int c = c0; c <= c1; ++c) {
    const float2 ml = *reinterpret_cast<const float2 *>(part(c) + kAtMaxRows * 16 * kHeadDim + 2 * at);
    const float4 y = *reinterpret_cast<const float4 *>(part(c) + at * kHeadDim + 4 * lane);
    const float f = ml.x == -INFINITY && ml.y == 0.f ? 0.f : ml.x == top ? 1.f : ex2_approx(ml.x - top);
    sum += f * ml.y;
    if (f != 0.f) acc.x += f * y.x, acc.y += f * y.y, acc.z += f * y.z, acc.w += f * y.w;
  }
  const float inv = sum == 0.f ? 0.f : a.out_scale / sum;
  const int64_t m = (int64_t)r * a.q_len + row0 + row;
  *reinterpret_cast<uint2 *>(a.out + m * a.out_stride + (int64_t)(h * a.group + head) * kHeadDim + 4 * lane) =
      make_uint2(bf16x2_bits(acc.x * inv, acc.y * inv), bf16x2_bits(acc.z * inv, acc.w * inv));
}

// Rows an item of q_len rows takes, and items a (request, KV head).
static inline void attn_rows(int q_len, int *groups, int *rows) {
  *groups = (q_len + kAtMaxRows - 1) / kAtMaxRows;
  *rows = (q_len + *groups - 1) / *groups;
}

template <int FMT>
static cudaError_t launch_attn(const AttnParams &a, int sms, bool pdl, cudaStream_t stream) {
  using Kern = void (*)(const AttnParams);
  Kern kern = pa_attn_kernel<FMT, 1>;
  int smem = attn_smem<FMT, 1>();
  if (a.rows_per == 1) kern = pa_attn_kernel<FMT, 8>, smem = attn_smem<FMT, 8>();
  else if (a.rows_per == 2) kern = pa_attn_kernel<FMT, 4>, smem = attn_smem<FMT, 4>();
  else if (a.rows_per <= 4) kern = pa_attn_kernel<FMT, 2>, smem = attn_smem<FMT, 2>();
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(kern), smem);
  if (e != cudaSuccess) return e;
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
  e = cudaLaunchKernelEx(&cfg, kern, a);
  if (e != cudaSuccess || !a.sliced || a.test_timeout) return e;
  cfg.gridDim = dim3(a.items * a.rows_per, (a.group + 3) / 4);
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, pa_attn_join_kernel, a, sms);
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
    if (x.block_size != 16 || (kps != 0 && kps < 8) || c.num_pages16 < 1) return PA_ERR_CONFIG;
    if (!aligned(c.k_cache, 16) || !aligned(c.v_cache, 16) || !aligned(c.k_scale, 16) || !aligned(c.v_scale, 16))
      return PA_ERR_ALIGN;
    if (kps == 0) kps = 8;
  } else {
    if (!c.kv_cache) return PA_ERR_NULL;
    const int bs = x.block_size;
    if (bs < 4 || bs % 4 || bs > 1024 || c.kv_pages < 1) return PA_ERR_CONFIG;
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
  pa::attn_rows(x.q_len, &a.row_groups, &a.rows_per);
  a.items = x.R * a.row_groups * x.n_kv_heads;
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
