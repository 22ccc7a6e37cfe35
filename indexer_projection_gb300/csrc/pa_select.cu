// Block selection from indexer scores (pre_attn_select_blocks): per (row,
// index head) the maximum of each block's 128 score columns, then the pinned
// blocks and the largest of the others, topk in all, ties to the lower block.
//
// The scores are read once (4 bytes a key: HBM bounds the whole, latency the
// small calls).  A cluster of CTAs takes one (row, head), each CTA a run of
// its blocks; a block's maximum becomes a 32-bit key whose unsigned order is
// the scores' (0: not selectable, all ones: pinned) in the first CTA's shared
// memory.  That CTA finds the last key to be taken by radix selection (8 bits
// a pass from the highest bit in which the keys differ, until a digit is
// taken whole) and writes the blocks above it, and the first of those equal
// to it, in block order.
//
// One GB300, calls back to back: 64 requests x 7 rows x 2 heads, lengths up to
// 32767, 61 MB in 13.7 us (4.4 TB/s, 0.65 of the measured copy rate; the
// selection behind the last loads is what is left); 3 rows x 4 heads of 131072
// keys 6.8 us, 8 rows of up to 32768 3.7 us, latency.
#include <cstdint>

#include "../../include/pre_attn.h"
#include "pa_device.cuh"
#include "pa_launch.h"

namespace pa {

constexpr int kSelThreads = 256;
constexpr int kSelMaxWidth = 16384;
constexpr int kSelMaxTopk = 256;

struct SelectParams {
  const float *scores;
  int64_t score_stride, head_stride;
  int n_heads;
  const int32_t *seq_lens;
  int R, q_len, bt_width, init_blocks, local_blocks, topk;
  int32_t *blocks, *counts;
  uint32_t *status;
  const int32_t *block_table;  // or null
  int64_t num_blocks;
};

// Order-preserving key of a block's maximum: greater score, greater key;
// -0 and +0 alike; 0 for -inf (nothing to select).
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x == -INFINITY) return 0u;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u >> 31) ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads, 6) pa_select_kernel(const __grid_constant__ SelectParams a) {
  extern __shared__ uint32_t keys[];  // [bt_width], of the cluster's first CTA
  __shared__ uint32_t hist[2][256];
  __shared__ int3 pick;               // the digit found, what remains to take in it, what it holds
  __shared__ uint4 warp_range[kSelThreads / 32];
  __shared__ int warp_sum[2][kSelThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t ctas, rank;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ctas));
  rank = cta_rank();
  cluster_arrive_relaxed();  // the first CTA runs before the others store to it
  const int item = blockIdx.x / ctas, m = item / a.n_heads, h = item - m * a.n_heads;
  const int r = m / a.q_len, i = m - r * a.q_len;
  pdl_wait();
  pdl_trigger();
  const int seq = __ldg(a.seq_lens + r);
  int nb = 0;
  if (seq >= a.q_len && (seq - 1) / 128 + 1 <= a.bt_width) nb = (seq - a.q_len + i) / 128 + 1;
  else if (seq > 0 && rank == 0 && tid == 0) set_status(a.status, kDevSlotRange);
  const float *row = a.scores + (int64_t)h * a.head_stride + (int64_t)m * a.score_stride;
  const uint32_t keys0 = mapa(smem_u32(keys), 0);
  cluster_wait();
  // eight lanes a block, four blocks a warp: each lane has four 16-byte loads
  // of its block in flight, twice (blocks b and b + 32)
  const int b0 = (int)((int64_t)nb * rank / ctas), b1 = (int)((int64_t)nb * (rank + 1) / ctas);
  const int sub = lane & 7;
  constexpr int kStep = kSelThreads / 8;
  for (int b = b0 + (tid >> 3); b < b1 + (tid >> 3); b += 2 * kStep) {  // the same number of turns for a warp's lanes
    float4 v[2][4];
    bool scored[2], lost[2];  // lost: scored columns that no scorer wrote
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int bu = b + u * kStep;
      scored[u] = bu < b1 && bu >= a.init_blocks && bu < nb - a.local_blocks;
      lost[u] = false;
      if (a.block_table && scored[u]) {
        const int64_t id = __ldg(a.block_table + (int64_t)r * a.bt_width + bu);
        lost[u] = id < 0 || id >= a.num_blocks;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        v[u][k] = scored[u] ? __ldg(reinterpret_cast<const float4 *>(row + bu * 128) + 8 * k + sub)
                          : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int bu = b + u * kStep;
      float x = -INFINITY;  // fmaxf leaves NaN out
#pragma unroll
      for (int k = 0; k < 4; ++k) x = fmaxf(fmaxf(fmaxf(x, v[u][k].x), fmaxf(v[u][k].y, v[u][k].z)), v[u][k].w);
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
      if (lost[u]) x = -INFINITY;
      if (sub == 0 && bu < b1) {
        if (lost[u]) set_status(a.status, kDevSlotRange);
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(keys0 + 4 * bu), "r"(scored[u] ? score_key(x) : 0xffffffffu)
                     : "memory");
      }
    }
  }
  cluster_sync();
  if (rank != 0) return;
  // what is to be found: of the keys that are neither pinned nor 0, the
  // `need` largest; how many there are, and their range
  int pins = 0;
  uint32_t most = 0, least = 0xffffffffu;
  int some = 0;
  for (int b = tid; b < nb; b += kSelThreads) {
    const uint32_t k = keys[b];
    if (k == 0xffffffffu) ++pins;
    else if (k != 0) ++some, most = max(most, k), least = min(least, k);
  }
  pins = __reduce_add_sync(0xffffffffu, pins), some = __reduce_add_sync(0xffffffffu, some);
  most = __reduce_max_sync(0xffffffffu, most), least = __reduce_min_sync(0xffffffffu, least);
  if (lane == 0) warp_range[warp] = make_uint4(pins, some, most, least);
  hist[0][tid] = 0;
  __syncthreads();
  pins = some = 0;
#pragma unroll
  for (int w = 0; w < kSelThreads / 32; ++w) {
    const uint4 r4 = warp_range[w];
    pins += r4.x, some += r4.y, most = max(most, r4.z), least = min(least, r4.w);
  }
  // the need-th largest key: radix selection from the highest bit in which
  // they differ, 8 bits a pass, until a digit's keys are all taken.  In the
  // end a block is taken if its key is above T, or is T and among the first
  // `need` such
  int need = a.topk - pins;
  uint32_t T = 0;
  if (need <= 0) T = 0xfffffffeu, need = 0;
  else if (some <= need) need = 0;
  else {
    int left = 32 - __clz(most ^ least);  // bits not settled yet
    T = left < 32 ? most >> left << left : 0u;
    for (int pass = 0; left > 0; ++pass) {
      const int bits = min(left, 8), shift = left - bits;
      uint32_t *h0 = hist[pass & 1];
      for (int b = tid; b < nb; b += kSelThreads) {
        const uint32_t k = keys[b];
        if (k != 0 && k != 0xffffffffu && (left == 32 || ((k ^ T) >> left) == 0))
          atomicAdd(&h0[(k >> shift) & ((1u << bits) - 1u)], 1u);
      }
      __syncthreads();
      if (warp == 0) {  // digits from the top: lane l holds 255 - 8 l .. 248 - 8 l
        int c[8], sum = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) sum += c[k] = (int)h0[255 - 8 * lane - k];
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
        int before = incl - sum;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (before < need && before + c[k] >= need) pick = make_int3(255 - 8 * lane - k, need - before, c[k]);
          before += c[k];
        }
      } else if (tid >= 32) {
        for (int k = tid - 32; k < 256; k += kSelThreads - 32) hist[(pass + 1) & 1][k] = 0;
      }
      __syncthreads();
      T |= (uint32_t)pick.x << shift;
      need = pick.y;
      left = shift;
      if (pick.y == pick.z) {  // the whole digit
        T -= 1, need = 0;
        break;
      }
    }
  }
  int32_t *out = a.blocks + (int64_t)item * a.topk;
  int taken = 0, equal = 0;  // before this chunk
  for (int c0 = 0; c0 < nb; c0 += kSelThreads) {
    const int b = c0 + tid;
    const uint32_t key = b < nb ? keys[b] : 0u;
    bool take = key > T;
    if (need > 0) {  // the same for the CTA
      const uint32_t eq = __ballot_sync(0xffffffffu, key == T);
      if (lane == 0) warp_sum[0][warp] = __popc(eq);
      __syncthreads();
      int e = equal + __popc(eq & ((1u << lane) - 1u));
#pragma unroll
      for (int w = 0; w < kSelThreads / 32; ++w) {
        const int v = warp_sum[0][w];
        if (w < warp) e += v;
        equal += v;
      }
      take |= key == T && e < need;
    }
    const uint32_t tk = __ballot_sync(0xffffffffu, take);
    if (lane == 0) warp_sum[1][warp] = __popc(tk);
    __syncthreads();
    int at = taken + __popc(tk & ((1u << lane) - 1u));
#pragma unroll
    for (int w = 0; w < kSelThreads / 32; ++w) {
      const int v = warp_sum[1][w];
      if (w < warp) at += v;
      taken += v;
    }
    if (take) out[at] = b;
    if (c0 + kSelThreads < nb) __syncthreads();
  }
  for (int k = taken + tid; k < a.topk; k += kSelThreads) out[k] = -1;
  if (tid == 0) a.counts[item] = taken;
}

static cudaError_t launch_select(const SelectParams &a, cudaStream_t stream) {
  const int smem = a.bt_width * 4;
  const cudaError_t e0 = ensure_smem_attr(reinterpret_cast<const void *>(pa_select_kernel), kSelMaxWidth * 4);
  if (e0 != cudaSuccess) return e0;
  const int64_t items = (int64_t)a.R * a.q_len * a.n_heads;
  const int sms = current_device_sms();
  // CTAs a (row, head): more while the grid is less than two CTAs an SM and
  // each has 16 blocks to read (1, 2, 4, 8 CTAs: 12 (row, head)s of 1024
  // blocks 13.6, 9.6, 7.7, 6.7 us; 8 of up to 256 5.1, 4.2, 3.8, 3.6)
  int ctas = 1;
  while (ctas < 8 && items * ctas < 2 * sms && a.bt_width >= 32 * ctas) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cfg.stream = stream;
  cfg.gridDim = dim3((unsigned)(items * ctas));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  return cudaLaunchKernelEx(&cfg, pa_select_kernel, a);
}

}  // namespace pa

extern "C" int pre_attn_select_blocks(const pa_select_args *in, void *stream) {
  if (!in) return PA_ERR_NULL;
  const pa_select_args &x = *in;
  auto aligned = [](const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
  if (!x.scores || !x.seq_lens || !x.blocks || !x.counts || !x.status) return PA_ERR_NULL;
  if (x.R < 0 || x.R > 65535 || x.q_len < 1 || x.q_len > 16 || x.n_heads < 1 || x.n_heads > 64 || x.bt_width < 1 ||
      x.bt_width > pa::kSelMaxWidth || x.topk < 1 || x.topk > pa::kSelMaxTopk)
    return PA_ERR_SHAPE;
  if (x.init_blocks < 0 || x.local_blocks < 0 || (int64_t)x.init_blocks + x.local_blocks > x.topk) return PA_ERR_CONFIG;
  if (x.score_stride < (int64_t)x.bt_width * 128 ||
      (x.n_heads > 1 && x.score_head_stride < (int64_t)x.R * x.q_len * x.score_stride) ||
      (x.block_table && x.num_blocks < 1))
    return PA_ERR_SHAPE;
  if (!aligned(x.scores, 16) || x.score_stride % 4 || x.score_head_stride % 4 || !aligned(x.seq_lens, 4) ||
      !aligned(x.blocks, 4) || !aligned(x.counts, 4) || !aligned(x.status, 4) || !aligned(x.block_table, 4))
    return PA_ERR_ALIGN;
  if (x.R == 0) return PA_OK;
  pa::SelectParams a;
  a.scores = x.scores;
  a.score_stride = x.score_stride;
  a.head_stride = x.score_head_stride;
  a.n_heads = x.n_heads;
  a.seq_lens = x.seq_lens;
  a.R = x.R;
  a.q_len = x.q_len;
  a.bt_width = x.bt_width;
  a.init_blocks = x.init_blocks;
  a.local_blocks = x.local_blocks;
  a.topk = x.topk;
  a.blocks = x.blocks;
  a.counts = x.counts;
  a.status = x.status;
  a.block_table = x.block_table;
  a.num_blocks = x.num_blocks;
  const cudaError_t e = pa::launch_select(a, (cudaStream_t)stream);
  return e == cudaSuccess ? PA_OK : pa::record_cuda_error(e);
}
