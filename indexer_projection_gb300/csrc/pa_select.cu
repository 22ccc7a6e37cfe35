// Block selection from indexer scores (pre_attn_select_blocks): per (row,
// index head) the maximum of each block's 128 score columns, then the pinned
// blocks and the largest of the others, topk in all, ties to the lower block.
//
// The scores are read once (4 bytes a key: HBM bounds the whole, latency the
// small calls).  A cluster of CTAs takes one (row, head), each CTA a run of
// its blocks; a block's maximum becomes a 32-bit key whose unsigned order is
// the scores' (0: not selectable, all ones: pinned) in the first CTA's shared
// memory.  That CTA finds the topk-th key by radix selection (8 bits a pass)
// and writes the blocks above it, and the first of those equal to it, in
// block order.
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
};

// Order-preserving key of a block's maximum: greater score, greater key;
// -0 and +0 alike; 0 for -inf (nothing to select).
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x == -INFINITY) return 0u;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u >> 31) ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads) pa_select_kernel(const __grid_constant__ SelectParams a) {
  extern __shared__ uint32_t keys[];  // [bt_width], of the cluster's first CTA
  __shared__ uint32_t hist[256];
  __shared__ uint32_t pick[2];        // the digit found, what remains to take in it
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
  const int b1 = (int)((int64_t)nb * (rank + 1) / ctas);
  for (int b = (int)((int64_t)nb * rank / ctas) + warp; b < b1; b += kSelThreads / 32) {
    const bool pinned = b < a.init_blocks || b >= nb - a.local_blocks;
    uint32_t key = 0xffffffffu;
    if (!pinned) {
      const float4 v = __ldg(reinterpret_cast<const float4 *>(row + b * 128) + lane);
      float x = fmaxf(fmaxf(fmaxf(-INFINITY, v.x), fmaxf(-INFINITY, v.y)), fmaxf(fmaxf(-INFINITY, v.z), fmaxf(-INFINITY, v.w)));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
      key = score_key(x);
    }
    if (lane == 0) asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(keys0 + 4 * b), "r"(key) : "memory");
  }
  cluster_sync();
  if (rank != 0) return;
  // the topk-th largest key: T, of whose holders `need` are taken
  uint32_t T = 0, need = (uint32_t)a.topk;
  for (int shift = 24; shift >= 0; shift -= 8) {
    hist[tid] = 0;
    __syncthreads();
    for (int b = tid; b < nb; b += kSelThreads)
      if (shift == 24 || (keys[b] >> (shift + 8)) == (T >> (shift + 8))) atomicAdd(&hist[(keys[b] >> shift) & 255u], 1u);
    __syncthreads();
    if (warp == 0) {
      // digits from the top: lane l holds 255 - 8 l .. 248 - 8 l
      uint32_t c[8], sum = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) sum += c[k] = hist[255 - 8 * lane - k];
      uint32_t incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      uint32_t before = incl - sum;
      if (lane == 31 && incl < need) pick[0] = 0, pick[1] = hist[0];  // fewer blocks than topk: all of them
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (before < need && before + c[k] >= need) pick[0] = 255 - 8 * lane - k, pick[1] = need - before;
        before += c[k];
      }
    }
    __syncthreads();
    T |= pick[0] << shift;
    need = pick[1];
    __syncthreads();
  }
  // blocks above T, and the first `need` equal to it (none where T is 0: not selectable)
  if (T == 0) need = 0;
  int32_t *out = a.blocks + (int64_t)item * a.topk;
  int taken = 0, equal = 0;  // before this chunk
  for (int b0 = 0; b0 < nb; b0 += kSelThreads) {
    const int b = b0 + tid;
    const uint32_t key = b < nb ? keys[b] : 0u;
    const uint32_t eq = __ballot_sync(0xffffffffu, key == T && key != 0u);
    if (lane == 0) warp_sum[0][warp] = __popc(eq);
    __syncthreads();
    int e = equal + __popc(eq & ((1u << lane) - 1u));
    for (int w = 0; w < warp; ++w) e += warp_sum[0][w];
    for (int w = 0; w < kSelThreads / 32; ++w) equal += warp_sum[0][w];
    const bool take = key > T || (key == T && key != 0u && e < (int)need);
    const uint32_t tk = __ballot_sync(0xffffffffu, take);
    if (lane == 0) warp_sum[1][warp] = __popc(tk);
    __syncthreads();
    int at = taken + __popc(tk & ((1u << lane) - 1u));
    for (int w = 0; w < warp; ++w) at += warp_sum[1][w];
    for (int w = 0; w < kSelThreads / 32; ++w) taken += warp_sum[1][w];
    if (take) out[at] = b;
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
  int ctas = 1;  // a (row, head): while the grid is less than two CTAs an SM and each has 16 blocks to read
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
      (x.n_heads > 1 && x.score_head_stride < (int64_t)x.R * x.q_len * x.score_stride))
    return PA_ERR_SHAPE;
  if (!aligned(x.scores, 16) || x.score_stride % 4 || x.score_head_stride % 4 || !aligned(x.seq_lens, 4) ||
      !aligned(x.blocks, 4) || !aligned(x.counts, 4) || !aligned(x.status, 4))
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
  const cudaError_t e = pa::launch_select(a, (cudaStream_t)stream);
  return e == cudaSuccess ? PA_OK : pa::record_cuda_error(e);
}
