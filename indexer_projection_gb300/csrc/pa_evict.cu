// Eviction of a request's blocks with the least accumulated attention weight
// (pre_attn_evict_blocks): of nb > keep blocks the pinned ones (the first, the
// last) stay and of the others the largest weights, ties to the lower block;
// the rows of the block table and of the weights move up over the evicted.
//
// A CTA takes a request, its entries in registers: warp w owns 32 K
// consecutive ones, of which lane l holds every 32nd, so that loads are
// coalesced and an order over the row takes ballots and one exchange of the
// warps' counts.  The last key to stay is found by radix selection (8 bits a
// pass from the highest bit in which the keys differ, until a digit stays
// whole).
//
// Measured: 64 requests of up to 256 blocks 3.0 us (a launch, then 0.5 for the
// length and the row, 1 for the radix passes); 3 of up to 8192 blocks 9.5 us, of
// which the row's loads are 1, the radix passes 3 to 4, the order 1 and the
// stores 2.  Eight counters a digit, by the lane, took 10.4 (more to clear and
// add up than the additions to one counter cost).  The bytes, 16 a block, are
// 0.04 us of HBM: latency on one SM a request bounds it.
#include <cstdint>

#include "../../include/pre_attn.h"
#include "pa_device.cuh"
#include "pa_launch.h"

namespace pa {

constexpr int kEvMaxWidth = 16384;
constexpr int kEvMaxThreads = 1024;

struct EvictParams {
  const float *weights;
  int64_t stride;
  const int32_t *table, *seq_lens;
  int R, W, keep, init, local;
  float *weights_out;
  int64_t stride_out;
  int32_t *table_out, *lens_out, *evicted, *counts;
  uint32_t *status;
};

// Order-preserving key of a weight: greater weight, greater key; -0 and +0
// alike, NaN as -inf; neither 0 nor all ones.
__device__ __forceinline__ uint32_t weight_key(float x) {
  if (!(x == x)) x = -INFINITY;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u >> 31) ? ~u : u | 0x80000000u;
}

// The sum over the warps' counts (one a warp, in `c`), and those before this warp's.
__device__ __forceinline__ int warps_before(const int *c, int warps, int warp, int *all) {
  const int lane = threadIdx.x & 31;
  const int v = lane < warps ? c[lane] : 0;
  *all = __reduce_add_sync(0xffffffffu, v);
  return __reduce_add_sync(0xffffffffu, lane < warp ? v : 0);
}

template <int K>  // entries a thread
__global__ void __launch_bounds__(kEvMaxThreads) pa_evict_kernel(const __grid_constant__ EvictParams a) {
  __shared__ uint32_t hist[2][256];
  __shared__ int3 pick;  // the digit found, what remains to stay in it, what it holds
  __shared__ uint2 warp_range[32];
  __shared__ int warp_count[2][32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
  const int r = blockIdx.x;
  const int first = warp * 32 * K + lane;  // entry k of the thread: first + 32 k
  for (int d = tid; d < 512; d += blockDim.x) hist[d >> 8][d & 255] = 0;
  pdl_wait();
  pdl_trigger();
  const int n = a.seq_lens[r];  // (plain loads: the outputs may be the inputs)
  float w[K];
  int32_t id[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int b = first + 32 * k;
    w[k] = b < a.W ? a.weights[r * a.stride + b] : 0.f;
    id[k] = b < a.W ? a.table[(int64_t)r * a.W + b] : -1;
  }
  int nb = n > 0 ? (n - 1) / 128 + 1 : 0;
  if (nb > a.W) {
    if (tid == 0) set_status(a.status, kDevSlotRange);
    nb = 0;
  }
  const int gone = max(nb - a.keep, 0);  // the same for the CTA
  uint32_t key[K];                       // all ones: stays (pinned, or behind the last block)
  uint32_t most = 0, least = 0xffffffffu;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int b = first + 32 * k;
    key[k] = 0xffffffffu;
    if (gone > 0 && b >= a.init && b < nb - a.local) {
      key[k] = weight_key(w[k]);
      most = max(most, key[k]), least = min(least, key[k]);
    }
  }
  // the smallest key that stays, T, and how many of those equal to it do
  uint32_t T = 0;
  int need = 0;
  if (gone > 0) {
    need = nb - a.init - a.local - gone;  // of the keys that are not pinned
    most = __reduce_max_sync(0xffffffffu, most), least = __reduce_min_sync(0xffffffffu, least);
    if (lane == 0) warp_range[warp] = make_uint2(most, least);
    __syncthreads();
    {
      const uint2 v = lane < warps ? warp_range[lane] : make_uint2(0u, 0xffffffffu);
      most = __reduce_max_sync(0xffffffffu, v.x), least = __reduce_min_sync(0xffffffffu, v.y);
    }
    if (need <= 0) {  // only the pinned ones
      T = 0xfffffffeu, need = 0;
    } else {
      int left = 32 - __clz(most ^ least);  // bits not settled yet
      T = left < 32 ? most >> left << left : 0u;
      for (int pass = 0; left > 0; ++pass) {
        const int bits = min(left, 8), shift = left - bits;
        uint32_t *h0 = hist[pass & 1];
#pragma unroll
        for (int k = 0; k < K; ++k)
          if (key[k] != 0xffffffffu && (left == 32 || ((key[k] ^ T) >> left) == 0))
            atomicAdd(&h0[(key[k] >> shift) & ((1u << bits) - 1u)], 1u);
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
        }
        __syncthreads();
        T |= (uint32_t)pick.x << shift;
        need = pick.y;
        left = shift;
        if (pick.y == pick.z) {  // the whole digit
          T -= 1, need = 0;
          break;
        }
        for (int d = tid; d < 256; d += blockDim.x) h0[d] = 0;  // (used again two passes on)
      }
    }
  }
  // which entries stay, and where the row's order puts them
  uint32_t stay[K];  // ballots
  int kept = 0;      // of the warp
  {
    int equal = 0;  // of the warp, then before the entry
    if (need > 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) equal += __popc(__ballot_sync(0xffffffffu, key[k] == T));
      if (lane == 0) warp_count[0][warp] = equal;
      __syncthreads();
      int all;
      equal = warps_before(warp_count[0], warps, warp, &all);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      bool in = key[k] > T;
      if (need > 0) {
        const uint32_t eq = __ballot_sync(0xffffffffu, key[k] == T);
        in |= key[k] == T && equal + __popc(eq & ((1u << lane) - 1u)) < need;
        equal += __popc(eq);
      }
      stay[k] = __ballot_sync(0xffffffffu, in && first + 32 * k < a.W);
      kept += __popc(stay[k]);
    }
  }
  if (lane == 0) warp_count[1][warp] = kept;
  __syncthreads();  // (and every entry has been read: the outputs may be the inputs)
  int all;
  int at = warps_before(warp_count[1], warps, warp, &all);
  int32_t *table = a.table_out + (int64_t)r * a.W, *out = a.evicted + (int64_t)r * a.W;
  float *weights = a.weights_out + r * a.stride_out;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int b = first + 32 * k, pos = at + __popc(stay[k] & ((1u << lane) - 1u));
    if (b < a.W) {
      if ((stay[k] >> lane) & 1u) table[pos] = id[k], weights[pos] = w[k];
      else out[b - pos] = id[k];
      if (b >= a.W - gone) table[b] = -1, weights[b] = 0.f;
      if (b >= gone) out[b] = -1;
    }
    at += __popc(stay[k]);
  }
  if (tid == 0) a.counts[r] = gone, a.lens_out[r] = n - 128 * gone;
}

static cudaError_t launch_evict(const EvictParams &a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  cfg.gridDim = dim3((unsigned)a.R);
  int per = 1;  // entries a thread
  while (per * kEvMaxThreads < a.W) per *= 2;
  cfg.blockDim = dim3((unsigned)((a.W + 32 * per - 1) / (32 * per) * 32));
  switch (per) {
    case 1: return cudaLaunchKernelEx(&cfg, pa_evict_kernel<1>, a);
    case 2: return cudaLaunchKernelEx(&cfg, pa_evict_kernel<2>, a);
    case 4: return cudaLaunchKernelEx(&cfg, pa_evict_kernel<4>, a);
    case 8: return cudaLaunchKernelEx(&cfg, pa_evict_kernel<8>, a);
    default: return cudaLaunchKernelEx(&cfg, pa_evict_kernel<16>, a);
  }
}

}  // namespace pa

extern "C" int pre_attn_evict_blocks(const pa_evict_args *in, void *stream) {
  if (!in) return PA_ERR_NULL;
  const pa_evict_args &x = *in;
  auto aligned = [](const void *p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; };
  if (!x.weights || !x.block_table || !x.seq_lens || !x.weights_out || !x.block_table_out || !x.seq_lens_out ||
      !x.evicted || !x.counts || !x.status)
    return PA_ERR_NULL;
  if (x.R < 0 || x.R > 65535 || x.bt_width < 1 || x.bt_width > pa::kEvMaxWidth || x.weights_stride < x.bt_width ||
      x.weights_out_stride < x.bt_width)
    return PA_ERR_SHAPE;
  const int local = x.local_blocks > 1 ? x.local_blocks : 1;
  if (x.init_blocks < 0 || x.local_blocks < 0 || (int64_t)x.init_blocks + local > x.keep) return PA_ERR_CONFIG;
  if (!aligned(x.weights) || !aligned(x.block_table) || !aligned(x.seq_lens) || !aligned(x.weights_out) ||
      !aligned(x.block_table_out) || !aligned(x.seq_lens_out) || !aligned(x.evicted) || !aligned(x.counts) ||
      !aligned(x.status))
    return PA_ERR_ALIGN;
  if (x.R == 0) return PA_OK;
  {  // the spans of the tensors, inputs first: only an output on its own input may overlap
    struct Span {
      uintptr_t p, n;
    };
    auto rows = [&](int64_t stride) { return (uintptr_t)((x.R - 1) * stride + x.bt_width) * 4; };
    const Span s[8] = {{reinterpret_cast<uintptr_t>(x.weights), rows(x.weights_stride)},
                       {reinterpret_cast<uintptr_t>(x.block_table), rows(x.bt_width)},
                       {reinterpret_cast<uintptr_t>(x.seq_lens), (uintptr_t)x.R * 4},
                       {reinterpret_cast<uintptr_t>(x.weights_out), rows(x.weights_out_stride)},
                       {reinterpret_cast<uintptr_t>(x.block_table_out), rows(x.bt_width)},
                       {reinterpret_cast<uintptr_t>(x.seq_lens_out), (uintptr_t)x.R * 4},
                       {reinterpret_cast<uintptr_t>(x.evicted), rows(x.bt_width)},
                       {reinterpret_cast<uintptr_t>(x.counts), (uintptr_t)x.R * 4}};
    for (int o = 3; o < 8; ++o)
      for (int i = 0; i < o; ++i) {
        const bool in_place = i == o - 3 && o < 6 && s[i].p == s[o].p &&
                              (o != 3 || x.weights_stride == x.weights_out_stride);
        if (!in_place && s[i].p < s[o].p + s[o].n && s[o].p < s[i].p + s[i].n) return PA_ERR_ALIAS;
      }
  }
  pa::EvictParams a;
  a.weights = x.weights;
  a.stride = x.weights_stride;
  a.table = x.block_table;
  a.seq_lens = x.seq_lens;
  a.R = x.R;
  a.W = x.bt_width;
  a.keep = x.keep;
  a.init = x.init_blocks;
  a.local = local;
  a.weights_out = x.weights_out;
  a.stride_out = x.weights_out_stride;
  a.table_out = x.block_table_out;
  a.lens_out = x.seq_lens_out;
  a.evicted = x.evicted;
  a.counts = x.counts;
  a.status = x.status;
  const cudaError_t e = pa::launch_evict(a, (cudaStream_t)stream);
  return e == cudaSuccess ? PA_OK : pa::record_cuda_error(e);
}
