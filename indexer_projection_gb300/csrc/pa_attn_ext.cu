// Attention over the paged caches within a sliding window and with the weight
// that each block got (pre_attn_attention_ext).
//
// The window.  A row at position p sees key j <= p if j > p - window or
// j < sinks, so an item's rows (pa_attn.cu) read the first blocks up to the
// sinks' last and those from the window's first on; the dealing of blocks to
// CTAs counts these alone, and the blocks in which a window, the sinks or the
// row's position end are masked key by key.
//
// The weights.  weights[b] = sum over the request's rows and query heads of
// the softmax weights of block b's keys.  The attention kernel has a block's
// weights in registers, as exp2(s - m) under its running reference m: it
// writes log2 of their sum plus m, one number a block, row and head (for a
// block that P warps share P of them; 0.2% to 3% of the cache bytes read).
// pa_weights_kernel then takes a request on a cluster of CTAs, each a run of
// the blocks: the sum of all blocks gives each (row, head)'s softmax sum, and
// with it each block's share.  The caches are not read again, and every sum
// has an order of its own: no atomics.
//
// Measured with / without weights: 8 requests of one row, 16 heads, up to 8192
// keys 14.2 / 9.7 us (latency: partial sums, the cluster's exchange, the sums
// again); 32 of one row, 2 KV heads, up to 32768 keys, FP8, 68 / 57 us (4.1 TB/s
// of K and V with them).
#include <cmath>
#include <cstdint>

#include "../../include/pre_attn.h"
#include "pa_attn_kernel.cuh"

namespace pa {

constexpr int kWgThreads = 32 * kJoinWarps;
constexpr int kWgWarps = kWgThreads / 32;
constexpr int kWgMaxCtas = 8;     // a cluster
constexpr int kWgMaxPairs = 64;   // (row, KV head)s of a request
constexpr int kWgMaxRun = 2048;   // blocks a CTA
// Sums that a CTA reads, at least, before a request gets more CTAs.  64 / 512 /
// 4096 / all on one CTA, us of the whole call: 8 requests of one row 14.1 / 14.2 /
// 15.3 / 15.3, 32 of one row 68.8 / 68.0 / 69.0 / 99.9, 64 of 7 rows the same 61.4
// but for one CTA, 94.7.
constexpr int kWgValues = 512;

struct WeightParams {
  const float *part;  // [R][row][KV head][W][2^lg_v]: parts x heads
  int lg_heads, lg_v;
  CacheAttnParams at;
  int64_t num_blocks;  // ids of the cache: below this
  float *weights;
  int64_t stride;
  const float *before;  // or null
  int64_t before_stride;
  float decay;
  int words;         // of a pair's bit set
  int ctas;          // a request
  int join, join_x;  // CTAs behind the requests' that join partial results, in rows of join_x
  int sms;
};

// s 2^m with the maximum m of several, and its s.
struct Scaled {
  float m, s;
};
__device__ __forceinline__ Scaled join_scaled(Scaled a, Scaled b) {
  const float top = fmaxf(a.m, b.m);
  return {top, (a.m == top ? a.s : a.s * ex2_approx(a.m - top)) + (b.m == top ? b.s : b.s * ex2_approx(b.m - top))};
}

__device__ __forceinline__ void block_weights(const WeightParams &w) {
  extern __shared__ uint32_t bits[];  // [pairs][words] blocks that the pair's row attends
  __shared__ uint32_t held[kWgMaxRun / 32 + 1];
  __shared__ float2 way_ms[kWgWarps][16];
  __shared__ float2 col_ms[kWgMaxPairs * 16];  // of this CTA's blocks
  __shared__ float lse[kWgMaxPairs * 16];      // log2 of the (row, head)'s sum
  __shared__ float old[kWgMaxRun + 1];         // of the blocks' weights, what they had
  const CacheAttnParams &a = w.at;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = cta_rank(), r = blockIdx.x / w.ctas;
  // What the attention did not write can be read before the wait on it: the
  // attention lets this kernel in when the kernels before it are done (loads
  // that go to L2, which has what those wrote).
  const int seq = __ldcg(a.seq_lens + r);
  const bool none = seq < a.q_len || (seq - 1) / 128 + 1 > a.bt_width;  // without keys (the attention flags it)
  const int nb = none ? 0 : (seq - 1) / 128 + 1, first = seq - a.q_len;
  const int c0 = (int)((int64_t)nb * rank / w.ctas), c1 = (int)((int64_t)nb * (rank + 1) / w.ctas), n = c1 - c0;
  const int pairs = a.q_len * a.n_kv, heads = 1 << w.lg_heads, v = 1 << w.lg_v;
  // the blocks that the attention has summed
  for (int wi = warp; 32 * wi < n; wi += kWgWarps) {
    const int b = c0 + 32 * wi + lane;
    const int64_t id = b < c1 ? __ldcg(a.block_table + (int64_t)r * a.bt_width + b) : -1;
    const bool in = id >= 0 && id < w.num_blocks;
    if (a.topk) {
      const uint32_t all = __ballot_sync(0xffffffffu, in);
      if (lane == 0) held[wi] = all;
      for (int k = lane; k < pairs; k += 32) bits[k * w.words + wi] = 0;
    } else {
      for (int i = 0; i < a.q_len; ++i) {
        const uint32_t all = __ballot_sync(0xffffffffu, in && b <= (first + i) / 128 && attn_sees<true>(a, first + i, b));
        if (lane < a.n_kv) bits[(i * a.n_kv + lane) * w.words + wi] = all;
      }
    }
  }
  const float *before = w.before && w.decay != 0.f ? w.before + r * w.before_stride : nullptr;
  for (int b = tid; b < n; b += kWgThreads) old[b] = before ? w.decay * __ldcg(before + c0 + b) : 0.f;
  __syncthreads();
  if (a.topk && n > 0) {
    const int64_t at = (int64_t)r * pairs;
    for (int e = tid; e < pairs * a.topk; e += kWgThreads) {
      const int k = e / a.topk, b = __ldcg(a.blocks + at * a.topk + e);
      if (e - k * a.topk < __ldcg(a.counts + at + k) && b >= c0 && b < c1 && b <= (first + k / a.n_kv) / 128 &&
          ((held[(b - c0) >> 5] >> ((b - c0) & 31)) & 1u))
        atomicOr(&bits[k * w.words + ((b - c0) >> 5)], 1u << ((b - c0) & 31));
    }
    __syncthreads();
  }
  pdl_wait();
  pdl_trigger();
  if (none) return;  // the whole cluster
  // the (row, head)s' sums over this CTA's blocks: a warp a (row, KV head),
  // or several of them a part of its blocks each
  const float *base = w.part + (((int64_t)r * pairs * a.bt_width + c0) << w.lg_v);
  const int64_t pair_stride = (int64_t)a.bt_width << w.lg_v;
  const int ways = max(kWgWarps / pairs, 1);
  for (int job = warp; job < pairs * ways; job += kWgWarps) {
    const int pair = job / ways, way = job - pair * ways;
    const float *src = base + pair * pair_stride;
    const uint32_t *mine = bits + pair * w.words;
    const int e1 = (n * (way + 1) / ways) << w.lg_v;
    Scaled z = {-INFINITY, 0.f};
    constexpr int kIn = 16;
    for (int e = ((n * way / ways) << w.lg_v) + lane; e < e1; e += 32 * kIn) {
      float x[kIn];
      float top = z.m;
#pragma unroll
      for (int k = 0; k < kIn; ++k) {
        const int ek = e + 32 * k, b = ek >> w.lg_v;
        x[k] = ek < e1 && (ek & (heads - 1)) < a.group && ((mine[b >> 5] >> (b & 31)) & 1u) ? src[ek] : -INFINITY;
      }
#pragma unroll
      for (int k = 0; k < kIn; ++k) top = fmaxf(top, x[k]);
      if (top == -INFINITY) continue;  // no weight yet
      z.s = z.m == top ? z.s : z.s * ex2_approx(z.m - top);
      z.m = top;
#pragma unroll
      for (int k = 0; k < kIn; ++k) z.s += ex2_approx(x[k] - top);
    }
    for (int o = 16; o >= heads; o >>= 1)
      z = join_scaled(z, Scaled{__shfl_xor_sync(0xffffffffu, z.m, o), __shfl_xor_sync(0xffffffffu, z.s, o)});
    if (lane < heads) {
      if (ways == 1) col_ms[(pair << w.lg_heads) + lane] = make_float2(z.m, z.s);
      else way_ms[job][lane] = make_float2(z.m, z.s);
    }
  }
  __syncthreads();
  const int cols = pairs << w.lg_heads;
  // several parts of a column, all read before they are joined
  auto joined = [](auto part, int parts) {
    float2 y[8];
    float top = -INFINITY, s = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = k < parts ? part(k) : make_float2(-INFINITY, 0.f);
#pragma unroll
    for (int k = 0; k < 8; ++k) top = fmaxf(top, y[k].x);
#pragma unroll
    for (int k = 0; k < 8; ++k) s += y[k].x == top ? y[k].y : y[k].y * ex2_approx(y[k].x - top);
    return make_float2(top, s);
  };
  static_assert(kWgWarps <= 8 && kWgMaxCtas <= 8, "parts of a column");
  auto finish = [&](int c, float2 y) { lse[c] = y.x == -INFINITY ? INFINITY : y.x + lg2_approx(y.y); };  // none: no weight anywhere
  for (int c = tid; c < cols; c += kWgThreads) {
    const int pair = c >> w.lg_heads, head = c & (heads - 1);
    const float2 y = ways > 1 ? joined([&](int k) { return way_ms[pair * ways + k][head]; }, ways) : col_ms[c];
    if (w.ctas == 1) finish(c, y);
    else col_ms[c] = y;
  }
  if (w.ctas > 1) {
    cluster_sync();
    for (int c = tid; c < cols; c += kWgThreads)
      finish(c, joined(
                    [&](int k) {
                      float2 y;
                      asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                                   : "=f"(y.x), "=f"(y.y)
                                   : "r"(mapa(smem_u32(col_ms + c), k)));
                      return y;
                    },
                    w.ctas));
  }
  __syncthreads();
  if (w.ctas > 1) cluster_arrive_relaxed();  // (the others' sums have been read)
  // the blocks' shares, a warp four blocks at a time
  float *out = w.weights + r * w.stride;
  const int all = pairs << w.lg_v;
  constexpr int kAt = 4;
  for (int b = warp; b < n; b += kAt * kWgWarps) {
    float sum[kAt];
#pragma unroll
    for (int k = 0; k < kAt; ++k) sum[k] = 0.f;
#pragma unroll 2
    for (int f = lane; f < all; f += 32) {
      const int pair = f >> w.lg_v, off = f & (v - 1), head = off & (heads - 1);
      const float *src = base + pair * pair_stride + off;
      const float ref = lse[(pair << w.lg_heads) + head];
      float x[kAt];
#pragma unroll
      for (int k = 0; k < kAt; ++k) {
        const int bk = b + k * kWgWarps;
        x[k] = bk < n && head < a.group && ((bits[pair * w.words + (bk >> 5)] >> (bk & 31)) & 1u) ? src[(int64_t)bk << w.lg_v]
                                                                                               : -INFINITY;
      }
#pragma unroll
      for (int k = 0; k < kAt; ++k) sum[k] += x[k] == -INFINITY ? 0.f : ex2_approx(x[k] - ref);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < kAt; ++k) sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], o);
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < kAt; ++k)
        if (b + k * kWgWarps < n) out[c0 + b + k * kWgWarps] = old[b + k * kWgWarps] + sum[k];
  }
  for (int b = nb + rank * kWgThreads + tid; b < a.bt_width; b += w.ctas * kWgThreads) out[b] = 0.f;
  if (w.ctas > 1) cluster_wait();
}

// The requests' weights, and beside them what pa_attn_join_kernel would do:
// neither needs the other.
template <bool BY_HEAD>
__global__ void __launch_bounds__(kWgThreads, BY_HEAD ? 3 : 5) pa_weights_kernel(const __grid_constant__ WeightParams w) {
  const int to_weigh = w.at.R * w.ctas;
  if ((int)blockIdx.x < to_weigh) return block_weights(w);
  pdl_trigger();
  pdl_wait();
  const int k = blockIdx.x - to_weigh;
  if (k >= w.join) return;  // (the grid is whole clusters)
  attn_join<BY_HEAD ? kJoinWarps : 1>(w.at, w.sms, k % w.join_x, k / w.join_x);
}

static cudaError_t launch_weights(WeightParams w, int sms, bool pdl, bool to_join, cudaStream_t stream) {
  const int W = w.at.bt_width;
  const int64_t values = (int64_t)w.at.q_len * w.at.n_kv * W << w.lg_v;  // of a request
  w.ctas = 1;
  while (w.ctas < kWgMaxCtas && (W > w.ctas * kWgMaxRun || (w.at.R * w.ctas < 2 * sms && values > (int64_t)w.ctas * kWgValues)))
    w.ctas *= 2;
  w.words = ((W + w.ctas - 1) / w.ctas + 31) / 32;
  w.sms = sms;
  const bool by_head = join_by_head(w.at, sms);
  const dim3 g = join_grid(w.at, by_head);
  w.join_x = g.x;
  w.join = to_join ? g.x * g.y : 0;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = w.ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cfg.stream = stream;
  cfg.gridDim = dim3((unsigned)(w.at.R * w.ctas + (w.join + w.ctas - 1) / w.ctas * w.ctas));
  cfg.blockDim = dim3(kWgThreads);
  cfg.dynamicSmemBytes = (size_t)w.at.q_len * w.at.n_kv * w.words * 4;
  return cudaLaunchKernelEx(&cfg, by_head && to_join ? pa_weights_kernel<true> : pa_weights_kernel<false>, w);
}

// log2 of the heads that a (row, KV head) has in the partial sums.
static int lg_heads_of(int group) {
  int lg = 0;
  while ((1 << lg) < group) ++lg;
  return lg;
}

}  // namespace pa

extern "C" size_t pre_attn_attention_weights_bytes(int R, int q_len, int n_q_heads, int n_kv_heads, int bt_width) {
  if (R < 0 || R > 65535 || q_len < 1 || q_len > 16 || bt_width < 1 || bt_width > pa::kAtMaxWidth) return 0;
  if (n_kv_heads != 1 && n_kv_heads != 2 && n_kv_heads != 4) return 0;
  if (n_q_heads < 1 || n_q_heads % n_kv_heads || n_q_heads / n_kv_heads > 16) return 0;
  // parts of a block: the warps that share it, at most (pa_attn_kernel.cuh, AttnSplit)
  const size_t parts = q_len <= 2 ? 4 : q_len <= 4 ? 2 : 1;
  return std::max<size_t>((size_t)R * q_len * n_kv_heads * bt_width * (parts << pa::lg_heads_of(n_q_heads / n_kv_heads)) * 4, 4);
}

namespace pa {

// The checks of pre_attn_attention_ext and the kernels' parameters; a.R is 0
// where there is nothing to do, and *plain whether it is pre_attn_attention.
static int ext_params(const pa_attention_args *in, const pa_attention_ext *ext, CacheAttnParams &a, int *sms, bool *plain) {
  if (!in || !ext) return PA_ERR_NULL;
  if (ext->window < 0 || ext->sinks < 0 || (ext->sinks > 0 && ext->window == 0)) return PA_ERR_CONFIG;
  if (ext->weights && (!(ext->decay >= 0.0f) || !std::isfinite(ext->decay))) return PA_ERR_CONFIG;
  const int st = attn_params(*in, a, sms);
  if (st != PA_OK) return st;
  if (ext->window && in->blocks) return PA_ERR_UNSUPPORTED;
  if (ext->weights) {
    auto aligned = [](const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
    if (ext->weights_stride < in->bt_width || (ext->weights_before && ext->before_stride < in->bt_width)) return PA_ERR_SHAPE;
    if (!aligned(ext->weights, 4) || !aligned(ext->weights_before, 4)) return PA_ERR_ALIGN;
    if (a.R > 0) {
      struct Span {
        uintptr_t p, n;
      };
      const uintptr_t M1 = (uintptr_t)a.R * a.q_len - 1, cols = (uintptr_t)in->n_q_heads * 128;
      const Span w = {reinterpret_cast<uintptr_t>(ext->weights), (uintptr_t)((a.R - 1) * ext->weights_stride + in->bt_width) * 4};
      const Span old = {reinterpret_cast<uintptr_t>(ext->weights_before),
                        ext->weights_before ? (uintptr_t)((a.R - 1) * ext->before_stride + in->bt_width) * 4 : 0};
      const Span q = {reinterpret_cast<uintptr_t>(a.q), (M1 * in->q_stride + cols) * (in->q ? 2u : 1u)};
      const Span out = {reinterpret_cast<uintptr_t>(in->out), (M1 * in->out_stride + cols) * 2u};
      auto meet = [](const Span &s, const Span &t) { return s.n && t.n && s.p < t.p + t.n && t.p < s.p + s.n; };
      if (meet(w, q) || meet(w, out) || meet(old, out) ||
          (meet(w, old) && (w.p != old.p || ext->weights_stride != ext->before_stride)))
        return PA_ERR_ALIAS;
      if (!ext->workspace || ext->workspace_bytes < pre_attn_attention_weights_bytes(a.R, a.q_len, in->n_q_heads,
                                                                                     in->n_kv_heads, in->bt_width))
        return PA_ERR_WORKSPACE;
      if (!aligned(ext->workspace, 256)) return PA_ERR_ALIGN;
    }
  }
  if (a.R == 0) return PA_OK;
  const int keys = in->bt_width * 128;  // a window of that many is none
  if (ext->window < keys) a.window = ext->window, a.sinks = std::min(ext->sinks, keys);
  *plain = a.window == 0 && !ext->weights;
  a.wpart = ext->weights ? static_cast<float *>(ext->workspace) : nullptr;
  a.lg_heads = lg_heads_of(a.group);
  return PA_OK;
}

}  // namespace pa

extern "C" int pre_attn_attention_path(const pa_attention_args *in, const pa_attention_ext *ext) {
  if (!in) return -PA_ERR_NULL;
  pa::CacheAttnParams a;
  int sms = 0, path = 0;
  bool plain = true;
  const int st = ext ? pa::ext_params(in, ext, a, &sms, &plain) : pa::attn_params(*in, a, &sms);
  if (st != PA_OK) return -st;
  if (a.R == 0) return -PA_ERR_SHAPE;
  const bool fp8 = in->cache_format == PA_CACHE_FP8;
  const cudaError_t e = plain ? pa::plain_attn_path(a, fp8 ? 0 : 1, sms, &path)
                        : fp8 ? pa::launch_attn<0, true>(a, sms, true, nullptr, nullptr, &path)
                              : pa::launch_attn<1, true>(a, sms, true, nullptr, nullptr, &path);
  return e == cudaSuccess ? path : -pa::record_cuda_error(e);
}

extern "C" int pre_attn_attention_ext(const pa_attention_args *in, const pa_attention_ext *ext, void *stream) {
  pa::CacheAttnParams a;
  int sms = 0;
  bool plain = false;
  const int st = pa::ext_params(in, ext, a, &sms, &plain);
  if (st != PA_OK || a.R == 0) return st;
  if (plain) return pre_attn_attention(in, stream);
  const bool pdl = !(in->flags & PA_FLAG_NO_PDL), fp8 = in->cache_format == PA_CACHE_FP8;
  pa::AttnLaunched did;
  pa::AttnLaunched *done = ext->weights ? &did : nullptr;  // (then the weights' kernel joins)
  cudaError_t e = fp8 ? pa::launch_attn<0, true>(a, sms, pdl, (cudaStream_t)stream, done)
                      : pa::launch_attn<1, true>(a, sms, pdl, (cudaStream_t)stream, done);
  if (e == cudaSuccess && done && !a.test_timeout) {
    pa::WeightParams w = {};
    w.part = a.wpart;
    w.lg_heads = a.lg_heads;
    w.lg_v = a.lg_heads + (did.parts == 4 ? 2 : did.parts - 1);
    w.at = did.a;
    w.num_blocks = fp8 ? (a.num_pages16 >= 8 ? (a.num_pages16 - 8) / a.kps + 1 : 0) : a.kv_pages * a.bs / 128;
    w.weights = ext->weights;
    w.stride = ext->weights_stride;
    w.before = ext->weights_before;
    w.before_stride = ext->before_stride;
    w.decay = ext->decay;
    e = pa::launch_weights(w, sms, pdl, did.to_join, (cudaStream_t)stream);
  }
  return e == cudaSuccess ? PA_OK : pa::record_cuda_error(e);
}
