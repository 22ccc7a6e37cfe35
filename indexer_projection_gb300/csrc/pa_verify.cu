// Verification of drafted tokens (pre_attn_verify_drafts): per request the
// drafts up to the first with u q(x) >= p(x), then one token drawn from
// max(p - q, 0), or from p where every draft was accepted, by its running sum.
//
// The drafts' test takes a few scattered loads, the draw one row of p and one
// of q (4 or 2 bytes a token and row: HBM bounds large batches, a chain of
// latencies the small ones).  A cluster of CTAs takes a request; each CTA
// finds the row by itself and sums its part of the vocabulary, a warp a
// contiguous run; the warps' sums go to every CTA of the cluster, whose warps
// then know which run the drawn token lies in, and that run's warp reads it
// again (from L2) and finds it.
//
// A weight is held in 64-bit fixed point, in units of 2^-62: a probability in
// [2^-38, 1] exactly (24 bits of mantissa), so that the difference p - q and
// all sums are exact, whatever their order, and equal inputs give equal tokens
// for any split.  (f32 sums of a vocabulary of 2^17 would move the drawn token
// in about one draw of a hundred; f64 adds run at a sixty-fourth of the f32
// rate here.)
#include <cstdint>

#include "../../include/pre_attn.h"
#include "pa_device.cuh"
#include "pa_launch.h"

namespace pa {

constexpr int kVfThreads = 256;
constexpr int kVfWarps = kVfThreads / 32;
constexpr int kVfCluster = 8;  // CTAs a request
constexpr int kVfRuns = kVfCluster * kVfWarps;

struct VerifyParams {
  const void *target, *draft;  // draft: or null
  int64_t target_stride, draft_stride;
  const int32_t *drafts;
  const float *uniforms;
  int R, q_len, vocab;
  int32_t *tokens, *accepted;
  uint32_t *status;
};

__device__ __forceinline__ float prob(const float *p) { return __ldg(p); }
__device__ __forceinline__ float prob(const __nv_bfloat16 *p) {
  return bf16_to_f32(__ldg(reinterpret_cast<const uint16_t *>(p)));
}

// floor(x 2^(32 + BITS)) of x in [0, 1] (BITS 30) or [0, 1) (BITS 32): its
// integer part at 2^BITS, then the rest's at 2^32; each step is exact.
template <int BITS>
__device__ __forceinline__ uint64_t fixed(float x) {
  const float y = x * (BITS == 30 ? 0x1p30f : 0x1p32f);
  const uint32_t hi = __float2uint_rz(y);
  const uint32_t lo = __float2uint_rz((y - __uint2float_rz(hi)) * 0x1p32f);
  return (uint64_t)hi << 32 | lo;
}
__device__ __forceinline__ uint64_t fixed_prob(float p) { return fixed<30>(fminf(fmaxf(p, 0.f), 1.f)); }

__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
// sums over the lanes up to and with this one
__device__ __forceinline__ uint64_t warp_running(uint64_t x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

template <typename TP, typename TQ>
__global__ void __launch_bounds__(kVfThreads) pa_verify_kernel(const __grid_constant__ VerifyParams a) {
  __shared__ uint64_t sums[2][kVfRuns];  // the runs' sums, in vocabulary order
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cta_rank();
  const int r = blockIdx.x / kVfCluster, k = a.q_len - 1, V = a.vocab;
  const TP *target = static_cast<const TP *>(a.target) + (int64_t)r * a.q_len * a.target_stride;
  const TQ *draft = static_cast<const TQ *>(a.draft);
  if (draft) draft += (int64_t)r * k * a.draft_stride;
  cluster_arrive_relaxed();  // the others' sums come once this CTA runs
  pdl_wait();
  pdl_trigger();
  // every warp: the drafts, one a lane
  int x = -1;
  bool good = false;
  if (lane < k) {
    x = __ldg(a.drafts + (int64_t)r * k + lane);
    if (x >= 0 && x < V) {
      const float p = prob(target + lane * a.target_stride + x);
      const float q = draft ? prob(draft + lane * a.draft_stride + x) : 1.f;
      good = (double)__ldg(a.uniforms + (int64_t)r * a.q_len + lane) * (double)q < (double)p;  // 24 x 24 bits: exact
    }
  }
  const float u = __ldg(a.uniforms + (int64_t)r * a.q_len + k);
  const int drafts = __ffs(__ballot_sync(0xffffffffu, x < 0)) - 1;  // lane k has none
  const int acc = __ffs(~__ballot_sync(0xffffffffu, good)) - 1;     // <= drafts
  const int xa = __shfl_sync(0xffffffffu, x, acc);
  if (rank == 0 && warp == 0) {
    if (__any_sync(0xffffffffu, lane < drafts && x >= V) && lane == 0) set_status(a.status, kDevTokenRange);
    if (lane < a.q_len && lane != acc) a.tokens[(int64_t)r * a.q_len + lane] = lane < acc ? x : -1;
    if (lane == 0) a.accepted[r] = acc;
  }
  const TP *P = target + acc * a.target_stride;
  const TQ *Q = draft ? draft + acc * a.draft_stride : nullptr;
  bool rest = acc < drafts;  // draw from what the drafter leaves
  auto weight = [&](int v) -> uint64_t {
    const uint64_t p = fixed_prob(prob(P + v));
    if (!rest) return p;
    const uint64_t q = Q ? fixed_prob(prob(Q + v)) : (v == xa ? ~0ull >> 1 : 0ull);
    return p > q ? p - q : 0ull;
  };
  // this warp's run of the vocabulary
  const int run = rank * kVfWarps + warp;
  const int v0 = (int)((int64_t)V * run / kVfRuns), v1 = (int)((int64_t)V * (run + 1) / kVfRuns);
  cluster_wait();
  for (int round = 0;; ++round) {
    uint64_t sum = 0;
    constexpr int kIn = 8;
    int v = v0 + lane;
    for (; v + 32 * (kIn - 1) < v1; v += 32 * kIn) {
      uint64_t w[kIn];
#pragma unroll
      for (int i = 0; i < kIn; ++i) w[i] = weight(v + 32 * i);
#pragma unroll
      for (int i = 0; i < kIn; ++i) sum += w[i];
    }
    for (; v < v1; v += 32) sum += weight(v);
    sum = warp_sum(sum);
    if (lane < kVfCluster)
      asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(mapa(smem_u32(&sums[round][run]), lane)), "l"(sum) : "memory");
    cluster_sync();
    // the runs in order, two a lane
    static_assert(kVfRuns == 64, "two runs a lane");
    const uint64_t s0 = sums[round][2 * lane], s1 = sums[round][2 * lane + 1];
    const uint64_t upto = warp_running(s0 + s1);
    const uint64_t total = __shfl_sync(0xffffffffu, upto, 31);
    if (total == 0) {
      if (rest) {  // the drafter leaves nothing: from the target's own
        rest = false;
        continue;
      }
      if (rank == 0 && tid == 0) {
        a.tokens[(int64_t)r * a.q_len + acc] = -1;
        set_status(a.status, kDevNoToken);
      }
      return;
    }
    // the running sum has to exceed u x total
    const uint64_t bar = __umul64hi(u >= 1.f ? ~0ull : fixed<32>(fmaxf(u, 0.f)), total);
    const int at = __ffs(__ballot_sync(0xffffffffu, upto > bar)) - 1;  // two runs
    uint64_t before = __shfl_sync(0xffffffffu, upto - s0 - s1, at);
    const uint64_t half = __shfl_sync(0xffffffffu, s0, at);
    const bool second = before + half <= bar;
    if (second) before += half;
    if (run != 2 * at + second) return;
    // the drawn token is in this warp's run
    int found = -1;
    for (v = v0 + lane; v - lane < v1; v += 32) {
      const uint64_t upto_v = before + warp_running(v < v1 ? weight(v) : 0ull);
      const uint32_t over = __ballot_sync(0xffffffffu, upto_v > bar);
      if (over) {
        found = v - lane + __ffs(over) - 1;
        break;
      }
      before = __shfl_sync(0xffffffffu, upto_v, 31);
    }
    if (lane == 0) {
      a.tokens[(int64_t)r * a.q_len + acc] = found;
      if (found < 0) set_status(a.status, kDevNoToken);
    }
    return;
  }
}

static cudaError_t launch_verify(const VerifyParams &a, bool target_bf16, bool draft_bf16, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kVfCluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cfg.stream = stream;
  cfg.gridDim = dim3((unsigned)a.R * kVfCluster);
  cfg.blockDim = dim3(kVfThreads);
  using bf = __nv_bfloat16;
  if (target_bf16)
    return draft_bf16 ? cudaLaunchKernelEx(&cfg, pa_verify_kernel<bf, bf>, a)
                      : cudaLaunchKernelEx(&cfg, pa_verify_kernel<bf, float>, a);
  return draft_bf16 ? cudaLaunchKernelEx(&cfg, pa_verify_kernel<float, bf>, a)
                    : cudaLaunchKernelEx(&cfg, pa_verify_kernel<float, float>, a);
}

}  // namespace pa

extern "C" int pre_attn_verify_drafts(const pa_verify_args *in, void *stream) {
  if (!in) return PA_ERR_NULL;
  const pa_verify_args &x = *in;
  auto aligned = [](const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
  if (!x.target || !x.uniforms || !x.tokens || !x.accepted || !x.status) return PA_ERR_NULL;
  if (x.R < 0 || x.R > 65535 || x.q_len < 1 || x.q_len > 16 || x.vocab < 1 || x.vocab > (1 << 24) ||
      x.target_stride < x.vocab || (x.draft_probs && x.draft_stride < x.vocab))
    return PA_ERR_SHAPE;
  if (x.q_len > 1 && !x.drafts) return PA_ERR_NULL;
  auto known = [](int t) { return t == PA_PROB_F32 || t == PA_PROB_BF16; };
  if (!known(x.target_type) || (x.draft_probs && !known(x.draft_type))) return PA_ERR_CONFIG;
  const bool target_bf16 = x.target_type == PA_PROB_BF16, draft_bf16 = x.draft_probs && x.draft_type == PA_PROB_BF16;
  if (!aligned(x.target, target_bf16 ? 2 : 4) || !aligned(x.draft_probs, draft_bf16 ? 2 : 4) || !aligned(x.drafts, 4) ||
      !aligned(x.uniforms, 4) || !aligned(x.tokens, 4) || !aligned(x.accepted, 4) || !aligned(x.status, 4))
    return PA_ERR_ALIGN;
  if (x.R == 0) return PA_OK;
  {  // the outputs apart from each other and from what other CTAs read
    struct Span {
      uintptr_t p, n;
    };
    const uintptr_t R = (uintptr_t)x.R, k = (uintptr_t)x.q_len - 1;
    auto rows = [&](uintptr_t n, int64_t stride, bool bf16) { return ((n - 1) * stride + x.vocab) * (bf16 ? 2u : 4u); };
    const Span s[6] = {{reinterpret_cast<uintptr_t>(x.target), rows(R * x.q_len, x.target_stride, target_bf16)},
                       {reinterpret_cast<uintptr_t>(x.draft_probs),
                        x.draft_probs && k ? rows(R * k, x.draft_stride, draft_bf16) : 0},
                       {reinterpret_cast<uintptr_t>(x.drafts), R * k * 4},
                       {reinterpret_cast<uintptr_t>(x.uniforms), R * x.q_len * 4},
                       {reinterpret_cast<uintptr_t>(x.tokens), R * x.q_len * 4},
                       {reinterpret_cast<uintptr_t>(x.accepted), R * 4}};
    for (int o = 4; o < 6; ++o)
      for (int i = 0; i < o; ++i)
        if (s[i].n && s[i].p < s[o].p + s[o].n && s[o].p < s[i].p + s[i].n) return PA_ERR_ALIAS;
  }
  pa::VerifyParams a;
  a.target = x.target;
  a.draft = x.draft_probs;
  a.target_stride = x.target_stride;
  a.draft_stride = x.draft_probs ? x.draft_stride : 0;
  a.drafts = x.drafts;
  a.uniforms = x.uniforms;
  a.R = x.R;
  a.q_len = x.q_len;
  a.vocab = x.vocab;
  a.tokens = x.tokens;
  a.accepted = x.accepted;
  a.status = x.status;
  const cudaError_t e = pa::launch_verify(a, target_bf16, draft_bf16, (cudaStream_t)stream);
  return e == cudaSuccess ? PA_OK : pa::record_cuda_error(e);
}
