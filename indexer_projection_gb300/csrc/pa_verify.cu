// Verification of drafted tokens (pre_attn_verify_drafts): per request the
// drafts up to the first with u q(x) >= p(x), then one token drawn from
// max(p - q, 0), or from p where every draft was accepted, by its running sum.
//
// The drafts' test takes a few scattered loads, the draw one row of p and one
// of q (4 or 2 bytes a token and row).  A cluster of CTAs takes a request; each
// CTA finds the row by itself and sums its part of the vocabulary, a warp a
// contiguous run; the warps' sums go to every CTA of the cluster, whose warps
// then know which run the drawn token lies in, and the CTA of that run reads it
// again (from L2), 256 tokens a warp, and finds it.
//
// A weight is held in 64-bit fixed point, in units of 2^-62: a probability in
// [2^-38, 1] exactly (24 bits of mantissa), so that the difference p - q and
// all sums are exact, whatever their order, and equal inputs give equal tokens
// for any split.  (f32 sums of a vocabulary of 2^17 would move the drawn token
// in about one draw of a hundred; f64 adds run at a sixty-fourth of the f32
// rate here.)  Where all probabilities have 8 bits of mantissa the units are
// 2^-46, what [2^-38, 1] takes, and the last of the three digits below is left
// out.
//
// Measured: 1 request of 32000 tokens 5.0 us (a launch and five dependent
// latencies: drafts, rows, sums, the cluster's exchange, the run again); 64 of
// 129281, f32 p and q, 17.5 us, 3.6 TB/s, of which the latencies, that nothing
// runs beside, are about 7 (a vocabulary of 1000 on as many CTAs) and the rows 10;
// 128 of 200064, bf16 p, 18.9 us, 2.7 TB/s (the same, and a 16-bit value costs
// as many additions as a 32-bit one; rows that begin off a 16-byte boundary 23).
// 64 registers (four CTAs an SM) do not hold everything where p is bf16: spills of
// 60 bytes a thread with bf16 q or none, off a 16-byte boundary 476, there with f32
// q 64.
#include <algorithm>
#include <cstdint>

#include "../../include/pre_attn.h"
#include "pa_device.cuh"
#include "pa_f16.cuh"
#include "pa_launch.h"

namespace pa {

constexpr int kVfThreads = 256;
constexpr int kVfWarps = kVfThreads / 32;
constexpr int kVfMaxCtas = 8;  // CTAs a request, a cluster
constexpr int kVfPerSm = 4;    // CTAs an SM holds

struct VerifyParams {
  const void *target, *draft;  // draft: or null
  int64_t target_stride, draft_stride;
  const int32_t *drafts;
  const float *uniforms;
  int R, q_len, vocab;
  int ctas;  // a request
  int32_t *tokens, *accepted;
  uint32_t *status;
};

__device__ __forceinline__ float prob(const float *p) { return __ldg(p); }
__device__ __forceinline__ float prob(const __nv_bfloat16 *p) {
  return bf16_to_f32(__ldg(reinterpret_cast<const uint16_t *>(p)));
}

// floor(x 2^64) of x in [0, 1): its first 32 bits, then the rest's; each step is exact.
__device__ __forceinline__ uint64_t fraction(float x) {
  const float y = x * 0x1p32f;
  const uint32_t hi = __float2uint_rz(y);
  return (uint64_t)hi << 32 | __float2uint_rz((y - __uint2float_rz(hi)) * 0x1p32f);
}

// floor(p 2^62) of p in [0, 1] as digits of 23, 23 and 16 bits, each with a
// constant beside it: p + 1, rounded down, has its last place at 2^-23, so its
// bits count p's 2^-23s; what that leaves of p (exact) likewise with 2^-23 for
// 1, and the rest of that with 2^-39.  Seven additions, two tokens' in one
// packed instruction, where a conversion to 64 bits takes a 64-bit shift or
// three conversions at a quarter of their rate.
__device__ __forceinline__ f32x2 add2_down(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rm.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
struct Digits {
  uint32_t d[3][2];  // of two tokens; sums and differences modulo 2^32
};
// N 2: the last digit left out.
template <int N>
__device__ __forceinline__ Digits digits_of(float p0, float p1) {
  const f32x2 c1 = pack2(1.f, 1.f), c2 = pack2(0x1p-23f, 0x1p-23f), c3 = pack2(0x1p-39f, 0x1p-39f);
  const f32x2 m1 = pack2(-1.f, -1.f), m2 = pack2(-0x1p-23f, -0x1p-23f);
  f32x2 p = pack2(p0, p1);
  const f32x2 r1 = add2_down(p, c1);
  p = fma2(add2(r1, m1), m1, p);  // (exact: multiples of 2^-23 below 2)
  const f32x2 r2 = add2_down(p, c2);
  if constexpr (N == 3) p = fma2(add2(r2, m2), m1, p);
  const f32x2 r3 = N == 3 ? add2_down(p, c3) : c3;
  const float2 a = unpack2(r1), b = unpack2(r2), c = unpack2(r3);
  return Digits{{{__float_as_uint(a.x), __float_as_uint(a.y)},
                 {__float_as_uint(b.x), __float_as_uint(b.y)},
                 {__float_as_uint(c.x), __float_as_uint(c.y)}}};
}
// (digits' differences are small, of either sign)
__device__ __forceinline__ int64_t value_of(uint32_t d1, uint32_t d2, uint32_t d3) {
  return (int64_t)(int)d1 * (1ll << 39) + (int64_t)(int)d2 * (1ll << 16) + (int)d3;
}
// a probability as it counts: [0, 1], 0 for a NaN
__device__ __forceinline__ float counted(float p) { return __saturatef(p); }

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

// A lane's IN values of a row in a step, as loaded: E consecutive tokens a
// load, its value i that of token v + 32 E (i / E) + E lane + i % E.
template <typename T, int E, int IN>
struct ProbRow;
template <typename T, int IN>
struct ProbRow<T, 1, IN> {
  T x[IN];
  __device__ __forceinline__ void load(const T *p) {
#pragma unroll
    for (int i = 0; i < IN; ++i) x[i] = __ldg(p + 32 * i + (threadIdx.x & 31));
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 2) return bf16_to_f32(__bfloat16_as_ushort(x[i]));
    else return x[i];
  }
};
template <int E, int IN>
struct ProbRowF32 {
  float4 x[IN / 4];
  __device__ __forceinline__ void load(const float *p) {  // (E 8: beside a row of 16-bit values)
#pragma unroll
    for (int i = 0; i < IN / 4; ++i)
      x[i] = __ldg(reinterpret_cast<const float4 *>(p + 32 * E * (4 * i / E) + E * (threadIdx.x & 31) + 4 * i % E));
  }
  __device__ __forceinline__ float get(int i) const {
    const float4 y = x[i / 4];
    return i % 4 == 0 ? y.x : i % 4 == 1 ? y.y : i % 4 == 2 ? y.z : y.w;
  }
};
template <int IN>
struct ProbRow<float, 4, IN> : ProbRowF32<4, IN> {};
template <int IN>
struct ProbRow<float, 8, IN> : ProbRowF32<8, IN> {};
template <int IN>
struct ProbRow<__nv_bfloat16, 8, IN> {
  uint4 x[IN / 8];
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
#pragma unroll
    for (int i = 0; i < IN / 8; ++i) x[i] = __ldg(reinterpret_cast<const uint4 *>(p + 256 * i + 8 * (threadIdx.x & 31)));
  }
  __device__ __forceinline__ float get(int i) const {
    const uint4 y = x[i / 8];
    const uint32_t w = i % 8 < 2 ? y.x : i % 8 < 4 ? y.y : i % 8 < 6 ? y.z : y.w;
    return __uint_as_float(i % 2 ? w & 0xffff0000u : w << 16);
  }
};

// The rows that a request's token is drawn from.
template <typename TP, typename TQ, int E>
struct Draw {
  static constexpr int kDigits = sizeof(TP) == 2 && sizeof(TQ) == 2 ? 2 : 3;  // (16-bit values: see the head of this file)
  static __device__ __forceinline__ Digits digits(float p0, float p1) { return digits_of<kDigits>(p0, p1); }
  const TP *P;
  const TQ *Q;         // or null
  int without;         // the token that weighs nothing, or -1
  int drafts, acc, x;  // the request's drafts, how many are accepted, the lane's

  // By a warp, the drafts one a lane.
  __device__ __forceinline__ void accept(const VerifyParams &a, int r) {
    const int lane = threadIdx.x & 31, k = a.q_len - 1;
    const TP *target = static_cast<const TP *>(a.target) + (int64_t)r * a.q_len * a.target_stride;
    const TQ *draft = static_cast<const TQ *>(a.draft);
    if (draft) draft += (int64_t)r * k * a.draft_stride;
    x = -1;
    bool good = false;
    if (lane < k) {
      x = __ldg(a.drafts + (int64_t)r * k + lane);
      const float u = __ldg(a.uniforms + (int64_t)r * a.q_len + lane);
      if (x >= 0 && x < a.vocab) {
        const float p = prob(target + lane * a.target_stride + x);
        const float q = draft ? prob(draft + lane * a.draft_stride + x) : 1.f;
        good = (double)u * (double)q < (double)p;  // 24 x 24 bits: exact
      }
    }
    drafts = __ffs(__ballot_sync(0xffffffffu, x < 0)) - 1;  // lane k has none
    acc = __ffs(~__ballot_sync(0xffffffffu, good)) - 1;     // <= drafts
    const int xa = __shfl_sync(0xffffffffu, x, acc);
    // from what the drafter leaves of the target's row: less its own, or without the token
    P = target + acc * a.target_stride;
    Q = draft && acc < drafts ? draft + acc * a.draft_stride : nullptr;
    without = !draft && acc < drafts ? xa : -1;
  }

  // IN tokens of a lane: token i of a warp's step at v
  static __device__ __forceinline__ int token(int v, int i) { return v + 32 * E * (i / E) + E * (threadIdx.x & 31) + i % E; }
  // What token v weighs as p - q, q not above p; 0 from v1 on.
  __device__ __forceinline__ void weigh(int v, int v1, float &p, float &q) const {
    const bool in = v < v1 && v != without;
    p = in ? prob(P + v) : 0.f;
    q = in && Q ? prob(Q + v) : 0.f;
  }
  static __device__ __forceinline__ void clamp(float &p, float &q) {
    p = counted(p);
    q = fminf(counted(q), p);
  }

  // The lane's sum over the tokens v0 .. v1 of its warp, a step's loads ahead
  // of the sums (64 bytes a lane of them).
  template <bool DRAFT>
  __device__ __forceinline__ uint64_t run(int v0, int v1) const {
    constexpr int kMost = 64 / (sizeof(TP) + (DRAFT ? sizeof(TQ) : 0)) / 8 * 8, IN = E == 1 && kMost > 16 ? 16 : kMost, kStep = 32 * IN;
    struct Loaded {
      ProbRow<TP, E, IN> p;
      ProbRow<TQ, E, DRAFT ? IN : E> q;
    };
    auto load = [&](Loaded &x, int v) {
      x.p.load(P + v);
      if constexpr (DRAFT) x.q.load(Q + v);
    };
    uint64_t sum = 0;
    Loaded next;
    int v = v0;
    if (v + kStep <= v1) load(next, v);
    for (; v + kStep <= v1; v += kStep) {
      const Loaded x = next;
      if (v + 2 * kStep <= v1) load(next, v + kStep);
      // (without a draft row its digits are the constants')
      const Digits none = digits(0.f, 0.f);
      uint32_t d[3];
#pragma unroll
      for (int k = 0; k < 3; ++k) d[k] = DRAFT ? 0u : 0u - (uint32_t)IN * none.d[k][0];
#pragma unroll
      for (int i = 0; i < IN; i += 2) {
        float p0 = counted(x.p.get(i)), p1 = counted(x.p.get(i + 1));
        const Digits s = digits(p0, p1);
        if constexpr (DRAFT) {
          const Digits y = digits(fminf(counted(x.q.get(i)), p0), fminf(counted(x.q.get(i + 1)), p1));
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            d[k] += s.d[k][0] - y.d[k][0];
            d[k] += s.d[k][1] - y.d[k][1];
          }
        } else {
#pragma unroll
          for (int k = 0; k < 3; ++k) d[k] += s.d[k][0] + s.d[k][1];
        }
      }
      sum += value_of(d[0], d[1], d[2]);
    }
    // `without` is among them: its weight once
    if (!DRAFT && without >= v0 && without < v && (threadIdx.x & 31) == 0) {
      const Digits y = digits(counted(prob(P + without)), 0.f);
      sum -= value_of(y.d[0][0] - y.d[0][1], y.d[1][0] - y.d[1][1], y.d[2][0] - y.d[2][1]);
    }
    for (; v < v1; v += 32 * 8) sum += part(v, v1);
    return sum;
  }
  // .. of 8 tokens, v + lane + 32 i; what each of them weighs
  __device__ __forceinline__ uint64_t part(int v, int v1) const {
    uint64_t each[8], sum = 0;
    part(v, v1, each);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += each[i];
    return sum;
  }
  __device__ __forceinline__ void part(int v, int v1, uint64_t (&each)[8]) const {
    float p[8], q[8];
    v += threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 8; ++i) weigh(v + 32 * i, v1, p[i], q[i]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      clamp(p[i], q[i]);
      const Digits s = digits(p[i], q[i]);
      each[i] = value_of(s.d[0][0] - s.d[0][1], s.d[1][0] - s.d[1][1], s.d[2][0] - s.d[2][1]);
    }
  }
  __device__ __forceinline__ uint64_t any(int v0, int v1) const { return Q ? run<true>(v0, v1) : run<false>(v0, v1); }
};

template <typename TP, typename TQ, int E>
__global__ void __launch_bounds__(kVfThreads, kVfPerSm) pa_verify_kernel(const __grid_constant__ VerifyParams a) {
  __shared__ uint64_t sums[2][kVfMaxCtas * kVfWarps];  // the runs' sums, in vocabulary order
  __shared__ uint64_t step_sums[2][kVfWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = cta_rank(), r = blockIdx.x / a.ctas, V = a.vocab, runs = a.ctas * kVfWarps;
  cluster_arrive_relaxed();  // the others' sums come once this CTA runs
  pdl_wait();
  pdl_trigger();
  Draw<TP, TQ, E> w;
  w.accept(a, r);
  const float u = __ldg(a.uniforms + (int64_t)r * a.q_len + a.q_len - 1);
  int32_t *tokens = a.tokens + (int64_t)r * a.q_len;
  if (rank == 0 && warp == 0) {
    if (__any_sync(0xffffffffu, lane < w.drafts && w.x >= V) && lane == 0) set_status(a.status, kDevTokenRange);
    if (lane < a.q_len && lane != w.acc) tokens[lane] = lane < w.acc ? w.x : -1;
    if (lane == 0) a.accepted[r] = w.acc;
  }
  // run i of the vocabulary, a warp's
  auto begin = [&](int i) { return i == runs ? V : (int)((int64_t)V * i / runs) & -8; };
  const int run = rank * kVfWarps + warp;
  cluster_wait();
  for (int round = 0;; ++round) {
    const uint64_t sum = warp_sum(w.any(begin(run), begin(run + 1)));
    if (lane < a.ctas)
      asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(mapa(smem_u32(&sums[round][run]), lane)), "l"(sum) : "memory");
    cluster_sync();
    // the runs in order, two a lane
    static_assert(kVfMaxCtas * kVfWarps == 64, "two runs a lane");
    const uint64_t s0 = 2 * lane < runs ? sums[round][2 * lane] : 0, s1 = 2 * lane < runs ? sums[round][2 * lane + 1] : 0;
    const uint64_t upto = warp_running(s0 + s1);
    const uint64_t total = __shfl_sync(0xffffffffu, upto, 31);
    if (total == 0) {
      if (w.acc < w.drafts && round == 0) {  // the drafter leaves nothing: from the target's own
        w.Q = nullptr;
        w.without = -1;
        continue;
      }
      if (rank == 0 && tid == 0) {
        tokens[w.acc] = -1;
        set_status(a.status, kDevNoToken);
      }
      return;
    }
    // the running sum has to exceed u x total
    const uint64_t bar = __umul64hi(u >= 1.f ? ~0ull : fraction(fmaxf(u, 0.f)), total);
    int at = 2 * (__ffs(__ballot_sync(0xffffffffu, upto > bar)) - 1);
    uint64_t before = __shfl_sync(0xffffffffu, upto - s0 - s1, at / 2);
    const uint64_t half = __shfl_sync(0xffffffffu, s0, at / 2);
    if (before + half <= bar) before += half, ++at;
    if (at / kVfWarps != rank) return;
    // the drawn token is in run `at`, one of this CTA's: its warps read the run
    // again, 256 tokens each
    const int v1 = begin(at + 1);
    for (int v0 = begin(at), turn = 0; v0 < v1; v0 += 256 * kVfWarps, ++turn) {
      const int v = v0 + warp * 256;
      uint64_t each[8], mine = 0;
      w.part(v, v1, each);
#pragma unroll
      for (int i = 0; i < 8; ++i) mine += each[i];
      mine = warp_sum(mine);
      if (lane == 0) step_sums[turn & 1][warp] = mine;
      __syncthreads();
      int hit = -1;  // the warp whose tokens have it, the same for every warp
      uint64_t first = 0;
#pragma unroll
      for (int i = 0; i < kVfWarps; ++i) {
        const uint64_t y = step_sums[turn & 1][i];
        if (hit < 0 && before <= bar && bar < before + y) hit = i, first = before;
        before += y;
      }
      if (hit >= 0) {
        if (hit == warp) {
          int found = -1;
#pragma unroll
          for (int i = 0; i < 8; ++i) each[i] = warp_running(each[i]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t over = __ballot_sync(0xffffffffu, first + each[i] > bar);
            if (over && found < 0) found = v + 32 * i + __ffs(over) - 1;
            first += __shfl_sync(0xffffffffu, each[i], 31);
          }
          if (lane == 0) tokens[w.acc] = found;
        }
        return;
      }
    }
    if (tid == 0) {  // (sums that wrapped)
      tokens[w.acc] = -1;
      set_status(a.status, kDevNoToken);
    }
    return;
  }
}

template <typename TP, typename TQ>
static cudaError_t launch_verify(VerifyParams a, int sms, cudaStream_t stream) {
  // As many CTAs a request as are resident at once.  2 / 4 / 8 of them, us: 1
  // request 6.9 / 5.6 / 5.0, 64 requests 31.4 / 20.6 / 17.5 (512 CTAs of 608), 128
  // requests 22.6 / 18.8 / 21.4 (8: two turns)
  // .. while a CTA has 2048 tokens or, beyond one an SM, 8192 (512 CTAs take 3 us
  // more than 64 to start and join): 64 requests of 4000 tokens 7.5 on eight CTAs,
  // 4.6 on two, 16000 tokens 7.5 on eight, 5.8 on two; 1 request of 16000 4.4 on
  // eight, 5.4 on two.
  auto least = [&] { return a.R * a.ctas > sms ? 8192 : 2048; };
  a.ctas = kVfMaxCtas;
  while (a.ctas > 1 && (a.R * a.ctas > sms * kVfPerSm || a.vocab < (a.ctas - 1) * least())) --a.ctas;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cfg.stream = stream;
  cfg.gridDim = dim3((unsigned)a.R * a.ctas);
  cfg.blockDim = dim3(kVfThreads);
  // 16-byte loads where every row begins on such a boundary
  auto rows16 = [](const void *p, int64_t stride, size_t es) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * es % 16 == 0;
  };
  constexpr int E = sizeof(TP) == 2 || sizeof(TQ) == 2 ? 8 : 4;
  const bool wide = rows16(a.target, a.target_stride, sizeof(TP)) && (!a.draft || rows16(a.draft, a.draft_stride, sizeof(TQ)));
  return cudaLaunchKernelEx(&cfg, wide ? pa_verify_kernel<TP, TQ, E> : pa_verify_kernel<TP, TQ, 1>, a);
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
  a.ctas = 0;
  a.tokens = x.tokens;
  a.accepted = x.accepted;
  a.status = x.status;
  using bf = __nv_bfloat16;
  const cudaStream_t s = (cudaStream_t)stream;
  const int sms = pa::current_device_sms();
  if (sms < 1) return pa::record_cuda_error(cudaGetLastError());
  const cudaError_t e = target_bf16 ? (draft_bf16 || !a.draft ? pa::launch_verify<bf, bf>(a, sms, s) : pa::launch_verify<bf, float>(a, sms, s))
                                    : (draft_bf16 ? pa::launch_verify<float, bf>(a, sms, s) : pa::launch_verify<float, float>(a, sms, s));
  return e == cudaSuccess ? PA_OK : pa::record_cuda_error(e);
}
