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
// attend it.  Three ways to deal items to CTAs (launch_attn): a cluster of
// CTAs an item, each sending its parts to the CTA that joins them (small calls); a
// persistent grid that walks the list of all items' blocks in even contiguous
// slices, an item that several CTAs share leaving partial sums in the
// workspace for pa_attn_join_kernel; a CTA an item where there are more items
// than the slices' list holds.  In a CTA one warp resolves the lists and block
// tables ahead, one thread keeps a ring of 128-key blocks in flight with
// tensor-map copies (pa_attn.cuh); a query row's (up to 16) heads are the 16
// rows of mma.sync m16n8k16, and the eight compute warps are dealt to the
// item's rows: WPR = 8, 4, 2 or 1 warps a row, each with its part of the keys.
//
// Arithmetic.  E4M3 codes and E2M1 code x E4M3 scale are f16 values, so keys
// and values are converted exactly in registers and multiplied on the f16
// tensor path with f32 sums.  A query head row is scaled by a power of two to
// a maximum in [2^14, 2^15) first, so its bf16 values are f16 values too
// unless they are 2^-29 of that maximum or less.  The per-token K scale
// multiplies the score, the per-token V scale the weight.  For the second
// product a weight (NVFP4), or a weight times its key's V scale (FP8), rounds
// to f16: 2^-11 relative while it is within 2^-23 of the largest so far, below
// that half of f16's smallest step, 2^-34 of the largest.  For FP8 "the
// largest" is that of weight x V scale, a reference apart from the softmax's:
// neither a key of large values that has no weight nor a row of zeros (which
// its writer gives the scale 1) costs the others their bits.  The sum of the
// weights is taken in f32 before that rounding.
//
// Bound and figures (one GB300, calls back to back; the floor is the keys'
// bytes at the measured copy rate).  Dense decode, ragged lengths up to 32768:
// FP8, 32 requests x 2 KV heads, 277 MB in 57.9 us (4.8 TB/s, 0.71 of the
// copy rate); NVFP4, 64 x 4, 606 MB in 171 us (3.6 TB/s, 0.52).  FP8 is bound
// by the stream and the ends of its slices, NVFP4 by the compute warps: 750
// instructions a warp for 32 keys (340 of them convert codes), where two warps
// a scheduler reach 1.8 a clock against fixed-latency waits and the ALU (35%)
// and tensor (35%) pipes.  Several rows on blocks of their choice (64 x 7 rows,
// 2 KV heads, 16 blocks: FP8 76 us, NVFP4 100) wait for the ring as much as
// they compute (FP8 1.3 instructions a clock, NVFP4 1.6): a stage is free when
// the warps of every row have passed it, so a block of one row holds up the
// others (none, 4 or 11 of a row's 16 blocks its own: FP8 67, 77, 98 us, NVFP4
// 87, 100, 110, at the same products).  Small calls (8 requests on 16 blocks
// each: 7.5 us) are a chain of latencies: list and table, first block, its
// products, the join.
//
// Measured and kept out: the rows of an item as one tcgen05 tile (FP8 spec
// rows 128 us against 77: softmax latency, instruction cache); two rows a warp
// sharing converted codes (114 against 77 where rows pick blocks of their own,
// 70 against 77 on every block); the value products of a step issued behind
// the next step's scores (179 to 186); twelve compute warps of 144 registers.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/pre_attn.h"
#include "pa_attn.cuh"

namespace pa {

constexpr int kAtThreads = 32 * (kAtWarps + 4);  // and the producers' warpgroup, of which two warps work
// Registers a thread after the split (setmaxnreg): the compute warps hold o,
// the queries and the step's scores and codes (twelve compute warps of 144
// registers were slower).  The sum must not exceed what the CTA was launched
// with, which launch_attn checks.
constexpr int kAtComputeRegs = 200, kAtProducerRegs = 96;

template <int ROWS, int MEET>  // MEET: warps whose parts meet here
struct AttnShared : AttnRing<ROWS> {
  uint64_t recv;   // kAtCluster: the other CTAs' partial results are here
  uint64_t fin;    // the compute warps among themselves: partial results are there
  uint64_t read;   // .. have been read
  uint64_t never;  // testing: nothing arrives on it
  float2 ml[MEET][16];
};

// A warp takes 16 Y keys at a time and at least those of a block; a row's
// warps beyond that take alternate entries of the ring, in kGroups groups.
// (64 keys a step were 7% faster than 32 for FP8 rows that share a CTA, slower
// for NVFP4, whose codes then cannot be read ahead of the softmax.)
template <int FMT, int WPR, bool CLUSTER>
struct AttnSplit {
  static constexpr int Y = FMT == 0 && !CLUSTER && WPR < 8 ? 4 : 2, kMost = 128 / (16 * Y);
  static constexpr int kParts = WPR > kMost ? kMost : WPR, kGroups = WPR / kParts, kKeys = 128 / kParts;
};

template <int FMT, int WPR, bool CLUSTER>
struct AttnSmem {  // stages, then the queries, the buffer where a row's warps meet, the rest
  static constexpr int kRows = kAtWarps / WPR, kQ = kRows * 16 * kHeadDim * 2, kMeet = kAtWarps * 8192;
  // where the warps meet: a place of its own, with a cluster and few warps a
  // row the stages, which are free by then
  static constexpr bool kMeetInRing = CLUSTER && WPR <= 2;
  static constexpr bool kDirect = !CLUSTER && WPR <= 2;  // (see the segment's result)
  static constexpr int kJoint = kMeetInRing || WPR == 1 ? 0 : kDirect ? kMeet / 2 : kMeet;
  // kAtCluster: partial results of the (row, head)s that this CTA joins, from
  // up to eight CTAs, o then (m, l)
  static constexpr int kRecvs = CLUSTER ? kRows * 16 + kAtMaxSplit : 0, kRecv = kRecvs * (kHeadDim * 4 + 16);
  // (places for one warp where none meet: a warp a row has its fifth FP8 stage by a few hundred bytes)
  using Shared = AttnShared<kRows, (kJoint > 0 || kMeetInRing) ? kAtWarps : 1>;
  static constexpr int kRest = kQ + kJoint + kRecv + (int)sizeof(Shared) + 128;
  static constexpr int kFit = (kAtSmem - kRest) / AttnStage<FMT>::kBytes;
  // a stage belongs to one group, which sees each of its phases (a wait names
  // a phase by its parity alone)
  static constexpr int kGroups = AttnSplit<FMT, WPR, CLUSTER>::kGroups;
  static constexpr int kStages = (kFit < kAtMaxStages ? kFit : kAtMaxStages) / kGroups * kGroups;
  static constexpr int kBytes = kStages * AttnStage<FMT>::kBytes + kRest;
};

template <int FMT, int WPR, bool CLUSTER>  // CLUSTER: mode kAtCluster
__global__ void __launch_bounds__(kAtThreads, 1) pa_attn_kernel(const __grid_constant__ AttnMaps maps,
                                                                const __grid_constant__ CacheAttnParams a) {
  using St = AttnStage<FMT>;
  using Sm = AttnSmem<FMT, WPR, CLUSTER>;
  using Sp = AttnSplit<FMT, WPR, CLUSTER>;
  static_assert(Sm::kBytes <= kAtSmem && Sm::kStages >= (CLUSTER ? 2 : 3), "shared memory of a CTA");
  static_assert(!Sm::kMeetInRing || Sm::kMeet <= Sm::kStages * St::kBytes, "the warps' meeting place");
  constexpr int kStages = Sm::kStages;
  constexpr int Y = Sp::Y, kParts = Sp::kParts, kGroups = Sp::kGroups, kKeys = Sp::kKeys;
  constexpr bool kEarly = Y == 2;
  static_assert(Sm::kStages >= 2 * kGroups, "two stages a group");
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = smem_raw + ((128 - (smem_u32(smem_raw) & 127)) & 127);
  uint8_t *q_smem = ring + kStages * St::kBytes;  // [row][group][128], as q holds them
  // where the warps meet: [warp][16 heads][128], in chunks of 4 as joint_at says
  float *joint = reinterpret_cast<float *>(Sm::kMeetInRing ? ring : q_smem + Sm::kQ);
  typename Sm::Shared &sh = *reinterpret_cast<typename Sm::Shared *>(q_smem + Sm::kQ + Sm::kJoint + Sm::kRecv);
  float *recv = reinterpret_cast<float *>(q_smem + Sm::kQ + Sm::kJoint);  // [CTA][its share of the (row, head)s][128]
  float4 *recv_ml = reinterpret_cast<float4 *>(recv + Sm::kRecvs * kHeadDim);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int mode = CLUSTER ? (int)kAtCluster : a.mode;
  if (warp == kAtWarps && (FMT == 0 ? lane < 4 : lane == 0 && a.bs <= 128))
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.m[lane])) : "memory");
  if (warp == kAtWarps + 1) attn_prefetch(a, mode);
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], kAtWarps / kGroups);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sh.batch_full[s], 1);
      mbar_init(&sh.batch_empty[s], 1);
    }
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.q_empty, kAtWarps);
    mbar_init(&sh.fin, kAtWarps);
    mbar_init(&sh.read, kAtWarps);
    mbar_init(&sh.never, 1);
    if constexpr (CLUSTER) mbar_init(&sh.recv, 1);
    fence_mbar_init();
  }
  // kAtCluster: CTA c joins the item's (row, head)s c, c + split, ..; what
  // rank `of` has to join of an item of `rows`
  auto to_join = [&](int rows, int of) { return (rows * a.group - of + a.split - 1) / a.split; };
  if constexpr (CLUSTER) {
    if (tid == 0)
      mbar_expect_tx(&sh.recv, to_join(attn_place(a, blockIdx.x / a.split).rows, cta_rank()) * a.split *
                                   (kHeadDim * 4 + 16));
    __syncwarp();
    cluster_arrive_relaxed();  // (a CTA sends when the others' barriers are there)
  }
  pdl_wait();  // queries, caches and lists come from the previous kernels
  pdl_trigger();
  if constexpr (CLUSTER) cluster_wait();
  const AttnSlice sl = attn_slice<kAtWarps>(a, sh, mode);
  if (sl.none) return;
  if (warp >= kAtWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kAtProducerRegs));
    if (warp == kAtWarps && lane == 0) attn_copies<FMT, kStages, kGroups>(a, maps, sh, sl, ring, q_smem);
    if (warp == kAtWarps + 1) attn_resolve<FMT>(a, sh, sl, mode);
    return;
  }

  // ----------------------------------------------------------------- compute
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kAtComputeRegs));
  const int row = warp / WPR, part = warp % WPR;
  const int key0 = part % kParts * kKeys;
  const int pt = min(a.bs, 128);  // NVFP4: tokens a piece of a stage
  // the warp's next entry: its number, stage and phase, and whether it is
  // known to be there (asked for while the one before is worked on)
  int next = kGroups > 1 ? part / kParts : 0, stage = next;
  uint32_t phase = 0;
  bool ready = false;
  auto peek = [&]() { ready = __all_sync(0xffffffffu, mbar_try_wait(smem_u32(&sh.full[stage]), phase)); };
  uint32_t nq = 0, nfin = 0;  // items begun; segments whose warps have met
  // A wait ran out: what this warp leaves out, the status tells.  Its CTA of a
  // cluster stays until no other can send to it (those have all they wait for
  // and are gone, or have given up too).
  auto give_up = [&]() {
    if constexpr (CLUSTER) cluster_sync();
  };
  int v0, v1, v;
  for (int it = sl.first; sl.segment(a, sh, it, v0, v1, v); ++it) {
    AttnItem x = attn_place(a, it);
    {
      const bool got = mbar_wait(&sh.q_full, nq & 1, a.status, a.lim);
      if (!__all_sync(0xffffffffu, got)) return give_up();
      ++nq;
    }
    x.first = sh.q_item.x, x.seq = sh.q_item.y;
    const bool live = row < x.rows && x.seq > 0;
    const int p = x.first + row;
    // the row's queries as A fragments: heads g and g + 8, k-step ks holding
    // dims dim0(ks) .. + 3 of this thread (an order of the dims that the key
    // fragments follow: 16 ks + 4 t for FP8 pages, 32 t + 4 ks for NVFP4)
    uint32_t qf[8][4];
    float sc[2];  // score = product * sc (* the key's scale)
    {
      float qv[2][32];
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int head = g + 8 * hh;
        const bool have = live && head < a.group;
        const int at = (row * a.group + head) * kHeadDim;
        float top = 0.f;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          const int d = FMT == 0 ? 16 * ks + 4 * t : 32 * t + 4 * ks;
          if (a.q_is_fp8) {
            const uint32_t w = have ? *reinterpret_cast<const uint32_t *>(q_smem + at + d) : 0u;
            const uint2 h2 = e4m3x4_f16(w);
            const float2 f0 = __half22float2(*reinterpret_cast<const __half2 *>(&h2.x));
            const float2 f1 = __half22float2(*reinterpret_cast<const __half2 *>(&h2.y));
            qv[hh][4 * ks] = f0.x, qv[hh][4 * ks + 1] = f0.y, qv[hh][4 * ks + 2] = f1.x, qv[hh][4 * ks + 3] = f1.y;
          } else {
            const uint2 w = have ? *reinterpret_cast<const uint2 *>(q_smem + 2 * (at + d)) : make_uint2(0u, 0u);
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
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_empty);
    }
    float o[16][4];  // n8 tile n: FP8 dims 8 n + 2 t + e, NVFP4 dims 16 (2 t + e) + n; heads g (0, 1) and g + 8 (2, 3)
#pragma unroll
    for (int n = 0; n < 16; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
    float mref[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    // When the reference moves.  NVFP4: a lifted score is above the limit.
    // FP8: a lane's weights of a step sum to more than it (or none is known)
    float glimit[2] = {FMT == 0 ? -1.f : -INFINITY, FMT == 0 ? -1.f : -INFINITY};
    // FP8: o is the sum of weight x V scale x unit x code, and the largest
    // weight x V scale x unit so far 2^kAtLift or more (2^kAtUnit while that
    // would take more)
    float unit[2] = {pow2i(kAtUnit), pow2i(kAtUnit)};
    if (a.test_timeout) {
      const bool got = mbar_wait(&sh.never, 0, a.status, a.lim);
      if (!__all_sync(0xffffffffu, got)) return give_up();
    }
    while (true) {
      if (!ready) {
        const bool got = mbar_wait(&sh.full[stage], phase, a.status, a.lim);
        if (!__all_sync(0xffffffffu, got)) return give_up();  // the warp gives up; the others' waits are bounded too
      }
      ready = false;
      const int s = stage;
      const int2 info = sh.info[next % kAtInfo];
      next += kGroups;
      stage += kGroups;
      if (stage >= kStages) stage -= kStages, phase ^= 1u;
      if (info.x >= 0 && ((info.y >> row) & 1)) {
        const uint8_t *st = ring + s * St::kBytes;
        const bool cut = info.x * 128 + 127 > p;  // keys after the row's position
#pragma unroll 1
        for (int k0 = key0; k0 < key0 + kKeys; k0 += 16 * Y) {
          // scores of 16 Y keys: of each 16, this thread's are 4 t + (e + rot) % 4, e = 0 .. 3
          float c[2 * Y][4];
#pragma unroll
          for (int nt = 0; nt < 2 * Y; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) c[nt][e] = 0.f;
          if constexpr (FMT == 0) {
            // a page is [8 chunks of 16 dims][16 tokens][16 bytes].  Column n
            // of tile nt is key 4 (n / 2) + 2 nt + n % 2 (the rows of an 8x8
            // tile meet in a bank two at a time; an order without that cost
            // 16 selects a step and was slower)
            const int n = lane & 7, nt = (lane >> 3) & 1;
            const int tok = 4 * (n >> 1) + 2 * nt + (n & 1);
            const uint32_t at = smem_u32(st) + (k0 >> 4) * 2048 + (lane >> 4) * 256 + tok * 16;
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) {
              uint32_t w[Y][4];
#pragma unroll
              for (int y = 0; y < Y; ++y) ldsm_x4(at + y * 2048 + cc * 512, w[y]);
#pragma unroll
              for (int z = 0; z < 2; ++z)
#pragma unroll
                for (int y = 0; y < Y; ++y)
#pragma unroll
                  for (int u = 0; u < 2; ++u) {
                    const uint2 k2 = e4m3x4_f16(w[y][2 * z + u]);
                    mma_f16(c[2 * y + u], qf[2 * cc + z], k2.x, k2.y);
                  }
            }
          } else {
            // a token is 64 bytes of codes; thread t takes the 16 of dims
            // 32 t .. + 31 (two scale groups).  Column n of tile nt is key
            // 4 (n / 2) + (2 nt + n % 2 + n / 2) % 4: with that rotation the
            // value reads below meet in a bank two at a time, not four
            uint32_t f0[2 * Y], f1[2 * Y];
            uint4 kw[2 * Y];
#pragma unroll
            for (int nt = 0; nt < 2 * Y; ++nt) {
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
              for (int nt = 0; nt < 2 * Y; ++nt) {
                uint32_t h[4];
                e2m1x8_f16(y == 0 ? kw[nt].x : y == 1 ? kw[nt].y : y == 2 ? kw[nt].z : kw[nt].w, h);
                const uint32_t f = y < 2 ? f0[nt] : f1[nt];
                mma_f16(c[nt], qf[2 * y], mul_f16x2(h[0], f), mul_f16x2(h[1], f));
                mma_f16(c[nt], qf[2 * y + 1], mul_f16x2(h[2], f), mul_f16x2(h[3], f));
              }
          }
          // the value codes, where registers allow before the softmax needs
          // the scores: as the products below take them
          uint32_t vraw[kEarly ? 16 * Y : 1], vsf[kEarly ? Y : 1];
          auto read_v = [&](int y, uint32_t *w, uint32_t &f4) {
            if constexpr (FMT == 0) {  // a page of values is [128 dims][16 tokens]
              const uint32_t vat = smem_u32(st) + St::kV + ((k0 >> 4) + y) * 2048 + lane * 16;
#pragma unroll
              for (int q4 = 0; q4 < 4; ++q4) {
                uint32_t r[4];
                ldsm_x4(vat + q4 * 512, r);
#pragma unroll
                for (int n = 0; n < 4; ++n) w[4 * q4 + n] = r[n];
              }
            } else {  // thread g takes dims 16 g .. + 15 (one scale group) of its tokens
              const int quad = k0 + 16 * y + 4 * t, in = quad & (pt - 1);
              const uint8_t *vp = st + (quad - in) * 144 + pt * 72;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint2 w2 = *reinterpret_cast<const uint2 *>(vp + (in + ((e + t) & 3)) * 64 + 8 * g);
                w[2 * e] = w2.x, w[2 * e + 1] = w2.y;
              }
              f4 = *reinterpret_cast<const uint32_t *>(vp + pt * 64 + in * 8 + 4 * g);
            }
          };
          if constexpr (kEarly)
#pragma unroll
            for (int y = 0; y < Y; ++y) read_v(y, vraw + 16 * y, vsf[y]);
          // x = score - reference (in log2 units, lifted by kAtLift; the score
          // itself while there is none), pairs of keys
          f32x2 x[2][2 * Y], vs2[2 * Y];
          float off[2];
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) off[hh] = mref[hh] == -INFINITY ? 0.f : kAtLift - mref[hh];
#pragma unroll
          for (int y = 0; y < Y; ++y) {
            f32x2 ks[2];
            if constexpr (FMT == 0) {
              const float4 k4 = *reinterpret_cast<const float4 *>(st + St::kKs + (k0 + 16 * y + 4 * t) * 4);
              const float4 v4 = *reinterpret_cast<const float4 *>(st + St::kVs + (k0 + 16 * y + 4 * t) * 4);
              ks[0] = pack2(k4.x, k4.y), ks[1] = pack2(k4.z, k4.w);
              vs2[2 * y] = pack2(v4.x, v4.y), vs2[2 * y + 1] = pack2(v4.z, v4.w);
            }
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                f32x2 f = pack2(sc[hh], sc[hh]);
                if constexpr (FMT == 0) f = mul2(f, ks[u]);
                x[hh][2 * y + u] = fma2(pack2(c[2 * y + u][2 * hh], c[2 * y + u][2 * hh + 1]), f, pack2(off[hh], off[hh]));
              }
          }
          // of this thread's four keys of 16, the last that counts
          auto last_of = [&](int y) { return p - info.x * 128 - k0 - 16 * y - 4 * t; };
          auto mask_v = [&](int left, uint32_t *w, uint32_t &f4) {
            const uint32_t keep = left >= 3 ? 0xffffffffu : left < 0 ? 0u : (256u << (8 * left)) - 1u;
            if constexpr (FMT == 0) {
#pragma unroll
              for (int n = 0; n < 16; ++n) w[n] &= keep;
            } else {
              f4 &= keep;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (((e + t) & 3) > left) w[2 * e] = w[2 * e + 1] = 0u;
            }
          };
          if (cut) {  // keys after the row's position: no weight, no value (whatever the cache holds there)
#pragma unroll
            for (int y = 0; y < Y; ++y) {
              const int left = last_of(y);
              if constexpr (kEarly) mask_v(left, vraw + 16 * y, vsf[y]);
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const bool ok0 = (FMT == 0 ? 2 * u : (2 * u + t) & 3) <= left;
                const bool ok1 = (FMT == 0 ? 2 * u + 1 : (2 * u + 1 + t) & 3) <= left;
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                  const float2 z = unpack2(x[hh][2 * y + u]);
                  x[hh][2 * y + u] = pack2(ok0 ? z.x : -INFINITY, ok1 ? z.y : -INFINITY);
                }
                if constexpr (FMT == 0) {
                  const float2 z = unpack2(vs2[2 * y + u]);
                  vs2[2 * y + u] = pack2(ok0 ? z.x : 0.f, ok1 ? z.y : 0.f);
                }
              }
            }
          }
          uint32_t pa[Y][4];
          float sum[2];
          auto weigh = [&]() {
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              f32x2 s2 = pack2(0.f, 0.f);
#pragma unroll
              for (int k = 0; k < 2 * Y; ++k) {
                const float2 u = unpack2(x[hh][k]);
                f32x2 w = pack2(ex2_approx(u.x), ex2_approx(u.y));
                s2 = add2(s2, w);
                if constexpr (FMT == 0) w = mul2(mul2(w, vs2[k]), pack2(unit[hh], unit[hh]));
                const float2 r = unpack2(w);
                pa[k >> 1][(k & 1) * 2 + hh] = f16x2_bits(r.x, r.y);
              }
              const float2 u = unpack2(s2);
              sum[hh] = u.x + u.y;
            }
          };
          auto highest = [&](int hh) {
            float top = -INFINITY;
#pragma unroll
            for (int k = 0; k < 2 * Y; ++k) {
              const float2 u = unpack2(x[hh][k]);
              top = fmaxf(top, fmaxf(u.x, u.y));
            }
            return top;
          };
          if constexpr (FMT == 0) {
            // The references move only where a product has outgrown f16 (a NaN
            // does not count) or the weights their sum; then the step is
            // weighed again
#pragma unroll 1
            for (bool again = false;; again = true) {
              weigh();
              uint32_t most = abs_f16x2(pa[0][0]);
#pragma unroll
              for (int k = 1; k < 4 * Y; ++k) most = max_f16x2(most, abs_f16x2(pa[k >> 2][k & 3]));
              // above 2^15 in either half: its bits are above 0x7800
              const bool grow = ((most + 0x07ff07ffu) & 0x80008000u) != 0u || sum[0] > glimit[0] || sum[1] > glimit[1];
              if (again || !__any_sync(0xffffffffu, grow)) break;
              // rows of zeros count for nothing, whatever their scale
#pragma unroll
              for (int y = 0; y < Y; ++y) {
                uint32_t late[kEarly ? 1 : 16], none = 0, some = 0;
                if constexpr (!kEarly) read_v(y, late, none);
#pragma unroll
                for (int n = 0; n < 16; ++n) some |= kEarly ? vraw[16 * y + n] : late[n];
                some |= __shfl_xor_sync(0xffffffffu, some, 4);
                some |= __shfl_xor_sync(0xffffffffu, some, 8);
                some |= __shfl_xor_sync(0xffffffffu, some, 16);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                  const float2 z = unpack2(vs2[2 * y + u]);
                  const bool zero0 = ((some >> (16 * u)) & 0x7fu) == 0u, zero1 = ((some >> (16 * u)) & 0x7f00u) == 0u;
                  vs2[2 * y + u] = pack2(zero0 && fabsf(z.x) < INFINITY ? 0.f : z.x, zero1 && fabsf(z.y) < INFINITY ? 0.f : z.y);
                }
              }
#pragma unroll
              for (int hh = 0; hh < 2; ++hh) {
                // the softmax's reference: up to the largest score, by whole powers of two
                const float was = mref[hh], tm = quad_max(highest(hh));
                const float nm = fmaxf(was, was == -INFINITY ? ceilf(tm) : was + ceilf(tm - kAtLift));
                const float by = nm == was ? 0.f : was == -INFINITY ? kAtLift - nm : was - nm;
                const int down = nm == was || was == -INFINITY ? 0 : (int)fminf(nm - was, 1000.f);
                float pv = 0.f;  // the largest weight x V scale, / 2^10
#pragma unroll
                for (int k = 0; k < 2 * Y; ++k) {
                  x[hh][k] = add2(x[hh][k], pack2(by, by));
                  const float2 u = unpack2(x[hh][k]), z = unpack2(vs2[k]);
                  pv = fmaxf(pv, fmaxf(ex2_approx(u.x) * (fabsf(z.x) * pow2i(-10)), ex2_approx(u.y) * (fabsf(z.y) * pow2i(-10))));
                }
                pv = quad_max(pv);
                mref[hh] = nm;
                glimit[hh] = nm == -INFINITY ? -1.f : kAtMostSum;
                l[hh] *= down > 126 ? 0.f : pow2i(-down);
                // the unit: the largest product, of this step or before it
                // (then 2^down lower than it was), at 2^kAtLift
                const int at = exponent_of(unit[hh]);
                int rise = down;
                if (pv > 0.f) rise = min(rise, (int)kAtLift - 10 - exponent_of(pv) - at);
                const int to = max(min(at + rise, kAtUnit), -126);
                unit[hh] = pow2i(to);
                const int by_o = to - at - down;  // <= 0
                const float f = by_o < -126 ? 0.f : pow2i(by_o);
#pragma unroll
                for (int n = 0; n < 16; ++n) o[n][2 * hh] *= f, o[n][2 * hh + 1] *= f;
              }
            }
          } else {
            // the reference moves only when a score has outgrown it, or there is none yet
            const float top[2] = {highest(0), highest(1)};
            if (__any_sync(0xffffffffu, top[0] > glimit[0] || top[1] > glimit[1])) {
#pragma unroll
              for (int hh = 0; hh < 2; ++hh) {
                const float was = mref[hh], tm = quad_max(top[hh]);
                const float now = was == -INFINITY ? tm : was + (tm - kAtLift);
                const float nm = fmaxf(was, now);
                const float al = nm == was ? 1.f : ex2_approx(was - nm);
                const float by = nm == was ? 0.f : was == -INFINITY ? kAtLift - nm : was - nm;
#pragma unroll
                for (int k = 0; k < 2 * Y; ++k) x[hh][k] = add2(x[hh][k], pack2(by, by));
                mref[hh] = nm;
                glimit[hh] = nm == -INFINITY ? -INFINITY : kAtLift + kAtSlack;
                l[hh] *= al;
#pragma unroll
                for (int n = 0; n < 16; ++n) o[n][2 * hh] *= al, o[n][2 * hh + 1] *= al;
              }
            }
            weigh();
          }
          l[0] += sum[0], l[1] += sum[1];
          peek();
          // o += weights . values
#pragma unroll
          for (int y = 0; y < Y; ++y) {
            uint32_t late[kEarly ? 1 : 16], late_sf = 0;
            if constexpr (!kEarly) read_v(y, late, late_sf);
            uint32_t *w = kEarly ? vraw + 16 * y : late;
            uint32_t f4 = kEarly ? vsf[y] : late_sf;
            if constexpr (!kEarly)
              if (cut) mask_v(last_of(y), w, f4);
            if constexpr (FMT == 0) {
#pragma unroll
              for (int n = 0; n < 16; ++n) {
                const uint2 v2 = e4m3x4_f16(w[n]);
                mma_f16(o[n], pa[y], v2.x, v2.y);
              }
            } else {
              // nibbles of two tokens are paired before the conversion
              const uint2 f = e4m3x4_f16(__funnelshift_r(f4, f4, 8 * t));
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
      // o leaves its unit, with l near 2^-kAtSumDown (where the values are not
      // tiny): then no sum of parts exceeds the largest value, however near
      // that is to the largest float
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int eu = exponent_of(unit[hh]);
        const int el = l[hh] > 0.f && l[hh] < INFINITY ? min(exponent_of(l[hh]) + kAtSumDown, 126 - eu) : 0;
        const float up = pow2i(-eu - el);
        mref[hh] += (float)el;
        l[hh] *= pow2i(-el);
#pragma unroll
        for (int n = 0; n < 16; ++n) o[n][2 * hh] *= up, o[n][2 * hh + 1] *= up;
      }
    }
    const bool whole = v0 == 0 && v1 == v;
    float *pp = nullptr;  // the segment's partial result: [row][head][128], then (m, l)
    if (!whole && mode == kAtSliced) {
      const bool head_seg = v0 > 0;  // the item began in an earlier CTA
      pp = a.part + (int64_t)(2 * sl.cta + (head_seg ? 0 : 1)) * kAtPartFloats;
      if (!head_seg && tid == 0) {
        const int last = sh.offs[it + 1] - 1;
        a.shares[it] = make_int2(sl.cta, (int)((((int64_t)last + 1) * sl.ctas - 1) / sl.total));
      }
    } else if (mode == kAtSliced && tid == 0) {
      a.shares[it] = make_int2(0, 0);
    }
    if constexpr (Sm::kDirect) {
      // a row has a warp or two: the second hands its part to the first, which
      // writes the result as it holds it (all rows' parts through shared memory,
      // as below, took two of nine stages: 5% of a dense call of four NVFP4 rows)
      if constexpr (WPR == 2) {
        float2 *box = reinterpret_cast<float2 *>(joint) + warp / 2 * 1024 + lane;  // [32][lane]
        if (nfin > 0) {  // the segment before has been read
          const bool got = mbar_wait(&sh.read, (nfin - 1) & 1, a.status, a.lim);
          if (!__all_sync(0xffffffffu, got)) return give_up();
        }
        if (part == 1) {
#pragma unroll
          for (int n = 0; n < 16; ++n)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) box[(2 * n + hh) * 32] = make_float2(o[n][2 * hh], o[n][2 * hh + 1]);
          if (t == 0) sh.ml[warp][g] = make_float2(mref[0], l[0]), sh.ml[warp][g + 8] = make_float2(mref[1], l[1]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.fin);
        const bool got = mbar_wait(&sh.fin, nfin & 1, a.status, a.lim);
        if (!__all_sync(0xffffffffu, got)) return give_up();
        if (part == 0) {
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const float2 ml = sh.ml[warp + 1][g + 8 * hh];
            const float top = fmaxf(mref[hh], ml.x);
            const float f0 = mref[hh] == top ? 1.f : ex2_approx(mref[hh] - top);
            const float f1 = ml.x == top ? 1.f : ex2_approx(ml.x - top);
            mref[hh] = top;
            l[hh] = f0 * l[hh] + f1 * ml.y;
#pragma unroll
            for (int n = 0; n < 16; ++n) {
              const float2 y = box[(2 * n + hh) * 32];
              o[n][2 * hh] = f0 * o[n][2 * hh] + f1 * y.x;
              o[n][2 * hh + 1] = f0 * o[n][2 * hh + 1] + f1 * y.y;
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.read);
        ++nfin;
      }
      const int64_t m = (int64_t)x.r * a.q_len + x.row0 + row;
      if (part == 0 && row < x.rows) {
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
      const int share = CLUSTER ? to_join(x.rows, 0) : 0;  // places a CTA's parts take in another
      // a (row, head)'s result and its place, dims 4 lane .. + 3
      auto store = [&](int i, int head, float sum, float4 y) {
        const float inv = sum == 0.f ? 0.f : a.out_scale / sum;
        const int64_t mi = (int64_t)x.r * a.q_len + x.row0 + i;
        *reinterpret_cast<uint2 *>(a.out + mi * a.out_stride + (int64_t)(x.h * a.group + head) * kHeadDim + 4 * lane) =
            make_uint2(bf16x2_bits(y.x * inv, y.y * inv), bf16x2_bits(y.z * inv, y.w * inv));
      };
      auto put = [&](int i, int head, float m, float sum, float4 y) {
        if constexpr (CLUSTER) {  // to the CTA that joins it
          const int k = i * a.group + head, at = sl.lo * share + k / a.split, to = k % a.split;
          const uint32_t bar = mapa(smem_u32(&sh.recv), to);
          st_async_v4(mapa(smem_u32(recv + at * kHeadDim + 4 * lane), to), y, bar);
          if (lane == 0) st_async_v4(mapa(smem_u32(recv_ml + at), to), make_float4(m, sum, 0.f, 0.f), bar);
        } else if (whole) {
          store(i, head, sum, y);
        } else {
          *reinterpret_cast<float4 *>(pp + (i * 16 + head) * kHeadDim + 4 * lane) = y;
          if (lane == 0)
            *reinterpret_cast<float2 *>(pp + kAtMaxRows * 16 * kHeadDim + (i * 16 + head) * 2) = make_float2(m, sum);
        }
      };
      // o, m and l go to the warp's slot in shared memory; chunk c (4 dims) of a
      // head sits at c ^ key, so that neither the fragments' writes nor the rows'
      // reads meet in a bank
      auto joint_at = [&](int slot, int head, int c) {
        const int key = FMT == 0 ? (head & 3) << 1 : ((c >> 3) & 3) | (head & 1) << 2;
        return joint + (slot * 16 + head) * kHeadDim + 4 * (c ^ key);
      };
      if constexpr (Sm::kMeetInRing) {  // the one segment's stages have been read
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.read);
        const bool got = mbar_wait(&sh.read, 0, a.status, a.lim);
        if (!__all_sync(0xffffffffu, got)) return give_up();
      } else if (nfin > 0) {  // the segment before has been read
        const bool got = mbar_wait(&sh.read, (nfin - 1) & 1, a.status, a.lim);
        if (!__all_sync(0xffffffffu, got)) return give_up();
      }
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int head = g + 8 * hh;
        if constexpr (FMT == 0) {
#pragma unroll
          for (int n = 0; n < 16; ++n)
            *reinterpret_cast<float2 *>(joint_at(warp, head, 2 * n + (t >> 1)) + 2 * (t & 1)) =
                make_float2(o[n][2 * hh], o[n][2 * hh + 1]);
        } else {
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int n = 0; n < 16; n += 4)
              *reinterpret_cast<float4 *>(joint_at(warp, head, 8 * t + 4 * e + n / 4)) =
                  make_float4(o[n][2 * hh + e], o[n + 1][2 * hh + e], o[n + 2][2 * hh + e], o[n + 3][2 * hh + e]);
        }
        if (t == 0) sh.ml[warp][head] = make_float2(mref[hh], l[hh]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.fin);
      {
        const bool got = mbar_wait(&sh.fin, nfin & 1, a.status, a.lim);
        if (!__all_sync(0xffffffffu, got)) return give_up();
      }
      // a warp a (row, head): its warps' parts added up in order
      for (int k = warp; k < x.rows * 16; k += kAtWarps) {
        const int i = k >> 4, head = k & 15;
        if (head >= a.group) continue;
        float2 ml[WPR];
        float4 y[WPR];
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int c = 0; c < WPR; ++c) {
          ml[c] = sh.ml[i * WPR + c][head];
          y[c] = *reinterpret_cast<const float4 *>(joint_at(i * WPR + c, head, lane));
          top = fmaxf(top, ml[c].x);
        }
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int c = 0; c < WPR; ++c) {
          const float f = ml[c].x == top ? 1.f : ex2_approx(ml[c].x - top);
          sum += f * ml[c].y;
          acc.x += f * y[c].x, acc.y += f * y[c].y, acc.z += f * y[c].z, acc.w += f * y[c].w;
        }
        put(i, head, top, sum, acc);
      }
      if constexpr (CLUSTER) {
        const bool got = mbar_wait_cluster(&sh.recv, 0, a.status, a.lim);
        if (!__all_sync(0xffffffffu, got)) return give_up();
        const int mine = to_join(x.rows, sl.lo);
        for (int k = warp; k < mine; k += kAtWarps) {  // a warp a (row, head), the CTAs' parts in order
          float2 ml[kAtMaxSplit];
          float top = -INFINITY, sum = 0.f;
#pragma unroll
          for (int c = 0; c < kAtMaxSplit; ++c)
            if (c < a.split) {
              const float4 u = recv_ml[c * share + k];
              ml[c] = make_float2(u.x, u.y);
              top = fmaxf(top, u.x);
            }
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int c = 0; c < kAtMaxSplit; ++c)
            if (c < a.split) {
              const float f = ml[c].x == top ? 1.f : ex2_approx(ml[c].x - top);
              const float4 y = *reinterpret_cast<const float4 *>(recv + (c * share + k) * kHeadDim + 4 * lane);
              sum += f * ml[c].y;
              acc.x += f * y.x, acc.y += f * y.y, acc.z += f * y.z, acc.w += f * y.w;
            }
          const int pair = sl.lo + k * a.split;
          store(pair / a.group, pair % a.group, sum, acc);
        }
        return;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.read);
      ++nfin;
    }
  }
}

// Join the partial results of items that several CTAs share, in CTA order:
// W warps a (item, row, head), each every W-th partial, several of them in
// flight a lane (four dims); the W sums meet in shared memory.  The first CTA's
// partial is its slot 1 (the item starts there), the others' their slot 0.
constexpr int kJoinWarps = 8;
template <int W>
__global__ void __launch_bounds__(32 * kJoinWarps) pa_attn_join_kernel(const __grid_constant__ CacheAttnParams a, int grid) {
  __shared__ float4 acc_s[kJoinWarps][32];
  __shared__ float2 ml_s[kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int it = blockIdx.x / a.rows_per, row = blockIdx.x % a.rows_per;
  const int head = blockIdx.y * (kJoinWarps / W) + warp / W;
  const int h = it & (a.n_kv - 1), rg = it >> a.lg_kv, r = rg >> a.lg_groups;
  const int row0 = (rg - (r << a.lg_groups)) * a.rows_per;
  pdl_trigger();  // the next kernel's CTAs fit beside these; it waits for this grid's end
  pdl_wait();
  const int2 s = a.shares[it];
  const int c0 = max(s.x, 0), c1 = min(s.y, grid - 1);
  if (c1 <= c0 || row0 + row >= a.q_len) return;  // the same for the whole CTA
  const bool have = head < a.group;
  const float *base = a.part + (int64_t)2 * c0 * kAtPartFloats + (row * 16 + (have ? head : 0)) * kHeadDim + 4 * lane;
  const float *mls = a.part + (int64_t)2 * c0 * kAtPartFloats + kAtMaxRows * 16 * kHeadDim + (row * 16 + (have ? head : 0)) * 2;
  float top = -INFINITY, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kIn = W > 1 ? 16 : 4;
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

static bool attn_maps(AttnMaps *maps, const CacheAttnParams &a, int fmt) {
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
static cudaError_t launch_attn(const CacheAttnParams &a0, int sms, bool pdl, cudaStream_t stream) {
  AttnMaps maps;
  if (!attn_maps(&maps, a0, FMT)) return cudaErrorInvalidValue;
  CacheAttnParams a = a0;
  using Kern = void (*)(const AttnMaps, const CacheAttnParams);
  struct Variant {
    Kern kern;
    int smem;
  };
  static const Variant kSliced[4] = {{pa_attn_kernel<FMT, 8, false>, AttnSmem<FMT, 8, false>::kBytes},
                                     {pa_attn_kernel<FMT, 4, false>, AttnSmem<FMT, 4, false>::kBytes},
                                     {pa_attn_kernel<FMT, 2, false>, AttnSmem<FMT, 2, false>::kBytes},
                                     {pa_attn_kernel<FMT, 1, false>, AttnSmem<FMT, 1, false>::kBytes}};
  static const Variant kClustered[4] = {{pa_attn_kernel<FMT, 8, true>, AttnSmem<FMT, 8, true>::kBytes},
                                        {pa_attn_kernel<FMT, 4, true>, AttnSmem<FMT, 4, true>::kBytes},
                                        {pa_attn_kernel<FMT, 2, true>, AttnSmem<FMT, 2, true>::kBytes},
                                        {pa_attn_kernel<FMT, 1, true>, AttnSmem<FMT, 1, true>::kBytes}};
  const int variant = a.rows_per == 1 ? 0 : a.rows_per == 2 ? 1 : a.rows_per <= 4 ? 2 : 3;
  cudaLaunchConfig_t cfg = {};
  // its shared memory, and that it holds the registers it splits
  auto use = [&](const Variant &v, std::atomic<int> &launch_regs) {
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(v.kern), v.smem);
    int regs = launch_regs.load(std::memory_order_relaxed);
    if (e == cudaSuccess && regs == 0) {
      cudaFuncAttributes at;
      e = cudaFuncGetAttributes(&at, reinterpret_cast<const void *>(v.kern));
      if (e == cudaSuccess) launch_regs.store(regs = at.numRegs, std::memory_order_relaxed);
    }
    if (e == cudaSuccess &&
        regs * kAtThreads < 32 * kAtWarps * kAtComputeRegs + (kAtThreads - 32 * kAtWarps) * kAtProducerRegs)
      e = cudaErrorInvalidConfiguration;
    cfg.blockDim = dim3(kAtThreads);
    cfg.dynamicSmemBytes = v.smem;
    return e;
  };
  static std::atomic<int> regs[2][4];  // of the kernels at launch
  cudaError_t e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  if (a.mode == kAtSliced) {
    // a cluster an item where all of them are resident at once and a CTA's
    // share of an item is short: then the scan and the second kernel cost more
    // than even slices save.  One FP8 row on 16 blocks: 7.2 us, sliced 11.4;
    // NVFP4, 24 blocks: 8.6, sliced 15.2.  On every block the two break even at
    // (blocks a CTA) x (rows) of 12 to 16 for 2 items (one row, 16 blocks a
    // CTA: 11.5 and 11.5 us; four rows, 4: 13.0 against 12.0) and of 25 to 35
    // for 8 and 16 (one row, 16: 17.2 against 20.9; four rows, 8: 20.9 against
    // 20.6; seven rows, 4: 22.4 against 26.0)
    const int longest = a.topk ? std::min(a.bt_width, a.topk * a.rows_per) : a.bt_width;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    static std::atomic<int> resident[4][64][kAtMaxSplit + 1];  // clusters of a size, by device; -1: none
    int dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    const Variant &v = kClustered[variant];
    if ((e = use(v, regs[1][variant])) != cudaSuccess) return e;
    for (int n = std::min(kAtMaxSplit, longest); n >= 2 && dev < 64; --n) {
      const int work = (longest + n - 1) / n * a.rows_per;
      if (a.items * n > sms || work > (a.items * n * 3 >= sms ? 2 : 1) * kAtClusterWork) continue;
      int held = resident[variant][dev][n].load(std::memory_order_relaxed);
      attr[1].val.clusterDim.x = n;
      if (held == 0) {
        cfg.gridDim = dim3(n);
        cfg.numAttrs = 2;
        int k = 0;
        held = cudaOccupancyMaxActiveClusters(&k, v.kern, &cfg) == cudaSuccess && k > 0 ? k : -1;
        resident[variant][dev][n].store(held, std::memory_order_relaxed);
      }
      if (held >= a.items) {
        a.mode = kAtCluster;
        a.split = n;
        cfg.gridDim = dim3(a.items * n);
        cfg.numAttrs = 2;
        return cudaLaunchKernelEx(&cfg, v.kern, maps, a);
      }
    }
    cfg.numAttrs = 1;
  }
  if ((e = use(kSliced[variant], regs[0][variant])) != cudaSuccess) return e;
  cfg.gridDim = dim3(a.mode == kAtSliced ? sms : a.items);
  e = cudaLaunchKernelEx(&cfg, kSliced[variant].kern, maps, a);
  if (e != cudaSuccess || a.mode != kAtSliced || a.test_timeout) return e;
  // few (item, row)s: many partials each, a CTA a head; else a warp a head.
  // Dense, whole calls with a CTA a head / a warp a head: 4 items x 4 rows 78 /
  // 92 us, 32 items x 1 row 35.9 / 36.9, 64 x 1 58.9 / 57.7, 32 x 4 548 / 543
  const bool many = a.items * a.rows_per * 4 <= sms;
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
    if (!(c.k_global_scale > 0.0f) || !(c.v_global_scale > 0.0f) || !std::isfinite(c.k_global_scale) ||
        !std::isfinite(c.v_global_scale))
      return PA_ERR_CONFIG;
    if (c.kv_page_bytes % 32 || !aligned(c.kv_cache, 32)) return PA_ERR_ALIGN;
  }
  // what a product of scaled queries and codes is multiplied by: a normal number
  const float score_scale = (float)((double)x.sm_scale * 1.4426950408889634 * (x.q ? 1.0 : (double)x.q_fp8_scale) *
                                    (fp8 ? 1.0 : (double)c.k_global_scale));
  if (!std::isnormal(score_scale)) return PA_ERR_CONFIG;
  if ((x.q && !aligned(x.q, 16)) || (x.q_fp8 && !aligned(x.q_fp8, 16)) || x.q_stride % 16 || !aligned(x.out, 16) ||
      x.out_stride % 8 || !aligned(x.block_table, 4) || !aligned(x.seq_lens, 4) || !aligned(x.blocks, 4) ||
      !aligned(x.counts, 4) || !aligned(x.status, 4))
    return PA_ERR_ALIGN;
  if (x.R == 0) return PA_OK;
  const int64_t M = (int64_t)x.R * x.q_len, cols = (int64_t)x.n_q_heads * 128;
  {
    const uintptr_t q0 = reinterpret_cast<uintptr_t>(x.q ? x.q : x.q_fp8), o0 = reinterpret_cast<uintptr_t>(x.out);
    const uintptr_t q1 = q0 + (uintptr_t)((M - 1) * x.q_stride + cols) * (x.q ? 2 : 1);
    const uintptr_t o1 = o0 + (uintptr_t)((M - 1) * x.out_stride + cols) * 2;
    if (q0 < o1 && o0 < q1) return PA_ERR_ALIAS;
  }
  const int sms = pa::current_device_sms();
  if (sms < 1) return pa::record_cuda_error(cudaGetLastError());
  if (!x.workspace || x.workspace_bytes < pre_attn_attention_workspace_bytes(x.R, x.q_len, x.n_kv_heads, sms))
    return PA_ERR_WORKSPACE;
  if (!aligned(x.workspace, 256)) return PA_ERR_ALIGN;
  pa::CacheAttnParams a = {};
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
  a.mode = a.items <= pa::kAtMaxItems ? pa::kAtSliced : pa::kAtWhole;
  a.score_scale = score_scale;
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
