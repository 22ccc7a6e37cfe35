// Indexer scores over an NVFP4 index cache (pre_attn_index_scores_nvfp4):
// the FP8 scorer's definition with the keys
//   key_j[d] = e2m1(code_j[d]) * e4m3(sf_j[d / 16])
// of the NVFP4 pages ("vllm.models.minimax_m3.nvidia.ops.
// qkv_index_fused_epilogue", _nvfp4_cache_views: 64 code bytes a token, then
// 8 scale bytes a token, linear).
//
// A skinny contraction over a key stream that HBM bounds (72 bytes a key in,
// 4 bytes a (row, key) out).  A warp takes half a 128-key block, straight from
// global memory into fragments: lane (g, t) reads the 16 code bytes of dims
// 32 t .. + 31 of keys 4 g .. 4 g + 3, so a load instruction covers whole
// 64-byte tokens and no byte passes through shared memory.  Row g of tile 0 /
// row g + 8 of tile 0 / row g of tile 1 / row g + 8 of tile 1 of the two
// m16n8k16 products are keys 4 g .. 4 g + 3: a thread ends with four
// consecutive keys of two query rows and stores 16 bytes at a time.  Code x
// scale is an f16 value and the query rows are f16 values after a power-of-two
// scaling to a maximum in [2^14, 2^15) (down to 2^-29 of it), so the products
// are exact; the sums are f32.
//
// One GB300, calls back to back: 64 requests x 7 rows, lengths up to 32767,
// 106 MB in 25 us (4.2 TB/s, 0.62 of the measured copy rate): each warp is a
// chain of length, table entry, codes, products and stores, and 20 warps an SM
// do not hide it wholly.  A warp that walks several half blocks with the next
// one's codes on their way needs the registers of a fifth CTA (25.4 us at four
// a warp, 30 at sixteen); 8 warps a CTA 30.6 us, 2 warps 25.3.  8 requests x 1
// row: 4.6 us, latency.
#include <cstdint>

#include <cuda_fp16.h>

#include "../../include/pre_attn.h"
#include "pa_device.cuh"
#include "pa_f16.cuh"
#include "pa_launch.h"

namespace pa {

constexpr int kI4Warps = 4;     // a CTA: half a 128-key block a warp
constexpr int kI4MaxWidth = 16384;

struct Index4Params {
  const __nv_bfloat16 *iq;
  int64_t iq_stride;
  int head;
  const uint8_t *idx_cache;
  int64_t idx_pages, idx_page_bytes;
  int bs;
  const int32_t *block_table, *seq_lens;
  int R, q_len, bt_width, init_blocks, local_blocks;
  float index_scale;
  float *scores;
  int64_t score_stride;
  uint32_t *status;
};

template <int NT>  // n8 tiles of query rows: q_len <= 8 * NT
__global__ void __launch_bounds__(32 * kI4Warps, NT == 1 ? 5 : 4)
    pa_index_scores_nvfp4_kernel(const __grid_constant__ Index4Params a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int r = blockIdx.y, unit = blockIdx.x * kI4Warps + warp;
  const int b = unit >> 1, half = unit & 1;  // the block's keys 64 half .. + 63
  pdl_wait();
  pdl_trigger();
  const int seq = __ldg(a.seq_lens + r);
  const int64_t blk = b < a.bt_width ? __ldg(a.block_table + (int64_t)r * a.bt_width + b) : -1;
  if (seq < 1) return;
  const int nb_max = (seq - 1) / 128 + 1;
  if (seq < a.q_len || nb_max > a.bt_width) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_status(a.status, kDevSlotRange);
    return;
  }
  if (b >= nb_max) return;
  const int p0 = seq - a.q_len;  // position of row 0
  // the rows that score the block: b < nb - local, nb = p / 128 + 1, and b >= init
  const bool scored_any = b >= a.init_blocks && b < (seq - 1) / 128 + 1 - a.local_blocks;
  if (scored_any) {
    if (blk < 0 || (blk + 1) * 128 > a.idx_pages * a.bs) {
      if (lane == 0) set_status(a.status, kDevSlotRange);
    } else {
      // the block's codes and scales, all on their way at once.  Its tokens
      // are pieces of pt = min(block_size, 128), a page each, from token t0
      const int pt = min(a.bs, 128), lg = 31 - __clz(pt);
      const int64_t page0 = a.bs <= 128 ? blk << (7 - lg) : blk * 128 / a.bs;
      const int t0 = a.bs <= 128 ? 0 : (int)(blk * 128 - page0 * a.bs);
      uint4 kw[2][4];
      uint32_t ksf[2][4];
#pragma unroll
      for (int z = 0; z < 2; ++z)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int off = 64 * half + 32 * z + 4 * g + u, tok = t0 + (off & (pt - 1));
          const uint8_t *base = a.idx_cache + (page0 + (off >> lg)) * a.idx_page_bytes;
          kw[z][u] = __ldg(reinterpret_cast<const uint4 *>(base + tok * 64 + 16 * t));
          ksf[z][u] = __ldg(reinterpret_cast<const uint16_t *>(base + a.bs * 64 + tok * 8 + 2 * t));
        }
      // query rows as B fragments: column g of tile nt is row 8 nt + g
      uint32_t qf[NT][8][2];
      float sc[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int i = 8 * nt + g;
        const __nv_bfloat16 *row = a.iq + ((int64_t)r * a.q_len + i) * a.iq_stride + a.head * kHeadDim + 32 * t;
        float qv[32], top = 0.f;
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          const uint2 w = i < a.q_len ? __ldg(reinterpret_cast<const uint2 *>(row + 4 * y)) : make_uint2(0u, 0u);
          qv[4 * y] = bf16_to_f32(w.x & 0xffffu), qv[4 * y + 1] = bf16_to_f32(w.x >> 16);
          qv[4 * y + 2] = bf16_to_f32(w.y & 0xffffu), qv[4 * y + 3] = bf16_to_f32(w.y >> 16);
#pragma unroll
          for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(qv[4 * y + e]));
        }
        const int ex = max(exponent_of(quad_max(top)), -110) - 14;
        const float down = pow2i(-ex), up = pow2i(ex);
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          qf[nt][y][0] = f16x2_bits(qv[4 * y] * down, qv[4 * y + 1] * down);
          qf[nt][y][1] = f16x2_bits(qv[4 * y + 2] * down, qv[4 * y + 3] * down);
        }
        // accumulator columns of this thread are rows 8 nt + 2 t + e: held by lanes g = 2 t + e
#pragma unroll
        for (int e = 0; e < 2; ++e) sc[nt][e] = a.index_scale * __shfl_sync(0xffffffffu, up, 4 * (2 * t + e));
      }
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const int k0 = 64 * half + 32 * z;
        const uint4 *w = kw[z];
        const uint32_t *sf = ksf[z];
        float c[2][NT][4];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) c[x][nt][e] = 0.f;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t f[2][2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t fh = e4m3x4_f16(sf[2 * x + u]).x;
            f[u][0] = __byte_perm(fh, fh, 0x1010), f[u][1] = __byte_perm(fh, fh, 0x3232);
          }
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            uint32_t h[2][4];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint4 ww = w[2 * x + u];
              e2m1x8_f16(y == 0 ? ww.x : y == 1 ? ww.y : y == 2 ? ww.z : ww.w, h[u]);
#pragma unroll
              for (int e = 0; e < 4; ++e) h[u][e] = mul_f16x2(h[u][e], f[u][y >> 1]);
            }
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const uint32_t af[4] = {h[0][2 * z], h[1][2 * z], h[0][2 * z + 1], h[1][2 * z + 1]};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_f16(c[x][nt], af, qf[nt][2 * y + z][0], qf[nt][2 * y + z][1]);
            }
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int i = 8 * nt + 2 * t + e, p = p0 + i, j = b * 128 + k0 + 4 * g;
            if (i >= a.q_len || b > p / 128) continue;
            const bool on = b >= a.init_blocks && b < p / 128 + 1 - a.local_blocks;
            const float s[4] = {c[0][nt][e], c[0][nt][2 + e], c[1][nt][e], c[1][nt][2 + e]};
            float4 v;
            v.x = on && j <= p ? s[0] * sc[nt][e] : -INFINITY;
            v.y = on && j + 1 <= p ? s[1] * sc[nt][e] : -INFINITY;
            v.z = on && j + 2 <= p ? s[2] * sc[nt][e] : -INFINITY;
            v.w = on && j + 3 <= p ? s[3] * sc[nt][e] : -INFINITY;
            *reinterpret_cast<float4 *>(a.scores + ((int64_t)r * a.q_len + i) * a.score_stride + j) = v;
          }
      }
      return;
    }
  }
  // no keys read: -inf where the block is pinned for the row (scored columns of a block outside the cache stay)
  for (int i = 0; i < a.q_len; ++i) {
    const int p = p0 + i;
    if (b > p / 128 || (b >= a.init_blocks && b < p / 128 + 1 - a.local_blocks)) continue;
    *reinterpret_cast<float2 *>(a.scores + ((int64_t)r * a.q_len + i) * a.score_stride + b * 128 + 64 * half + 2 * lane) =
        make_float2(-INFINITY, -INFINITY);
  }
}

static cudaError_t launch_index4(const Index4Params &a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  cfg.gridDim = dim3((2 * a.bt_width + kI4Warps - 1) / kI4Warps, a.R);
  cfg.blockDim = dim3(32 * kI4Warps);
  return a.q_len <= 8 ? cudaLaunchKernelEx(&cfg, pa_index_scores_nvfp4_kernel<1>, a)
                      : cudaLaunchKernelEx(&cfg, pa_index_scores_nvfp4_kernel<2>, a);
}

}  // namespace pa

extern "C" int pre_attn_index_scores_nvfp4(const pa_index_nvfp4_args *in, void *stream) {
  if (!in) return PA_ERR_NULL;
  const pa_index_nvfp4_args &x = *in;
  auto aligned = [](const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
  if (!x.iq || !x.idx_cache || !x.block_table || !x.seq_lens || !x.scores || !x.status) return PA_ERR_NULL;
  if (x.R < 0 || x.R > 65535 || x.q_len < 1 || x.q_len > 16 || x.bt_width < 1 || x.bt_width > pa::kI4MaxWidth ||
      x.head < 0 || x.idx_pages < 1)
    return PA_ERR_SHAPE;
  if (x.init_blocks < 0 || x.local_blocks < 0 || !(x.index_scale == x.index_scale)) return PA_ERR_CONFIG;
  if (x.block_size < 4 || x.block_size % 4 || x.block_size > 1024) return PA_ERR_CONFIG;
  if (128 % x.block_size && x.block_size % 128) return PA_ERR_UNSUPPORTED;
  if (x.iq_stride < ((int64_t)x.head + 1) * 128 || x.score_stride < (int64_t)x.bt_width * 128 ||
      x.idx_page_bytes < (int64_t)x.block_size * 72)
    return PA_ERR_SHAPE;
  if (!aligned(x.iq, 8) || x.iq_stride % 4 || !aligned(x.idx_cache, 32) || x.idx_page_bytes % 32 ||
      !aligned(x.scores, 16) || x.score_stride % 4 || !aligned(x.block_table, 4) || !aligned(x.seq_lens, 4) ||
      !aligned(x.status, 4))
    return PA_ERR_ALIGN;
  if (x.R == 0) return PA_OK;
  pa::Index4Params a;
  a.iq = static_cast<const __nv_bfloat16 *>(x.iq);
  a.iq_stride = x.iq_stride;
  a.head = x.head;
  a.idx_cache = static_cast<const uint8_t *>(x.idx_cache);
  a.idx_pages = x.idx_pages;
  a.idx_page_bytes = x.idx_page_bytes;
  a.bs = x.block_size;
  a.block_table = x.block_table;
  a.seq_lens = x.seq_lens;
  a.R = x.R;
  a.q_len = x.q_len;
  a.bt_width = x.bt_width;
  a.init_blocks = x.init_blocks;
  a.local_blocks = x.local_blocks;
  a.index_scale = x.index_scale;
  a.scores = x.scores;
  a.score_stride = x.score_stride;
  a.status = x.status;
  const cudaError_t e = pa::launch_index4(a, (cudaStream_t)stream);
  return e == cudaSuccess ? PA_OK : pa::record_cuda_error(e);
}
