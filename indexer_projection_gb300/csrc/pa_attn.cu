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
// Measured and kept out: the rows of an item as one tcgen05 tile in a first form
// (FP8 spec rows 128 us against 77: softmax latency, instruction cache; calls
// with a window or weights take a later one, pa_attn_tc.cu); two rows a warp
// sharing converted codes (114 against 77 where rows pick blocks of their own,
// 70 against 77 on every block); the value products of a step issued behind
// the next step's scores (179 to 186); twelve compute warps of 144 registers.
#include <cmath>
#include <cstdint>

#include "../../include/pre_attn.h"
#include "pa_attn_kernel.cuh"

namespace pa {

template <int W>
__global__ void __launch_bounds__(32 * kJoinWarps) pa_attn_join_kernel(const __grid_constant__ CacheAttnParams a, int grid) {
  pdl_trigger();  // the next kernel's CTAs fit beside these; it waits for this grid's end
  pdl_wait();
  attn_join<W>(a, grid, blockIdx.x, blockIdx.y);
}

cudaError_t launch_attn_join(const CacheAttnParams &a, int sms, bool pdl, cudaStream_t stream) {
  const bool many = join_by_head(a, sms);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  cfg.gridDim = join_grid(a, many);
  cfg.blockDim = dim3(32 * kJoinWarps);
  return cudaLaunchKernelEx(&cfg, many ? pa_attn_join_kernel<kJoinWarps> : pa_attn_join_kernel<1>, a, sms);
}

}  // namespace pa

extern "C" size_t pre_attn_attention_workspace_bytes(int R, int q_len, int n_kv_heads, int num_sms) {
  if (R < 0 || R > 65535 || q_len < 1 || q_len > 16 || num_sms < 1 || num_sms > 4096) return 0;
  if (n_kv_heads != 1 && n_kv_heads != 2 && n_kv_heads != 4) return 0;
  return (size_t)2 * num_sms * pa::kAtPartFloats * sizeof(float) + pa::kAtMaxItems * sizeof(int2);
}

namespace pa {

// The checks of a call's arguments and the kernels' parameters from them;
// a.R is 0 where there is nothing to do.
int attn_params(const pa_attention_args &x, CacheAttnParams &a, int *num_sms) {
  a = CacheAttnParams{};
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
  *num_sms = sms;
  return PA_OK;
}

cudaError_t plain_attn_path(const CacheAttnParams &a, int fmt, int sms, int *path) {
  return fmt == 0 ? launch_attn<0, false>(a, sms, true, nullptr, nullptr, path)
                  : launch_attn<1, false>(a, sms, true, nullptr, nullptr, path);
}

}  // namespace pa

extern "C" int pre_attn_attention(const pa_attention_args *in, void *stream) {
  if (!in) return PA_ERR_NULL;
  pa::CacheAttnParams a;
  int sms = 0;
  const int st = pa::attn_params(*in, a, &sms);
  if (st != PA_OK || a.R == 0) return st;
  const bool pdl = !(in->flags & PA_FLAG_NO_PDL);
  const cudaError_t e = in->cache_format == PA_CACHE_FP8
                            ? pa::launch_attn<0, false>(a, sms, pdl, (cudaStream_t)stream, nullptr)
                            : pa::launch_attn<1, false>(a, sms, pdl, (cudaStream_t)stream, nullptr);
  return e == cudaSuccess ? PA_OK : pa::record_cuda_error(e);
}
