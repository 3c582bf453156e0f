// Decode of a batch whose sequences share long prefixes: C ABI and the join
// of the prefix's partial results with each sequence's own.
//
// Sequence s of group g attends to its group's P_g prefix positions, then to
// its own L_s.  Softmax over both is joined from parts: with (m_i, l_i, o_i)
// an exponent near the maximum, and the sum and unnormalised output relative
// to it, of part i of the prefix, and
// (lse, o) of the sequence's own positions (base 2),
//   M = max(m_i, lse),  out = (sum 2^(m_i - M) o_i + 2^(lse - M) o) /
//                             (sum 2^(m_i - M) l_i + 2^(lse - M)).
// The prefix's pages are read once per group instead of once per sequence:
// prefix partials by prefill_tc5_kernel (SH instances; members x heads of
// a group fill the 128 score rows of a tensor-core tile), own positions by
// the paged decode.
#include <algorithm>
#include <cmath>

#include "kvq_host.h"
#include "kvq_launch.h"

namespace kvq {

namespace {

struct JoinArgs {
  const float* part;    // [num_seqs][nq][splits][hd]
  const float2* ml;
  const float* own;     // [num_seqs][nq][hd]
  const float* lse;     // [num_seqs][nq]
  const int32_t* cu_groups;
  const int32_t* prefix_lens;
  const int32_t* unordered;
  int32_t num_groups, num_seqs, nq, splits;
  void* out;
  int out_bf16;
};

// A warp per (sequence, head) row; the parts' maxima and sums meet across its
// lanes, so that the outputs are read without waiting for one another.
template <int HD>
__global__ void __launch_bounds__(128) shared_join_kernel(const JoinArgs a) {
  constexpr int E = HD / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= (int64_t)a.num_seqs * a.nq) return;
  const int seq = (int)(row / a.nq);
  // the last group that starts at or before seq
  int lo = 0, hi = a.num_groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.cu_groups[mid] <= seq) lo = mid; else hi = mid;
  }
  const bool grouped = *a.unordered == 0 && a.cu_groups[lo] <= seq && seq < a.cu_groups[lo + 1] && a.prefix_lens[lo] > 0;
  const int n = grouped ? a.splits : 0;   // at most 64
  const float lse = a.lse[row];
  // lane i has parts i and i + 32; a part without positions is (-inf, 0)
  float2 ml[2];
#pragma unroll
  for (int u = 0; u < 2; ++u)
    ml[u] = lane + 32 * u < n ? a.ml[row * a.splits + lane + 32 * u] : make_float2(-INFINITY, 0.f);
  float m = fmaxf(ml[0].x, ml[1].x);
#pragma unroll
  for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  m = fmaxf(m, lse);
  const float base = m == -INFINITY ? 0.f : m;
  float f[2], l = 0.f;
#pragma unroll
  for (int u = 0; u < 2; ++u) {   // (a NaN sum stays one)
    f[u] = ml[u].x == -INFINITY && ml[u].y == 0.f ? 0.f : exp2f(ml[u].x - base);
    l += f[u] * ml[u].y;
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  const float w = lse == -INFINITY ? 0.f : exp2f(lse - base);
  const float sum = l + w;
  float x[E];
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = lse == -INFINITY ? 0.f : w * a.own[row * HD + lane * E + e];
  // parts past the last with positions may not have been written
  const uint32_t b0 = __ballot_sync(0xffffffffu, f[0] != 0.f), b1 = __ballot_sync(0xffffffffu, f[1] != 0.f);
  const int last = b1 ? 64 - __clz(b1) : 32 - __clz(b0);
  const float* part = a.part + row * a.splits * HD + lane * E;
#pragma unroll 4
  for (int i = 0; i < last; ++i) {   // (those before that without positions hold zeros)
    const float g = __shfl_sync(0xffffffffu, i < 32 ? f[0] : f[1], i & 31);
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = fmaf(g, part[i * HD + e], x[e]);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int64_t o = row * HD + lane * E + e;
    const float y = x[e] * inv;
    if (a.out_bf16) reinterpret_cast<uint16_t*>(a.out)[o] = bf16_bits_from_float(y);
    else reinterpret_cast<float*>(a.out)[o] = y;
  }
}

struct SharedPlan {
  int slots, splits;
  size_t decode, own, lse, part, ml, unordered, total;   // byte offsets and the whole size
};

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// CTAs per kv head of the prefix kernel, which shares the ranges out over them:
// one per SM, or two per score-row tile where the tiles at most (groups' sizes
// are on the device) are more than half of that; and the ranges a prefix may
// be cut into (at most 64, the join's two per lane).
SharedPlan plan_shared(int32_t num_seqs, int32_t num_groups, int nq, int nkv, int hd, int bs,
                       int32_t max_prefix_blocks, int32_t max_blocks, int32_t window, kvq_format fmt) {
  SharedPlan p{};
  const int rp = rmax_for(nq / nkv), rows = hd == 256 ? 64 : 128, tok = hd == 256 ? 32 : 64, qt = rows / rp;
  const int64_t tiles = num_seqs / qt + std::min(num_groups, num_seqs);
  const int64_t steps = std::max<int64_t>(1, ((int64_t)max_prefix_blocks * bs + tok - 1) / tok);
  const int64_t one = std::max(1, sm_count()) / nkv;
  p.slots = (int)std::min<int64_t>(std::max<int64_t>({2 * tiles > one ? 2 * tiles : one, tiles, 1}), 0x7fffffff);
  p.splits = (int)std::min<int64_t>({64, (int64_t)p.slots, steps});
  const size_t rows_all = (size_t)num_seqs * nq;
  const size_t dec = kvq_decode_workspace_bytes(num_seqs, nq, nkv, hd, bs, max_blocks, window, fmt);
  if (dec == 0) return SharedPlan{};
  p.decode = 0;
  p.own = align256(dec);
  p.lse = p.own + align256(rows_all * hd * 4);
  p.part = p.lse + align256(rows_all * 4);
  p.ml = p.part + align256(rows_all * p.splits * hd * 4);
  p.unordered = p.ml + align256(rows_all * p.splits * 8);
  p.total = p.unordered + 256;
  return p;
}

}  // namespace

}  // namespace kvq

using namespace kvq;

extern "C" {

size_t kvq_shared_decode_workspace_bytes(int32_t num_seqs, int32_t num_groups, int32_t nq, int32_t nkv, int32_t hd,
                                         int32_t bs, int32_t max_prefix_blocks, int32_t max_blocks, int32_t window,
                                         kvq_format fmt) {
  if (!fmt_ok(fmt) || num_seqs < 1 || num_groups < 1 || nkv < 1 || nq < 1 || nq % nkv || !rmax_for(nq / nkv) ||
      (hd != 64 && hd != 128 && hd != 256) || (bs != 8 && bs != 16 && bs != 32) || max_prefix_blocks < 1 ||
      max_blocks < 1 || window < 0)
    return 0;
  return plan_shared(num_seqs, num_groups, nq, nkv, hd, bs, max_prefix_blocks, max_blocks, window, fmt).total;
}

kvq_status kvq_paged_decode_shared(const void* q, kvq_dtype q_dtype, int64_t q_stride, const void* k_cache,
                                   const void* v_cache, void* out, kvq_dtype out_dtype,
                                   const int32_t* prefix_tables, int32_t max_prefix_blocks,
                                   const int32_t* prefix_lens, const int32_t* cu_groups, int32_t num_groups,
                                   const int32_t* block_tables, int32_t max_blocks, const int32_t* seq_lens,
                                   int32_t num_seqs, int64_t num_blocks, int32_t nq, int32_t nkv, int32_t hd,
                                   int32_t bs, int64_t k_bstride, int64_t v_bstride, float sm_scale, float k_scale,
                                   float v_scale, int32_t window, void* workspace, size_t workspace_bytes,
                                   kvq_format fmt, int32_t* error_flag, void* stream) {
  if (!fmt_ok(fmt)) return fail(KVQ_ERR_FORMAT, "format %d out of range", (int)fmt);
  const int ks = side_of(fmt, 0), vs = side_of(fmt, 1);
  if ((q_dtype != KVQ_DTYPE_F32 && q_dtype != KVQ_DTYPE_BF16) ||
      (out_dtype != KVQ_DTYPE_F32 && out_dtype != KVQ_DTYPE_BF16))
    return fail(KVQ_ERR_FORMAT, "q/out dtype must be f32 or bf16");
  if (hd != 64 && hd != 128 && hd != 256) return fail(KVQ_ERR_SHAPE, "head_dim %d not in {64,128,256}", hd);
  if (bs != 8 && bs != 16 && bs != 32) return fail(KVQ_ERR_SHAPE, "block_size %d not in {8,16,32}", bs);
  if (nkv < 1 || nq < 1 || nq % nkv) return fail(KVQ_ERR_SHAPE, "num_q_heads must be a multiple of num_kv_heads");
  const int rep = nq / nkv, rp = rmax_for(rep);
  if (!rp) return fail(KVQ_ERR_SHAPE, "grouped-query ratio %d above 8", rep);
  if (nkv > 65535) return fail(KVQ_ERR_SHAPE, "num_kv_heads above 65535");
  if (num_seqs < 0 || num_blocks < 0 || window < 0) return fail(KVQ_ERR_ARG, "negative count");
  if (!std::isfinite(sm_scale)) return fail(KVQ_ERR_ARG, "sm_scale must be finite");
  if (num_seqs == 0) return ok();
  if (num_groups < 1) return fail(KVQ_ERR_ARG, "num_groups must be >= 1");
  if (max_blocks < 1 || max_prefix_blocks < 1) return fail(KVQ_ERR_ARG, "block tables need a column");
  if (!q || !k_cache || !v_cache || !out || !prefix_tables || !prefix_lens || !cu_groups || !block_tables ||
      !seq_lens || !workspace)
    return fail(KVQ_ERR_ARG, "null pointer");
  if (q_stride < (int64_t)nq * hd) return fail(KVQ_ERR_ARG, "q_stride smaller than num_q_heads*head_dim");
  const int64_t kb = kvq_block_bytes(fmt, 0, bs, nkv, hd), vb = kvq_block_bytes(fmt, 1, bs, nkv, hd);
  if (k_bstride < kb || v_bstride < vb) return fail(KVQ_ERR_ARG, "block stride below block bytes");
  if (k_bstride % 16 || v_bstride % 16 || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(workspace))
    return fail(KVQ_ERR_ALIGN, "caches, block strides and workspace must be 16-byte aligned");
  if ((ks == S_FP8 && !(k_scale > 0.f && std::isfinite(k_scale))) ||
      (vs == S_FP8 && !(v_scale > 0.f && std::isfinite(v_scale))))
    return fail(KVQ_ERR_ARG, "FP8 side needs a finite scale > 0");
  if ((int64_t)num_seqs * nq > (int64_t)0x7fffffff) return fail(KVQ_ERR_SHAPE, "num_seqs * num_q_heads must be below 2^31");
  const SharedPlan p = plan_shared(num_seqs, num_groups, nq, nkv, hd, bs, max_prefix_blocks, max_blocks, window, fmt);
  if (workspace_bytes < p.total)
    return fail(KVQ_ERR_WORKSPACE, "workspace %zu bytes, need %zu", workspace_bytes, p.total);
  uint8_t* ws = (uint8_t*)workspace;
  const cudaStream_t st = (cudaStream_t)stream;

  PrefillArgs a{};
  a.q = q;
  a.q_stride = q_stride;
  a.q_bf16 = q_dtype == KVQ_DTYPE_BF16;
  a.cu_q = cu_groups;
  a.k_cache = (const uint8_t*)k_cache;
  a.v_cache = (const uint8_t*)v_cache;
  a.block_tables = prefix_tables;
  a.max_blocks = max_prefix_blocks;
  a.seq_lens = prefix_lens;
  a.num_seqs = num_seqs;
  a.num_blocks = num_blocks;
  a.nq = nq;
  a.nkv = nkv;
  a.rep = rep;
  a.rp = rp;
  a.bs = bs;
  a.k_bstride = k_bstride;
  a.v_bstride = v_bstride;
  a.k_dsec = kvq_data_section_bytes(fmt, 0, bs, nkv, hd);
  a.v_dsec = kvq_data_section_bytes(fmt, 1, bs, nkv, hd);
  const double scale = sm_scale == 0.f ? 1.0 / std::sqrt((double)hd) : (double)sm_scale;
  a.score_scale = (float)(scale * M_LOG2E * (ks == S_FP8 ? (double)k_scale : 1.0));
  a.v_mult = vs == S_FP8 ? v_scale : 1.0f;
  a.inv_sqrt_hd = (float)(1.0 / std::sqrt((double)hd));
  a.window = window;
  a.err = error_flag;
  a.sh.num_groups = num_groups;
  a.sh.own_lens = seq_lens;
  a.sh.splits = p.splits;
  a.sh.q_mul = query_factor(ks, a.score_scale);
  a.sh.s_mul = a.score_scale / a.sh.q_mul;
  a.sh.part = (float*)(ws + p.part);
  a.sh.ml = (float2*)(ws + p.ml);
  // the decode wants its merge counters zero, whatever the workspace held
  const size_t dec = kvq_decode_workspace_bytes(num_seqs, nq, nkv, hd, bs, max_blocks, window, fmt);
  const size_t ctr = ((size_t)num_seqs * nkv * sizeof(int32_t) + 15) / 16 * 16;
  a.sh.counters = (int32_t*)(ws + dec - ctr);
  a.sh.num_counters = (int64_t)num_seqs * nkv;
  a.sh.unordered = (int32_t*)(ws + p.unordered);
  const Codebooks& cb = codebooks();
  cudaError_t e;
  switch (ks) {
    case S_BF16: e = launch_sh_k_bf16(vs, hd, a, cb, p.slots, st); break;
    case S_FP8: e = launch_sh_k_fp8(vs, hd, a, cb, p.slots, st); break;
    case S_T4: e = launch_sh_k_t4(vs, hd, a, cb, p.slots, st); break;
    case S_T3: e = launch_sh_k_t3(vs, hd, a, cb, p.slots, st); break;
    case S_T2: e = launch_sh_k_t2(vs, hd, a, cb, p.slots, st); break;
    case S_T8: e = launch_sh_k_t8(vs, hd, a, cb, p.slots, st); break;
    case S_NVFP4: e = launch_sh_k_nvfp4(vs, hd, a, cb, p.slots, st); break;
    default: e = cudaErrorInvalidValue;
  }
  if (e != cudaSuccess) return fail(KVQ_ERR_CUDA, "shared prefix launch: %s", cudaGetErrorString(e));
  const kvq_status s = decode_with_lse(q, q_dtype, q_stride, k_cache, v_cache, ws + p.own, KVQ_DTYPE_F32,
                                       (float*)(ws + p.lse), block_tables, max_blocks, seq_lens, num_seqs,
                                       num_blocks, nq, nkv, hd, bs, k_bstride, v_bstride, sm_scale, k_scale, v_scale,
                                       window, 0.f, ws + p.decode, dec, fmt, error_flag, stream);
  if (s != KVQ_OK) return s;
  JoinArgs j{a.sh.part, a.sh.ml, (const float*)(ws + p.own), (const float*)(ws + p.lse), cu_groups, prefix_lens,
             a.sh.unordered, num_groups, num_seqs, nq, p.splits, out, out_dtype == KVQ_DTYPE_BF16};
  const unsigned grid = (unsigned)(((int64_t)num_seqs * nq + 3) / 4);
  if (hd == 64) shared_join_kernel<64><<<grid, 128, 0, st>>>(j);
  else if (hd == 128) shared_join_kernel<128><<<grid, 128, 0, st>>>(j);
  else shared_join_kernel<256><<<grid, 128, 0, st>>>(j);
  e = cudaGetLastError();
  if (e != cudaSuccess) return fail(KVQ_ERR_CUDA, "shared join launch: %s", cudaGetErrorString(e));
  return ok();
}

}  // extern "C"
