// Attention mass: the C ABI entry points and the instances whose K side is
// stored as values (BF16, FP8, Turbo8).
#include <algorithm>
#include <cmath>

#include "kvq_host.h"
#include "kvq_mass_tc.cuh"

namespace kvq {

cudaError_t launch_mass_raw(int k_side, int hd, const MassArgs& a, const Codebooks& cb, cudaStream_t st) {
  switch (k_side) {
    case S_BF16: return launch_mass_side<S_BF16>(hd, a, cb, st);
    case S_FP8: return launch_mass_side<S_FP8>(hd, a, cb, st);
    case S_T8: return launch_mass_side<S_T8>(hd, a, cb, st);
    default: return cudaErrorInvalidValue;
  }
}

namespace {

// Few score rows: totals from the kept scores, a thread per position.
constexpr int kAddTile = 1024;

template <int RP>
__global__ void __launch_bounds__(256) mass_add_kernel(const MassArgs a) {
  __shared__ float lse_s[8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t seq = blockIdx.x / a.nkv;
  const int kvh = (int)(blockIdx.x - seq * a.nkv);
  const MassSeq sq = mass_seq(a, seq, false);
  const int t0 = blockIdx.y * kAddTile;
  if (t0 >= sq.len) return;
  if (warp < sq.rows) {   // a warp joins a row's ranges
    const int tiles = (sq.len + kMassTile - 1) / kMassTile, first = min(sq.lo / kMassTile, tiles);
    const int per = (tiles - first + a.splits1 - 1) / a.splits1;
    const int used = per > 0 ? (tiles - first + per - 1) / per : 0;
    const float2* st = a.stats + ((sq.q0 + warp / a.rep) * a.nq + kvh * a.rep + warp % a.rep) * a.splits1;
    const float2 x = lane < used ? st[lane] : make_float2(-CUDART_INF_F, 0.f);
    float mm = x.x;
#pragma unroll
    for (int d = 16; d; d >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, d));
    float ll = x.y * t5::ex2(x.x - (mm == -CUDART_INF_F ? 0.f : mm));
#pragma unroll
    for (int d = 16; d; d >>= 1) ll += __shfl_xor_sync(0xffffffffu, ll, d);
    // a row that attends to nothing adds nothing: 2^(s - inf) = 0
    if (lane == 0) lse_s[warp] = mm == -CUDART_INF_F && !(ll != ll) ? CUDART_INF_F : mm + log2f(ll);
  }
  __syncthreads();
  float lse[RP];
#pragma unroll
  for (int r = 0; r < RP; ++r) lse[r] = r < sq.rows ? lse_s[r] : CUDART_INF_F;
  const float* sc = a.scores + ((int64_t)blockIdx.x * a.max_blocks * a.bs) * RP;
#pragma unroll
  for (int k = 0; k < kAddTile / 256; ++k) {
    const int t = t0 + k * 256 + tid;
    if (t >= sq.len || t >= a.out_stride) continue;
    float sum = 0.f;
    if (t >= sq.lo && sq.rows > 0) {
      float s[RP];
#pragma unroll
      for (int r = 0; r < RP; r += 2) {
        const float2 x = *reinterpret_cast<const float2*>(sc + (int64_t)t * RP + r);
        s[r] = x.x;
        s[r + 1] = x.y;
      }
      // a masked score and a row without positions add nothing, whatever the other is
#pragma unroll
      for (int r = 0; r < RP; ++r)
        sum += lse[r] == CUDART_INF_F || s[r] == -CUDART_INF_F ? 0.f : t5::ex2(s[r] - lse[r]);
    }
    const float prev = a.mass_in ? a.mass_in[(int64_t)blockIdx.x * a.in_stride + t] : 0.f;
    a.mass_out[(int64_t)blockIdx.x * a.out_stride + t] = prev + sum;
  }
}

cudaError_t launch_mass_add(const MassArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)((int64_t)a.num_seqs * a.nkv), (unsigned)(((int64_t)a.max_blocks * a.bs + kAddTile - 1) / kAddTile));
  switch (a.row_pad) {
    case 2: mass_add_kernel<2><<<grid, 256, 0, st>>>(a); break;
    case 4: mass_add_kernel<4><<<grid, 256, 0, st>>>(a); break;
    case 6: mass_add_kernel<6><<<grid, 256, 0, st>>>(a); break;
    default: mass_add_kernel<8><<<grid, 256, 0, st>>>(a); break;
  }
  return cudaGetLastError();
}

// How a call is cut.  Few rows (up to 8, with room for their scores): enough
// ranges for about two waves of two CTAs per SM, at most 32 (a warp joins them
// lane by lane).  Many rows: one CTA per SM, or two ranges per (sequence, kv
// head) where those alone are more than half the SMs; the kernel balances the
// ranges over them.  Its statistics are no larger for a smaller total_q or
// max_chunk, so that a workspace of a larger chunk always serves: few rows
// then take the other kernel where their scores do not fit.
struct MassPlan {
  bool few;
  int splits1, slots, row_pad;
  size_t stats, total;   // bytes of the statistics, and of the workspace
};

MassPlan mass_plan(int64_t total_q, int32_t num_seqs, int32_t max_chunk, int nq, int nkv, int bs, int32_t max_blocks,
                   bool scores = true) {
  MassPlan p{};
  const int rep = nq / nkv;
  const int64_t rows = (int64_t)max_chunk * rep, units = (int64_t)num_seqs * nkv, max_pos = (int64_t)max_blocks * bs;
  const int64_t tiles = std::max<int64_t>(1, (max_pos + kMassTile - 1) / kMassTile), sms = std::max(sm_count(), 1);
  p.few = scores && rows <= 8;
  if (p.few) {
    p.row_pad = ((int)rows + 1) / 2 * 2;
    p.splits1 = (int)std::max<int64_t>(1, std::min<int64_t>({(4 * sms + units - 1) / units, tiles, 32}));
  } else {
    p.slots = (int)std::min<int64_t>(2 * units <= sms ? std::max<int64_t>(sms / nkv, num_seqs) : 2 * (int64_t)num_seqs,
                                     0x7fffffff / nkv);
    p.splits1 = (int)std::min<int64_t>(p.slots, tiles);
  }
  p.stats = ((size_t)total_q * nq * p.splits1 * sizeof(float2) + 255) / 256 * 256;
  p.total = p.stats + (p.few ? (size_t)units * max_pos * p.row_pad * sizeof(float) : 0);
  return p;
}

}  // namespace

}  // namespace kvq

using namespace kvq;

extern "C" {

size_t kvq_attention_mass_workspace_bytes(int64_t total_q, int32_t num_seqs, int32_t max_chunk, int32_t nq,
                                          int32_t nkv, int32_t bs, int32_t max_blocks) {
  if (total_q < 0 || num_seqs < 1 || max_chunk < 1 || nq < 1 || nkv < 1 || nq % nkv || bs < 1 || max_blocks < 1)
    return 0;
  return mass_plan(total_q, num_seqs, max_chunk, nq, nkv, bs, max_blocks).total;
}

kvq_status kvq_attention_mass(const void* q, kvq_dtype q_dtype, int64_t q_stride, const int32_t* cu_q,
                              int64_t total_q, int32_t max_chunk, const void* k_cache,
                              const int32_t* block_tables, int32_t max_blocks, const int32_t* seq_lens,
                              int32_t num_seqs, int64_t num_blocks, int32_t nq, int32_t nkv, int32_t hd,
                              int32_t bs, int64_t k_bstride, float sm_scale, float k_scale, int32_t window,
                              const float* mass_in, int64_t mass_in_stride, float* mass_out,
                              int64_t mass_out_stride, void* workspace, size_t workspace_bytes, kvq_format fmt,
                              int32_t* error_flag, void* stream) {
  if (!fmt_ok(fmt)) return fail(KVQ_ERR_FORMAT, "format %d out of range", (int)fmt);
  const int ks = side_of(fmt, 0);
  if (q_dtype != KVQ_DTYPE_F32 && q_dtype != KVQ_DTYPE_BF16) return fail(KVQ_ERR_FORMAT, "q dtype must be f32 or bf16");
  if (hd != 64 && hd != 128 && hd != 256) return fail(KVQ_ERR_SHAPE, "head_dim %d not in {64,128,256}", hd);
  if (bs != 8 && bs != 16 && bs != 32) return fail(KVQ_ERR_SHAPE, "block_size %d not in {8,16,32}", bs);
  if (nkv < 1 || nq < 1 || nq % nkv) return fail(KVQ_ERR_SHAPE, "num_q_heads must be a multiple of num_kv_heads");
  const int rep = nq / nkv;
  if (!rmax_for(rep)) return fail(KVQ_ERR_SHAPE, "grouped-query ratio %d above 8", rep);
  if (num_seqs < 0 || num_blocks < 0 || window < 0 || max_chunk < 0 || total_q < 0)
    return fail(KVQ_ERR_ARG, "negative count");
  if (!std::isfinite(sm_scale)) return fail(KVQ_ERR_ARG, "sm_scale must be finite");
  if (num_seqs == 0) return ok();
  if (max_blocks < 1) return fail(KVQ_ERR_ARG, "max_blocks_per_seq must be >= 1");
  if (max_chunk < 1) return fail(KVQ_ERR_ARG, "max_chunk must be >= 1");
  if ((int64_t)max_blocks * bs > (int64_t)65535 * kAddTile) return fail(KVQ_ERR_SHAPE, "max_blocks_per_seq too large");
  if ((int64_t)num_seqs * nkv > 0x7fffffff) return fail(KVQ_ERR_SHAPE, "num_seqs * num_kv_heads must be below 2^31");
  if ((int64_t)max_chunk * rep > (int64_t)65535 * 128) return fail(KVQ_ERR_SHAPE, "max_chunk too large (split the call)");
  if ((!q && total_q > 0) || !cu_q || !k_cache || !block_tables || !seq_lens || !mass_out)
    return fail(KVQ_ERR_ARG, "null pointer");
  if (q_stride < (int64_t)nq * hd) return fail(KVQ_ERR_ARG, "q_stride smaller than num_q_heads*head_dim");
  if (mass_out_stride < 1 || (mass_in && mass_in_stride < mass_out_stride && mass_in_stride < (int64_t)max_blocks * bs))
    return fail(KVQ_ERR_ARG, "mass rows too short");
  if (mass_in == mass_out && mass_in_stride != mass_out_stride)
    return fail(KVQ_ERR_ARG, "one mass array needs one stride");
  if (k_bstride < kvq_block_bytes(fmt, 0, bs, nkv, hd)) return fail(KVQ_ERR_ARG, "block stride below block bytes");
  if (k_bstride % 16 || !aligned16(k_cache)) return fail(KVQ_ERR_ALIGN, "cache and block stride must be 16-byte aligned");
  if (ks == S_FP8 && !(k_scale > 0.f && std::isfinite(k_scale)))
    return fail(KVQ_ERR_ARG, "FP8 side needs a finite scale > 0");
  MassPlan p = mass_plan(total_q, num_seqs, max_chunk, nq, nkv, bs, max_blocks);
  if (p.few && workspace_bytes < p.total) p = mass_plan(total_q, num_seqs, max_chunk, nq, nkv, bs, max_blocks, false);
  const size_t need = p.total;
  if (need > 0 && !workspace) return fail(KVQ_ERR_ARG, "null pointer");
  if (workspace_bytes < need) return fail(KVQ_ERR_WORKSPACE, "workspace %zu bytes, need %zu", workspace_bytes, need);
  if (!aligned16(workspace)) return fail(KVQ_ERR_ALIGN, "workspace must be 16-byte aligned");
  MassArgs a{};
  a.q = q;
  a.q_stride = q_stride;
  a.q_bf16 = q_dtype == KVQ_DTYPE_BF16;
  a.q_vec = total_q > 0 && aligned16(q) && q_stride * 2 % 16 == 0;
  a.cu_q = cu_q;
  a.total_q = total_q;
  a.max_chunk = max_chunk;
  a.k_cache = (const uint8_t*)k_cache;
  a.block_tables = block_tables;
  a.max_blocks = max_blocks;
  a.seq_lens = seq_lens;
  a.num_seqs = num_seqs;
  a.num_blocks = num_blocks;
  a.nq = nq;
  a.nkv = nkv;
  a.rep = rep;
  a.bs = bs;
  a.lbs = __builtin_ctz((unsigned)bs);
  a.k_bstride = k_bstride;
  a.k_dsec = kvq_data_section_bytes(fmt, 0, bs, nkv, hd);
  const double scale = sm_scale == 0.f ? 1.0 / std::sqrt((double)hd) : (double)sm_scale;
  const float score_scale = (float)(scale * M_LOG2E * (ks == S_FP8 ? (double)k_scale : 1.0));
  a.q_mul = query_factor(ks, score_scale);
  a.score_scale = score_scale / a.q_mul;
  a.inv_sqrt_hd = (float)(1.0 / std::sqrt((double)hd));
  a.window = window;
  a.splits1 = p.splits1;
  a.slots = p.slots;
  a.row_pad = p.row_pad;
  a.stats = (float2*)workspace;
  a.scores = p.few ? (float*)((uint8_t*)workspace + p.stats) : nullptr;
  a.mass_in = mass_in;
  a.mass_out = mass_out;
  a.in_stride = mass_in_stride;
  a.out_stride = mass_out_stride;
  a.err = error_flag;
  const bool codes = side_codebook(ks);
  cudaError_t e = codes ? launch_mass_codes(ks, hd, a, codebooks(), (cudaStream_t)stream)
                        : launch_mass_raw(ks, hd, a, codebooks(), (cudaStream_t)stream);
  if (e == cudaSuccess && p.few) e = launch_mass_add(a, (cudaStream_t)stream);
  if (e != cudaSuccess) return fail(KVQ_ERR_CUDA, "attention mass launch: %s", cudaGetErrorString(e));
  return ok();
}

}  // extern "C"
