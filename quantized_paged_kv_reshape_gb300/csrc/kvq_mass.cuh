// Attention weight per cached position, summed over the queries of a chunk
// and the query heads of a kv head, added to running totals.
//
// "combs_models/kv.rs" attend (scores, causal mask, softmax) with repeat_kv;
// query i of sequence s's chunk sits at p = L - C + i and attends to
// [max(0, p + 1 - W), p] as in the chunked prefill.  With s_rt the score of
// score row r = (i, head) at position t:
//   lse_r = log sum_t exp(s_rt),   mass_t += sum_r exp(s_rt - lse_r).
//
// Up to 8 score rows per kv head (a decode step): mass_rows_kernel reads K
// once, keeps every score (fp32, 4 bytes a row and position) and writes each
// range's running maximum and sum (base 2); mass_add_kernel joins the ranges
// and adds 2^(s - lse) up.  Eight rows' scores are 64 bytes a position written
// and read, beside a K row of 256 (BF16, head_dim 128) but also of 20 (Turbo2,
// 64); what is saved is the row's dequantization and its products.  GB300, 32
// sequences of 4096 positions and 8 kv heads, kept against mass_tc_kernel: BF16
// 4 rows 76 / 429 us, Turbo2 at 64 8 rows 61 / 420 us.  More rows:
// mass_tc_kernel (kvq_mass_tc.cuh), which computes the scores twice.  A
// position's total is one thread's sum, so nothing is added atomically and
// results do not depend on scheduling.
//
// Scores: S[16 positions x 8 rows] = K . q^T per warp with mma.sync
// m16n8k16.  A dot product does not depend on the order of its dims, so lane
// (g, c) reads dims of rows g and g + 8 straight from the page as one run of
// head_dim / 4 elements (BF16: runs of 8, whole sectors per quad), already
// in operand order, with no staging; q is laid out to match.  Where one
// 16-bit value is not exact, q and K carry hi + lo fp16 parts (22 bits): the
// totals are fp32 and add up over many steps, so the decode's 14-bit levels
// (whose error its 16-bit outputs hide) are not used here.  fp16 queries
// are kept in range by a power of two (query_factor).
#pragma once

#include "kvq_prefill_tc5.cuh"

namespace kvq {

struct MassArgs {
  const void* q;
  int64_t q_stride;
  int q_bf16, q_vec;           // q_vec: rows start on 16-byte boundaries
  const int32_t* cu_q;
  int64_t total_q;
  int32_t max_chunk;
  const uint8_t* k_cache;
  const int32_t* block_tables;
  int32_t max_blocks;
  const int32_t* seq_lens;
  int32_t num_seqs;
  int64_t num_blocks;
  int32_t nq, nkv, rep, bs, lbs;
  int64_t k_bstride, k_dsec;
  float score_scale, q_mul, inv_sqrt_hd;   // scores = score_scale * (q_mul * q).k
  int32_t window;
  int32_t splits1;             // position ranges per (sequence, kv head)
  int32_t slots;               // CTAs per kv head (mass_tc_kernel)
  float2* stats;               // [total_q][nq][splits1] (max, sum)
  float* scores;               // mass_rows_kernel: [num_seqs][nkv][max_blocks * bs][row_pad]
  int32_t row_pad;             // score rows of a sequence and kv head, rounded up to 2
  const float* mass_in;
  float* mass_out;
  int64_t in_stride, out_stride;   // elements per (sequence, kv head) row
  int32_t* err;
};

constexpr int kMassWarps = 8, kMassTile = 16 * kMassWarps;

template <int S, int HD>
struct MassSide {
  static constexpr int D = HD / 4;                        // dims per lane and row
  static constexpr int NK = HD / 16;                      // k-steps
  static constexpr int BYTES = D * side_bits(S) / 8;      // raw bytes per lane and row
  static constexpr int WORDS = (BYTES + 3) / 4;
  static constexpr int SBYTES = D / kGroup * side_scale_bytes(S);
  static constexpr int SWORDS = (SBYTES + 3) / 4;
  static constexpr int PLANES = PfSide<S>::PLANES;
  static constexpr bool BF = S == S_BF16;
};

template <int S, int HD>
struct MassRaw {   // a lane's bytes of one row
  uint32_t w[MassSide<S, HD>::WORDS];
  uint32_t s[MassSide<S, HD>::SWORDS > 0 ? MassSide<S, HD>::SWORDS : 1];
};

template <int BYTES>
__device__ __forceinline__ void load_bytes(const uint8_t* p, uint32_t* w) {
  if constexpr (BYTES >= 16) {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
      const uint4 x = *reinterpret_cast<const uint4*>(p + 16 * i);
      w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
    }
    if constexpr (BYTES % 16 == 8) {
      const uint2 x = *reinterpret_cast<const uint2*>(p + BYTES / 16 * 16);
      w[BYTES / 16 * 4] = x.x; w[BYTES / 16 * 4 + 1] = x.y;
    }
  } else if constexpr (BYTES == 12) {
#pragma unroll
    for (int i = 0; i < 3; ++i) w[i] = *reinterpret_cast<const uint32_t*>(p + 4 * i);
  } else if constexpr (BYTES == 8) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    w[0] = x.x; w[1] = x.y;
  } else if constexpr (BYTES == 6) {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
    w[0] = (uint32_t)h[0] | ((uint32_t)h[1] << 16);
    w[1] = h[2];
  } else if constexpr (BYTES == 4) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (BYTES == 2) {
    w[0] = *reinterpret_cast<const uint16_t*>(p);
  } else if constexpr (BYTES == 1) {
    w[0] = *p;
  }
}

// Turbo3 rows of 24 bytes per lane start on 8-byte boundaries only.
template <int S, int HD>
__device__ __forceinline__ void mass_load(MassRaw<S, HD>& r, const uint8_t* row, const uint8_t* srow, int c) {
  using M = MassSide<S, HD>;
  if constexpr (S == S_BF16) {
#pragma unroll
    for (int n = 0; n < HD / 32; ++n) load_bytes<16>(row + 2 * (32 * n + 8 * c), r.w + 4 * n);
  } else if constexpr (M::BYTES == 24) {
#pragma unroll
    for (int n = 0; n < 3; ++n) load_bytes<8>(row + 24 * c + 8 * n, r.w + 2 * n);
  } else {
    load_bytes<M::BYTES>(row + M::BYTES * c, r.w);
  }
  if constexpr (M::SBYTES > 0) load_bytes<M::SBYTES>(srow + M::SBYTES * c, r.s);
}

// A row's elements as 16-bit pairs (hi, and lo where PLANES == 2).  Levels
// come one code at a time from `lv` (fp32, at most 16 entries): every entry
// has its own bank, so the lanes' look-ups never conflict (a table of code
// pairs halves the look-ups, but its lanes conflict: 107 against 92 us for 128
// rows over 35k Turbo4 positions of 8 heads).
template <int S, int HD>
__device__ __forceinline__ void mass_dequant(const MassRaw<S, HD>& r, const float* lv, uint32_t (&hi)[HD / 8],
                                             uint32_t (&lo)[HD / 8]) {
  constexpr int D = HD / 4;
  if constexpr (S == S_BF16) {
#pragma unroll
    for (int i = 0; i < D / 2; ++i) hi[i] = r.w[i];
  } else if constexpr (S == S_FP8) {
#pragma unroll
    for (int i = 0; i < D / 2; ++i) hi[i] = tc::e4m3x2_f16x2((r.w[i / 2] >> (16 * (i & 1))) & 0xffffu);
  } else if constexpr (S == S_T8) {
#pragma unroll
    for (int i = 0; i < D / 2; ++i) {
      const int gi = 2 * i / kGroup;
      const float sc = bf16_bits_to_float((r.s[gi / 2] >> (16 * (gi & 1))) & 0xffffu);
      const float2 e = e4m3x2_to_float2((uint16_t)(r.w[i / 2] >> (16 * (i & 1))));
      tc::split2<false>(e.x * sc, e.y * sc, hi[i], lo[i]);
    }
  } else {
    constexpr int B = code_bits(S);
    auto level = [&](int i) {   // of the i-th code
      const int bit = B * i, w = bit / 32, off = bit % 32;
      uint32_t x = r.w[w] >> off;
      if (off + B > 32) x |= r.w[w + 1] << (32 - off);
      return lv[x & ((1u << B) - 1u)];
    };
#pragma unroll
    for (int i = 0; i < D / 2; ++i) {
      const int gi = 2 * i / kGroup;
      const float sc = e4m3_to_float((uint8_t)(r.s[gi / 4] >> (8 * (gi & 3))));
      const float x0 = level(2 * i) * sc, x1 = level(2 * i + 1) * sc;
      if constexpr (MassSide<S, HD>::PLANES == 2) tc::split2<false>(x0, x1, hi[i], lo[i]);
      else hi[i] = tc::pack2<false>(x0, x1);   // E2M1 values times the scale: exact
    }
  }
}

template <int S>
__device__ __forceinline__ void mass_fill_levels(float* lv, const Codebooks& cb, int tid) {
  if constexpr (side_codebook(S)) {
    if (tid < (1 << code_bits(S))) lv[tid] = side_levels<S>(cb)[tid];
  }
}

// Per sequence: cached positions, chunk, first attended position.
struct MassSeq {
  int len, pbase, rows, lo;
  int64_t q0;
};
__device__ __forceinline__ MassSeq mass_seq(const MassArgs& a, int64_t seq, bool flag) {
  MassSeq x;
  const int64_t cap = (int64_t)a.max_blocks * a.bs;
  int len = a.seq_lens[seq];
  int64_t q0 = a.cu_q[seq], q1 = a.cu_q[seq + 1];
  bool cut = false;
  if (q0 < 0 || q1 > a.total_q || q1 < q0) {
    cut = true;
    q0 = max((int64_t)0, min(q0, a.total_q));
    q1 = max(q0, min(q1, a.total_q));
  }
  const int cq = (int)(q1 - q0);   // the chunk's queries are the last cq positions
  if (flag && a.err) {
    if (cut || cq > a.max_chunk || len > a.out_stride) atomicOr(a.err, KVQ_DEVERR_RANGE);
    if (len > cap) atomicOr(a.err, KVQ_DEVERR_BLOCK);
  }
  if (len > cap) len = (int)cap;
  x.len = max(len, 0);
  x.pbase = x.len - cq;            // position of query 0
  x.rows = min(cq, a.max_chunk) * a.rep;
  x.lo = a.window > 0 ? max(0, max(x.pbase, 0) + 1 - a.window) : 0;
  x.q0 = q0;
  return x;
}

// Scores and statistics of up to 8 rows: a warp takes 16 positions of the
// CTA's 128-position tiles; rows, codes and queries stay in registers.
template <int S, int HD>
__global__ void __launch_bounds__(32 * kMassWarps) mass_rows_kernel(const MassArgs a, const Codebooks cb) {
  using M = MassSide<S, HD>;
  constexpr int NK = M::NK, E = HD / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int64_t seq = blockIdx.x / a.nkv;
  const int kvh = (int)(blockIdx.x - seq * a.nkv);
  extern __shared__ __align__(128) uint8_t smem[];
  uint4* qf = reinterpret_cast<uint4*>(smem);                  // [NK][32 lanes] (hi0, hi1, lo0, lo1)
  __shared__ float2 red_s[kMassWarps][8];
  __shared__ float lv[16];

  const MassSeq sq = mass_seq(a, seq, tid == 0 && blockIdx.y == 0);
  const int len = sq.len, pbase = sq.pbase, rows = sq.rows, lo_all = sq.lo;
  const int tiles = (len + kMassTile - 1) / kMassTile, first = min(lo_all / kMassTile, tiles);
  const int per = (tiles - first + a.splits1 - 1) / a.splits1;
  const int tile0 = min(tiles, first + (int)blockIdx.y * per), tile1 = min(tiles, tile0 + per);
  if (tile0 >= tile1 || rows == 0) return;

  mass_fill_levels<S>(lv, cb, tid);
  const bool q_lo = side_rotated(S) || !a.q_bf16;
  {   // a warp per score row, into operand order
    const int r = warp;
    float x[E];
    if (r < rows) {
      const int64_t off = (sq.q0 + r / a.rep) * a.q_stride + (int64_t)(kvh * a.rep + r % a.rep) * HD + lane * E;
#pragma unroll
      for (int i = 0; i < E; ++i)
        x[i] = a.q_bf16 ? bf16_bits_to_float(reinterpret_cast<const uint16_t*>(a.q)[off + i])
                        : reinterpret_cast<const float*>(a.q)[off + i];
      if constexpr (side_rotated(S)) fwht_warp<E>(x, lane, a.inv_sqrt_hd);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      const int d = lane * E + i;
      const int qc = S == S_BF16 ? (d % 32) / 8 : d / (HD / 4);
      const int idx = S == S_BF16 ? d / 32 * 8 + d % 8 : d % (HD / 4);
      uint32_t h, l;
      tc::split2<M::BF>(x[i] * a.q_mul, x[i + 1] * a.q_mul, h, l);
      uint32_t* dst = reinterpret_cast<uint32_t*>(qf + (idx / 4) * 32 + r * 4 + qc);
      dst[(idx % 4) / 2] = h;
      dst[2 + (idx % 4) / 2] = l;
    }
  }
  __syncthreads();

  // raw rows of a tile: lane rows g and g + 8 of this warp's 16 positions
  const int32_t* tab = a.block_tables + seq * a.max_blocks;
  MassRaw<S, HD> raw[2];
  bool rok[2];
  int32_t bid[2];
  auto ids = [&](int tile) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int t = tile * kMassTile + warp * 16 + g + 8 * e;
      bid[e] = tile < tile1 && t < len && t >= lo_all ? tab[t >> a.lbs] : -2;
    }
  };
  auto fetch = [&](int tile) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int t = tile * kMassTile + warp * 16 + g + 8 * e;
      rok[e] = bid[e] >= 0 && (a.num_blocks <= 0 || bid[e] < a.num_blocks);
      if (!rok[e] && bid[e] != -2 && a.err) atomicOr(a.err, KVQ_DEVERR_BLOCK);
      if (rok[e]) {
        const int64_t rr = (int64_t)(t & (a.bs - 1)) * a.nkv + kvh;
        const uint8_t* p = a.k_cache + bid[e] * a.k_bstride;
        mass_load<S, HD>(raw[e], p + rr * (HD * side_bits(S) / 8),
                         p + a.k_dsec + rr * (HD / kGroup * side_scale_bytes(S)), c);
      } else {
#pragma unroll
        for (int i = 0; i < M::WORDS; ++i) raw[e].w[i] = 0u;
#pragma unroll
        for (int i = 0; i < (M::SWORDS > 0 ? M::SWORDS : 1); ++i) raw[e].s[i] = 0u;
      }
    }
  };
  // positions this lane's two score rows (2c, 2c + 1) attend to: (p - W, p]
  const int p0 = 2 * c < rows ? pbase + 2 * c / a.rep : -1, p1 = 2 * c + 1 < rows ? pbase + (2 * c + 1) / a.rep : -1;
  const int w0 = a.window > 0 ? p0 - a.window : -1, w1 = a.window > 0 ? p1 - a.window : -1;
  float m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.f, 0.f};
  float* sc_out = a.scores + ((int64_t)blockIdx.x * a.max_blocks * a.bs) * a.row_pad;
  ids(tile0);
  fetch(tile0);
  ids(tile0 + 1);
  for (int tile = tile0; tile < tile1; ++tile) {
    uint32_t kh[2][HD / 8], kl[2][HD / 8];
    mass_dequant<S, HD>(raw[0], lv, kh[0], kl[0]);
    mass_dequant<S, HD>(raw[1], lv, kh[1], kl[1]);
    const bool ok0 = rok[0], ok1 = rok[1];
    if (tile + 1 < tile1) {
      fetch(tile + 1);
      ids(tile + 2);
    }
    // sv[0], sv[1] = position g, rows 2c, 2c + 1; sv[2], sv[3] = position g + 8
    float sv[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NK; ++j) {
      const uint4 b = qf[j * 32 + lane];
      tc::mma<M::BF>(sv, kh[0][2 * j], kh[1][2 * j], kh[0][2 * j + 1], kh[1][2 * j + 1], b.x, b.y);
      if (q_lo) tc::mma<M::BF>(sv, kh[0][2 * j], kh[1][2 * j], kh[0][2 * j + 1], kh[1][2 * j + 1], b.z, b.w);
      if constexpr (M::PLANES == 2)
        tc::mma<M::BF>(sv, kl[0][2 * j], kl[1][2 * j], kl[0][2 * j + 1], kl[1][2 * j + 1], b.x, b.y);
    }
    const int ta = tile * kMassTile + warp * 16 + g, tb = ta + 8;
    sv[0] = ok0 && ta <= p0 && ta > w0 ? sv[0] * a.score_scale : -CUDART_INF_F;
    sv[1] = ok0 && ta <= p1 && ta > w1 ? sv[1] * a.score_scale : -CUDART_INF_F;
    sv[2] = ok1 && tb <= p0 && tb > w0 ? sv[2] * a.score_scale : -CUDART_INF_F;
    sv[3] = ok1 && tb <= p1 && tb > w1 ? sv[3] * a.score_scale : -CUDART_INF_F;
    if (2 * c < a.row_pad) {
      if (ta < len) *reinterpret_cast<float2*>(sc_out + (int64_t)ta * a.row_pad + 2 * c) = make_float2(sv[0], sv[1]);
      if (tb < len) *reinterpret_cast<float2*>(sc_out + (int64_t)tb * a.row_pad + 2 * c) = make_float2(sv[2], sv[3]);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float mn = fmaxf(m[e], fmaxf(sv[e], sv[e + 2]));
      const float base = mn == -CUDART_INF_F ? 0.f : mn;   // all masked so far: (-inf, 0) stays
      l[e] = l[e] * t5::ex2(m[e] - base) + t5::ex2(sv[e] - base) + t5::ex2(sv[e + 2] - base);
      m[e] = mn;
    }
  }
  // join the lanes of a row (g), then the warps
#pragma unroll
  for (int e = 0; e < 2; ++e) {
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      const float mo = __shfl_xor_sync(0xffffffffu, m[e], d);
      const float lo = __shfl_xor_sync(0xffffffffu, l[e], d);
      const float mn = fmaxf(m[e], mo), base = mn == -CUDART_INF_F ? 0.f : mn;
      l[e] = l[e] * t5::ex2(m[e] - base) + lo * t5::ex2(mo - base);
      m[e] = mn;
    }
    if (g == 0) red_s[warp][2 * c + e] = make_float2(m[e], l[e]);
  }
  __syncthreads();
  if (tid < rows) {
    float mm = -CUDART_INF_F, ll = 0.f;
    for (int w = 0; w < kMassWarps; ++w) mm = fmaxf(mm, red_s[w][tid].x);
    const float base = mm == -CUDART_INF_F ? 0.f : mm;
    for (int w = 0; w < kMassWarps; ++w) ll += red_s[w][tid].y * t5::ex2(red_s[w][tid].x - base);
    a.stats[((sq.q0 + tid / a.rep) * a.nq + kvh * a.rep + tid % a.rep) * a.splits1 + blockIdx.y] = make_float2(mm, ll);
  }
}

template <int S, int HD>
cudaError_t launch_mass_rows(const MassArgs& a, const Codebooks& cb, cudaStream_t st) {
  constexpr int SMEM = (HD / 16) * 512;
  mass_rows_kernel<S, HD><<<dim3((unsigned)((int64_t)a.num_seqs * a.nkv), a.splits1), 32 * kMassWarps, SMEM, st>>>(a, cb);
  return cudaGetLastError();
}

cudaError_t launch_mass_raw(int k_side, int hd, const MassArgs& a, const Codebooks& cb, cudaStream_t st);
cudaError_t launch_mass_codes(int k_side, int hd, const MassArgs& a, const Codebooks& cb, cudaStream_t st);

}  // namespace kvq
