// Chunked-prefill attention on the 5th-generation tensor cores (tcgen05,
// accumulators in tensor memory), head_dim 64, 128 and 256.
//
// "combs_models/kv.rs" attend with the causal / window mask and repeat_kv,
// "spark_runtime/kv_cache.rs" is_wht_rotated bookends: query i of sequence
// s's chunk sits at p = L - C + i and attends to [max(0, p + 1 - W), p].
//
// One CTA (16 warps) per (tile of R score rows = QT query tokens x RP
// heads, kv head, sequence), R = 128 for head_dim 64/128 and R = 64 for
// head_dim 256 (whose planes would not fit a 128-row tile).  With R = 128
// score row r is tensor-memory lane r, held by threads r + 128 i, i = 0..3,
// each with a quarter of its columns; with R = 64 (M = 64 accumulators) row
// r sits in lane 32 floor(r / 16) + r mod 16, so the first 16 lanes of each
// warp hold rows.  Per step of T KV positions (T = 64, or 32 for head_dim
// 256; raw cache rows staged by cp.async two steps ahead):
//   one thread issues S[R x T] = Q . K^T (tcgen05.mma kind::f16, fp32 in
//   tensor memory; K dequantized during the previous step) and commits it
//   to an mbarrier;
//   meanwhile all threads dequantize V into the V [T x hd] operand plane
//   (16-bit hi + lo parts where one 16-bit value is not exact);
//   each thread reads its quarter score row (tcgen05.ld), masks it (only on
//   steps that cut a row's range); the quarters' maxima meet in shared
//   memory; it writes its quarter P row (hi + lo) to shared memory; the O
//   accumulator in tensor memory is rescaled only when a row's maximum grew
//   by more than 2^8 since the last rescale (P <= 2^8 otherwise: exact
//   enough in fp32 and in the 16-bit parts);
//   one thread issues O[R x hd] += P . V, and meanwhile all threads
//   dequantize the next step's K into the K [T x hd] plane.
// q (scaled by the score scale) and P carry hi + lo 16-bit parts like the
// decode.  Operands lie in 128-byte-swizzled planes (t5::sw); V, stored
// token by token as it comes, is the MN-major operand.
#pragma once

#include <math_constants.h>

#include "kvq_prefill.cuh"
#include "kvq_tc5_issue.cuh"

namespace kvq {

namespace t5 {

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
// Instruction descriptor of kind::f16: fp32 accumulator, A and B both bf16
// or both fp16, both K-major, M x N.
__host__ __device__ constexpr uint32_t idesc(bool bf, int M, int N) {
  return (1u << 4) | ((bf ? 1u : 0u) << 7) | ((bf ? 1u : 0u) << 10) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void commit(uint32_t mbar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(mbar)
               : "memory");
}
// Bounded wait for the completion of phase `parity` of an mbarrier.
__device__ __forceinline__ bool wait(uint32_t mbar, uint32_t parity) {
  for (int it = 0; it < (1 << 24); ++it) {
    uint32_t done;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        "selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(mbar), "r"(parity)
        : "memory");
    if (done) return true;
  }
  return false;
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
}
// Generic-proxy shared-memory writes made visible to the tensor cores.
__device__ __forceinline__ void fence_smem_async() {
  asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
}
__device__ __forceinline__ void ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, "
      "[%16];\n"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]),
        "=r"(v[15])
      : "r"(taddr));
}
__device__ __forceinline__ void ld8(uint32_t taddr, uint32_t (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
                 "=r"(v[7])
               : "r"(taddr));
}
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16};\n" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]));
}
// 2^x (PTX ex2.approx.ftz: relative error ~2^-22; 2^-inf = 0).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
// Maximum that keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// Operand planes: rows of 64 16-bit elements (128 bytes) with the 128-byte
// swizzle (16-byte chunk c of row r at c ^ (r mod 8)), 64-element blocks of R
// rows one after another.  The same plane is a K-major operand (rows x K) or
// an MN-major one (K x columns), so V needs no transpose.  Element offset
// (16-bit units) of (row r, column d):
template <int R>
__device__ __forceinline__ int sw(int r, int d) {
  return (d / 64) * (R * 64) + r * 64 + ((((d % 64) / 8) ^ (r & 7)) << 3) + d % 8;
}
// 16-byte steps of a K-major operand's k-step j (16 columns).
template <int R>
constexpr uint32_t kstep(int j) { return (uint32_t)((j / 4 * R * 128 + j % 4 * 32) / 16); }

}  // namespace t5

// Codebook sides (Turbo2/3/4, NVFP4): a table of the levels, entry c = hi(c) |
// lo(c) << 16 with the level split into two fp16 parts of 7 significant bits.
// A part times an E4M3 group scale (4 significant bits) is exact in fp16.
// Every entry has its own bank, so look-ups never conflict (a table of code
// pairs needs half of them, but they conflict: a step's Turbo4 K tile took
// 1600 cycles with it, 1050 so).
template <int S>
__device__ __forceinline__ void t5_fill_levels(uint32_t* lut, const Codebooks& cb, int tid) {
  if constexpr (side_codebook(S)) {
    if (tid < (1 << code_bits(S))) {
      const float c = side_levels<S>(cb)[tid], h = tc::round_sig7(c);
      lut[tid] = tc::pack2<false>(h, tc::round_sig7(c - h));
    }
  }
}

// Elements d0 .. d0 + 7 (d0 % 8 == 0, one scale group) of a staged codebook
// row as fp16x2 hi / lo pairs, scaled in fp16.
template <int S>
__device__ __forceinline__ void t5_dequant_codes(const uint8_t* row, const uint8_t* srow, int d0,
                                                 const uint32_t* lut, uint32_t (&hw)[4], uint32_t (&lw)[4]) {
  constexpr int B = code_bits(S);
  uint32_t w;
  if constexpr (B == 4) {
    w = *reinterpret_cast<const uint32_t*>(row + d0 / 2);
  } else if constexpr (B == 2) {
    w = *reinterpret_cast<const uint16_t*>(row + d0 / 4);
  } else {   // 3-bit codes: 24 bits from byte 3 d0 / 8
    const uint8_t* p = row + 3 * (d0 / 8);
    w = (uint32_t)p[0] | ((uint32_t)p[1] << 8) | ((uint32_t)p[2] << 16);
  }
  const uint32_t sb = srow[d0 / kGroup];
  const uint32_t sc2 = tc::e4m3x2_f16x2(sb | (sb << 8));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t e0 = lut[(w >> (2 * B * i)) & ((1u << B) - 1u)];
    const uint32_t e1 = lut[(w >> (2 * B * i + B)) & ((1u << B) - 1u)];
    hw[i] = tc::hmul2(tc::prmt(e0, e1, 0x5410u), sc2);
    lw[i] = PfSide<S>::PLANES == 2 ? tc::hmul2(tc::prmt(e0, e1, 0x7632u), sc2) : 0u;
  }
}

template <int KS, int VS, int HD, bool SH = false>
struct T5Cfg {
  static_assert(HD == 64 || HD == 128 || HD == 256, "tensor-memory prefill: head_dim 64, 128 or 256");
  // M of the accumulators (score rows per tile) and KV positions per step;
  // NSPLIT column parts per row (the four warps of a lane quadrant)
  static constexpr int NT = 512, ROWS = HD == 256 ? 64 : 128, TOK = HD == 256 ? 32 : 64, NSPLIT = 4;
  static constexpr int KPL = PfSide<KS>::PLANES, VPL = PfSide<VS>::PLANES;
  static constexpr int KROW = SideGeom<KS, HD>::ROW, KSROW = SideGeom<KS, HD>::SROW;
  static constexpr int VROW = SideGeom<VS, HD>::ROW, VSROW = SideGeom<VS, HD>::SROW;
  static constexpr int R_KS = align_up(TOK * KROW, 16);
  static constexpr int R_V = R_KS + align_up(TOK * KSROW, 16);
  static constexpr int R_VS = R_V + align_up(TOK * VROW, 16);
  static constexpr int RAW = R_VS + align_up(TOK * VSROW, 16);
  static constexpr int QB = ROWS * HD * 2, KB = TOK * HD * 2, VB = TOK * HD * 2;
  static constexpr int PB = ROWS * 128;               // (half of each row unused with TOK = 32)
  static constexpr int OFF_Q = 0;                     // q hi, q lo
  static constexpr int OFF_K = OFF_Q + 2 * QB;        // K planes [TOK x HD]
  static constexpr int OFF_V = OFF_K + KPL * KB;      // V planes [TOK x HD]
  static constexpr int OFF_P = OFF_V + VPL * VB;      // P hi, lo [ROWS x TOK]
  static constexpr int OFF_RAW = OFF_P + 2 * PB;      // raw rows, two buffers
  static constexpr int OFF_VROW = OFF_RAW + 2 * RAW;  // [2][TOK] row valid flags
  static constexpr int OFF_LV = OFF_VROW + 2 * TOK;   // level tables [2][2][16] fp32, [2][16] fp16 parts
  static constexpr int OFF_MX = OFF_LV + 384;  // [NSPLIT][ROWS] part-row maxima / sums
  static constexpr int OFF_BAR = OFF_MX + NSPLIT * ROWS * 4;  // 2 mbarriers, tensor-memory address
  // Block ids of the tile's first BLKC pages staged in shared memory at the
  // start (measured on GB300, 8 x 4096 with 512-token chunks: Turbo4 1359 ->
  // 1335 us, head_dim 256 BF16 / Turbo2 / Turbo8 4142 / 5958 / 5668 -> 4047 /
  // 5866 / 5628 us); BF16 and FP8 K at head_dim 64/128 load them at the
  // copies' issue (staged: 896 -> 903 and 893 -> 903 us).
  static constexpr int BLKC = (SH || HD == 256 || side_codebook(KS)) ? 1024 : 0;
  static_assert(BLKC % NT == 0, "block ids per thread");
  static constexpr int OFF_BLKC = OFF_BAR + 32;
  static constexpr int SMEM_MAIN = OFF_BLKC + BLKC * 4;
  static constexpr int OUTB = ROWS * (HD + 4) * 4;    // output staging (fp32), reuses the planes
  static constexpr int SMEM = SMEM_MAIN > OUTB ? SMEM_MAIN : OUTB;
  static constexpr int S_COL = 0, O_COL = TOK;         // tensor-memory columns of S and O
  static constexpr int TCOLS = TOK + HD <= 128 ? 128 : TOK + HD <= 256 ? 256 : 512;
};

// SH false: the chunked prefill.  SH true: partial attention over prefixes
// that groups of sequences share.  cu_q, block_tables and seq_lens then
// describe the groups (members cu_q[g] .. cu_q[g + 1] - 1, pages and length
// of the prefix); a tile's rows are QT members x RP heads, each member's one
// query attending the whole prefix (from its window's start, where one
// reaches into it).  Each tile's prefix is cut into ranges of `per` steps, the
// least that gives no more ranges than CTAs per kv head (grid x), found by
// bisection from the groups' sizes and lengths, so that one wave of CTAs
// carries about equal shares whatever the groups are; each row's
// unnormalised output, maximum and sum of a range go to the partials.
template <int KS, int VS, int HD, bool SH = false>
__global__ void __launch_bounds__(512, 1)
prefill_tc5_kernel(const PrefillArgs a, const Codebooks cb) {
  using C = T5Cfg<KS, VS, HD, SH>;
  using KP = PfSide<KS>;
  using VP = PfSide<VS>;
  constexpr int NT = C::NT, TOK = C::TOK;
  constexpr int E = HD / 32;
  extern __shared__ __align__(1024) uint8_t tma_smem[];   // (the name and alignment the TMA kernels declare)
  uint8_t* const smem = tma_smem;
  if (t5::smem_addr(smem) & 1023u) {   // the swizzle needs it; dynamic shared memory starts at 1 KB
    if (threadIdx.x == 0 && a.err) atomicOr(a.err, 4);
    return;
  }
  uint16_t* qh_s = reinterpret_cast<uint16_t*>(smem + C::OFF_Q);
  uint16_t* ql_s = reinterpret_cast<uint16_t*>(smem + C::OFF_Q + C::QB);
  uint16_t* k_s = reinterpret_cast<uint16_t*>(smem + C::OFF_K);   // plane p at + p * KB bytes
  uint16_t* v_s = reinterpret_cast<uint16_t*>(smem + C::OFF_V);   // plane p at + p * VB bytes
  uint16_t* ph_s = reinterpret_cast<uint16_t*>(smem + C::OFF_P);
  uint16_t* pl_s = reinterpret_cast<uint16_t*>(smem + C::OFF_P + C::PB);
  uint8_t* raw = smem + C::OFF_RAW;
  uint8_t* vrow_s = smem + C::OFF_VROW;
  float* lv = reinterpret_cast<float*>(smem + C::OFF_LV);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + 16);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int warp_u = __shfl_sync(0xffffffffu, warp, 0);   // (known to be the same in a warp)
  const int rp = a.rp, qt = C::ROWS / rp;
  const int kvh = blockIdx.y;
  int tile = blockIdx.x, seq = blockIdx.z;
  [[maybe_unused]] int split = 0, per = 1, used = 1;
  if constexpr (SH) {
    const int64_t cta = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    for (int64_t i = cta * NT + tid; i < a.sh.num_counters; i += (int64_t)gridDim.x * gridDim.y * NT)
      a.sh.counters[i] = 0;
    // Decreasing offsets have no groups (overlapping ones could need more
    // ranges than there are CTAs): the join then takes the own positions alone.
    bool dec = false, cut = false;
    for (int g = lane; g < a.sh.num_groups; g += 32) {
      const int m0 = a.cu_q[g], m1 = a.cu_q[g + 1];
      dec |= m1 < m0;
      cut |= m0 < 0 || m1 > a.num_seqs;
    }
    dec = __any_sync(0xffffffffu, dec);
    cut = __any_sync(0xffffffffu, cut);
    if (cta == 0 && tid == 0) {
      *a.sh.unordered = dec;
      if ((dec || cut) && a.err) atomicOr(a.err, 8);   // KVQ_DEVERR_RANGE
    }
    if (dec) return;
    const int64_t room = (int64_t)a.max_blocks * a.bs;
    auto group = [&](int g, int& tiles, int& steps) {   // tiles of its members, steps of its prefix
      const int m0 = max(a.cu_q[g], 0), m1 = min(a.cu_q[g + 1], a.num_seqs);
      tiles = m1 > m0 ? (m1 - m0 + qt - 1) / qt : 0;
      steps = (int)((min((int64_t)max(a.seq_lens[g], 0), room) + TOK - 1) / TOK);
    };
    int my_tiles = 0, my_steps = 0;
    if (lane < a.sh.num_groups) group(lane, my_tiles, my_steps);
    auto ranges = [&](int per) {   // of all groups (per warp)
      int n = my_tiles * ((my_steps + per - 1) / per);
      for (int g = lane + 32; g < a.sh.num_groups; g += 32) {
        int t, s;
        group(g, t, s);
        n += t * ((s + per - 1) / per);
      }
      return (int)__reduce_add_sync(0xffffffffu, n);
    };
    const int longest = (int)((room + TOK - 1) / TOK);
    int lo = (longest - 1) / a.sh.splits, hi = max(longest, 1);   // hi fits: no more tiles than CTAs
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (ranges(mid) <= (int)gridDim.x) hi = mid; else lo = mid;
    }
    per = hi;
    // the group whose ranges hold this CTA's, 32 groups per look
    for (int g0 = 0;; g0 += 32) {
      if (g0 >= a.sh.num_groups) return;
      int t = 0, s = 0;
      if (g0 + lane < a.sh.num_groups) group(g0 + lane, t, s);
      const int r = (s + per - 1) / per, n = t * r;
      int incl = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, incl > tile);
      if (past) {
        const int l = __ffs(past) - 1;
        seq = g0 + l;
        tile -= __shfl_sync(0xffffffffu, incl - n, l);
        used = __shfl_sync(0xffffffffu, r, l);
        split = tile % used;
        tile /= used;
        break;
      }
      tile -= __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  const int q0 = SH ? max(a.cu_q[seq], 0) : a.cu_q[seq];
  const int cq = (SH ? min(a.cu_q[seq + 1], a.num_seqs) : a.cu_q[seq + 1]) - q0;
  const int t0 = tile * qt;
  if (t0 >= cq) return;
  const int nq_tile = min(qt, cq - t0);
  int len = a.seq_lens[seq];
  const int64_t cap = (int64_t)a.max_blocks * a.bs;
  if (len > cap) {
    if (tid == 0 && tile == 0 && kvh == 0 && a.err) atomicOr(a.err, 2);
    len = (int)cap;
  }
  // a shared prefix is attended whole: the mask's upper end is its last position
  const int pbase = SH ? len - 1 : len - cq + t0;
  const int p_last = SH ? len - 1 : pbase + nq_tile - 1;
  [[maybe_unused]] int sh_lo_min = 0, sh_lo_max = 0;   // window starts of the tile's members
  if constexpr (SH) {
    if (a.window > 0) {
      sh_lo_min = 0x7fffffff;
      for (int i = 0; i < nq_tile; ++i) {
        const int64_t lo = (int64_t)len + max(a.sh.own_lens[q0 + t0 + i], 0) - a.window;
        const int l = (int)max((int64_t)0, min(lo, (int64_t)len));
        sh_lo_min = min(sh_lo_min, l);
        sh_lo_max = max(sh_lo_max, l);
      }
    }
  }
  const int lbs = 31 - __clz(a.bs);
  const int64_t tab = (int64_t)seq * a.max_blocks;
  // steps of the tile's attended positions, and the block ids of its first
  // BLKC pages, requested now (they are staged in shared memory after the
  // queries, before the first copies; -1 where the table holds no valid id)
  const int p_first = max(pbase, 0);
  const int lo_first = SH ? sh_lo_min : a.window > 0 ? max(0, p_first + 1 - a.window) : 0;
  int st_begin = lo_first / TOK;
  int st_end = p_last >= 0 ? p_last / TOK + 1 : st_begin;
  if constexpr (SH) {   // this CTA's range of the steps
    st_end = min(st_end, (split + 1) * per);
    st_begin = min(st_end, max(st_begin, split * per));
  }
  const int pg0 = (st_begin * TOK) >> lbs;
  const int npg = st_end > st_begin ? min(((st_end * TOK - 1) >> lbs) + 1 - pg0, C::BLKC) : 0;
  constexpr int BPT = C::BLKC / NT;
  int64_t bq[BPT > 0 ? BPT : 1];
#pragma unroll
  for (int k = 0; k < BPT; ++k) {
    const int i = tid + k * NT, pg = pg0 + i;
    bq[k] = (i < npg && pg < a.max_blocks) ? a.block_tables[tab + pg] : -1;
  }

  // ---- tensor memory and mbarriers
  const uint32_t bar_s = t5::smem_addr(bars), bar_o = t5::smem_addr(bars + 1);
  if (tid == 0) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;\n" ::"r"(bar_s));
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;\n" ::"r"(bar_o));
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(
                     t5::smem_addr(tslot)),
                 "r"(C::TCOLS));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  }

  // Shared prefixes, where products bound a step more than here: a BF16 q
  // that is not rotated needs no lo part.  It is the operand as it is, or,
  // where that is fp16 (FP8, NVFP4 keys) and the score scale far from one,
  // times a power of two (query_factor); the score scale's rest is taken after
  // the products.  In fp16 its 8 bits are exact from 2^-17 to 65504, below that
  // it is off by 2^-25 at most, as hi + lo parts are.
  [[maybe_unused]] bool q_exact = false;
  float q_mul = a.score_scale;
  if constexpr (SH) {
    q_exact = !side_rotated(KS) && a.q_bf16;
    if (q_exact) q_mul = a.sh.q_mul;
  }
  // ---- queries of the tile (rotated when K is), hi/lo planes in K's type
  for (int r = warp; r < C::ROWS; r += NT / 32) {
    const int qi = r / rp, hj = r - qi * rp;
    float x[E];
    if (qi < nq_tile && hj < a.rep) {
      const int64_t off = (int64_t)(q0 + t0 + qi) * a.q_stride + (int64_t)(kvh * a.rep + hj) * HD + lane * E;
#pragma unroll
      for (int i = 0; i < E; ++i)
        x[i] = a.q_bf16 ? bf16_bits_to_float(reinterpret_cast<const uint16_t*>(a.q)[off + i])
                        : reinterpret_cast<const float*>(a.q)[off + i];
      if constexpr (side_rotated(KS)) fwht_warp<E>(x, lane, a.inv_sqrt_hd);
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] *= q_mul;   // scores come out scaled (or are below)
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      uint32_t h, l;
      tc::split2<KP::BF>(x[i], x[i + 1], h, l);
      const int o_ = t5::sw<C::ROWS>(r, lane * E + i);
      *reinterpret_cast<uint32_t*>(qh_s + o_) = h;
      *reinterpret_cast<uint32_t*>(ql_s + o_) = l;
    }
  }
  pf_fill_levels<KS>(lv, lv + 16, cb, tid, NT);
  pf_fill_levels<VS>(lv + 32, lv + 48, cb, tid, NT);
  uint32_t* lut_k = reinterpret_cast<uint32_t*>(lv + 64);
  uint32_t* lut_v = lut_k + 16;
  t5_fill_levels<KS>(lut_k, cb, tid);
  t5_fill_levels<VS>(lut_v, cb, tid);

  // ---- raw rows of step st (positions TOK st .. TOK st + TOK - 1) into buffer b
  int* blkc = reinterpret_cast<int*>(smem + C::OFF_BLKC);
#pragma unroll
  for (int k = 0; k < BPT; ++k) {
    const int i = tid + k * NT;
    if (i < npg) blkc[i] = (bq[k] < 0 || bq[k] > 0x7fffffff) ? -1 : (int)bq[k];
  }
  // Block id of this thread's row of step st (-1: no row there).  With the
  // short steps of head_dim 256 it is read at the top of the step that
  // issues the copies.
  auto row_block = [&](int st) -> int64_t {
    const int pos = st * TOK + tid / (NT / TOK);
    if (st >= st_end || pos < 0 || pos >= len) return -1;
    const int i = (pos >> lbs) - pg0;
    if (C::BLKC > 0 && i < C::BLKC) return blkc[i];
    return a.block_tables[tab + (pos >> lbs)];
  };
  // Thread (row t = tid / PARTS, part = tid % PARTS) looks the row's block
  // up once and copies chunks part, part + PARTS, ... of its four rows:
  // consecutive threads write consecutive 16-byte chunks of one row.
  constexpr int PARTS = NT / TOK;
  auto copy_row = [&](uint8_t* dst, const uint8_t* src, const uint8_t* base, bool ok, int part,
                      auto rowbytes_c, auto chunk_c) {
    constexpr int RB = decltype(rowbytes_c)::value, CHB = decltype(chunk_c)::value;
    if constexpr (RB > 0) {
#pragma unroll
      for (int ch = part; ch < RB / CHB; ch += PARTS)
        cp_async<CHB>(dst + ch * CHB, (ok ? src : base) + ch * CHB, ok);
    }
  };
  auto issue = [&](int st, int b, int64_t blk) {
    uint8_t* rb = raw + b * C::RAW;
    using KG = SideGeom<KS, HD>;
    using VG = SideGeom<VS, HD>;
    const int t = tid / PARTS, part = tid % PARTS;
    const bool ok = blk >= 0 && (a.num_blocks <= 0 || blk < a.num_blocks);
    const int64_t rr = (int64_t)((st * TOK + t) & (a.bs - 1)) * a.nkv + kvh;
    if constexpr (SH) {   // (a first step may begin before the lowest window start, where pages may be gone)
      const int pos = st * TOK + t;
      if (!ok && pos >= lo_first && pos < len && part == 0 && a.err) atomicOr(a.err, 2);   // KVQ_DEVERR_BLOCK
    }
    if (!ok) blk = 0;
    const uint8_t* kb = a.k_cache + blk * a.k_bstride;
    const uint8_t* vb = a.v_cache + blk * a.v_bstride;
    copy_row(rb + t * KG::ROW, kb + rr * KG::ROW, a.k_cache, ok, part,
             std::integral_constant<int, KG::ROW>{}, std::integral_constant<int, KG::CH>{});
    copy_row(rb + C::R_KS + t * KG::SROW, kb + a.k_dsec + rr * KG::SROW, a.k_cache, ok, part,
             std::integral_constant<int, KG::SROW>{}, std::integral_constant<int, (KG::SCH > 0 ? KG::SCH : 1)>{});
    copy_row(rb + C::R_V + t * VG::ROW, vb + rr * VG::ROW, a.v_cache, ok, part,
             std::integral_constant<int, VG::ROW>{}, std::integral_constant<int, VG::CH>{});
    copy_row(rb + C::R_VS + t * VG::SROW, vb + a.v_dsec + rr * VG::SROW, a.v_cache, ok, part,
             std::integral_constant<int, VG::SROW>{}, std::integral_constant<int, (VG::SCH > 0 ? VG::SCH : 1)>{});
    if (part == 0) vrow_s[b * TOK + t] = ok ? 1 : 0;
  };

  t5::fence_before();
  __syncthreads();   // q planes, level tables, mbarrier init and the tensor-memory address visible
  t5::fence_after();
  const uint32_t tmem = *tslot;
  constexpr int NS = C::NSPLIT, SC = TOK / NS, OC = HD / NS;   // columns per thread of S, of O
  constexpr bool M64 = C::ROWS == 64;
  // score row and column part: lane 32 (warp & 3) + lane of tensor memory
  // holds row 32 (warp & 3) + lane (M = 128), or row 16 (warp & 3) + lane
  // for lanes 0-15 (M = 64; lanes 16-31 hold no row)
  const bool has_row = !M64 || lane < 16;
  const int row = M64 ? 16 * (warp & 3) + (lane & 15) : tid & (C::ROWS - 1);
  const int hf = warp >> 2;
  const uint32_t t_lane = (uint32_t)(32 * (warp & 3)) << 16;   // this warp's lanes (rows)
  const uint32_t s_tm = tmem + C::S_COL + hf * SC, o_tm = tmem + C::O_COL;
  float* mx_s = reinterpret_cast<float*>(smem + C::OFF_MX);    // [NS][ROWS]

  // per-row softmax state (both threads of a row keep the same m_used)
  const int qi_r = row / rp, hj_r = row - qi_r * rp;
  const bool row_ok = has_row && qi_r < nq_tile && hj_r < a.rep;
  const int p_r = SH ? pbase : pbase + qi_r;
  int lo_r = a.window > 0 ? p_r + 1 - a.window : 0;
  if constexpr (SH) {
    lo_r = 0;
    if (a.window > 0 && row_ok)
      lo_r = (int)max((int64_t)0, min((int64_t)len, (int64_t)len + max(a.sh.own_lens[q0 + t0 + qi_r], 0) - a.window));
  }
  float m_used = -CUDART_INF_F, l_sum = 0.f;
  bool ok_all = true;
  // positions every row of the tile attends: [all_lo, all_hi]
  const int all_hi = pbase;
  const int all_lo = SH ? sh_lo_max : a.window > 0 ? p_last + 1 - a.window : 0;

  // K of a staged step into the K plane: thread = 8 dims of a token.
  auto dequant_k = [&](int b) {
    const uint8_t* rb = raw + b * C::RAW;
    for (int q = tid; q < TOK * (HD / 8); q += NT) {
      const int t = q / (HD / 8), d0 = (q % (HD / 8)) * 8;
      uint32_t hw[4], lw[4];
      if constexpr (side_codebook(KS))
        t5_dequant_codes<KS>(rb + t * C::KROW, rb + C::R_KS + t * C::KSROW, d0, lut_k, hw, lw);
      else
        pf_dequant<KS, HD, 8>(rb + t * C::KROW, rb + C::R_KS + t * C::KSROW, d0, lv, lv + 16, hw, lw);
      const int o_ = t5::sw<TOK>(t, d0);
      *reinterpret_cast<uint4*>(k_s + o_) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
      if constexpr (C::KPL == 2)
        *reinterpret_cast<uint4*>(k_s + C::KB / 2 + o_) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
    }
  };
  // V of a staged step into the V plane: thread = 8 dims of a token.
  [[maybe_unused]] bool v_nonfinite = false;   // this thread wrote a NaN or infinite value
  auto dequant_v = [&](int b) {
    const uint8_t* rb = raw + b * C::RAW;
    for (int q = tid; q < TOK * (HD / 8); q += NT) {
      const int t = q / (HD / 8), d0 = (q % (HD / 8)) * 8;
      uint32_t hw[4], lw[4];
      if constexpr (side_codebook(VS))
        t5_dequant_codes<VS>(rb + C::R_V + t * C::VROW, rb + C::R_VS + t * C::VSROW, d0, lut_v, hw, lw);
      else
        pf_dequant<VS, HD, 8>(rb + C::R_V + t * C::VROW, rb + C::R_VS + t * C::VSROW, d0, lv + 32, lv + 48, hw, lw);
      if constexpr (SH) {
        constexpr uint32_t EX = VP::BF ? 0x7f80u : 0x7c00u;
#pragma unroll
        for (int i = 0; i < 4; ++i) v_nonfinite |= (hw[i] & EX) == EX || ((hw[i] >> 16) & EX) == EX;
      }
      const int o_ = t5::sw<TOK>(t, d0);
      *reinterpret_cast<uint4*>(v_s + o_) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
      if constexpr (C::VPL == 2)
        *reinterpret_cast<uint4*>(v_s + C::VB / 2 + o_) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
    }
  };

  // prologue: raw rows of the first two steps in flight, K of the first step
  if (st_begin < st_end) issue(st_begin, 0, row_block(st_begin));
  cp_async_commit();
  if (st_begin + 1 < st_end) issue(st_begin + 1, 1, row_block(st_begin + 1));
  cp_async_commit();
  cp_async_wait<1>();
  __syncthreads();
  if (st_begin < st_end) dequant_k(0);
  t5::fence_smem_async();

  for (int st = st_begin; st < st_end; ++st) {
    const int b = (st - st_begin) & 1;
    const uint32_t par = (uint32_t)((st - st_begin) & 1);
    __syncthreads();   // K of step st in its plane; raw rows of step st visible
    int64_t blk2 = -1;
    if constexpr (HD == 256) blk2 = row_block(st + 2);   // used by the copies issued at the end
    // ---- S = Q . K^T (q hi x K hi, q lo x K hi, q hi x K lo)
    if (warp_u == 0 && tc5::elect_one()) {
      t5::fence_after();
      constexpr uint32_t ID = t5::idesc(KP::BF, C::ROWS, TOK), HI = tc5::desc_hi(1024, true);
      const uint32_t qa = tc5::desc_lo(t5::smem_addr(qh_s), 16), qb = tc5::desc_lo(t5::smem_addr(ql_s), 16);
      const uint32_t ka = tc5::desc_lo(t5::smem_addr(k_s), 16), kb = tc5::desc_lo(t5::smem_addr(k_s) + C::KB, 16);
#pragma unroll
      for (int j = 0; j < HD / 16; ++j) {
        const uint32_t oq = t5::kstep<C::ROWS>(j), ok = t5::kstep<TOK>(j);
        tc5::mma_ss<HI>(tmem + C::S_COL, qa + oq, ka + ok, ID, j > 0);
        if (!SH || !q_exact) tc5::mma_ss<HI>(tmem + C::S_COL, qb + oq, ka + ok, ID, 1);
        if constexpr (C::KPL == 2) tc5::mma_ss<HI>(tmem + C::S_COL, qa + oq, kb + ok, ID, 1);
      }
      t5::commit(bar_s);
    }
    __syncwarp();
    // ---- meanwhile V of this step (its plane is free once O of the previous step is done)
    if (st > st_begin && !t5::wait(bar_o, par ^ 1u)) ok_all = false;
    dequant_v(b);
    t5::fence_smem_async();
    // A step that some member's window cuts: a weight of zero does not keep
    // a NaN or infinite value out of a product, so such a step (found while
    // its V plane is written) is added on the CUDA cores below.
    [[maybe_unused]] bool by_hand = false;
    if constexpr (SH) {
      if (st * TOK < sh_lo_max) by_hand = __syncthreads_or(v_nonfinite);
      v_nonfinite = false;
    }
    if (!t5::wait(bar_s, par)) ok_all = false;
    __syncwarp();   // each lane waited by itself; tensor-memory accesses are the whole warp's
    t5::fence_after();

    // ---- this part of the score row, masked only where the step cuts a range
    static_assert(SC == 16 || SC == 8, "one tensor-memory load per thread");
    float sv[SC];
    {
      uint32_t v0[SC];
      if constexpr (SC == 16) t5::ld16(s_tm + t_lane, v0);
      else t5::ld8(s_tm + t_lane, v0);
      t5::wait_ld();
#pragma unroll
      for (int j = 0; j < SC; ++j) sv[j] = __uint_as_float(v0[j]);
      if constexpr (SH) {
        if (q_exact) {
#pragma unroll
          for (int j = 0; j < SC; ++j) sv[j] *= a.sh.s_mul;
        }
      }
    }
    const int tbase = st * TOK + hf * SC;
    const uint32_t* vr4 = reinterpret_cast<const uint32_t*>(vrow_s + b * TOK + hf * SC);
    uint32_t vand = 0x01010101u;
#pragma unroll
    for (int w4 = 0; w4 < SC / 4; ++w4) vand &= vr4[w4];
    // (rows of no query count as full: nothing of them is stored, and masking
    // them cost their warps 850 cycles a step)
    const bool full = st * TOK >= all_lo && st * TOK + TOK - 1 <= all_hi && vand == 0x01010101u;
    float mx = -CUDART_INF_F;
    if (full) {
#pragma unroll
      for (int j = 0; j < SC; ++j) mx = SH ? t5::max_nan(mx, sv[j]) : fmaxf(mx, sv[j]);
    } else {
      const uint8_t* vr = vrow_s + b * TOK + hf * SC;
#pragma unroll
      for (int j = 0; j < SC; ++j) {
        const int t = tbase + j;
        const bool ok = row_ok && t <= p_r && t >= lo_r && vr[j];
        sv[j] = ok ? sv[j] : -CUDART_INF_F;
        mx = SH ? t5::max_nan(mx, sv[j]) : fmaxf(mx, sv[j]);
      }
    }
    if (has_row) mx_s[hf * C::ROWS + row] = mx;
    if (!__syncthreads_and(ok_all)) break;   // maxima and the V plane visible
#pragma unroll
    for (int i = 0; i < NS; ++i)
      mx = SH ? t5::max_nan(mx, mx_s[i * C::ROWS + row]) : fmaxf(mx, mx_s[i * C::ROWS + row]);
    // fp16 weights of a shared prefix are held 2^7 above their size (at most
    // 2^15, where a row's maximum has grown by 2^8): those of 2^-21 beside the
    // maximum stay normal numbers and none above 2^-32 is lost, which a long
    // prefix beside one large weight would add up (l_sum counts them all).
    // (hi + lo parts for 16-bit outputs too: the hi part alone is off by 2^-11
    // of a weight, which turns the rounding of some outputs, for 3% of the time.)
    constexpr float UP = SH && !VP::BF ? 7.f : 0.f;
    float alpha = 1.f;
    bool resc = false;
    if (mx != -CUDART_INF_F) {
      if (m_used == -CUDART_INF_F) {
        m_used = mx - UP;
      } else if (mx > m_used + (8.f + UP)) {
        alpha = t5::ex2(m_used - (mx - UP));
        resc = true;
        l_sum *= alpha;
        m_used = mx - UP;
      }
    }
    const bool live = m_used != -CUDART_INF_F;   // else every score so far is masked: P = 0
#pragma unroll
    for (int c8 = 0; c8 < SC; c8 += 8) {
      uint32_t h[4], l[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x0 = live ? t5::ex2(sv[c8 + 2 * i] - m_used) : 0.f;
        const float x1 = live ? t5::ex2(sv[c8 + 2 * i + 1] - m_used) : 0.f;
        l_sum += x0 + x1;
        tc::split2<VP::BF>(x0, x1, h[i], l[i]);
      }
      const int o_ = t5::sw<C::ROWS>(row, hf * SC + c8);
      if (has_row) {
        *reinterpret_cast<uint4*>(ph_s + o_) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(pl_s + o_) = make_uint4(l[0], l[1], l[2], l[3]);
      }
    }
    // rescale this part of the O rows whose maximum grew (warp-collective accesses)
    if (st > st_begin && __any_sync(0xffffffffu, resc)) {
#pragma unroll 1
      for (int c0 = hf * OC; c0 < (hf + 1) * OC; c0 += 16) {
        uint32_t v[16];
        t5::ld16(o_tm + t_lane + c0, v);
        t5::wait_ld();
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * alpha);
        t5::st16(o_tm + t_lane + c0, v);
      }
      t5::wait_st();
    }
    cp_async_wait<0>();   // the next step's raw rows (issued at the end of the previous step)
    t5::fence_smem_async();
    t5::fence_before();
    __syncthreads();   // P plane and the next step's raw rows visible

    if constexpr (SH) {
      if (by_hand) {   // O += P . V over the attended positions only
#pragma unroll 1
        for (int c0 = hf * OC; c0 < (hf + 1) * OC; c0 += 16) {
          uint32_t v[16];
          if (st > st_begin) {
            t5::ld16(o_tm + t_lane + c0, v);
            t5::wait_ld();
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = 0u;
          }
#pragma unroll 1
          for (int t = 0; t < TOK; ++t) {   // (no branch of a lane's own: tensor-memory accesses are the whole warp's)
            const int pos = st * TOK + t;
            const bool in = row_ok && pos <= p_r && pos >= lo_r && vrow_s[b * TOK + t];
            if (!__any_sync(0xffffffffu, in)) continue;   // (warp-uniform)
            const int o_ = t5::sw<C::ROWS>(row, t);
            const float p = tc::unpack2<VP::BF>(ph_s[o_]).x + tc::unpack2<VP::BF>(pl_s[o_]).x;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int ov = t5::sw<TOK>(t, c0 + j);
              float y = tc::unpack2<VP::BF>(v_s[ov]).x;
              if constexpr (C::VPL == 2) y += tc::unpack2<VP::BF>(v_s[C::VB / 2 + ov]).x;
              const float z = fmaf(p, y, __uint_as_float(v[j]));
              v[j] = in ? __float_as_uint(z) : v[j];
            }
          }
          t5::st16(o_tm + t_lane + c0, v);
        }
        t5::wait_st();
        t5::fence_before();
        __syncthreads();
      }
    }

    // ---- O += P . V (P hi x V hi, P lo x V hi, P hi x V lo)
    if (warp_u == 0 && tc5::elect_one()) {
      t5::fence_after();
      // V as the MN-major operand: 64-dim blocks TOK rows apart (the leading
      // offset), 16 tokens a k-step
      constexpr uint32_t ID = t5::idesc(VP::BF, C::ROWS, HD) | (1u << 16), HI = tc5::desc_hi(1024, true);
      const uint32_t pa = tc5::desc_lo(t5::smem_addr(ph_s), 16), pb = tc5::desc_lo(t5::smem_addr(pl_s), 16);
      const uint32_t va = tc5::desc_lo(t5::smem_addr(v_s), TOK * 128), vb = tc5::desc_lo(t5::smem_addr(v_s) + C::VB, TOK * 128);
      bool products = true;
      if constexpr (SH) products = !by_hand;
      if (products) {
#pragma unroll
        for (int j = 0; j < TOK / 16; ++j) {
          const uint32_t op = t5::kstep<C::ROWS>(j), ov = (uint32_t)(j * 2048 / 16);
          tc5::mma_ss<HI>(o_tm, pa + op, va + ov, ID, (st > st_begin || j > 0) ? 1u : 0u);
          tc5::mma_ss<HI>(o_tm, pb + op, va + ov, ID, 1);
          if constexpr (C::VPL == 2) tc5::mma_ss<HI>(o_tm, pa + op, vb + ov, ID, 1);
        }
      }
      t5::commit(bar_o);
    }
    __syncwarp();
    // ---- meanwhile K of the next step (the K plane is free: S of this step is done)
    if (st + 1 < st_end) dequant_k(b ^ 1);
    t5::fence_smem_async();
    // raw rows two steps ahead into this step's buffer (its K and V are in
    // their planes), issued after this step's last proxy fence: a proxy fence
    // also waits for the copies in flight (measured on GB300)
    if (st + 2 < st_end) issue(st + 2, b, HD == 256 ? blk2 : row_block(st + 2));
    cp_async_commit();
  }
  cp_async_wait<0>();
  if (st_end > st_begin && ok_all) {
    if (!t5::wait(bar_o, (uint32_t)((st_end - 1 - st_begin) & 1))) ok_all = false;
  }
  if (!ok_all && tid == 0 && a.err) atomicOr(a.err, 4);
  t5::fence_after();
  if (has_row) mx_s[hf * C::ROWS + row] = l_sum;
  __syncthreads();   // every plane read is done: the output staging reuses them
  l_sum = 0.f;
#pragma unroll
  for (int i = 0; i < NS; ++i) l_sum += mx_s[i * C::ROWS + row];

  // ---- normalise row `row` (this thread's part) from tensor memory, stage,
  // rotate back, store
  float* os = reinterpret_cast<float*>(smem);   // [ROWS][HD + 4]
  {
    const float inv = SH ? a.v_mult : l_sum > 0.f ? a.v_mult / l_sum : 0.f;
    const bool have_o = st_end > st_begin && ok_all;
#pragma unroll 1
    for (int c0 = hf * OC; c0 < (hf + 1) * OC; c0 += 16) {
      uint32_t v[16];
      if (have_o) {
        t5::ld16(o_tm + t_lane + c0, v);
        t5::wait_ld();
      }
      if (has_row) {
#pragma unroll
        for (int j = 0; j < 16; ++j) os[row * (HD + 4) + c0 + j] = have_o ? __uint_as_float(v[j]) * inv : 0.f;
      }
      __syncwarp();   // the next load is the whole warp's
    }
  }
  if constexpr (SH) {
    if (row_ok && hf == 0) {
      const int64_t r_ = (int64_t)(q0 + t0 + qi_r) * a.nq + kvh * a.rep + hj_r;
      a.sh.ml[r_ * a.sh.splits + split] = make_float2(ok_all ? m_used : -CUDART_INF_F, ok_all ? l_sum : 0.f);
      if (split == 0)   // ranges this group has not
        for (int i = used; i < a.sh.splits; ++i) a.sh.ml[r_ * a.sh.splits + i] = make_float2(-CUDART_INF_F, 0.f);
    }
  }
  t5::fence_before();
  __syncthreads();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(C::TCOLS));
  for (int r = warp; r < C::ROWS; r += NT / 32) {
    const int qi = r / rp, hj = r - qi * rp;
    if (qi >= nq_tile || hj >= a.rep) continue;   // warp-uniform
    float x[E];
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = os[r * (HD + 4) + lane * E + i];
    if constexpr (side_rotated(VS)) fwht_warp<E>(x, lane, a.inv_sqrt_hd);
    if constexpr (SH) {
      float* po = a.sh.part + (((int64_t)(q0 + t0 + qi) * a.nq + kvh * a.rep + hj) * a.sh.splits + split) * HD + lane * E;
#pragma unroll
      for (int i = 0; i < E; ++i) po[i] = x[i];
      continue;
    }
    const int64_t o_ = ((int64_t)(q0 + t0 + qi) * a.nq + kvh * a.rep + hj) * HD + lane * E;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      if (a.out_bf16) reinterpret_cast<uint16_t*>(a.out)[o_ + i] = bf16_bits_from_float(x[i]);
      else reinterpret_cast<float*>(a.out)[o_ + i] = x[i];
    }
  }
}

template <int KS, int VS, int HD>
cudaError_t launch_prefill_tc5(const PrefillArgs& a, const Codebooks& cb, int max_chunk, cudaStream_t st) {
  using C = T5Cfg<KS, VS, HD>;
  static_assert(C::SMEM <= 227 * 1024, "shared memory budget");
  auto kern = prefill_tc5_kernel<KS, VS, HD>;
  if (C::SMEM > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
  }
  const int qt = C::ROWS / a.rp;
  dim3 grid((max_chunk + qt - 1) / qt, a.nkv, a.num_seqs);
  kern<<<grid, C::NT, C::SMEM, st>>>(a, cb);
  return cudaGetLastError();
}

template <int KS, int VS, int HD>
cudaError_t launch_shared_tc5(const PrefillArgs& a, const Codebooks& cb, int slots, cudaStream_t st) {
  using C = T5Cfg<KS, VS, HD, true>;
  static_assert(C::SMEM <= 227 * 1024, "shared memory budget");
  auto kern = prefill_tc5_kernel<KS, VS, HD, true>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  kern<<<dim3((unsigned)slots, a.nkv), C::NT, C::SMEM, st>>>(a, cb);
  return cudaGetLastError();
}

template <int KS, int VS>
cudaError_t launch_shared_pair(int hd, const PrefillArgs& a, const Codebooks& cb, int slots, cudaStream_t st) {
  switch (hd) {
    case 64: return launch_shared_tc5<KS, VS, 64>(a, cb, slots, st);
    case 128: return launch_shared_tc5<KS, VS, 128>(a, cb, slots, st);
    case 256: return launch_shared_tc5<KS, VS, 256>(a, cb, slots, st);
    default: return cudaErrorInvalidValue;
  }
}

template <int KS, int VS>
cudaError_t launch_prefill_pair(int hd, const PrefillArgs& a, const Codebooks& cb, int max_chunk,
                                cudaStream_t st) {
  switch (hd) {
    case 64: return launch_prefill_tc5<KS, VS, 64>(a, cb, max_chunk, st);
    case 128: return launch_prefill_tc5<KS, VS, 128>(a, cb, max_chunk, st);
    case 256: return launch_prefill_tc5<KS, VS, 256>(a, cb, max_chunk, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvq
