// Attention mass of many score rows (a chunk's queries x the heads of a kv
// head) on the 5th-generation tensor cores.
//
// Two passes over K, statistics and then sums, with a CTA of 16 warps (and one
// that issues the products) per range of positions of one (sequence, kv
// head).  Each lane of a 128-lane accumulator wants its reduction along
// columns, so the passes transpose each other:
//   pass 1: S[128 rows x TP positions] = Q K^T, lane = row: a thread keeps its
//     row's running maximum and sum over its quarter of the columns;
//   pass 2: S^T[128 positions x QR rows] = K Q^T, lane = position: a thread
//     adds 2^(s - lse) over its quarter of the rows.
// Both operands are K-major planes in shared memory (128-byte swizzle), so one
// set of planes serves as A in one pass and as B in the other.  K rows come
// from the pages into registers a tile ahead, become hi + lo fp16 parts
// (22 bits) in the planes, and while the products of a tile run the threads
// work on the tile before (two accumulators in tensor memory).
// Measured on GB300: 32 queries x 4 heads over 35k Turbo4 positions of 8 kv
// heads 92 us (504 us with mma.sync); a tile's dequantization (about 1300
// cycles) and its 24 products (1550) alternate, which bounds it.
#pragma once

#include "kvq_decode_tma.cuh"
#include "kvq_mass.cuh"
#include "kvq_tc5_issue.cuh"

namespace kvq {

template <int S, int HD, int PASS>
struct MtCfg {
  static constexpr int QR = PASS == 2 && HD == 256 ? 64 : 128;    // score rows per block
  static constexpr int TP = PASS == 1 && HD == 256 ? 64 : 128;    // positions per tile
  static constexpr int KPL = PfSide<S>::PLANES;
  static constexpr int QB = QR * HD * 2, KB = TP * HD * 2;        // a plane: 64-dim blocks of 128-byte rows
  static constexpr int OFF_K = 2 * QB;
  static constexpr int OFF_LV = OFF_K + KPL * KB;                 // level table
  static constexpr int OFF_X = OFF_LV + 64;                       // joins of the quarters
  static constexpr int OFF_L = OFF_X + 2 * 4 * 128 * 4;           // [QR] lse (pass 2)
  static constexpr int OFF_OK = OFF_L + 128 * 4;                  // [3][TP] position valid
  static constexpr int OFF_BAR = OFF_OK + 3 * 128;
  static constexpr int SMEM = OFF_BAR + 32;
  static constexpr int LPR = 512 / TP;                            // threads per K row
  static constexpr int D = HD / LPR, HP = 4 * D;                  // dims per thread; a row of HP dims has 4 such parts
  static constexpr int COLS = PASS == 1 ? TP : QR;
  static constexpr int NC = COLS / 4;                             // columns per thread
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
};

// Byte of (row r, dim d) in a plane of R rows: 128-byte swizzle, 64-dim
// blocks one after another.
template <int R>
__device__ __forceinline__ int sw(int r, int d) {
  return (d / 64) * (R * 128) + r * 128 + ((((d % 64) / 8) ^ (r & 7)) << 4) + (d % 8) * 2;
}

template <int S, int HD, int PASS>
__global__ void __launch_bounds__(544, 1) mass_tc_kernel(const MassArgs a, const Codebooks cb) {
  using C = MtCfg<S, HD, PASS>;
  constexpr bool BF = S == S_BF16;
  constexpr int E = HD / 32, NC = C::NC, TP = C::TP, QR = C::QR;
  extern __shared__ __align__(1024) uint8_t tma_smem[];   // (its own name: other kernels declare 128-byte alignment)
  uint8_t* const smem = tma_smem;
  const uint32_t sb = t5::smem_addr(smem);
  if (sb & 1023u) {   // the swizzle needs it; dynamic shared memory starts at 1 KB
    if (threadIdx.x == 0 && a.err) atomicOr(a.err, KVQ_DEVERR_TIMEOUT);
    return;
  }
  float* lv = reinterpret_cast<float*>(smem + C::OFF_LV);
  float* xs = reinterpret_cast<float*>(smem + C::OFF_X);
  float* lse_s = reinterpret_cast<float*>(smem + C::OFF_L);
  uint8_t* ok_s = smem + C::OFF_OK;
  const uint32_t bar = sb + C::OFF_BAR;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + 8);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

  // ---- this CTA's share: the sequences' 128-position units are cut into
  // ranges of `per`, the least that gives no more ranges than CTAs (found by
  // bisection; every CTA of both passes finds the same)
  auto unit_count = [&](int s) {
    return (int)((min((int64_t)max(a.seq_lens[s], 0), (int64_t)a.max_blocks * a.bs) + 127) / 128);
  };
  const int my_units = lane < a.num_seqs ? unit_count(lane) : 0;
  auto ranges_before = [&](int per, int upto) {   // ranges of the sequences before `upto`, of one kv head (per warp)
    int n = lane < upto ? (my_units + per - 1) / per : 0;
    for (int s = lane + 32; s < upto; s += 32) n += (unit_count(s) + per - 1) / per;
    return (int)__reduce_add_sync(0xffffffffu, n);
  };
  if (PASS == 1 && blockIdx.x == 0 && blockIdx.z == 0)
    for (int s = tid; s < a.num_seqs; s += 544) mass_seq(a, s, true);   // flags
  int per = 1, range = 0;
  int64_t seq = -1;
  const int kvh = (int)(blockIdx.x % a.nkv), slot0 = (int)(blockIdx.x / a.nkv), slots = (int)(gridDim.x / a.nkv);
  {
    int lo = 0, hi = (int)(((int64_t)a.max_blocks * a.bs + 127) / 128);   // hi always fits: slots >= num_seqs
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (ranges_before(mid, a.num_seqs) <= slots) hi = mid; else lo = mid;
    }
    per = hi;
    // the sequence that holds range `slot0`: bisection over the prefix counts
    if (ranges_before(per, a.num_seqs) <= slot0) return;
    int s0 = 0, s1 = a.num_seqs;   // ranges before s0 <= slot0 < ranges before s1
    while (s1 - s0 > 1) {
      const int mid = (s0 + s1) / 2;
      if (ranges_before(per, mid) <= slot0) s0 = mid; else s1 = mid;
    }
    seq = s0;
    range = slot0 - ranges_before(per, s0);
  }
  const MassSeq sq = mass_seq(a, seq, false);
  const int len = sq.len, pbase = sq.pbase, rows_all = sq.rows, lo_all = sq.lo;
  const int last = pbase + rows_all / a.rep - 1;   // position of the last query
  const int64_t q0 = sq.q0;
  const int nblk = (rows_all + QR - 1) / QR;
  const int units = (len + 127) / 128, used1 = (units + per - 1) / per;
  const int u0 = min(units, range * per), u1 = min(units, u0 + per);
  if (PASS == 1 && (int)blockIdx.z >= nblk) return;
  const int tile1 = min(u1 * (128 / TP), (len + TP - 1) / TP);
  const int tile0 = PASS == 1 ? min(tile1, max(u0 * (128 / TP), lo_all / TP)) : u0 * (128 / TP);
  if (PASS == 1 && tile0 >= tile1) {   // no window reaches this range
    const int r = blockIdx.z * QR + tid;
    if (tid < QR && r < rows_all)
      a.stats[((q0 + r / a.rep) * a.nq + kvh * a.rep + r % a.rep) * a.splits1 + range] = make_float2(-CUDART_INF_F, 0.f);
    return;
  }

  if (tid == 0) {
    tm::bar_init(bar);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 256;\n" ::"r"(t5::smem_addr(tslot)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  }
  mass_fill_levels<S>(lv, cb, tid);
  t5::fence_before();
  __syncthreads();
  t5::fence_after();
  const uint32_t tmem = *tslot;
  const bool q_lo = side_rotated(S) || !a.q_bf16;
  // (the sign goes into the queries: scores then scale by a positive factor)
  const float scale = fabsf(a.score_scale), q_mul = a.score_scale < 0.f ? -a.q_mul : a.q_mul;

  auto load_q = [&](int blk) {   // score rows blk * QR .. into the q planes, 4 rows of a warp at a time
#pragma unroll 1
    for (int r0 = warp; r0 < QR; r0 += 64) {
      float x[4][E];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int rr = blk * QR + r0 + 16 * u;
        const bool ok = r0 + 16 * u < QR && rr < rows_all;
        const int64_t off = ok ? (q0 + rr / a.rep) * a.q_stride + (int64_t)(kvh * a.rep + rr % a.rep) * HD + lane * E : 0;
        if (a.q_vec && a.q_bf16) {
          uint32_t w[E / 2];
          load_bytes<2 * E>(reinterpret_cast<const uint8_t*>(a.q) + 2 * off, w);
#pragma unroll
          for (int i = 0; i < E; ++i)
            x[u][i] = ok ? bf16_bits_to_float((w[i / 2] >> (16 * (i & 1))) & 0xffffu) : 0.f;
        } else {
#pragma unroll
          for (int i = 0; i < E; ++i)
            x[u][i] = !ok ? 0.f : a.q_bf16 ? bf16_bits_to_float(reinterpret_cast<const uint16_t*>(a.q)[off + i])
                                           : reinterpret_cast<const float*>(a.q)[off + i];
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int r = r0 + 16 * u;
        if (r >= QR) break;
        if constexpr (side_rotated(S)) fwht_warp<E>(x[u], lane, a.inv_sqrt_hd);
#pragma unroll
        for (int i = 0; i < E; i += 2) {
          uint32_t h, l;
          tc::split2<BF>(x[u][i] * q_mul, x[u][i + 1] * q_mul, h, l);
          const int o = sw<QR>(r, lane * E + i);
          *reinterpret_cast<uint32_t*>(smem + o) = h;
          *reinterpret_cast<uint32_t*>(smem + C::QB + o) = l;
        }
      }
    }
  };

  // ---- K rows of a tile: LPR threads per position, each D dims (one wide
  // load and one table look-up a tile); block ids a tile ahead of the rows
  constexpr int LPR = C::LPR, D = C::D, HP = C::HP;
  const int pc = (tid & 511) % LPR, pt = (tid & 511) / LPR;
  const int rowb = HD * side_bits(S) / 8, srowb = HD / kGroup * side_scale_bytes(S);
  // (BF16: a part's 8-dim runs alternate within 128 dims)
  const int part = S == S_BF16 ? pc % 4 : pc, blk128 = S == S_BF16 ? pc / 4 : 0;
  const uint8_t* kbase = a.k_cache + (int64_t)kvh * rowb + blk128 * 256;
  const uint8_t* sbase = a.k_cache + a.k_dsec + (int64_t)kvh * srowb;
  const int32_t* tab = a.block_tables + seq * a.max_blocks;
  int32_t bid = -2;
  MassRaw<S, HP> raw;
  bool rok = false;
  auto ids = [&](int tile) {
    const int t = tile * TP + pt;
    bid = tile < tile1 && t < len && t >= lo_all ? tab[t >> a.lbs] : -2;
  };
  auto fetch = [&](int tile) {
    const int t = tile * TP + pt;
    rok = bid >= 0 && (a.num_blocks <= 0 || bid < a.num_blocks);
    if (PASS == 1 && !rok && bid != -2 && pc == 0 && a.err) atomicOr(a.err, KVQ_DEVERR_BLOCK);
    if (rok) {
      const int64_t page = bid * a.k_bstride;
      const int rr = (t & (a.bs - 1)) * a.nkv;   // (a page stays below 2^31 bytes a section)
      mass_load<S, HP>(raw, kbase + page + (int64_t)rr * rowb, sbase + page + (int64_t)rr * srowb, part);
    } else {
#pragma unroll
      for (int i = 0; i < (int)(sizeof(raw.w) / 4); ++i) raw.w[i] = 0u;
#pragma unroll
      for (int i = 0; i < (int)(sizeof(raw.s) / 4); ++i) raw.s[i] = 0u;
    }
  };
  bool ok_run = true;
  uint32_t phase = 0;
  const uint32_t d_row = (uint32_t)(32 * (warp & 3)) << 16;
  const int ln = tid & 127, hf = (tid >> 7) & 3;   // accumulator lane, column quarter
  const bool worker = warp < 16;                    // the 17th warp issues the products

  for (int blk = PASS == 1 ? blockIdx.z : 0; blk < (PASS == 1 ? (int)blockIdx.z + 1 : max(nblk, 1)) && ok_run; ++blk) {
    if (worker) load_q(blk);
    if constexpr (PASS == 2) {
      constexpr int TPR = 512 / QR;   // threads that join a row's ranges
      const int r = (tid & 511) / TPR, rr = blk * QR + r;
      float mm = -CUDART_INF_F, ll = 0.f;
      if (worker && rr < rows_all) {
        const float2* st = a.stats + ((q0 + rr / a.rep) * a.nq + kvh * a.rep + rr % a.rep) * a.splits1;
#pragma unroll 4
        for (int i = tid % TPR; i < used1; i += TPR) {
          const float2 x = st[i];
          const float mn = fmaxf(mm, x.x), base = mn == -CUDART_INF_F ? 0.f : mn;
          ll = ll * t5::ex2((mm - base) * scale) + x.y * t5::ex2((x.x - base) * scale);
          mm = mn;
        }
      }
#pragma unroll
      for (int d = 1; d < TPR; d <<= 1) {
        const float mo = __shfl_xor_sync(0xffffffffu, mm, d), lo = __shfl_xor_sync(0xffffffffu, ll, d);
        const float mn = fmaxf(mm, mo), base = mn == -CUDART_INF_F ? 0.f : mn;
        ll = ll * t5::ex2((mm - base) * scale) + lo * t5::ex2((mo - base) * scale);
        mm = mn;
      }
      if (worker && tid % TPR == 0)
        lse_s[r] = mm == -CUDART_INF_F && !(ll != ll) ? -CUDART_INF_F : -fmaf(mm, scale, log2f(ll));
    }
    const int rows_blk = min(QR, rows_all - blk * QR);
    const int row = blk * QR + ln;                             // pass 1: this lane's score row
    const int p_row = pbase + row / a.rep;
    float m = -CUDART_INF_F, l = 0.f;
    bool full_prev = false;

    // one tile's scores: pass 1 into (m, l); pass 2 into the totals
    // (validity flags in three slots: a fast thread writes the next tile's
    // while a slow one still reads the last's)
    auto consume = [&](int tile, int buf, bool valid) {
      const uint32_t src = tmem + d_row + buf * 128 + hf * NC;
      const int t0 = tile * TP, t1 = t0 + TP - 1;
      const bool full = valid && t0 >= lo_all && t1 < len && t1 <= pbase &&
                        (a.window <= 0 || t0 > last - a.window);
      const uint8_t* okb = ok_s + (tile - tile0) % 3 * 128;
      uint32_t s[NC];
      __syncwarp();   // (lanes fetched and stored different rows; the load is the whole warp's)
#pragma unroll
      for (int c = 0; c < NC; c += 16) t5::ld16(src + c, *reinterpret_cast<uint32_t(*)[16]>(s + c));
      t5::wait_ld();
      const uint64_t sc2 = f2::pack(scale, scale);
      if constexpr (PASS == 1) {
        if (!full) {
#pragma unroll
          for (int e = 0; e < NC; ++e) {
            const int t = t0 + hf * NC + e;
            if (!(okb[hf * NC + e] && t <= p_row && (a.window <= 0 || t > p_row - a.window))) s[e] = 0xff800000u;
          }
        }
        // (m in units of the raw scores)
        float x0 = m, x1 = m;
#pragma unroll
        for (int e = 0; e < NC; e += 4) {
          x0 = f2::max3(x0, __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
          x1 = f2::max3(x1, __uint_as_float(s[e + 2]), __uint_as_float(s[e + 3]));
        }
        const float mx = fmaxf(x0, x1), neg = mx == -CUDART_INF_F ? 0.f : -mx * scale;
        const uint64_t neg2 = f2::pack(neg, neg);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < NC; e += 2) {
          const float2 x = f2::unpack(f2::fma(f2::pack(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), sc2, neg2));
          sum[(e >> 1) & 1] = f2::add(sum[(e >> 1) & 1], f2::pack(t5::ex2(x.x), t5::ex2(x.y)));
        }
        const float2 y = f2::unpack(f2::add(sum[0], sum[1]));
        l = l * t5::ex2(fmaf(m, scale, neg)) + (y.x + y.y);
        m = mx;
      } else {   // lse_s holds -lse; -inf for a row that attends to nothing
        const int t = t0 + ln;
        uint64_t acc[2] = {0, 0};
        if (full && rows_blk == QR) {
#pragma unroll
          for (int e = 0; e < NC; e += 4) {
            const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(lse_s + hf * NC + e);
            const float2 x0 = f2::unpack(f2::fma(f2::pack(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), sc2, y.x));
            const float2 x1 = f2::unpack(f2::fma(f2::pack(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3])), sc2, y.y));
            acc[0] = f2::add(acc[0], f2::pack(t5::ex2(x0.x), t5::ex2(x0.y)));
            acc[1] = f2::add(acc[1], f2::pack(t5::ex2(x1.x), t5::ex2(x1.y)));
          }
        } else {
          const bool ok = okb[ln];
          float part = 0.f;
#pragma unroll
          for (int e = 0; e < NC; ++e) {
            const int r = hf * NC + e, p = pbase + (blk * QR + r) / a.rep;
            const float y = lse_s[r];
            const bool in = ok && r < rows_blk && t <= p && (a.window <= 0 || t > p - a.window) && y != -CUDART_INF_F;
            part += in ? t5::ex2(fmaf(__uint_as_float(s[e]), scale, y)) : 0.f;
          }
          acc[0] = f2::pack(part, 0.f);
        }
        const float2 y = f2::unpack(f2::add(acc[0], acc[1]));
        const float sum = y.x + y.y;
        xs[(buf * 4 + hf) * 128 + ln] = sum;
      }
    };
    // pass 2: a tile's quarters meet, after a barrier; what is already in the
    // total was requested two tiles earlier
    float prev[2] = {0.f, 0.f};
    const int64_t mrow = seq * a.nkv + kvh;
    auto before = [&](int tile) {
      const int t = tile * TP + ln;
      if (PASS != 2 || !worker || hf != 0 || t >= len || t >= a.out_stride) return 0.f;
      return blk > 0 ? a.mass_out[mrow * a.out_stride + t] : a.mass_in ? a.mass_in[mrow * a.in_stride + t] : 0.f;
    };
    auto store = [&](int tile, int buf, float was) {
      if constexpr (PASS == 2) {
        const int t = tile * TP + ln;
        if (worker && hf == 0 && t < len && t < a.out_stride) {
          const float* x = xs + buf * 512 + ln;
          a.mass_out[mrow * a.out_stride + t] = was + ((x[0] + x[128]) + (x[256] + x[384]));
        }
      }
    };
    auto one_tile = [&](int tile, int buf, float& was) {   // (`was` by the tile's parity)
      if (tile > tile0) {   // the planes are free once the last products are done
        if (worker) ok_run = t5::wait(bar, phase) && ok_run;
        phase ^= 1;
        t5::fence_after();
      }
      if (worker) {
        uint32_t h[HP / 8], lw[HP / 8];
        mass_dequant<S, HP>(raw, lv, h, lw);
        uint8_t* kh = smem + C::OFF_K;
#pragma unroll
        for (int k = 0; k < D / 8; ++k) {
          const int o = sw<TP>(pt, S == S_BF16 ? blk128 * 128 + 32 * k + 8 * part : pc * D + 8 * k);
          *reinterpret_cast<uint4*>(kh + o) = make_uint4(h[4 * k], h[4 * k + 1], h[4 * k + 2], h[4 * k + 3]);
          if constexpr (C::KPL == 2)
            *reinterpret_cast<uint4*>(kh + C::KB + o) = make_uint4(lw[4 * k], lw[4 * k + 1], lw[4 * k + 2], lw[4 * k + 3]);
        }
        if (pc == 0) ok_s[(tile - tile0) % 3 * 128 + pt] = rok;
      }
      const bool mine = !worker || rok;
      t5::fence_smem_async();
      t5::fence_before();
      const bool valid = __syncthreads_and(mine && ok_run);
      if (!worker) {
        if (tc5::elect_one()) {
          t5::fence_after();
          constexpr uint32_t ID = t5::idesc(BF, 128, PASS == 1 ? TP : QR), HI = tc5::desc_hi(1024, true);
          const uint32_t dq = tc5::desc_lo(sb, 16), dk = tc5::desc_lo(sb + C::OFF_K, 16);
          const uint32_t d = tmem + buf * 128;
#pragma unroll
          for (int j = 0; j < HD / 16; ++j) {
            const uint32_t oq = (j / 4 * QR * 128 + j % 4 * 32) / 16, ok = (j / 4 * TP * 128 + j % 4 * 32) / 16;
            const uint32_t x = PASS == 1 ? dq + oq : dk + ok, y = PASS == 1 ? dk + ok : dq + oq;
            tc5::mma_ss<HI>(d, x, y, ID, j > 0);
            if (q_lo) tc5::mma_ss<HI>(d, x + (PASS == 1 ? C::QB / 16 : 0), y + (PASS == 1 ? 0 : C::QB / 16), ID, 1);
            if constexpr (C::KPL == 2)
              tc5::mma_ss<HI>(d, x + (PASS == 1 ? 0 : C::KB / 16), y + (PASS == 1 ? C::KB / 16 : 0), ID, 1);
          }
          t5::commit(bar);
        }
        __syncwarp();
      } else {
        if (tile + 1 < tile1) {
          fetch(tile + 1);
          ids(tile + 2);
        }
        if (tile > tile0 + 1) store(tile - 2, buf, was);
        was = before(tile);
        if (tile > tile0) consume(tile - 1, buf ^ 1, full_prev);
      }
      full_prev = valid;
    };

    if (worker) {
      ids(tile0);
      fetch(tile0);
      ids(tile0 + 1);
    }
    for (int tile = tile0; tile < tile1; tile += 2) {
      one_tile(tile, 0, prev[0]);
      if (tile + 1 < tile1) one_tile(tile + 1, 1, prev[1]);
    }
    ok_run = t5::wait(bar, phase) && ok_run;
    phase ^= 1;
    t5::fence_after();
    __syncthreads();
    const int nt = tile1 - tile0;
    if (nt > 1) store(tile1 - 2, nt & 1, nt & 1 ? prev[1] : prev[0]);
    if (worker) consume(tile1 - 1, (nt - 1) & 1, full_prev);
    t5::fence_before();
    __syncthreads();
    t5::fence_after();
    store(tile1 - 1, (nt - 1) & 1, (nt - 1) & 1 ? prev[1] : prev[0]);
    if constexpr (PASS == 1) {   // join the quarters of a row
      float2* x2 = reinterpret_cast<float2*>(xs);
      if (worker) x2[hf * 128 + ln] = make_float2(m, l);
      __syncthreads();
      if (worker && hf == 0 && row < rows_all) {
        float mm = -CUDART_INF_F, ll = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) mm = fmaxf(mm, x2[i * 128 + ln].x);
        const float base = mm == -CUDART_INF_F ? 0.f : mm;
#pragma unroll
        for (int i = 0; i < 4; ++i) ll += x2[i * 128 + ln].y * t5::ex2((x2[i * 128 + ln].x - base) * scale);
        a.stats[((q0 + row / a.rep) * a.nq + kvh * a.rep + row % a.rep) * a.splits1 + range] = make_float2(mm, ll);
      }
    }
    if (!ok_run && tid == 0 && a.err) atomicOr(a.err, KVQ_DEVERR_TIMEOUT);
  }
  t5::fence_before();
  __syncthreads();
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 256;\n" ::"r"(tmem));
}

template <int S, int HD>
cudaError_t launch_mass_tc(const MassArgs& a, const Codebooks& cb, cudaStream_t st) {
  auto k1 = mass_tc_kernel<S, HD, 1>;
  auto k2 = mass_tc_kernel<S, HD, 2>;
  cudaError_t e = cudaFuncSetAttribute(k1, cudaFuncAttributeMaxDynamicSharedMemorySize, MtCfg<S, HD, 1>::SMEM);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(k2, cudaFuncAttributeMaxDynamicSharedMemorySize, MtCfg<S, HD, 2>::SMEM);
  if (e != cudaSuccess) return e;
  const unsigned ctas = (unsigned)((int64_t)a.slots * a.nkv);
  const int nblk = (int)(((int64_t)a.max_chunk * a.rep + 127) / 128);
  k1<<<dim3(ctas, 1, nblk), 544, MtCfg<S, HD, 1>::SMEM, st>>>(a, cb);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  k2<<<ctas, 544, MtCfg<S, HD, 2>::SMEM, st>>>(a, cb);
  return cudaGetLastError();
}

template <int S>
cudaError_t launch_mass_side(int hd, const MassArgs& a, const Codebooks& cb, cudaStream_t st) {
  const bool few = a.scores != nullptr;
  switch (hd) {
    case 64: return few ? launch_mass_rows<S, 64>(a, cb, st) : launch_mass_tc<S, 64>(a, cb, st);
    case 128: return few ? launch_mass_rows<S, 128>(a, cb, st) : launch_mass_tc<S, 128>(a, cb, st);
    case 256: return few ? launch_mass_rows<S, 256>(a, cb, st) : launch_mass_tc<S, 256>(a, cb, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvq
