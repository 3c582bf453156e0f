// Prompt attention on the 5th-generation tensor cores (BF16 rows).
//
// "combs_models/kv.rs" attend with its causal mask + repeat_kv: for a tile of
// 128 score rows, S = Q K^T, P = 2^(S scale - m), O = sum P V with a running
// maximum and sum per row.
//
// Score rows: RP heads of one kv head x 128 / RP consecutive queries (RP =
// the largest power of two that divides the GQA ratio, at most 16), so that
// short prompts fill the rows and the heads share the K/V tiles.  A CTA
// takes NQ such row tiles (2; 1 at head_dim 256, whose accumulator fills
// half of tensor memory) and walks 128-position K/V tiles.
//
// Roles: eight softmax warps per row tile (two threads per row, half of a
// tile's positions and of O's columns each), a matrix warp per row tile, a
// warp for the copies.
//   copies: Q once; K and V tiles by TMA (128-byte swizzle, 64 dims x 128
//     positions a box) through a ring of NST stages, K and V in turn (at
//     head_dim 256 a ring each); a tile's row bytes are used as they lie in
//     memory: K as the K-major operand, V as the MN-major one, nothing is
//     transposed.
//   matrix: S_q (128 x 128 fp32 in tensor memory) = Q_q K^T; then O_q += P_q V
//     with P_q read from tensor memory, where the softmax writes it over S_q
//     (bf16, two positions a column).  The two row tiles take turns: while
//     one is in its softmax the other's products run; at head_dim 256 the one
//     tile has two S buffers and the next S runs ahead instead.
//   softmax: a thread reads its half row (tcgen05.ld), masks it where the
//     tile cuts the row's range, and computes the weights with the maximum of
//     the tiles before while its maximum and the other half's meet in shared
//     memory; only if the row's grew by more than 2^8 (P <= 2^8 otherwise) is
//     O rescaled and the weights computed again.
// One prompt of 16384 tokens, 32 query / 8 kv heads, GB300: head_dim 128
// 1.38 to 1.52 ms, cold to back to back (1.45 to 1.59 PFLOP/s algorithmic, 75
// to 83% of a cuBLAS burst), 64 1.17 to 1.20 ms; 16 heads of 256 2.05 to 2.11
// ms.  Bound by each row tile's chain softmax (about 1600 cycles) -> products
// (1024) -> hand-over (500).
// P is rounded to bf16 (relative 2^-8 a weight, the size of the output's own
// rounding: 2.1e-3 rms of the output's size where the output's rounding alone
// gives 1.6e-3); for an fp32 output it carries hi + lo parts, two products
// (2.46 ms at head_dim 128, 1.69 at 64, 2.64 at 256).
//
// A weight of zero does not keep a NaN or infinite value out of a product,
// so where a tile is cut the warpgroup looks the V tile over and, if it holds
// one, adds the attended positions on the CUDA cores instead.
#include <math_constants.h>

#include <cstring>

#include "kvq_host.h"
#include "kvq_prefill_tc5.cuh"
#include "kvq_decode_tma.cuh"
#include "kvq_prompt.h"
#include "kvq_tc5_issue.cuh"
#include "kvq_tma_host.h"

namespace kvq {

namespace {

struct PromptMaps {
  CUtensorMap q, k, v;
};

template <int HD>
struct PtCfg {
  static constexpr int NQ = HD == 256 ? 1 : 2;      // row tiles
  static constexpr int NSB = HD == 256 ? 2 : 1;     // S buffers per row tile
  static constexpr int DP = HD == 256 ? 2 : 1;      // parts of a K or V tile, one stage each
  static constexpr int PBLK = HD / 64 / DP;         // 64-dim blocks per part
  static constexpr int BLK = 128 * 128;             // bytes of a block: 128 rows x 64 dims
  static constexpr int STAGE = PBLK * BLK;
  static constexpr int NST = HD == 64 ? 8 : 5;
  static constexpr int QB = HD / 64 * BLK;
  static constexpr int OFF_KV = NQ * QB;
  static constexpr int OFF_BAR = OFF_KV + NST * STAGE;
  static constexpr int OFF_X = OFF_BAR + 512;         // [2 S buffers][2 halves][128 rows] row maxima, then sums
  static constexpr int SMEM = OFF_X + 2048;
  static constexpr int SOFT = NQ * 8;                 // softmax warps
  static constexpr int THREADS = (SOFT + 4) * 32;     // + a warpgroup of one copy and NQ matrix warps
  // registers a thread: 96 at the launch of 640 threads, then 32 and 112
  // (4 x 32 x 64 given back, 16 x 32 x 16 taken up)
  static constexpr bool SPLIT_REGS = NQ == 2;
  static constexpr int O_COL = 256;
  static constexpr int OROW = HD == 64 ? 64 : 128;  // bytes of a row a warp stages at a time for its stores
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
};

constexpr int kListed = 1024;   // sequences whose tile counts fit where the row maxima go

// Descriptors (low words) of 128-byte-swizzled operands.  K-major: 8-row
// groups 1 KB apart.  MN-major: 64-element blocks 16 KB apart (the leading
// offset), 8-deep groups 1 KB apart.
__device__ __forceinline__ uint32_t desc_k(uint32_t addr) { return tc5::desc_lo(addr, 16); }
__device__ __forceinline__ uint32_t desc_mn(uint32_t addr) { return tc5::desc_lo(addr, 16384); }
constexpr uint32_t kDescHi = tc5::desc_hi(1024, true);
__device__ __forceinline__ bool try_bar(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}
__device__ __forceinline__ void ld32(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
      "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
        "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
        "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr));
}
__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
template <int HD, bool SPLIT>
__global__ void __launch_bounds__(PtCfg<HD>::THREADS, 1)
prompt_tc_kernel(const PromptArgs a, const __grid_constant__ PromptMaps maps, int rp, int listed) {
  using C = PtCfg<HD>;
  constexpr int NQ = C::NQ, NSB = C::NSB, DP = C::DP, PBLK = C::PBLK, NST = C::NST;
  extern __shared__ __align__(1024) uint8_t tma_smem[];
  uint8_t* const smem = tma_smem;
  const uint32_t sbase = tm::saddr(smem);
  const int tid = threadIdx.x, lane = tid & 31;
  // (from one lane: the roles below then branch by whole warps)
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (sbase & 1023u) {   // the swizzled tiles need it; dynamic shared memory starts at 1 KB
    if (tid == 0 && a.err) atomicOr(a.err, KVQ_DEVERR_TIMEOUT);
    return;
  }

  // ---- the CTA's rows
  const int subs = a.nq / rp;                           // head groups
  const int hg = (int)(blockIdx.x % subs);
  const int head0 = hg * rp, kvh = head0 / a.rep;
  const int lrp = 31 - __clz(rp), lqt = 7 - lrp;        // rp is a power of two
  const int qt = 1 << lqt;                              // queries per row tile
  // The longest rows start first: tile index from the highest down, sequences
  // in order.  Listed: CTA `item` finds its tile among those there are; else
  // every sequence has a CTA for each tile of the longest one.
  int64_t seq = blockIdx.x / subs, t0 = 0;
  int tile = gridDim.y - 1 - blockIdx.y, len = 0;
  int* found = reinterpret_cast<int*>(smem + C::OFF_BAR + 352);   // sequence, tile
  if (!listed) {
    prompt_range(a, seq, tid == 0 && tile == 0 && hg == 0, t0, len);
    if (tile * NQ * qt >= min(len, a.max_len)) return;
  } else if (warp == 0) {
    const int item = (int)seq;
    uint16_t* tiles = reinterpret_cast<uint16_t*>(smem + C::OFF_X);   // per sequence
    int most = 0;
    for (int s = lane; s < a.num_seqs; s += 32) {
      prompt_range(a, s, blockIdx.x == 0, t0, len);
      const int x = (min(len, a.max_len) + NQ * qt - 1) >> (lqt + NQ - 1);
      tiles[s] = (uint16_t)x;
      most = max(most, x);
    }
    __syncwarp();
    // tiles at or above index x, of all sequences
    auto above = [&](int x) {
      int c = 0;
#pragma unroll 1
      for (int s = lane; s < a.num_seqs; s += 32) c += max(0, (int)tiles[s] - x);
      return __reduce_add_sync(0xffffffffu, c);
    };
    int lo = -1, hi = __reduce_max_sync(0xffffffffu, most), more = 0;   // lo: the highest x with above(x) > item
#pragma unroll 1
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1, c = above(mid);
      if (c > item) {
        lo = mid;
      } else {
        hi = mid;
        more = c;
      }
    }
    int rem = item - more;   // sequences with tile `lo` before this one
    if (lane == 0) found[1] = lo;   // -1: no tile left
#pragma unroll 1
    for (int s0 = 0; s0 < a.num_seqs && lo >= 0 && rem >= 0; s0 += 32) {
      const bool mine = s0 + lane < a.num_seqs && (int)tiles[s0 + lane] > lo;
      const uint32_t has = __ballot_sync(0xffffffffu, mine);
      if (mine && rem == __popc(has & ((1u << lane) - 1u))) found[0] = s0 + lane;
      rem -= __popc(has);
    }
  }
  // ---- barriers and tensor memory
  const uint32_t bar = sbase + C::OFF_BAR;
  auto full = [&](int s) { return bar + 8 * s; };              // a stage's copy landed
  auto freed = [&](int e) { return bar + 64 + 8 * e; };        // see the copies
  auto s_full = [&](int b) { return bar + 128 + 8 * b; };       // S written
  auto p_ready = [&](int b) { return bar + 144 + 8 * b; };     // S read, P written (per S buffer)
  auto o_done = [&](int q) { return bar + 160 + 8 * q; };      // O += P V done
  auto m_end = [&](int q) { return bar + 176 + 8 * q; };       // every product done
  auto v_seen = [&](int q) { return bar + 192 + 8 * q; };      // a cut tile's V looked over
  auto by_done = [&](int q) { return bar + 208 + 8 * q; };     // and added by hand
  auto pair = [&](int q, int w) { return bar + 224 + 8 * (4 * q + w); };   // the two warps of 32 rows
  auto turn = [&](int q) { return bar + 288 + 8 * q; };        // the matrix warps' turns
  const uint32_t q_full = bar + 304;
  volatile uint32_t* skip = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_BAR + 312);    // [2] per S buffer
  volatile uint32_t* failed = skip + 2;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + 324);
  volatile uint32_t* v_bad = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_BAR + 328);   // [2][3]
  if (tid == 64) {
    auto init = [&](uint32_t b, int count) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(b), "r"(count));
    };
    for (int s = 0; s < NST; ++s) init(full(s), 1);
    for (int e = 0; e < (NSB == 1 ? 4 : NST); ++e) init(freed(e), NQ);
    for (int b = 0; b < 2; ++b) {
      init(s_full(b), 1);
      init(p_ready(b), 256);
      init(o_done(b), 1);
      init(m_end(b), 1);
      init(v_seen(b), 256);
      init(by_done(b), 256);
      init(turn(b), 1);
      for (int w = 0; w < 4; ++w) init(pair(b, w), 64);
      skip[b] = 0;
    }
    for (int b = 0; b < 6; ++b) v_bad[b] = 0;
    init(q_full, 1);
    *failed = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (tid >= 96 && tid < 99)
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(tid == 96 ? &maps.q : tid == 97 ? &maps.k : &maps.v) : "memory");
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(tm::saddr(tslot)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  }
  t5::fence_before();
  __syncthreads();
  t5::fence_after();
  const uint32_t tmem = *tslot;
  auto free_tmem = [&]() {
    if (warp == 1)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem));
  };
  if (listed) {
    seq = found[0];
    tile = found[1];
    if (tile < 0) return free_tmem();
    prompt_range(a, seq, false, t0, len);
  }
  // (a warp reduction leaves its result in a uniform register: as values of
  // each thread these cost the softmax warps 22 spilled registers)
  tile = (int)__reduce_max_sync(0xffffffffu, tile);
  t0 = (int)__reduce_max_sync(0xffffffffu, (int)t0);
  len = (int)__reduce_max_sync(0xffffffffu, len);
  const int n = min(len, a.max_len), i0 = tile << (lqt + NQ - 1);
  const int W = a.window;
  // K/V tiles of each row tile: [jb, je), empty for a tile without queries
  int jb[NQ], je[NQ], J0 = 0x7fffffff, J1 = 0;
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    const int f = i0 + q * qt, l = min(f + qt, n) - 1;
    jb[q] = f < n && W > 0 ? max(0, f + 1 - W) / 128 : 0;
    je[q] = f < n ? l / 128 + 1 : 0;
    if (f < n) {
      J0 = min(J0, jb[q]);
      J1 = max(J1, je[q]);
    }
  }

  auto await = [&](uint32_t b, uint32_t parity) {
    for (int x = 0; x < (1 << 18); ++x) {
#pragma unroll 1
      for (int y = 0; y < 16; ++y)
        if (try_bar(b, parity)) return true;
      if (*failed) return false;
    }
    *failed = 1;
    return false;
  };
  // (warp-uniform: what follows a wait is collective)
  auto await_all = [&](uint32_t b, uint32_t parity) { return __all_sync(0xffffffffu, await(b, parity)); };

  // head_dim 256: the K parts take turns in two stages and the V parts in
  // three, each ring filled by a thread of its own, so that the next K tile
  // does not wait for room behind a V tile.  Part x of K (v = 0) or V.
  auto ring_stage = [&](int v, int x) { return v ? 2 + x % 3 : x % 2; };
  auto ring_parity = [&](int v, int x) { return (uint32_t)(v ? x / 3 : x / 2) & 1u; };
  auto copy_ring = [&](int v) {
    const int total = (J1 - J0) * DP, depth = v ? 3 : 2;
    int issued = 0;
    for (int x = 0; x < total; ++x) {
      const int s = ring_stage(v, x);
      if (x >= depth && !await(freed(s), ring_parity(v, x - depth))) break;
      tm::bar_expect(full(s), C::STAGE);
      for (int b = 0; b < PBLK; ++b)
        tm::tma3(sbase + C::OFF_KV + s * C::STAGE + b * C::BLK, v ? &maps.v : &maps.k, (x % DP * PBLK + b) * 64, kvh,
                 (int)(t0 + (J0 + x / DP) * 128), full(s));
      issued = x + 1;
    }
    for (int x = max(0, issued - depth); x < issued; ++x) tm::bar_wait(full(ring_stage(v, x)), ring_parity(v, x));
  };
  if constexpr (C::SPLIT_REGS) {
    if (warp >= C::SOFT) asm volatile("setmaxnreg.dec.sync.aligned.u32 32;\n");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 112;\n");
  }
  if (warp == C::SOFT) {
    // ---------------------------------------------------------------- copies
    if (lane == 0) {
      int bytes = 0;
#pragma unroll
      for (int q = 0; q < NQ; ++q) bytes += je[q] > 0 ? C::QB : 0;
      tm::bar_expect(q_full, bytes);
#pragma unroll
      for (int q = 0; q < NQ; ++q)
        if (je[q] > 0)
          for (int b = 0; b < HD / 64; ++b)
            tm::tma3(sbase + q * C::QB + b * C::BLK, &maps.q, b * 64, head0, (int)(t0 + i0 + q * qt), q_full);
      if constexpr (NSB == 1) {
        // One ring.  Event e: the products that read K tile e (from J0) and V
        // tile e - 1 are done.  Stage i % NST last held ring position i - NST.
        const int total = (J1 - J0) * 2;
        int issued = 0;
        for (int i = 0; i < total; ++i) {
          const int s = i % NST, v = i % 2, j = J0 + i / 2;
          if (i >= NST) {
            const int e = (i - NST) / 2 + (i - NST) % 2;
            if (!await(freed(e & 3), (uint32_t)(e / 4) & 1u)) break;
          }
          tm::bar_expect(full(s), C::STAGE);
          for (int b = 0; b < PBLK; ++b)
            tm::tma3(sbase + C::OFF_KV + s * C::STAGE + b * C::BLK, v ? &maps.v : &maps.k, b * 64, kvh,
                     (int)(t0 + j * 128), full(s));
          issued = i + 1;
        }
        // no copy may be in flight when the CTA's shared memory goes
        tm::bar_wait(q_full, 0);
        for (int i = max(0, issued - NST); i < issued; ++i) tm::bar_wait(full(i % NST), (uint32_t)(i / NST) & 1u);
      } else {
        copy_ring(0);
        tm::bar_wait(q_full, 0);
      }
    }
  } else if (warp > C::SOFT + NQ) {
    // the second ring's copies, or nothing (fills the warpgroup)
    if (NSB == 2 && warp == C::SOFT + NQ + 1 && lane == 0) copy_ring(1);
  } else if (warp > C::SOFT) {
    // ------------------------------------------- matrix: a warp per row tile
    constexpr uint32_t ID_S = t5::idesc(true, 128, 128);
    constexpr uint32_t ID_O = t5::idesc(true, 128, 64 * PBLK) | (1u << 16);   // B MN-major
    // (a warp reduction leaves its result in a uniform register)
    auto uni = [](int x) { return (int)__reduce_max_sync(0xffffffffu, x); };
    const int q = uni(warp - C::SOFT - 1);
    const uint32_t tm_u = (uint32_t)uni((int)tmem);
    const int first = uni(J0), tiles = uni(J1) - first;
    const int qb = uni(q ? jb[NQ - 1] : jb[0]) - first, qe = uni(q ? je[NQ - 1] : je[0]) - first;
    const uint32_t d_o = tm_u + C::O_COL + q * HD, q_s = sbase + q * C::QB;
    const int f_q = i0 + q * qt, l_q = min(f_q + qt, n) - 1;   // the row tile's queries
    int rs = 0, rph = 0;    // next ring stage to be read and its phase
    bool ok = await_all(q_full, 0);
    int ks[DP], vs[DP];     // stages of the K tile and the V tile in hand
    auto landed = [&](int (&st)[DP]) {
#pragma unroll
      for (int p = 0; p < DP; ++p) {
        ok = ok && await_all(full(rs), (uint32_t)rph);
        st[p] = rs;
        if (++rs == NST) {
          rs = 0;
          rph ^= 1;
        }
      }
      t5::fence_after();
    };
    auto ring_landed = [&](int v, int t, int (&st)[DP]) {   // head_dim 256: tile t's parts
#pragma unroll
      for (int p = 0; p < DP; ++p) {
        const int x = t * DP + p;
        ok = ok && await_all(full(ring_stage(v, x)), ring_parity(v, x));
        st[p] = ring_stage(v, x);
      }
      t5::fence_after();
    };
    auto commit = [&](uint32_t b) {
      if (tc5::elect_one()) t5::commit(b);
    };
    auto qk = [&](int buf) {
      if (!tc5::elect_one()) return;
#pragma unroll
      for (int p = 0; p < DP; ++p) {
        const uint32_t qd = desc_k(q_s + p * PBLK * C::BLK);
        const uint32_t kd = desc_k(sbase + C::OFF_KV + ks[p] * C::STAGE);
#pragma unroll
        for (int b = 0; b < PBLK; ++b)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc5::mma_ss<kDescHi>(tm_u + buf * 128, qd + (b * C::BLK + k * 32) / 16, kd + (b * C::BLK + k * 32) / 16, ID_S,
                   p > 0 || b > 0 || k > 0);
        if (NSB == 2) t5::commit(freed(ks[p]));
      }
      t5::commit(s_full(buf));
    };
    auto cut = [&](int t) {   // as the softmax sees tile t
      const int kv0 = (first + t) * 128;
      return kv0 + 127 > f_q || (W > 0 && kv0 < l_q + 1 - W);
    };
    // (the softmax waits for a product with V only where S runs ahead of it,
    // to rescale O, and for the last)
    auto pv = [&](int buf, int t) {
      const bool by_hand = cut(t) && skip[buf] != 0;
      if (!tc5::elect_one()) return;
      if (!by_hand) {
        const uint32_t acc = t > qb;
#pragma unroll
        for (int p = 0; p < DP; ++p) {
          const uint32_t vd = desc_mn(sbase + C::OFF_KV + vs[p] * C::STAGE);
          const uint32_t d = d_o + p * 128, pa = tm_u + buf * 128;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            // P of positions 0 .. 63 in columns 0 .. 31, of 64 .. 127 in 64 .. 95
            const uint32_t pk = pa + (k & 3) * 8 + (k >> 2) * 64;
            tc5::mma_ts<kDescHi>(d, pk, vd + k * 2048 / 16, ID_O, k > 0 ? 1u : acc);
            if constexpr (SPLIT) tc5::mma_ts<kDescHi>(d, pk + 32, vd + k * 2048 / 16, ID_O, 1);
          }
          if (NSB == 2) t5::commit(freed(vs[p]));
        }
      } else if (NSB == 2) {
#pragma unroll
        for (int p = 0; p < DP; ++p) t5::commit(freed(vs[p]));
      }
      if (NSB == 2) t5::commit(o_done(q));
    };
    // The two row tiles' products take turns, so that one tile's softmax runs
    // under the other's products (issued side by side they would end together
    // and leave the tensor cores idle during both softmaxes).
    auto my_turn = [&](int t) {
      if constexpr (NQ == 2) {
        if (q == 1 || t > 0) ok = ok && await_all(turn(q), (uint32_t)(q ? t : t - 1) & 1u);
      }
    };
    auto pass_turn = [&]() {
      if constexpr (NQ == 2) {
        if (tc5::elect_one()) arrive(turn(q ^ 1));
      }
    };
    auto in = [&](int t) { return qb <= t && t < qe; };
    auto p_wait = [&](int t) {
      // (per S buffer: where S runs ahead, the softmax may hand over two tiles
      // before the first is waited for)
      ok = ok && (NSB == 1 ? await_all(p_ready(q), (uint32_t)(t - qb) & 1u)
                           : await_all(p_ready(t & 1), (uint32_t)(t >> 1) & 1u));
      t5::fence_after();
    };
    if constexpr (NSB == 1) {
      // turn 0: the first S; turn t + 1: tile t's product with V, then the next S
      landed(ks);
      my_turn(0);
      if (ok && in(0)) qk(q);
      pass_turn();
      commit(freed(0));
      for (int t = 0; ok && t < tiles; ++t) {
        landed(vs);
        if (t + 1 < tiles) landed(ks);
        my_turn(t + 1);
        if (in(t)) p_wait(t);
        if (!ok) break;
        if (in(t)) pv(q, t);
        if (t + 1 < tiles && in(t + 1)) qk(q);
        pass_turn();
        commit(freed((t + 1) & 3));
      }
    } else {
      ring_landed(0, 0, ks);
      if (ok) qk(0);
      for (int t = 0; ok && t < tiles; ++t) {
        // The softmax of a cut tile waits for its V tile by itself, and a
        // barrier's parity tells a phase only from the one before: the V tile
        // before it, whose stage it may follow into, has to have landed when
        // that softmax starts.
        const bool early = t + 1 < tiles && cut(t + 1);
        if (early) ring_landed(1, t, vs);
        if (t + 1 < tiles) {   // the next S runs under this tile's softmax
          ring_landed(0, t + 1, ks);
          if (ok) qk((t + 1) & 1);
        }
        if (!early) ring_landed(1, t, vs);
        p_wait(t);
        if (ok) pv(t & 1, t);
      }
    }
    // no product may be in flight when the CTA's memory goes
    commit(m_end(q));
    tm::bar_wait(m_end(q), 0);
  } else {
    // ------------------- softmax: 8 warps per row tile, two threads per row,
    // each with half of a tile's positions and half of O's columns
    constexpr int HC = HD / 2;
    const int q = warp >> 3, half = (warp >> 2) & 1, quad = warp & 3, row = quad * 32 + lane;
    const int f = i0 + q * qt;
    const int qb = NQ == 2 && q ? jb[NQ - 1] : jb[0], qe = NQ == 2 && q ? je[NQ - 1] : je[0];
    const int i = f + (row >> lrp);                         // this row's query
    const int last = min(f + qt, n) - 1;
    const int lo = W > 0 ? max(0, i + 1 - W) : 0;
    const uint32_t t_lane = (uint32_t)(32 * quad) << 16;
    const uint32_t o_tm = tmem + C::O_COL + q * HD + t_lane;
    const float sc = a.scale2, lazy = 8.f / a.scale2;
    const uint64_t sc2 = f2::pack(sc, sc);
    float* xs = reinterpret_cast<float*>(smem + C::OFF_X);
    float m = -CUDART_INF_F, l = 0.f;    // maximum of the row, sum of this half
    bool ok = true;
    int cuts = 0, hands = 0;
    for (int j = qb; j < qe; ++j) {
      const int it = j - qb, buf = NSB == 1 ? q : it & 1;
      const uint32_t s_tm = tmem + buf * 128 + t_lane, h_tm = s_tm + 64 * half;   // the row's scores, this half's
      ok = await_all(s_full(buf), (uint32_t)(NSB == 1 ? it : it >> 1) & 1u);
      if (!ok) break;
      t5::fence_after();
      const int kv0 = j * 128;
      // does the tile hold a position some query of the row tile does not attend to?
      const bool cut = kv0 + 127 > f || (W > 0 && kv0 < last + 1 - W);
      bool by_hand = false;
      if (cut) {
        // values of the V tile, every row: is one NaN or infinite?
        uint32_t top = 0;   // the largest of the bits without signs, two values at a time
#pragma unroll 1
        for (int p = 0; p < DP; ++p) {
          const int r = NSB == 1 ? (j - J0) * 2 + 1 : (j - J0) * DP + p;   // ring position
          const int rs = NSB == 1 ? r % NST : ring_stage(1, r);
          ok = await_all(full(rs), NSB == 1 ? (uint32_t)(r / NST) & 1u : ring_parity(1, r)) && ok;
          const uint32_t v = sbase + C::OFF_KV + rs * C::STAGE + (128 * half + row) * 16;
#pragma unroll 4
          for (int x = 0; x < C::STAGE; x += 4096) {
            const uint4 w = tm::lds128(v + x);
            top = __vmaxu2(__vmaxu2(top, w.x & 0x7fff7fffu), w.y & 0x7fff7fffu);
            top = __vmaxu2(__vmaxu2(top, w.z & 0x7fff7fffu), w.w & 0x7fff7fffu);
          }
        }
        // one flag for the row tile's threads, three slots in turn: slot x is
        // cleared after barrier x + 1, when all have read it, and set again
        // only after barrier x + 2
        if ((top & 0xffffu) >= 0x7f80u || (top >> 16) >= 0x7f80u) v_bad[3 * q + cuts % 3] = 1;
        arrive(v_seen(q));
        ok = await_all(v_seen(q), (uint32_t)cuts & 1u) && ok;
        if (!ok) break;
        by_hand = v_bad[3 * q + cuts % 3] != 0;
        if ((tid & 255) == 0) v_bad[3 * q + (cuts + 2) % 3] = 0;
        ++cuts;
      }
      if ((tid & 255) == 0) skip[buf] = by_hand;
      __syncwarp();   // the loads below are the whole warp's
      // this half's scores, masked where the tile is cut
      const uint32_t m0 = (uint32_t)(lo - kv0 - 64 * half), span = (uint32_t)(i - lo);
      auto fetch = [&](uint32_t (&s)[64]) {
        ld32(h_tm, s);
        ld32(h_tm + 32, s + 32);
        t5::wait_ld();
        if (cut) {
#pragma unroll
          for (int e = 0; e < 64; ++e)
            if ((uint32_t)e - m0 > span) s[e] = 0xff800000u;
        }
      };
      // ---- weights with the maximum of the tiles before, while the halves'
      // maxima meet in shared memory; computed again in the rare case that a
      // row's maximum grew by more than 2^8
      uint32_t ph[32], pl[SPLIT ? 32 : 1];
      float lsum = 0.f, mt;
      auto weights = [&](const uint32_t (&s)[64]) {
        const float neg = m == -CUDART_INF_F ? 0.f : -m * sc;
        const uint64_t neg2 = f2::pack(neg, neg);
        uint64_t sum2[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float2 x = f2::unpack(f2::fma(f2::pack(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), sc2, neg2));
          const float y0 = t5::ex2(x.x), y1 = t5::ex2(x.y);
          sum2[e & 1] = f2::add(sum2[e & 1], f2::pack(y0, y1));
          if constexpr (SPLIT) tc::split2<true>(y0, y1, ph[e], pl[e]);
          else ph[e] = tc::pack2<true>(y0, y1);
        }
        const float2 sa = f2::unpack(f2::add(sum2[0], sum2[1]));
        lsum = sa.x + sa.y;
      };
      auto again = [&]() {   // (32 positions at a time: fewer registers on the rare path)
        const float neg = m == -CUDART_INF_F ? 0.f : -m * sc;
        lsum = 0.f;
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          uint32_t s[32];
          ld32(h_tm + c, s);
          t5::wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float x0 = fmaf(__uint_as_float(s[2 * e]), sc, neg), x1 = fmaf(__uint_as_float(s[2 * e + 1]), sc, neg);
            if (cut && (uint32_t)(c + 2 * e) - m0 > span) x0 = -CUDART_INF_F;
            if (cut && (uint32_t)(c + 2 * e + 1) - m0 > span) x1 = -CUDART_INF_F;
            const float y0 = t5::ex2(x0), y1 = t5::ex2(x1);
            lsum += y0 + y1;
            if constexpr (SPLIT) tc::split2<true>(y0, y1, ph[c / 2 + e], pl[c / 2 + e]);
            else ph[c / 2 + e] = tc::pack2<true>(y0, y1);
          }
        }
      };
      {
        uint32_t s[64];
        fetch(s);
        float x0 = -CUDART_INF_F, x1 = x0;
#pragma unroll
        for (int e = 0; e < 64; e += 4) {
          x0 = f2::max3(x0, __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
          x1 = f2::max3(x1, __uint_as_float(s[e + 2]), __uint_as_float(s[e + 3]));
        }
        mt = t5::max_nan(x0, x1);
        xs[(2 * buf + half) * 128 + row] = mt;
        arrive(pair(q, quad));
        if (it > 0) weights(s);
      }
      ok = await_all(pair(q, quad), (uint32_t)it & 1u);
      if (!ok) break;
      mt = t5::max_nan(mt, xs[(2 * buf + 1 - half) * 128 + row]);
      bool resc = false;
      float alpha = 1.f;
      // (a row that is NaN already stays as it is)
      if (__any_sync(0xffffffffu, it == 0 || (!(mt <= m + lazy) && m == m))) {
        if (!(mt <= m + lazy)) {
          alpha = m == -CUDART_INF_F ? 0.f : t5::ex2((m - mt) * sc);
          resc = it > 0 && m != -CUDART_INF_F;
          l *= alpha;
          m = mt;
        }
        resc = __any_sync(0xffffffffu, resc);
        again();
      }
      l += lsum;
      if (NSB == 2 && (resc || by_hand) && it > 0) {   // O is read below: the last product is done
        ok = await_all(o_done(q), (uint32_t)(it - 1) & 1u);
        if (!ok) break;
        t5::fence_after();
      }
      if (resc) {
#pragma unroll 1
        for (int c = half * HC; c < half * HC + HC; c += 16) {
          uint32_t v[16];
          t5::ld16(o_tm + c, v);
          t5::wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
          t5::st16(o_tm + c, v);
        }
        t5::wait_st();
      }
      if (by_hand) {   // O += P . V over the attended positions only
        const float neg = m == -CUDART_INF_F ? 0.f : -m * sc;
#pragma unroll 1
        for (int c = half * HC; c < half * HC + HC; c += 16) {
          uint32_t v[16], sv[16];
          if (it > 0) {
            t5::ld16(o_tm + c, v);
            t5::wait_ld();
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = 0u;
          }
          const int blk = c / 64;
          const int r = NSB == 1 ? ((j - J0) * 2 + 1) % NST : ring_stage(1, (j - J0) * DP + blk / PBLK);
          const uint32_t vb = sbase + C::OFF_KV + r * C::STAGE + (blk % PBLK) * C::BLK;
#pragma unroll 1
          for (int x = 0; x < 128; x += 16) {
            __syncwarp();
            t5::ld16(s_tm + x, sv);
            t5::wait_ld();
#pragma unroll 1
            for (int e = 0; e < 16; ++e) {
              const int t = kv0 + x + e;
              float sx = 0.f;
#pragma unroll
              for (int y = 0; y < 16; ++y) sx = y == e ? __uint_as_float(sv[y]) : sx;
              if (t < lo || t > i) continue;
              const float p = t5::ex2(fmaf(sx, sc, neg));
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint4 w = tm::lds128(vb + (x + e) * 128 + (((c % 64) / 8 + h) ^ ((x + e) & 7)) * 16);
                const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  const float2 z = tc::unpack2<true>(ww[y]);
                  v[8 * h + 2 * y] = __float_as_uint(fmaf(p, z.x, __uint_as_float(v[8 * h + 2 * y])));
                  v[8 * h + 2 * y + 1] = __float_as_uint(fmaf(p, z.y, __uint_as_float(v[8 * h + 2 * y + 1])));
                }
              }
            }
          }
          __syncwarp();
          t5::st16(o_tm + c, v);
          t5::wait_st();
        }
        // both halves have read the scores before either's weights replace them
        arrive(by_done(q));
        ok = await_all(by_done(q), (uint32_t)hands & 1u);
        if (!ok) break;
        ++hands;
      }
#pragma unroll
      for (int c = 0; c < 32; c += 16) {
        t5::st16(h_tm + c, *reinterpret_cast<uint32_t(*)[16]>(ph + c));
        if constexpr (SPLIT) t5::st16(h_tm + 32 + c, *reinterpret_cast<uint32_t(*)[16]>(pl + c));
      }
      t5::wait_st();
      t5::fence_before();
      arrive(p_ready(buf));
    }
    // ---- the row's sum, then normalise and store this half's columns
    // (its own barrier: the last two products may both still run here, and
    // o_done's parity would not tell which of them is done)
    if (qe > qb && ok) ok = await_all(m_end(q), 0u);
    t5::fence_after();
    if (qe > qb && ok) {
      xs[(2 * q + half) * 128 + row] = l;   // every maximum is read: all weights are in
      arrive(pair(q, quad));
      ok = await_all(pair(q, quad), (uint32_t)(qe - qb) & 1u);
    }
    if (qe > qb && ok) {
      l += xs[(2 * q + 1 - half) * 128 + row];
      const float inv = 1.f / l;
      // Through shared memory (the queries are not needed any more), 4 KB per
      // warp, so that stores fill lines: 16 bytes per thread of a row each
      // took 3900 cycles a CTA, these 2000.
      constexpr int OSZ = SPLIT ? 4 : 2, CP = C::OROW / OSZ, CH = C::OROW / 16, RI = 32 / CH;
      const uint32_t stage = sbase + q * C::QB + (4 * half + quad) * 32 * C::OROW;
      auto slot = [&](int r, int c) { return stage + r * C::OROW + (c ^ (CH == 8 ? r & 7 : (r >> 1) & 3)) * 16; };
#pragma unroll 1
      for (int c = half * HC; c < half * HC + HC; c += CP) {
#pragma unroll
        for (int x = 0; x < CP; x += 16) {
          uint32_t v[16], w[16];
          t5::ld16(o_tm + c + x, v);
          t5::wait_ld();
#pragma unroll
          for (int e = 0; e < 16; e += OSZ == 2 ? 2 : 1) {
            if constexpr (SPLIT) w[e] = __float_as_uint(__uint_as_float(v[e]) * inv);
            else w[e / 2] = tc::pack2<true>(__uint_as_float(v[e]) * inv, __uint_as_float(v[e + 1]) * inv);
          }
#pragma unroll
          for (int e = 0; e < OSZ; ++e)
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(slot(lane, x * OSZ / 16 + e)), "r"(w[4 * e]),
                         "r"(w[4 * e + 1]), "r"(w[4 * e + 2]), "r"(w[4 * e + 3])
                         : "memory");
        }
        __syncwarp();
#pragma unroll 4
        for (int k = 0; k < CH; ++k) {
          const int r = k * RI + lane / CH, g = 32 * quad + r, iq = f + (g >> lrp);
          const uint4 w = tm::lds128(slot(r, lane % CH));
          if (iq < n)
            *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(a.out) +
                                      (((t0 + iq) * a.nq + head0 + (g & (rp - 1))) * HD + c) * OSZ + lane % CH * 16) = w;
        }
        __syncwarp();
      }
      if (i < n && a.lse && half == 0) a.lse[(t0 + i) * a.nq + head0 + (row & (rp - 1))] = fmaf(m, sc, log2f(l)) * CUDART_LN2_F;
    }
  }
  __syncwarp();
  t5::fence_before();
  __syncthreads();
  if (tid == 0 && *failed && a.err) atomicOr(a.err, KVQ_DEVERR_TIMEOUT);
  free_tmem();
}

// Rows [tokens][heads][hd] bf16: boxes of 64 dims x `heads_box` x `tok_box`.
bool row_map(CUtensorMap* m, const void* base, int hd, int heads, int64_t tokens, int64_t stride, int heads_box,
             int tok_box) {
  const cuuint64_t dim[3] = {(cuuint64_t)hd, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t str[2] = {(cuuint64_t)hd * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)heads_box, (cuuint32_t)tok_box};
  const cuuint32_t es[3] = {1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dim, str, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int HD, bool SPLIT>
cudaError_t launch_tc(const PromptArgs& a, const PromptMaps& maps, int rp, cudaStream_t st) {
  using C = PtCfg<HD>;
  auto kern = prompt_tc_kernel<HD, SPLIT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  const int per = C::NQ * 128 / rp;
  // Packed sequences of different lengths have at most total / per + num_seqs
  // tiles.  Where that is less than num_seqs times the longest one's, CTAs
  // look their tile up (2000 cycles) instead of starting in vain (2250 cycles
  // each, nothing else on the SM meanwhile): 24 prompts of 94 to 4096 tokens,
  // 9544 such CTAs of 12288, took 457 us, listed 383 us with the stores
  // staged.  The list holds kListed sequences' tile counts.
  const int64_t rows = (a.max_len + per - 1) / per, subs = a.nq / rp;
  const int64_t items = a.total / per + a.num_seqs;
  const bool listed = a.num_seqs <= kListed && items < rows * a.num_seqs && items * subs <= 0x7fffffff;
  kern<<<listed ? dim3((unsigned)(items * subs)) : dim3((unsigned)(subs * a.num_seqs), (unsigned)rows), C::THREADS,
         C::SMEM, st>>>(a, maps, rp, listed);
  return cudaGetLastError();
}

int rows_per_query(int rep) {
  int rp = 1;
  while (rp < 16 && rep % (2 * rp) == 0) rp *= 2;
  return rp;
}

}  // namespace

// BF16 rows on 16-byte boundaries (TMA) and a positive scale (the running
// maximum is taken of the raw scores); everything else runs prompt_fma_kernel.
bool prompt_tc_supported(int hd, const PromptArgs& a) {
  const int per = (hd == 256 ? 128 : 256) / rows_per_query(a.rep);
  return a.in_bf16 && a.vec && a.scale2 > 0.f && ((uintptr_t)a.out & 15) == 0 && encode_fn() != nullptr &&
         (a.max_len + per - 1) / per <= 65535 &&
         a.q_stride * 2 < ((int64_t)1 << 40) && a.k_stride * 2 < ((int64_t)1 << 40) && a.v_stride * 2 < ((int64_t)1 << 40);
}

cudaError_t launch_prompt_tc(int hd, const PromptArgs& a, cudaStream_t st) {
  PromptMaps maps;
  std::memset(&maps, 0, sizeof maps);
  const int rp = rows_per_query(a.rep);
  if (!row_map(&maps.q, a.q, hd, a.nq, a.total, a.q_stride, rp, 128 / rp) ||
      !row_map(&maps.k, a.k, hd, a.nkv, a.total, a.k_stride, 1, 128) ||
      !row_map(&maps.v, a.v, hd, a.nkv, a.total, a.v_stride, 1, 128))
    return cudaErrorInvalidValue;
  if (a.out_bf16)
    return hd == 64 ? launch_tc<64, false>(a, maps, rp, st) : hd == 128 ? launch_tc<128, false>(a, maps, rp, st)
                                                                       : launch_tc<256, false>(a, maps, rp, st);
  return hd == 64 ? launch_tc<64, true>(a, maps, rp, st) : hd == 128 ? launch_tc<128, true>(a, maps, rp, st)
                                                                    : launch_tc<256, true>(a, maps, rp, st);
}

}  // namespace kvq
