// attn_kv4_tc.cu -- verify attention over a 4-bit paged cache (format: kv4.cuh) on the
// fifth-generation tensor cores, for more query rows a KV head than attn_kv4.cu takes.
//
// The 4-bit rows reach the tensor cores as f16, which holds every value exactly: the codes
// come to shared memory by TMA, a warpgroup decodes each 128-key tile of K and of V into
// swizzled f16 operand tiles, and S = Q K^T and O += P V are tcgen05.mma kind::f16 with Q and P
// in TMEM. Units of 128 query rows, their line and the join: line.cuh, kv4_join. Two neighbouring
// CTAs take the two heads of a unit over the same keys, so that the second head's half of every
// 128-byte line comes from L2 (with heads read at other times, 8 sequences of 32768 positions
// and 8 heads took 700 MB from HBM where the codes and scales are 302).
//
//   warp 0       TMA producer: a stage is the K and V codes of a tile (boxes of one block each)
//   warp 1       S issuer           warp 3   P V issuer
//   warp 2       walks the line: the units of the CTA's range and where their rows lie in q and
//                out, a unit ahead, through a ring in shared memory that the others read
//   warps 4-11   softmax: warpgroup w owns keys [64 w, 64 w + 64) of every tile, with a score
//                buffer S_w, a probability buffer P_w, an accumulator O_w and a running
//                (reference, sum) of its own, so the two never wait for each other; they join
//                at the end of a unit. S_w of the next tile is issued as soon as this one's
//                scores are in registers.
//   warps 12-15  decode: a thread takes a key's row of K and of V. It fetches the row's block
//                scales itself (cp.async, three tiles ahead; nobody else reads them), zero for
//                keys outside the sequence, whose values are then zero whatever their codes.
// 16 warps, because 17 would leave a thread 96 registers (five warps on a scheduler) and a
// softmax thread holds 64 scores: with some 30 words spilled a tile took 3700 clocks, as next to
// 220 KB of shared memory L1 has nothing to hold them. At 128 registers 24 words are spilled still
// (d 128; none with d 64).
//
// Rounding: as in attn_kv4.cu (Q and P in f16, the sums those of the unrounded weights).
//
// At the end of a unit O goes out, and at its start Q comes in, through 2 KB of shared memory a
// warp, so that global memory sees 64-byte pieces of a row and not 16; the next unit's Q is
// requested before this unit's O is written. (Row by row in 16-byte pieces, a change of units
// took 20 thousand clocks, ten tiles' time.)
//
// Measured (d 128): a tile takes 2050 clocks, of which its MMAs take 1024 (issuing them alone
// would give 1.9 PFLOP/s); decoding and softmax warps issue 1200 instructions a scheduler a
// tile, half of their slots: the rest of its time is what its steps (S, scores to registers,
// exponentials, P V) wait for one another, as each warpgroup has one score buffer. 8 sequences of
// 32768 positions, 16 tokens, 64 query and 8 KV heads: 142 us with the join, 0.97 PFLOP/s; 16 of
// 8192, 32 tokens, 32 and 8 heads: 84 us, 0.82.
//
// TMEM columns: O_0, O_1 (128 each), S_0, S_1 (64 each), Q (64: f16 pairs), P_0, P_1 (32 each).
// Every wait is bounded as in attn_tc.cu.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.cuh"
#include "kv4.cuh"
#include "line.cuh"
#include "tc_util.cuh"

namespace sv {
namespace {

constexpr int KT = KV4_KT;        // keys per tile
constexpr int HK = KT / 2;        // keys per warpgroup per tile
constexpr int NR = 4;             // raw stages
constexpr int NSC = 4;            // tiles of block scales
constexpr int NCV = 2;            // decoded stages, K and V each
constexpr int NU = 4;             // units known ahead
constexpr int NTHREADS = 512;
constexpr int SOFT0 = 4, DEC0 = 12;  // first softmax and decoding warps
constexpr int NSOFT = 256, NDEC = 128;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t COL_O = 0, COL_S = 256, COL_Q = 384, COL_P = 448;
// Reference of a row: its largest score less SHIFT, so that f16 drops only weights below
// 2^-32 of the largest (attn_kv4.cu).
constexpr float SHIFT = 7.f;

struct __align__(8) Bars {
  uint64_t raw_full[NR], raw_empty[NR];
  uint64_t kc_full[NCV], kc_empty[NCV], vc_full[NCV], vc_empty[NCV];
  uint64_t s_full[2], s_free[2], p_full[2], o_done[2];
  uint64_t q_full, s_final, pv_final;
  uint32_t tmem_base;
  int abort;
  uint32_t qmax[2][128];  // start of a unit: each half row's largest magnitude
  uint64_t unit_full[NU], unit_empty[NU];
  struct Unit {
    int32_t live;         // 0: no more units
    int32_t b, g, T, D, j0, j1, kbase, rows, row0, begins, whole;
    int32_t row[MT];      // row of q and out, times Hq, plus its head
  } unit[NU];
  float xm[2][128], xl[2][128];  // end of a unit: each warpgroup's (reference, sum) per row
};

template <int HD>
struct Lay {
  static constexpr int RB = HD / 2;             // bytes of a row's codes
  static constexpr int SB = HD / 8;             // bytes of a row's block scales (K, then V)
  static constexpr int BLK = KT * 128;          // one 64-column block of a decoded tile
  static constexpr int TILE = KT * HD * 2;      // a decoded tile
  static constexpr int RAW = KT * RB;           // a tile's codes
  static constexpr int KC = 0;
  static constexpr int VC = KC + NCV * TILE;
  static constexpr int RK = VC + NCV * TILE;    // stage s: K codes at RK + 2 s RAW, V behind
  static constexpr int SC = RK + NR * 2 * RAW;
  static constexpr int STG = SC + NSC * KT * SB;  // 2 KB a softmax warp: 32 rows of 64 bytes
  static constexpr int BARS = STG + NSOFT / 32 * 2048;
  static constexpr size_t SMEM = (size_t)BARS + sizeof(Bars);
  static_assert(SMEM <= 227 * 1024, "dynamic shared memory above the per-CTA limit");
};

// True in one lane of a converged warp, always the same one.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(e));
  return e != 0;
}

// One arrival for a whole warp, after everything that its lanes did before.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if (elect_one()) mbar_arrive(bar);
}
template <int N>  // bytes: 16 or 8; not ok: zeros, nothing is read
__device__ __forceinline__ void cp_async_scales(uint32_t dst, const void* src, bool ok) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(ok ? 8 : 0) : "memory");
}

// Row r of a decoded tile from its codes (16-byte pieces, 32 elements each) and block scales, in
// the 128-byte swizzled layout of 64-column blocks.
template <int HD>
__device__ __forceinline__ void decode_row(uint8_t* tile, int r, const uint4 (&w)[HD / 32],
                                           const uint32_t (&scale)[HD / 64]) {
  using L = Lay<HD>;
  const uint32_t at = r * 128 + ((r & 7) << 4);  // 16-byte place c of the row: at ^ (c << 4)
#pragma unroll
  for (int c = 0; c < HD / 32; ++c) {
    const uint32_t f = e4m3x2_to_f16x2(c & 1 ? scale[c >> 1] >> 16 : scale[c >> 1] & 0xffffu);
    const uint32_t u[2] = {lo_twice(f), hi_twice(f)};  // the piece's two block scales, each twice
    const uint32_t q[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t h[4];
      e2m1x8_to_f16(q[e], h);
#pragma unroll
      for (int k = 0; k < 4; ++k) h[k] = hmul2(h[k], u[e >> 1]);
      *reinterpret_cast<uint4*>(tile + (at ^ (((c & 1) * 4 + e) << 4)) + (c >> 1) * L::BLK) =
          make_uint4(h[0], h[1], h[2], h[3]);
    }
  }
}

template <int HD>
__global__ void __launch_bounds__(NTHREADS, 1)
    attn_kv4_tc_kernel(const Kv4Attn p, const __grid_constant__ CUtensorMap tmk,
                       const __grid_constant__ CUtensorMap tmv) {
  using L = Lay<HD>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars* bars = (Bars*)(smem + L::BARS);
  volatile int* abort = &bars->abort;
  const Waiter wt{abort, p.flags, p.wait_limit > 0 ? p.wait_limit : TIMEOUT_CYCLES};
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform, and so are the roles
  pdl_wait();
  LineWalk walk;
  const int range = blockIdx.x / p.heads, hsel = blockIdx.x % p.heads;
  if (!line_begin<NTHREADS>(p, range, walk)) return;  // uniform across the CTA
  if (saddr(smem) & 1023) {      // the swizzle phases assume a 1 KiB-aligned base
    if (tid == 0) atomicOr(p.flags, FLAG_ATTN_SHAPE);
    return;
  }
  if (tid == 0) {
    for (int s = 0; s < NR; ++s) {
      mbar_init(&bars->raw_full[s], 1);
      mbar_init(&bars->raw_empty[s], NDEC / 32);
    }
    for (int s = 0; s < NCV; ++s) {
      mbar_init(&bars->kc_full[s], NDEC / 32);
      mbar_init(&bars->kc_empty[s], 1);
      mbar_init(&bars->vc_full[s], NDEC / 32);
      mbar_init(&bars->vc_empty[s], 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&bars->s_full[w], 1);
      mbar_init(&bars->s_free[w], NSOFT / 64);
      mbar_init(&bars->p_full[w], NSOFT / 64);
      mbar_init(&bars->o_done[w], 1);
    }
    mbar_init(&bars->q_full, NSOFT / 32);
    mbar_init(&bars->s_final, 1);
    mbar_init(&bars->pv_final, 1);
    for (int s = 0; s < NU; ++s) {
      mbar_init(&bars->unit_full[s], 1);
      mbar_init(&bars->unit_empty[s], NTHREADS / 32 - 1);
    }
    bars->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     saddr(&bars->tmem_base)),
                 "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bars->tmem_base, 0);
  auto wwait = [&](uint64_t* bar, uint32_t par) -> bool {  // by a whole warp
    return __all_sync(0xffffffffu, mbar_wait(bar, par, wt));
  };
  const int window = p.window;
  uint32_t it = 0, unit_i = 0;  // tiles and units that this warp has begun
  bool ok = true;
  Bars::Unit* s = nullptr;
  // The next unit, by a whole warp of any role but the walker's; false at the end. The unit
  // before is given back first.
  auto next_unit = [&]() -> bool {
    if (unit_i > 0) warp_arrive(&bars->unit_empty[(unit_i - 1) % NU]);
    s = &bars->unit[unit_i % NU];
    if (!wwait(&bars->unit_full[unit_i % NU], (unit_i / NU) & 1)) return false;
    ++unit_i;
    return s->live != 0;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    // A tile is KT / box boxes of box = min(block_size, KT) rows, lane n loading box n of K and
    // of V from the page its table entry names; entries are requested a group of tiles ahead,
    // one a lane. Boxes without a visible key load from a negative row, which fills them with
    // zeros.
    if (lane == 0) {
      asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&tmk) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&tmv) : "memory");
    }
    const int box = min(p.block_size, KT), nbox = KT / box, tg = 32 / nbox;
    while (ok && next_unit()) {
      const int T = s->T, nkeys = T + s->D + 1;
      const int kvis = first_visible_key(T, window);
      const int32_t* tab = p.block_table + (size_t)s->b * p.bt_stride;
      const int j0 = s->j0, j1 = s->j1, kbase = s->kbase, g = s->g;
      auto box_pos = [&](int j, int n) { return kbase + j * KT + n * box; };
      auto visible = [&](int pos) { return pos < nkeys && pos + box > kvis; };
      auto fetch = [&](int jg) -> int {  // this lane's entry of the group starting at tile jg
        const int j = jg + lane / nbox, pos = box_pos(j, lane % nbox);
        return j < j1 && visible(pos) ? __ldg(tab + (pos >> p.bs_log2)) : 0;
      };
      int ent_cur = fetch(j0), ent_nxt = fetch(j0 + tg);
      for (int j = j0; j < j1; ++j, ++it) {
        const uint32_t st = it % NR;
        const int q = (j - j0) % tg;
        if (q == 0 && j > j0) {
          ent_cur = ent_nxt;
          ent_nxt = fetch(j + tg);
        }
        const int blk = __shfl_sync(0xffffffffu, ent_cur, q * nbox + lane % nbox);
        int row = -box;
        if (lane < nbox && visible(box_pos(j, lane))) {
          if (blk >= 0 && blk < p.num_blocks)
            row = blk * p.block_size + (box_pos(j, lane) & (p.block_size - 1));
          else
            atomicOr(p.flags, FLAG_ATTN_SHAPE);  // a table entry outside the pool
        }
        if (it >= NR && !wwait(&bars->raw_empty[st], ((it / NR) - 1) & 1)) {
          ok = false;
          break;
        }
        const bool withheld = it == 0 && p.stall_first_tile;
        if (lane == 0 && !withheld) mbar_expect_tx(&bars->raw_full[st], 2 * L::RAW);
        __syncwarp();
        if (lane < nbox && !withheld) {
          const uint32_t dst = saddr(smem + L::RK + st * 2 * L::RAW) + lane * box * L::RB;
          tma_load_3d(dst, &tmk, &bars->raw_full[st], 0, g, row);
          tma_load_3d(dst + L::RAW, &tmv, &bars->raw_full[st], 0, g, row);
        }
      }
    }
    if (lane == 0) {  // leave no copy in flight (bounded)
      for (uint32_t st = p.stall_first_tile && it <= NR ? 1 : 0; st < NR && st < it; ++st) {
        const uint32_t par = ((it - 1 - st) / NR) & 1;
        const long long t0 = clock64();
        while (!mbar_try(&bars->raw_full[st], par) && clock64() - t0 < TIMEOUT_CYCLES) {
        }
      }
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ walker
    bool more = true;
    for (uint32_t n = 0; more; ++n) {
      LineSeg g;
      more = walk.next(p, g);
      if (n >= NU && !wwait(&bars->unit_empty[n % NU], ((n / NU) - 1) & 1)) break;
      Bars::Unit* d = &bars->unit[n % NU];
      if (more) {
        const int rows = min(MT, p.G * (g.D + 1) - g.mt * MT), head = g.g * p.heads + hsel;
        for (int i = lane; i < rows; i += 32) {
          const int rg = g.mt * MT + i;
          const int row = (int)((g.q_off + rg / p.G) * p.Hq + head * p.G + rg % p.G);
          d->row[i] = row;
#pragma unroll
          for (int c = 0; c < HD / 64; ++c)
            asm volatile("prefetch.global.L2 [%0];" ::"l"((const uint16_t*)p.q + (int64_t)row * HD + c * 64));
        }
        if (lane == 0) {
          d->b = g.b;
          d->g = head;
          d->T = g.T;
          d->D = g.D;
          d->j0 = g.j0;
          d->j1 = g.j1;
          d->kbase = g.kbase;
          d->rows = rows;
          d->row0 = g.mt * MT;
          d->begins = g.begins;
          d->whole = g.whole;
        }
      }
      if (lane == 0) d->live = more;
      warp_arrive(&bars->unit_full[n % NU]);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ S_w = Q K_w^T issuer
    constexpr uint32_t ID_S = idesc_f16(HK, 0);
    // K: K-major, 128-byte rows, 8-row groups 1024 B apart; 32 B per K step
    const uint64_t kdesc0 = smem_desc(saddr(smem + L::KC), 16, 1024);
    uint32_t seg_i = 0;
    while (ok && next_unit()) {
      if (!wwait(&bars->q_full, seg_i & 1)) break;
      fence_after();
      for (int n = s->j1 - s->j0; n > 0 && ok; --n, ++it) {
        const uint32_t st = it % NCV;
        ok = wwait(&bars->kc_full[st], (it / NCV) & 1);
        for (int w = 0; w < 2 && ok; ++w) {
          if (it >= 1 && !(ok = wwait(&bars->s_free[w], (it - 1) & 1))) break;
          fence_after();
          const uint64_t kd = kdesc0 + ((st * L::TILE + w * HK * 128) >> 4);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk)
              mma_ts(tmem + COL_S + w * HK, tmem + COL_Q + kk * 8,
                     kd + ((((kk >> 2) * L::BLK) + (kk & 3) * 32) >> 4), ID_S, kk > 0 ? 1u : 0u);
            mma_commit(&bars->s_full[w]);
            if (w == 1) mma_commit(&bars->kc_empty[st]);
          }
          __syncwarp();
        }
      }
      ++seg_i;
    }
    if (elect_one()) mma_commit(&bars->s_final);
    __syncwarp();
    const long long t0 = clock64();
    while (!mbar_try(&bars->s_final, 0) && clock64() - t0 < TIMEOUT_CYCLES) {
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------ O_w += P_w V_w issuer
    constexpr uint32_t ID_PV = idesc_f16(HD, 1);
    // V: MN-major, 64-column blocks L::BLK apart (LBO), 8-key groups 1024 B apart (SBO)
    const uint64_t vdesc0 = smem_desc(saddr(smem + L::VC), L::BLK, 1024);
    while (ok && next_unit()) {
      const int tiles = s->j1 - s->j0;
      for (int j = 0; j < tiles && ok; ++j, ++it) {
        const uint32_t st = it % NCV;
        ok = wwait(&bars->vc_full[st], (it / NCV) & 1);
        const uint64_t vd = vdesc0 + ((st * L::TILE) >> 4);
        for (int w = 0; w < 2 && ok; ++w) {
          if (!(ok = wwait(&bars->p_full[w], it & 1))) break;
          fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < HK / 16; ++kk)
              mma_ts(tmem + COL_O + w * 128, tmem + COL_P + w * (HK / 2) + kk * 8,
                     vd + (((w * HK + kk * 16) * 128) >> 4), ID_PV, (j == 0 && kk == 0) ? 0u : 1u);
            mma_commit(&bars->o_done[w]);
            if (w == 1) mma_commit(&bars->vc_empty[st]);
          }
          __syncwarp();
        }
      }
    }
    if (elect_one()) mma_commit(&bars->pv_final);
    __syncwarp();
    const long long t0 = clock64();
    while (!mbar_try(&bars->pv_final, 0) && clock64() - t0 < TIMEOUT_CYCLES) {
    }
  } else if (warp >= SOFT0 && warp < DEC0) {
    // ------------------------------------------------------------ softmax / epilogue
    const int wg = (warp - SOFT0) >> 2;
    const int r0w = (warp & 3) * 32;       // the warp's first query row = its quarter of the lanes
    const int r = r0w + lane;
    const uint32_t tq = tmem + ((uint32_t)r0w << 16);
    constexpr int OC = HD / 2;             // output columns of a warpgroup in the epilogue
    constexpr int QC = HD / 64;            // 64-byte pieces of its half of a Q row
    uint8_t* stg = smem + L::STG + (warp - SOFT0) * 2048;
    // 16-byte place c of row i in the staging area: rows are 64 bytes, pairs of rows exchange
    // places so that eight lanes, of one row each or four of two, meet every bank once
    auto place = [&](int i, int c) { return stg + i * 64 + ((c ^ ((i >> 1) & 3)) << 4); };
    const int si = lane >> 2, sc4 = lane & 3;  // row (of eight) and place of a coalesced access
    uint4 qv[QC][4];
    auto request_q = [&]() {  // of unit s
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = r0w + k * 8 + si;
        const bool have = i < s->rows;
        const uint4* src = reinterpret_cast<const uint4*>((const uint16_t*)p.q +
                                                          (int64_t)(have ? s->row[i] : 0) * HD + wg * (HD / 2)) + sc4;
#pragma unroll
        for (int c = 0; c < QC; ++c) qv[c][k] = have ? __ldg(src + c * 4) : make_uint4(0, 0, 0, 0);
      }
    };
    bool more = next_unit();
    if (more) request_q();
    while (true) {
      // The warpgroups leave together if a warp of either is without a unit (a wait gave up).
      if (!softmax_pair_and(more)) break;
      // Q row x 2^e -> f16 pairs in TMEM; each warpgroup writes its half, and they exchange the
      // halves' maxima
      uint32_t rq[HD / 4], amax = 0;
      {
#pragma unroll
        for (int c = 0; c < QC; ++c) {
#pragma unroll
          for (int k = 0; k < 4; ++k) *reinterpret_cast<uint4*>(place(k * 8 + si, sc4)) = qv[c][k];
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint4 v = *reinterpret_cast<const uint4*>(place(lane, k));
            rq[16 * c + 4 * k] = v.x;
            rq[16 * c + 4 * k + 1] = v.y;
            rq[16 * c + 4 * k + 2] = v.z;
            rq[16 * c + 4 * k + 3] = v.w;
          }
          __syncwarp();
        }
#pragma unroll
        for (int e = 0; e < HD / 4; ++e) amax = max(amax, max(rq[e] & 0x7fffu, (rq[e] >> 16) & 0x7fffu));
        bars->qmax[wg][r] = amax;
      }
      softmax_pair_and(true);
      amax = max(amax, bars->qmax[wg ^ 1][r]);
      const float f = exp2_of(q_exponent(amax));
#pragma unroll
      for (int e = 0; e < HD / 4; ++e)
        rq[e] = pack_f16(__uint_as_float(rq[e] << 16) * f, __uint_as_float(rq[e] & 0xffff0000u) * f);
      if constexpr (HD == 128)
        tmem_st32(tq + COL_Q + wg * 32, rq);
      else
        tmem_st16(tq + COL_Q + wg * 16, rq);
      tmem_wait_st();
      const float sc = q_row_scale(p.scale_log2 * p.kv_scale[s->g], amax);
      fence_before();
      warp_arrive(&bars->q_full);
      const int T = s->T - s->kbase;  // positions below: relative to kbase
      const int rows = s->rows, j0 = s->j0, j1 = s->j1;
      const int i_row = r < rows ? (s->row0 + r) / p.G : s->D;
      const int hi_row = T + i_row;            // the row's last visible key
      const int lo_row = hi_row + 1 - window;  // its first, under a sliding window

      float m_ref = -INFINITY, lh = 0.f;
      uint32_t it_last = 0;
      bool good = true;
      for (int j = j0; j < j1; ++j, ++it) {
        if (!good) continue;
        it_last = it;
        if (!(good = wwait(&bars->s_full[wg], it & 1))) continue;
        fence_after();
        float sv[HK];
        {
          uint32_t* raw = reinterpret_cast<uint32_t*>(sv);
#pragma unroll
          for (int c = 0; c < HK / 32; ++c) tmem_ld32(tq + COL_S + wg * HK + c * 32, raw + c * 32);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < HK / 32; ++c) reg_fence32(raw + c * 32);
        }
        fence_before();
        warp_arrive(&bars->s_free[wg]);  // the scores are in registers: the next S_w may start
        const int key0 = j * KT + wg * HK;
        if (key0 + HK - 1 > hi_row) {
          const int lim = hi_row - key0;
#pragma unroll
          for (int c = 0; c < HK; ++c)
            if (c > lim) sv[c] = -INFINITY;
        }
        if (window > 0 && key0 < lo_row) {
          const int low = lo_row - key0;
#pragma unroll
          for (int c = 0; c < HK; ++c)
            if (c < low) sv[c] = -INFINITY;
        }
        float m8[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          m8[e] = max3f(sv[e], sv[e + 8], sv[e + 16]);
          m8[e] = max3f(m8[e], sv[e + 24], sv[e + 32]);
          m8[e] = max3f(m8[e], sv[e + 40], sv[e + 48]);
          m8[e] = fmaxf(m8[e], sv[e + 56]);
        }
        const float mx = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])),
                               fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
        const float mt = mx * sc - SHIFT;  // this half tile's reference, log2 units (sc > 0)
        float alpha = 1.f;
        const bool grow = m_ref != -INFINITY && mt > m_ref + RESCALE_THRESHOLD;
        if (m_ref == -INFINITY) {
          m_ref = mt;  // O_w holds nothing yet for this row
        } else if (grow) {
          alpha = ex2(m_ref - mt);
          lh *= alpha;
          m_ref = mt;
        }
        const float nmu = m_ref == -INFINITY ? 0.f : -m_ref;
        float s8[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) s8[e] = 0.f;
#pragma unroll
        for (int e = 0; e < HK / 2; ++e) {
          fma2(sv[2 * e], sv[2 * e + 1], sc, nmu);
          sv[2 * e] = ex2(sv[2 * e]);
          sv[2 * e + 1] = ex2(sv[2 * e + 1]);
          add2(s8[(e & 3) * 2], s8[(e & 3) * 2 + 1], sv[2 * e], sv[2 * e + 1]);
        }
        lh += ((s8[0] + s8[1]) + (s8[2] + s8[3])) + ((s8[4] + s8[5]) + (s8[6] + s8[7]));
        uint32_t pk[HK / 2];
#pragma unroll
        for (int e = 0; e < HK / 2; ++e) pk[e] = pack_f16(sv[2 * e], sv[2 * e + 1]);
        // O_w and P_w are reused once this warpgroup's previous P V is complete
        if (it >= 1) {
          if (!(good = wwait(&bars->o_done[wg], (it - 1) & 1))) continue;
          fence_after();
        }
        if (__any_sync(0xffffffffu, grow)) {  // (never on a unit's first tile)
#pragma unroll 1
          for (int c = 0; c < HD / 16; ++c) {
            uint32_t ro[16];
            tmem_ld16(tq + COL_O + wg * 128 + c * 16, ro);
            tmem_wait_ld();
            reg_fence16(ro);
#pragma unroll
            for (int e = 0; e < 16; ++e) ro[e] = __float_as_uint(__uint_as_float(ro[e]) * alpha);
            tmem_st16(tq + COL_O + wg * 128 + c * 16, ro);
          }
        }
        tmem_st32(tq + COL_P + wg * (HK / 2), pk);
        tmem_wait_st();
        fence_before();
        warp_arrive(&bars->p_full[wg]);
      }
      if (good) {
        good = wwait(&bars->o_done[wg], it_last & 1);
        if (good) fence_after();
      }
      bars->xm[wg][r] = m_ref;
      bars->xl[wg][r] = lh;
      if (!softmax_pair_and(good)) break;
      fence_after();  // the other warpgroup's accumulator is complete too

      // ---- epilogue: join the two accumulators; this warpgroup's half of the columns
      const Bars::Unit* o = s;
      const bool whole = o->whole;
      const size_t part0 = ((size_t)(2 * range + o->begins) * p.heads + hsel) * MT;
      // (the unit is given back by next_unit: what is needed of it below is read first)
      int orow[4];  // the rows of this thread's coalesced accesses
#pragma unroll
      for (int k = 0; k < 4; ++k) orow[k] = o->row[min(r0w + k * 8 + si, rows - 1)];
      const int my_row = o->row[min(r, rows - 1)];
      const float vs = p.kv_scale[p.Hkv + o->g];
      more = next_unit();
      if (more) request_q();
      const float m0 = bars->xm[0][r], m1 = bars->xm[1][r];
      const float m = fmaxf(m0, m1);
      const float a0 = m0 == -INFINITY ? 0.f : ex2(m0 - m);
      const float a1 = m1 == -INFINITY ? 0.f : ex2(m1 - m);
      // (a sum without a reference is 0, or NaN, which stays)
      const float l = (m0 == -INFINITY ? bars->xl[0][r] : a0 * bars->xl[0][r]) +
                      (m1 == -INFINITY ? bars->xl[1][r] : a1 * bars->xl[1][r]);
      const float inv = whole ? vs / l : 1.f;
      auto joined = [&](int col, float (&v)[16]) {  // 16 columns of this thread's row
        uint32_t x0[16], x1[16];
        tmem_ld16(tq + COL_O + col, x0);
        tmem_ld16(tq + COL_O + 128 + col, x1);
        tmem_wait_ld();
        reg_fence16(x0);
        reg_fence16(x1);
#pragma unroll
        for (int e = 0; e < 16; ++e)  // an accumulator without keys is skipped
          v[e] = ((a0 != 0.f ? a0 * __uint_as_float(x0[e]) : 0.f) +
                  (a1 != 0.f ? a1 * __uint_as_float(x1[e]) : 0.f)) * inv;
      };
      // 64 bytes of each of the warp's rows: from the rows' threads to whole pieces
      auto flush = [&](uint8_t* base, int row_bytes, bool by_row) {
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = k * 8 + si;
          const uint4 v = *reinterpret_cast<const uint4*>(place(i, sc4));
          if (r0w + i < rows)
            *reinterpret_cast<uint4*>(base + (int64_t)(by_row ? r0w + i : orow[k]) * row_bytes + sc4 * 16) = v;
        }
        __syncwarp();
      };
      if (whole) {
#pragma unroll 1
        for (int c = 0; c < OC / 32; ++c) {  // 32 columns of bf16
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float v[16];
            joined(wg * OC + c * 32 + h * 16, v);
#pragma unroll
            for (int e = 0; e < 2; ++e)
              *reinterpret_cast<uint4*>(place(lane, 2 * h + e)) =
                  make_uint4(pack_bf16(v[8 * e], v[8 * e + 1]), pack_bf16(v[8 * e + 2], v[8 * e + 3]),
                             pack_bf16(v[8 * e + 4], v[8 * e + 5]), pack_bf16(v[8 * e + 6], v[8 * e + 7]));
          }
          flush((uint8_t*)p.out + (wg * OC + c * 32) * 2, HD * 2, false);
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < OC / 16; ++c) {
          float v[16];
          joined(wg * OC + c * 16, v);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<float4*>(place(lane, e)) = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
          flush((uint8_t*)(p.part_o + part0 * HD + wg * OC + c * 16), HD * 4, true);
        }
      }
      if (r < rows && wg == 0) {
        if (!whole) p.part_ml[part0 + r] = make_float2(m, l);
        else if (p.lse) p.lse[my_row] = (m + log2f(l)) * 0.6931471805599453f;
      }
      fence_before();  // TMEM reads above complete before the next unit's MMAs
    }
  } else if (warp >= DEC0) {
    // ------------------------------------------------------------ decode
    const int r = (warp - DEC0) * 32 + lane;  // this thread's key of every tile
    uint8_t* ssc = smem + L::SC + r * L::SB;
    const uint8_t* rsrc = smem + L::RK + r * L::RB;
    // codes' 16-byte pieces as TMA swizzled them: the piece's index XOR address bits 7.. (64-
    // byte rows: two bits, 32-byte rows: one)
    const int sw = HD == 128 ? (r >> 1) & 3 : (r >> 2) & 1;
    while (ok && next_unit()) {
      const int nkeys = s->T + s->D + 1;
      const int kvis = first_visible_key(s->T, window);
      const int32_t* tab = p.block_table + (size_t)s->b * p.bt_stride;
      const uint8_t* scales = (const uint8_t*)p.scales + s->g * L::SB;
      const int64_t row_bytes = (int64_t)p.Hkv * L::SB;
      const int j0 = s->j0, j1 = s->j1, pos0 = s->kbase + r;
      auto entry = [&](int j) -> int {  // the page of this thread's key of tile j
        const int pos = pos0 + j * KT;
        return j < j1 && pos < nkeys && pos >= kvis ? __ldg(tab + (pos >> p.bs_log2)) : -1;
      };
      auto fetch = [&](int j, int blk) {  // its block scales, into the ring
        const int pos = pos0 + j * KT;
        const bool have = blk >= 0 && blk < p.num_blocks;
        const int row = have ? (blk << p.bs_log2) + (pos & (p.block_size - 1)) : 0;
        cp_async_scales<L::SB>(saddr(ssc + (j % NSC) * KT * L::SB), scales + row * row_bytes, have);
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      {
        int e0[NSC - 1];
#pragma unroll
        for (int k = 0; k < NSC - 1; ++k) e0[k] = entry(j0 + k);
#pragma unroll
        for (int k = 0; k < NSC - 1; ++k) fetch(j0 + k, e0[k]);
      }
      int ent = entry(j0 + NSC - 1);
      for (int j = j0; j < j1; ++j, ++it) {
        const uint32_t rs = it % NR, cs = it % NCV;
        fetch(j + NSC - 1, ent);  // (its ring place was read a tile ago)
        ent = entry(j + NSC);
        const uint32_t free_par = ((it / NCV) - 1) & 1;
        if (!(ok = wwait(&bars->raw_full[rs], (it / NR) & 1) &&
                   (it < NCV || wwait(&bars->kc_empty[cs], free_par))))
          break;
        asm volatile("cp.async.wait_group %0;" ::"n"(NSC - 1) : "memory");
        uint32_t sk[HD / 64], sv[HD / 64];  // E4M3 scales of K and of V
        const uint8_t* sp = ssc + (j % NSC) * KT * L::SB;
        if constexpr (HD == 128) {
          const uint4 v = *reinterpret_cast<const uint4*>(sp);
          sk[0] = v.x;
          sk[1] = v.y;
          sv[0] = v.z;
          sv[1] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(sp);
          sk[0] = v.x;
          sv[0] = v.y;
        }
        uint4 wk[HD / 32], wv[HD / 32];
        const uint8_t* src = rsrc + rs * 2 * L::RAW;
#pragma unroll
        for (int c = 0; c < HD / 32; ++c) {
          wk[c] = *reinterpret_cast<const uint4*>(src + ((c ^ sw) << 4));
          wv[c] = *reinterpret_cast<const uint4*>(src + L::RAW + ((c ^ sw) << 4));
        }
        decode_row<HD>(smem + L::KC + cs * L::TILE, r, wk, sk);
        // for the MMAs, and for the TMA that writes the stage next: it may not overtake the reads
        // above (without a fence before this arrival it did, about once in a thousand units)
        fence_proxy_async();
        warp_arrive(&bars->kc_full[cs]);
        warp_arrive(&bars->raw_empty[rs]);
        if (!(ok = it < NCV || wwait(&bars->vc_empty[cs], free_par))) break;
        decode_row<HD>(smem + L::VC + cs * L::TILE, r, wv, sv);
        fence_proxy_async();
        warp_arrive(&bars->vc_full[cs]);
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
  }

  fence_before();
  __syncthreads();
  fence_after();
  pdl_trigger();
  if (warp == 1) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(TMEM_COLS)
                 : "memory");
  }
}

// ---------------------------------------------------------------- host side

template <int HD>
cudaError_t launch_hd(const Kv4Attn& p, cudaStream_t s) {
  using L = Lay<HD>;
  CUtensorMap mk, mv;
  const int box = min(p.block_size, KT);
  const int64_t rows = p.num_blocks * p.block_size;
  if (!kv4_tensor_map(&mk, p.k, rows, p.Hkv, HD, box) ||
      !kv4_tensor_map(&mv, p.v, rows, p.Hkv, HD, box))
    return cudaErrorInvalidValue;
  auto kernel = attn_kv4_tc_kernel<HD>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(p.n_ctas * p.heads), dim3(NTHREADS), L::SMEM, s, p, mk, mv);
}

}  // namespace

cudaError_t launch_attn_kv4_tc(const Kv4Attn& p, cudaStream_t s) {
  return p.d == 128 ? launch_hd<128>(p, s) : launch_hd<64>(p, s);
}

}  // namespace sv
