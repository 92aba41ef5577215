// attn_parts.cu -- attention over the parts of a shared-prefix call on the fifth-generation
// tensor cores (spec_verify_attn_shared; parts and units: internal.cuh, SharedSeq).
//
// A CTA works through a unit's keys in steps of 64. Row tile r (128 query rows) has a softmax
// warpgroup of its own, a score buffer S_r, a probability buffer P_r and an accumulator O_r
// in TMEM, and half of Q_r there; the other half of Q_r is in shared memory:
//   columns   O_r  128 each (64 used for d = 64)      P_r  32 each, 16-bit pairs
//             S_r   64 each                           Q_r  32 each: bf16 elements 0-63 of a
//                                                          row, or its E4M3 hi terms
// P has columns of its own, so S_r of the next step is issued as soon as the warpgroup has
// read this step's scores into registers, and runs under its softmax. What that leaves of
// TMEM holds half of Q; the score MMA reads the other half (bf16 elements 64-127, or the
// E4M3 lo terms) from shared memory. With both operands there an MMA of 64 columns takes 48
// clocks, with Q in TMEM 32 (measured; shared memory gives 128 bytes a clock).
//
//   RT = 2  the prefixes. Units of 256 rows, all 512 columns, one CTA per SM: each 128-key
//           K/V tile is read once for both row tiles, whose softmaxes alternate on the
//           tensor cores. Bound by those in this layout: a step of both row tiles is 1152
//           clocks of MMAs (bf16: 8 of the 16 score MMAs at 48 clocks, which with their half
//           of Q in TMEM would take 32: 128 clocks of the 1152), and takes 1150 to 1260; a
//           unit's start and end take 9 to 12 thousand more.
//   RT = 1  the sequences behind them. Units of 128 rows, 256 columns, 64-key tiles, two
//           independent lanes of work in a CTA (its halves, each with its own warps, shared
//           memory, TMEM and range of the line): the units are short (a few hundred keys) and
//           each starts with a read of Q and ends with a write of O, which the other half's
//           unit covers. Bound by neither HBM (2.5 TB/s alone in the first case below) nor
//           live tensor work: an MMA is issued for 128 rows however few of them live (36 at
//           most there), 576 clocks for a step of 64 keys, so 10.4 of the 18.8 thousand clocks
//           of a pair of units of nine tiles are MMAs, and 5.8 are starts and ends.
// The two run at the same time, each on a share of the SMs that the plan chooses (the one is
// bound by the tensor cores, the other by HBM): the sequences' kernel comes first, one CTA
// per SM, those without a range leave at once, and the prefixes' CTAs take the SMs that are
// free, the last of them those that the sequences leave. The sequences' CTAs come in pairs
// for the two SMs of a TPC: a CTA of the prefixes beside one of them took 15% longer.
//
//   warp 0   TMA producer of K tiles     warp 2   TMA producer of V tiles
//   warp 1   S issuer: S_r = Q_r K^T     warp 3   P V issuer: O_r += P_r V
//   then a softmax warpgroup per row tile: a thread owns one query row
//   then (E4M3 only) a warpgroup that decodes V tiles to f16
// A step's mathematics is that of attn_tc.cu (lazily rescaled online softmax, E4M3 keys met
// by Q as the exact sum of two E4M3 terms). The results are partials (O unnormalised, m, l)
// for combine_shared. Every wait is bounded as in attn_tc.cu.
//
// Measured (one after another, cold caches): 64 sequences of up to 1024 own positions over a
// prefix of 8192, Hq 32, Hkv 8, d 128, bf16: sequences 55-57 us (142 MB from HBM), prefixes 57
// us (36 MB, tensor pipe 61% busy); the whole call 65 us captured. 32 sequences of 16 rows over
// two prefixes of 32768, Hq 64, E4M3: prefixes 339 us (148 MB, tensor pipe 78% busy), the
// call 355-377 us (the power limit), 1.5 PFLOP/s.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.cuh"
#include "tc_util.cuh"

namespace sv {
namespace {

constexpr int HK = 64;  // keys per step
constexpr int SOFTMAX_WARP0 = 4;
constexpr int NST = 4;  // ring stages at most
constexpr int NCV = 2;  // E4M3: decoded V tiles

struct __align__(8) Bars {
  uint64_t k_full[NST], k_empty[NST], v_full[NST], v_empty[NST];
  uint64_t vc_full[NCV], vc_empty[NCV];
  uint64_t q_full[2], s_full[2], s_free[2], p_full[2], o_done[2];
  uint64_t s_final, pv_final;
  uint32_t tmem_base;
  int abort;
};

// The 128 threads of softmax warpgroup g meet; with `v`, whether it held for all of them.
__device__ __forceinline__ void wg_sync(int g) {
  asm volatile("barrier.sync %0, 128;" ::"r"(1 + g) : "memory");
}
__device__ __forceinline__ bool wg_and(int g, bool v) {
  __syncwarp();  // the reduction counts whole warps: arrive converged
  uint32_t o;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.red.and.pred q, %2, 128, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(o)
      : "r"((uint32_t)v), "r"(1 + g)
      : "memory");
  return o != 0;
}

template <int HD, bool F8, int RT>
struct Layout {
  static constexpr int KT = RT * HK;        // keys per tile
  static constexpr uint32_t COL_O = 0, COL_S = RT * 128, COL_P = RT * 192, COL_Q = RT * 224;
  static constexpr int CONV_WARP0 = SOFTMAX_WARP0 + 4 * RT;
  static constexpr int NCONV = 64 * RT;  // decoding threads
  static constexpr int BLK = KT * 128;      // one 128-byte-wide column block of a tile
  static constexpr int TILE = KT * HD * 2;  // one 16-bit tile
  static constexpr int RAW = F8 ? KT * HD : TILE;  // a tile as the cache has it
  static constexpr int HALVES = RT == 2 ? 1 : 2;
  static constexpr int NS = HD == 64 && RT == 2 ? 4 : 3;  // stages of each ring
  static constexpr int K = 0;
  static constexpr int V = K + NS * RAW;
  static constexpr int CV = V + NS * RAW;            // E4M3: decoded V tiles
  static constexpr int Q = CV + (F8 ? NCV * TILE : 0);
  static constexpr bool QS = F8 || HD == 128;        // part of Q is in shared memory
  static constexpr int QB = 128 * 128;               // bytes of it per row tile
  // a row tile's 128 bytes a row for reordering Q and O: its part of Q before that is
  // written and after it is used, or (E4M3, whose hi and lo terms come together) another
  static constexpr int STG = F8 ? Q + RT * QB : Q;
  static constexpr int TILES = (F8 ? STG : Q) + RT * QB;  // bytes of all that, per half
  static constexpr int BARS = HALVES * TILES;
  static constexpr int AMAX = BARS + HALVES * (int)sizeof(Bars);  // E4M3: each query row's
                                                                  // largest magnitude
  static constexpr size_t SMEM = (size_t)AMAX + (F8 ? HALVES * RT * 512 : 0);
  static_assert(!F8 || HD == 128, "E4M3 rows of one head are one 128-byte swizzle row");
  static_assert(TILES % 1024 == 0, "a half's tiles keep the swizzle's alignment");
  static_assert(SMEM <= 227 * 1024, "dynamic shared memory above the per-CTA limit");
  static constexpr int WARPS = CONV_WARP0 + (F8 ? NCONV / 32 : 0);  // of a half
  static constexpr int THREADS = 32 * WARPS * HALVES;
};

// D[tmem] (+)= A[smem] * B[smem], 16-bit and E4M3 operands
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}
__device__ __forceinline__ void mma_ss_e4m3(uint32_t d_tmem, uint64_t a, uint64_t b,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}

// True in one lane of a converged warp, always the same one.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(e));
  return e != 0;
}

// Two scaled Q elements (|x| < 256, at most 8 significant bits) as hi + lo E4M3 terms
// (attn_tc.cu, split_q_e4m3). f16 holds such an x and x - hi exactly down to its finest step
// of 2^-24; E4M3's is 2^-9.
__device__ __forceinline__ void split_q(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  asm("{\n .reg .b32 h, b;\n .reg .b16 c, d;\n cvt.rn.f16x2.f32 h, %3, %2;\n"
      " cvt.rn.satfinite.e4m3x2.f16x2 c, h;\n cvt.rn.f16x2.e4m3x2 b, c;\n"
      " sub.rn.f16x2 h, h, b;\n cvt.rn.satfinite.e4m3x2.f16x2 d, h;\n"
      " mov.b32 %0, {c, 0};\n mov.b32 %1, {d, 0};\n}\n"
      : "=r"(hi), "=r"(lo)
      : "f"(x0), "f"(x1));
}

// One unit's share of a CTA's range: its tiles [j0, j1).
struct Seg {
  SharedUnit d;
  int u, j0, j1;
};

// The units of a CTA's range [t0, t1) of the line, unit u0 holding its first tile. The first
// unit comes last: every CTA then begins at the first key of some unit (its whole units, then
// the head of the last, then the tail of the first, which begins about where the head ended),
// so that at any time all row tiles of a prefix are near the same keys and share them through
// L2. In the line's own order 128 prefix units of 134 MB read 1.0 GB from HBM.
struct Walk {
  int t0, t1, u0, u1;  // u1: the unit where the next range begins
  int k;               // units visited; -1: none is left
};

__device__ __forceinline__ bool seg_next(const AttnParams& p, int num_units, Walk& w, Seg& s) {
  if (w.k < 0) return false;
  for (int pass = 0; pass < 2; ++pass) {
    int u = w.u0 + 1 + w.k;
    if (pass == 1 || u > w.u1 || u >= num_units) {
      u = w.u0;
      w.k = -1;
    }
    const int4* src = reinterpret_cast<const int4*>(p.sunits + u);
    const int4 a = src[0], b = src[1], c = src[2];
    s.d = SharedUnit{(int64_t)(uint32_t)a.x | (int64_t)a.y << 32, a.z, a.w, b.x, b.y, b.z, b.w,
                     c.x, c.y, c.z, c.w};
    s.u = u;
    s.j0 = max(w.t0 - s.d.tile, 0);
    s.j1 = min(w.t1 - s.d.tile, s.d.nt);
    if (w.k < 0) break;
    if (s.j1 > 0) {  // (a unit at the very end of the range has no tile of it)
      ++w.k;
      break;
    }
  }
  return s.j1 > s.j0;
}
// Row tiles of a segment, and steps of its tile j.
template <int RT>
__device__ __forceinline__ int tiles_of(const Seg& s) {
  return RT == 2 && s.d.rows > MT ? 2 : 1;
}
template <int RT>
__device__ __forceinline__ int steps_of(const Seg& s, int j) {
  return RT == 2 && s.d.nkeys - j * RT * HK > HK ? 2 : 1;
}

template <int HD, bool F8, int RT>
__global__ void __launch_bounds__(Layout<HD, F8, RT>::THREADS, 1)
    attn_parts_kernel(const AttnParams p, const __grid_constant__ CUtensorMap tmk,
                      const __grid_constant__ CUtensorMap tmv) {
  using L = Layout<HD, F8, RT>;
  constexpr int KT = L::KT;
  constexpr uint32_t COL_O = L::COL_O, COL_S = L::COL_S,
                     COL_P = L::COL_P, COL_Q = L::COL_Q;
  extern __shared__ __align__(1024) uint8_t smem_cta[];  // 128-byte swizzled tiles: 1 KiB aligned
  const int cta_warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);  // uniform, and so are
  const int half = cta_warp / L::WARPS, warp = cta_warp % L::WARPS;    // the roles' branches
  const int tid = threadIdx.x - half * L::WARPS * 32, lane = tid & 31;
  const int worker = blockIdx.x * L::HALVES + half;  // whose range of the line this is
  uint8_t* smem = smem_cta + half * L::TILES;
  Bars* bars = (Bars*)(smem_cta + L::BARS) + half;
  volatile int* abort = &bars->abort;
  const Waiter wt{abort, p.flags, p.wait_limit > 0 ? p.wait_limit : TIMEOUT_CYCLES};
  // The sequences' kernel waits for the plan, hands what that wait made visible to it (the
  // plan, and the inputs, which are older) over to the prefixes' CTAs, and lets them start.
  // Those take it over before their first read, and wait for the sequences' kernel at their
  // end, so that the completion of theirs stands for both.
  if constexpr (RT == 1) {
    pdl_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) hand_over(p.handover, p.prefix_ctas);
    pdl_trigger();
  } else {
    pdl_trigger();
    bool late = false;
    if (threadIdx.x == 0 && !take_over(p.handover, wt.limit)) {
      atomicOr(p.flags, FLAG_TIMEOUT);
      late = true;
    }
    if (__syncthreads_or(late)) {
      pdl_wait();
      return;
    }
  }

  const int num_units = p.hdr->num_units;
  const int2 rb = p.cta_tab[worker], re = p.cta_tab[worker + 1];
  // a half without a range finds no unit
  const Walk walk0 = {rb.x, re.x, rb.y, re.y, rb.x < re.x && rb.y < num_units ? 0 : -1};
  const bool aligned = (saddr(smem_cta) & 1023) == 0;  // the swizzle phases below assume it
  const int cta_begin = p.cta_tab[blockIdx.x * L::HALVES].x;
  const int cta_end = p.cta_tab[(blockIdx.x + 1) * L::HALVES].x;
  if (cta_begin >= cta_end || !aligned) {
    if (!aligned && threadIdx.x == 0) atomicOr(p.flags, FLAG_ATTN_SHAPE);
    if constexpr (RT == 2) pdl_wait();
    return;  // uniform across the CTA
  }
  if (tid == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->k_empty[s], 1);  // the commit after the tile's last score MMA
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->v_empty[s], F8 ? L::NCONV : 1);  // decoded, or the last P V's commit
    }
    for (int s = 0; s < NCV; ++s) {
      mbar_init(&bars->vc_full[s], L::NCONV);
      mbar_init(&bars->vc_empty[s], 1);
    }
    for (int r = 0; r < 2; ++r) {
      mbar_init(&bars->q_full[r], 128);
      mbar_init(&bars->s_full[r], 1);
      mbar_init(&bars->s_free[r], 128);
      mbar_init(&bars->p_full[r], 128);
      mbar_init(&bars->o_done[r], 1);
    }
    mbar_init(&bars->s_final, 1);
    mbar_init(&bars->pv_final, 1);
    bars->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  Bars* bars0 = (Bars*)(smem_cta + L::BARS);
  if (cta_warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     saddr(&bars0->tmem_base)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem_cta = __shfl_sync(0xffffffffu, bars0->tmem_base, 0);
  const uint32_t tmem = tmem_cta + half * 256;
  auto wwait = [&](uint64_t* bar, uint32_t par) -> bool {  // by a whole warp
    return __all_sync(0xffffffffu, mbar_wait(bar, par, wt));
  };

  if (warp == 0 || warp == 2) {
    // ------------------------------------------------------------ TMA producers
    // A tile is KT / box boxes of box = min(block_size, KT) rows, lane n loading box n from
    // the page its table entry names. Entries are requested a group of tiles ahead (one per
    // lane); boxes without a key of the part load from a negative row, which fills them with
    // zeros.
    const bool is_k = warp == 0;
    const CUtensorMap* tm = is_k ? &tmk : &tmv;
    uint64_t* full = is_k ? bars->k_full : bars->v_full;
    uint64_t* empty = is_k ? bars->k_empty : bars->v_empty;
    const uint32_t ring = saddr(smem + (is_k ? L::K : L::V));
    if (lane == 0) asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)tm) : "memory");
    const int box = min(p.block_size, KT), nbox = KT / box, tg = 32 / nbox;
    const bool mine = lane < nbox;
    // A sequence's keys are read once, a prefix's by every row tile: the one stream must not
    // push the other out of L2.
    const uint64_t policy = RT == 1 ? policy_evict_first() : policy_evict_last();
    // test hook: the first tile of the range is never loaded, so every wait for it runs out
    const bool withhold = p.stall_first_tile != 0;
    if constexpr (RT == 2) fence_proxy_async_global();  // after take_over: K/V come by TMA
    Walk walk = walk0;
    Seg s;
    uint32_t it = 0;
    bool ok = true;
    while (ok && seg_next(p, num_units, walk, s)) {
      const int32_t* tab = p.block_table + (size_t)s.d.table_row * p.bt_stride;
      auto box_pos = [&](int j, int n) { return j * KT + n * box; };
      auto seen = [&](int pos) { return pos < s.d.nkeys && pos + box > s.d.start; };
      auto fetch = [&](int jg) -> int {  // this lane's entry of the group starting at tile jg
        const int j = jg + lane / nbox, pos = box_pos(j, lane % nbox);
        // (a plain load, as that of Q below: not the read-only path, which take_over does not order)
        return j < s.j1 && seen(pos) ? tab[(s.d.kbase + pos) >> p.bs_log2] : 0;
      };
      int ent_cur = fetch(s.j0), ent_nxt = fetch(s.j0 + tg);
      for (int j = s.j0; j < s.j1; ++j, ++it) {
        const uint32_t st = it % L::NS;
        const int q = (j - s.j0) % tg;
        if (q == 0 && j > s.j0) {  // the next group: its entries were requested tg tiles ago
          ent_cur = ent_nxt;
          ent_nxt = fetch(j + tg);
        }
        const int blk = __shfl_sync(0xffffffffu, ent_cur, q * nbox + lane % nbox);
        int grow = -box;
        const int pos = box_pos(j, lane % nbox);
        if (mine && seen(pos)) {
          if (blk < 0 || blk >= p.num_blocks) {  // a table entry outside the pool
            atomicOr(p.flags, FLAG_ATTN_SHAPE);
          } else {
            grow = blk * p.block_size + ((s.d.kbase + pos) & (p.block_size - 1));
          }
        }
        bool w = true;
        if (it >= L::NS && lane == 0) w = mbar_wait(&empty[st], ((it / L::NS) - 1) & 1, wt);
        if (!__shfl_sync(0xffffffffu, w, 0)) {
          ok = false;
          break;
        }
        if (withhold && it == 0) continue;
        if (lane == 0) mbar_expect_tx(&full[st], L::RAW);
        __syncwarp();
        if (mine) {
          const uint32_t dst = ring + st * L::RAW + lane * box * 128;
          if constexpr (F8) {
            tma_load_3d(dst, tm, &full[st], 0, s.d.g, grow, policy);
          } else {
#pragma unroll
            for (int c = 0; c < HD / 64; ++c)
              tma_load_3d(dst + c * L::BLK, tm, &full[st], c * 64, s.d.g, grow, policy);
          }
        }
      }
    }
    if (lane == 0) {
      // leave no copy in flight: wait (bounded) for the last fill of every stage
      for (uint32_t st = withhold ? 1 : 0; st < L::NS && st < it; ++st) {
        const uint32_t fills = (it - 1 - st) / L::NS + 1;
        const long long t0 = clock64();
        while (!mbar_try(&full[st], (fills - 1) & 1) && clock64() - t0 < TIMEOUT_CYCLES) {
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ S_r = Q_r K^T issuer
    // The whole warp walks the units and waits, and one elected lane issues: descriptors
    // stay in uniform registers. An issuer that is one divergent thread needs 45 clocks a
    // 64-column MMA, more than the 32 that the MMA takes.
    {
      constexpr uint32_t ID_S = F8 ? idesc_e4m3(HK) : idesc_bf16(HK, 0);
      // K and Q: K-major, 128-byte rows, 8-row groups 1024 B apart, 32 B per K step
      const uint64_t kdesc0 = smem_desc(saddr(smem + L::K), 16, 1024);
      const uint64_t qdesc0 = smem_desc(saddr(smem + L::Q), 16, 1024);
      Walk walk = walk0;
      Seg s;
      uint32_t it = 0, n[RT] = {}, units[RT] = {};
      bool ok = true;
      while (ok && seg_next(p, num_units, walk, s)) {
        if (lane == 0) {  // for the join: who holds the unit's first tile, who its last
          if (s.j0 == 0) p.unit_ctas[s.u].x = worker;
          if (s.j1 == s.d.nt) p.unit_ctas[s.u].y = worker;
        }
        __syncwarp();
        const int nr = tiles_of<RT>(s);
        for (int j = s.j0; ok && j < s.j1; ++j, ++it) {
          const uint32_t st = it % L::NS;
          if (!(ok = wwait(&bars->k_full[st], (it / L::NS) & 1))) break;
          const int steps = steps_of<RT>(s, j);
          for (int h = 0; ok && h < steps; ++h) {
            const uint64_t kd = kdesc0 + ((st * L::RAW + h * HK * 128) >> 4);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
              if (r >= nr) break;
              if ((j == s.j0 && h == 0 && !wwait(&bars->q_full[r], units[r] & 1)) ||
                  (n[r] >= 1 && !wwait(&bars->s_free[r], (n[r] - 1) & 1))) {
                ok = false;
                break;
              }
              fence_after();
              ++n[r];
              if (elect_one()) {
                const uint32_t d = tmem + COL_S + r * HK, a = tmem + COL_Q + r * 32;
                const uint64_t qd = qdesc0 + ((r * L::QB) >> 4);
                if constexpr (F8) {
#pragma unroll
                  for (int kk = 0; kk < HD / 32; ++kk) {
                    mma_ts_e4m3(d, a + kk * 8, kd + ((kk * 32) >> 4), ID_S, kk > 0 ? 1u : 0u);
                    mma_ss_e4m3(d, qd + ((kk * 32) >> 4), kd + ((kk * 32) >> 4), ID_S, 1u);
                  }
                } else {
#pragma unroll
                  for (int kk = 0; kk < HD / 16; ++kk) {
                    const uint64_t ko = ((kk >> 2) * L::BLK + (kk & 3) * 32) >> 4;
                    if (kk < 4)
                      mma_ts(d, a + kk * 8, kd + ko, ID_S, kk > 0 ? 1u : 0u);
                    else
                      mma_ss(d, qd + (((kk & 3) * 32) >> 4), kd + ko, ID_S, 1u);
                  }
                }
                mma_commit(&bars->s_full[r]);
              }
              __syncwarp();
            }
          }
          if (ok && elect_one()) mma_commit(&bars->k_empty[st]);
          __syncwarp();
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) units[r] += r < nr;
      }
      __syncwarp();
      if (elect_one()) {
        mma_commit(&bars->s_final);
        const long long t0 = clock64();
        while (!mbar_try(&bars->s_final, 0) && clock64() - t0 < TIMEOUT_CYCLES) {
        }
      }
      __syncwarp();
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------ O_r += P_r V issuer
    // In every step row tile 0 first: its warpgroup clears the V rows past the prefix.
    {
      constexpr uint32_t ID_PV = F8 ? idesc_f16(HD, 1) : idesc_bf16(HD, 1);
      // V: MN-major, 64-column blocks L::BLK apart (LBO), 8-key groups 1024 B apart (SBO)
      const uint64_t vdesc0 = smem_desc(saddr(smem + (F8 ? L::CV : L::V)), L::BLK, 1024);
      Walk walk = walk0;
      Seg s;
      uint32_t it = 0, n[RT] = {};
      bool ok = true;
      while (ok && seg_next(p, num_units, walk, s)) {
        const int nr = tiles_of<RT>(s);
        for (int j = s.j0; ok && j < s.j1; ++j, ++it) {
          constexpr uint32_t NV = F8 ? NCV : L::NS;
          const uint32_t st = it % NV;
          if (!(ok = wwait(F8 ? &bars->vc_full[st] : &bars->v_full[st], (it / NV) & 1))) break;
          const int steps = steps_of<RT>(s, j);
          for (int h = 0; ok && h < steps; ++h) {
            const uint64_t vd = vdesc0 + ((st * L::TILE + h * HK * 128) >> 4);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
              if (r >= nr) break;
              if (!(ok = wwait(&bars->p_full[r], n[r] & 1))) break;
              fence_after();
              ++n[r];
              if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < HK / 16; ++kk)
                  mma_ts(tmem + COL_O + r * 128, tmem + COL_P + r * 32 + kk * 8,
                         vd + ((kk * 16 * 128) >> 4), ID_PV,
                         (j == s.j0 && h == 0 && kk == 0) ? 0u : 1u);
                mma_commit(&bars->o_done[r]);
              }
              __syncwarp();
            }
          }
          if (ok && elect_one()) mma_commit(F8 ? &bars->vc_empty[st] : &bars->v_empty[st]);
          __syncwarp();
        }
      }
      __syncwarp();
      if (elect_one()) {
        mma_commit(&bars->pv_final);
        const long long t0 = clock64();
        while (!mbar_try(&bars->pv_final, 0) && clock64() - t0 < TIMEOUT_CYCLES) {
        }
      }
      __syncwarp();
    }
  } else if (warp < L::CONV_WARP0) {
    // ------------------------------------------------------------ softmax of row tile r
    const int r = (warp - SOFTMAX_WARP0) >> 2;
    const int wg = r + half;                // its barrier
    // the thread's row in its tile = its TMEM lane (a warp reaches the 32 lanes of its place
    // in the CTA modulo 4)
    const int rr = (cta_warp & 3) * 32 + lane;
    const uint32_t tq = tmem + ((uint32_t)((cta_warp & 3) * 32) << 16);
    Walk walk = walk0;
    Seg s;
    uint32_t it = 0, n = 0;  // tiles of the range; steps of this row tile
    bool ok = true;
    uint8_t* stg = smem + L::STG + r * L::QB;  // 128 bytes a row, 16-byte chunks swizzled
    uint8_t* qsm = smem + L::Q + r * L::QB;
    uint32_t* row_amax = reinterpret_cast<uint32_t*>(smem_cta + L::AMAX) + wg * MT;
    auto chunk_at = [](int row, int k) -> uint32_t { return row * 128 + ((k ^ (row & 7)) << 4); };
    // A warp whose wait failed stays until its warpgroup meets at the next unit, where all of
    // its warps leave together: none is left waiting at a barrier.
    while (seg_next(p, num_units, walk, s)) {
      if (r >= tiles_of<RT>(s)) {
        it += s.j1 - s.j0;
        continue;
      }
      if (!wg_and(wg, ok)) break;  // (and the staging rows of the last unit have been read)
      const int row = r * MT + rr;
      const bool live = row < s.d.rows;
      float sc = p.scale_log2;  // score scale in log2 units
      // ---- Q: 16-byte chunk qc of rows q0 + i * QI, whole rows side by side (coalesced);
      // rows that are none become zeros
      constexpr int QC = HD / 8, QI = 128 / QC;
      const int qc = rr % QC, q0 = rr / QC;
      // (window row, head of the group) of row q0 + i * QI, stepped from row to row
      int qw = (s.d.mt * RT * MT + r * MT + q0) / p.G, qh = (s.d.mt * RT * MT + r * MT + q0) % p.G;
      const int dw = QI / p.G, dh = QI % p.G;
      const uint4* qbase = reinterpret_cast<const uint4*>(
                               (const __nv_bfloat16*)p.q + (s.d.q_off * p.Hq + (int64_t)s.d.g * p.G) * HD) +
                           qc;
      auto load_q = [&](int i) -> uint4 {  // called for i = 0, 1, ..
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r * MT + q0 + i * QI < s.d.rows) v = qbase[(int64_t)(qw * p.Hq + qh) * QC];
        qw += dw;
        qh += dh;
        if (qh >= p.G) {
          qh -= p.G;
          ++qw;
        }
        return v;
      };
      if constexpr (F8) {
        // row x 2^e, its largest magnitude in [128, 256), as hi + lo (attn_tc.cu); 2^-e joins
        // the K scale in the score scale
#pragma unroll 1
        for (int i0 = 0; i0 < QC; i0 += 8) {
          uint4 v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = load_q(i0 + i);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            uint32_t amax = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) amax = max(amax, max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
            // the row's 16 lanes
            amax = lane < 16 ? __reduce_max_sync(0x0000ffffu, amax) : __reduce_max_sync(0xffff0000u, amax);
            const float f = exp2_of(q_exponent(amax));
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              split_q(__uint_as_float(w[k] << 16) * f, __uint_as_float(w[k] & 0xffff0000u) * f, hi[k], lo[k]);
            const int qr = q0 + (i0 + i) * QI;
            const uint32_t at = chunk_at(qr, qc >> 1) + (qc & 1) * 8;
            *reinterpret_cast<uint2*>(stg + at) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
            *reinterpret_cast<uint2*>(qsm + at) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
            if (qc == 0) row_amax[qr] = amax;
          }
        }
        wg_sync(wg);
        sc = q_row_scale(p.scale_log2 * p.kv_scale[s.d.g], row_amax[rr]);
      } else {
        uint4 v[QC];
#pragma unroll
        for (int i = 0; i < QC; ++i) v[i] = load_q(i);
        if (qc < 8) {
#pragma unroll
          for (int i = 0; i < QC; ++i)
            *reinterpret_cast<uint4*>(stg + chunk_at(q0 + i * QI, qc)) = v[i];
        }
        wg_sync(wg);
        if constexpr (L::QS) {  // the other half of the row waits for the first
          uint32_t rq[32];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<uint4*>(rq + 4 * k) = *reinterpret_cast<uint4*>(stg + chunk_at(rr, k));
          tmem_st32(tq + COL_Q + r * 32, rq);
          wg_sync(wg);
          if (qc >= 8) {
#pragma unroll
            for (int i = 0; i < QC; ++i)
              *reinterpret_cast<uint4*>(qsm + chunk_at(q0 + i * QI, qc - 8)) = v[i];
          }
        }
      }
      if constexpr (F8 || !L::QS) {
        uint32_t rq[32];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          *reinterpret_cast<uint4*>(rq + 4 * k) = *reinterpret_cast<uint4*>(stg + chunk_at(rr, k));
        tmem_st32(tq + COL_Q + r * 32, rq);
      }
      tmem_wait_st();
      if constexpr (L::QS) fence_proxy_async();
      fence_before();
      mbar_arrive(&bars->q_full[r]);
      // the row's last visible key (every row of a prefix sees all of it)
      const int last = RT == 2 ? s.d.nkeys - 1
                               : s.d.last0 + (s.d.mt * MT + (live ? row : 0)) / p.G;

      // V rows of step h of tile j that are no keys of the part
      auto clear_v = [&](int j, int h) -> bool {
        const int key0 = j * KT + h * HK;
        const int first = RT == 1 ? max(s.d.start - key0, 0) : 0, end = min(s.d.nkeys - key0, HK);
        if (!F8 && r == 0 && (first > 0 || end < HK)) {
          // V rows before and past the part's keys may hold any bits: zeros, so that P = 0
          // never meets non-finite data
          const uint32_t st = it % L::NS;
          if (!wwait(&bars->v_full[st], (it / L::NS) & 1)) return false;
          uint8_t* vt = smem + L::V + st * L::RAW + h * HK * 128;
          for (int q = rr; q < HK * 8 * (HD / 64); q += 128) {  // 16-byte chunks
            const int key = (q / 8) % HK;
            if (key < first || key >= end)
              *reinterpret_cast<uint4*>(vt + q / (8 * HK) * L::BLK + key * 128 + (q % 8) * 16) =
                  make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async();
        }
        return true;
      };

      float m_ref = -INFINITY, lh = 0.f;
      bool good = true;
      // A warp without a live row keeps the steps' order only: its rows of P are whatever they
      // were, and so its rows of O, which nobody reads. (A call of 128 sequences of 64 rows a
      // KV head 263 us instead of 266, one of 2 sequences 14.1 instead of 14.4. The same as a
      // condition inside the step's code cost 5%: it spilled.)
      int j = s.j0;
      if (RT == 1 && (cta_warp & 3) * 32 >= s.d.rows) {
        for (; good && j < s.j1; ++j, ++it, ++n) {
          good = wwait(&bars->s_full[r], n & 1);
          mbar_arrive(&bars->s_free[r]);
          if (good && n >= 1) good = wwait(&bars->o_done[r], (n - 1) & 1);
          if (good) good = clear_v(j, 0);
          if (good) mbar_arrive(&bars->p_full[r]);
        }
      }
      for (; good && j < s.j1; ++j, ++it) {
        const int steps = steps_of<RT>(s, j);
        for (int h = 0; h < steps; ++h, ++n) {
          if (!(good = wwait(&bars->s_full[r], n & 1))) break;
          fence_after();
          float x[HK];
          {
            uint32_t* raw = reinterpret_cast<uint32_t*>(x);
            tmem_ld32(tq + COL_S + r * HK, raw);
            tmem_ld32(tq + COL_S + r * HK + 32, raw + 32);
            tmem_wait_ld();
            reg_fence32(raw);
            reg_fence32(raw + 32);
          }
          fence_before();
          mbar_arrive(&bars->s_free[r]);  // the scores are in registers: the next S may start
          const int key0 = j * KT + h * HK;
          if (key0 + HK - 1 > last) {
            const int left = last - key0;
#pragma unroll
            for (int c = 0; c < HK; ++c)
              if (c > left) x[c] = -INFINITY;
          }
          if (RT == 1 && key0 < s.d.start) {
            const int low = s.d.start - key0;
#pragma unroll
            for (int c = 0; c < HK; ++c)
              if (c < low) x[c] = -INFINITY;
          }
          float m8[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            m8[e] = max3f(x[e], x[e + 8], x[e + 16]);
            m8[e] = max3f(m8[e], x[e + 24], x[e + 32]);
            m8[e] = max3f(m8[e], x[e + 40], x[e + 48]);
            m8[e] = fmaxf(m8[e], x[e + 56]);
          }
          const float mx = max3f(max3f(m8[0], m8[1], m8[2]), max3f(m8[3], m8[4], m8[5]),
                                 fmaxf(m8[6], m8[7]));
          const float mt = mx * sc;  // the step's maximum in log2 units (sc > 0)
          float alpha = 1.f;
          const bool grow = m_ref != -INFINITY && mt > m_ref + RESCALE_THRESHOLD;
          if (m_ref == -INFINITY) {
            m_ref = mt;
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
            fma2(x[2 * e], x[2 * e + 1], sc, nmu);
            x[2 * e] = ex2(x[2 * e]);
            x[2 * e + 1] = ex2(x[2 * e + 1]);
            add2(s8[(e & 3) * 2], s8[(e & 3) * 2 + 1], x[2 * e], x[2 * e + 1]);
          }
          lh += ((s8[0] + s8[1]) + (s8[2] + s8[3])) + ((s8[4] + s8[5]) + (s8[6] + s8[7]));
          uint32_t pk[HK / 2];
#pragma unroll
          for (int e = 0; e < HK / 2; ++e) pk[e] = pack_p<F8>(x[2 * e], x[2 * e + 1]);
          // P_r and O_r are free once the previous step's P V is complete
          if (n >= 1) {
            if (!(good = wwait(&bars->o_done[r], (n - 1) & 1))) break;
            fence_after();
          }
          if (__any_sync(0xffffffffu, grow)) {  // (never in a unit's first step)
#pragma unroll 1
            for (int c = 0; c < HD / 16; ++c) {
              uint32_t ro[16];
              tmem_ld16(tq + COL_O + r * 128 + c * 16, ro);
              tmem_wait_ld();
              reg_fence16(ro);
#pragma unroll
              for (int e = 0; e < 16; ++e) ro[e] = __float_as_uint(__uint_as_float(ro[e]) * alpha);
              tmem_st16(tq + COL_O + r * 128 + c * 16, ro);
            }
          }
          tmem_st32(tq + COL_P + r * 32, pk);
          tmem_wait_st();
          if (!(good = clear_v(j, h))) break;
          fence_before();
          mbar_arrive(&bars->p_full[r]);
        }
      }
      // the unit's last P V is complete: its partial result
      if (good) {
        good = wwait(&bars->o_done[r], (n - 1) & 1);
        fence_after();
      }
      if (!good) {
        ok = false;
        continue;
      }
      // 32 columns at a time through the staging rows (a warp's own 32), so that whole
      // 128-byte lines are written
      const size_t at = ((size_t)worker + s.u) * (RT * MT) + r * MT;
      const int w0 = (cta_warp & 3) * 32;
#pragma unroll 1
      for (int c = 0; c < HD / 32 && r * MT + w0 < s.d.rows; ++c) {  // (warps with live rows)
        uint32_t ro[32];
        tmem_ld32(tq + COL_O + r * 128 + c * 32, ro);
        tmem_wait_ld();
        reg_fence32(ro);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k)
          *reinterpret_cast<uint4*>(stg + chunk_at(rr, k)) = *reinterpret_cast<uint4*>(ro + 4 * k);
        __syncwarp();
        uint4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          v[i] = *reinterpret_cast<uint4*>(stg + chunk_at(w0 + i * 4 + lane / 8, lane % 8));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int o = w0 + i * 4 + lane / 8;
          if (r * MT + o < s.d.rows)
            *reinterpret_cast<uint4*>(p.part_o + (at + o) * HD + c * 32 + (lane % 8) * 4) = v[i];
        }
      }
      if (live) p.part_ml[at + rr] = make_float2(m_ref, lh);
      fence_before();  // TMEM reads above complete before the next unit's MMAs
    }
  }

  if constexpr (F8) {
    if (warp >= L::CONV_WARP0) {
      // ---------------------------------------------------------- E4M3 -> f16 V decoding
      // As in attn_tc.cu: raw 128-byte swizzled rows in, the 16-bit MN-major operand layout
      // out; rows that are no keys of the part become zeros.
      const int ct = (warp - L::CONV_WARP0) * 32 + lane;
      const int c = ct & 7;
      const int rw = (ct >> 3) ^ (c >> 2);
      const int ph = rw & 7;
      const uint32_t src_off = rw * 128 + ((c ^ ph) << 4);
      const uint32_t dst_off = (c >> 2) * L::BLK + rw * 128;
      const uint32_t w0 = ((2 * (c & 3)) ^ ph) << 4, w1 = ((2 * (c & 3) + 1) ^ ph) << 4;
      constexpr int CR = L::NCONV / 8, RSTEP = CR * 128;  // rows of a pass
      Walk walk = walk0;
      Seg s;
      uint32_t it = 0;
      bool ok = true;
      while (ok && seg_next(p, num_units, walk, s)) {
        for (int j = s.j0; j < s.j1; ++j, ++it) {
          const uint32_t rs = it % L::NS, cs = it % NCV;
          if (!mbar_wait(&bars->v_full[rs], (it / L::NS) & 1, wt) ||
              (it >= NCV && !mbar_wait(&bars->vc_empty[cs], ((it / NCV) - 1) & 1, wt))) {
            ok = false;
            break;
          }
          fence_after();
          const uint8_t* rsrc = smem + L::V + rs * L::RAW + src_off;
          uint8_t* cdst = smem + L::CV + cs * L::TILE + dst_off;
          uint4 w[KT / CR];
#pragma unroll
          for (int k = 0; k < KT / CR; ++k)
            w[k] = *reinterpret_cast<const uint4*>(rsrc + k * RSTEP);
          mbar_arrive(&bars->v_empty[rs]);
          const int lim = s.d.nkeys - j * KT, low = s.d.start - j * KT;  // the part's keys
#pragma unroll
          for (int k = 0; k < KT / CR; ++k) {
            uint32_t h[8];
            e4m3x4_to_f16x4(w[k].x, h[0], h[1]);
            e4m3x4_to_f16x4(w[k].y, h[2], h[3]);
            e4m3x4_to_f16x4(w[k].z, h[4], h[5]);
            e4m3x4_to_f16x4(w[k].w, h[6], h[7]);
            if (rw + CR * k >= lim || rw + CR * k < low) {
#pragma unroll
              for (int e = 0; e < 8; ++e) h[e] = 0u;
            }
            uint8_t* row = cdst + k * RSTEP;
            *reinterpret_cast<uint4*>(row + w0) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(row + w1) = make_uint4(h[4], h[5], h[6], h[7]);
          }
          fence_proxy_async();
          mbar_arrive(&bars->vc_full[cs]);
        }
      }
    }
  }

  fence_before();
  __syncthreads();
  fence_after();
  if (cta_warp == 1) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_cta),
                 "r"(512)
                 : "memory");
  }
  if constexpr (RT == 2) pdl_wait();
}

template <int HD, bool F8, int RT>
cudaError_t launch_hd(const AttnParams& p, cudaStream_t s) {
  using L = Layout<HD, F8, RT>;
  CUtensorMap mk, mv;
  const int box = p.block_size < L::KT ? p.block_size : L::KT;
  if (!kv_tensor_map(&mk, p.k, p.kv_rows, p.Hkv, HD, F8, box) ||
      !kv_tensor_map(&mv, p.v, p.kv_rows, p.Hkv, HD, F8, box))
    return cudaErrorInvalidValue;
  auto kernel = attn_parts_kernel<HD, F8, RT>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::SMEM);
  if (e != cudaSuccess) return e;
  if constexpr (RT == 1)
    return launch_pdl_pairs(kernel, dim3(p.n_ctas / 2), dim3(L::THREADS), L::SMEM, s, p, mk, mv);
  else
    return launch_pdl(kernel, dim3(p.n_ctas), dim3(L::THREADS), L::SMEM, s, p, mk, mv);
}

template <int RT>
cudaError_t launch_rt(const AttnParams& p, bool fp8, cudaStream_t s) {
  if (!attn_tc_supports(p.d, fp8) || p.block_size == 0) return cudaErrorNotSupported;
  if (fp8) return launch_hd<128, true, RT>(p, s);
  return p.d == 128 ? launch_hd<128, false, RT>(p, s) : launch_hd<64, false, RT>(p, s);
}

}  // namespace

cudaError_t launch_attn_prefixes(const AttnParams& p, bool fp8, cudaStream_t s) {
  return launch_rt<2>(p, fp8, s);
}
cudaError_t launch_attn_sequences(const AttnParams& p, bool fp8, cudaStream_t s) {
  return launch_rt<1>(p, fp8, s);
}

}  // namespace sv
