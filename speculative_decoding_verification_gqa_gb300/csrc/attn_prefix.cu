// attn_prefix.cu -- attention of a group's rows over their shared prefix on the
// fifth-generation tensor cores: the compute-bound part of spec_verify_attn_shared.
//
// A unit is (group, KV head, pair of 128-row tiles): up to 256 of the G * sum W query rows
// of the group's sequences. Its CTA reads each 128-key K/V tile once for both row tiles and
// works through it in steps of 64 keys. Row tile r has a softmax warpgroup of its own, a
// score buffer S_r, a probability buffer P_r and an accumulator O_r in TMEM:
//   columns   0-255  O_0, O_1 (128 each; 64 used for d = 64)
//           256-383  S_0, S_1 (64 each)      384-447  P_0, P_1 (32 each, 16-bit pairs)
//           448-511  Q_0, Q_1 (32 each): bf16 elements 0-63 of a row, or the E4M3 hi term
// P has columns of its own, so S_r of the next step is issued as soon as the warpgroup has
// read this step's scores into registers and runs under its softmax. What that leaves of
// TMEM holds half of Q; the other half (bf16 elements 64-127, or the E4M3 lo term) is read
// by the score MMA from shared memory. Both operands from shared memory would need 192 bytes
// a clock of it at N = 64, half of Q in TMEM brings a step's shared-memory traffic (scores,
// P V and the TMA writes) to about 128.
//
//   warp 0   TMA producer of K tiles     warp 2   TMA producer of V tiles
//   warp 1   S issuer: S_r = Q_r K^T, r = 0, 1 (one thread)
//   warp 3   P V issuer: O_r += P_r V, r = 0, 1 (one thread)
//   warps 4-7, 8-11   softmax of row tile 0, 1: a thread owns one query row
//   warps 12-15 (E4M3 only)  decode V tiles to f16
// A step's mathematics is that of attn_tc.cu (lazily rescaled online softmax, E4M3 keys met
// by Q as the exact sum of two E4M3 terms); the prefix needs no causal mask. The results are
// partials (O unnormalised, m, l) for combine_shared. Every wait is bounded as in attn_tc.cu.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.cuh"
#include "tc_util.cuh"

namespace sv {
namespace {

constexpr int KT = 128;  // keys per tile
constexpr int HK = 64;   // keys per step
constexpr int NTHREADS = 384;
constexpr int SOFTMAX_WARP0 = 4;
constexpr int CONV_WARP0 = 12;
constexpr int NCONV = 128;
constexpr int NST = 4;   // ring stages at most
constexpr int NCV = 2;   // E4M3: decoded V tiles
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t COL_O = 0, COL_S = 256, COL_P = 384, COL_Q = 448;

struct __align__(8) Bars {
  uint64_t k_full[NST], k_empty[NST], v_full[NST], v_empty[NST];
  uint64_t vc_full[NCV], vc_empty[NCV];
  uint64_t q_full[2], s_full[2], s_free[2], p_full[2], o_done[2];
  uint64_t s_final, pv_final;
  uint32_t tmem_base;
  int abort;
};

template <int HD, bool F8>
struct Layout {
  static constexpr int BLK = KT * 128;      // one 128-byte-wide column block of a tile
  static constexpr int TILE = KT * HD * 2;  // one 16-bit tile
  static constexpr int RAW = F8 ? KT * HD : TILE;  // a tile as the cache has it
  static constexpr int NS = (F8 || HD == 64) ? 4 : 3;  // stages of each ring
  static constexpr int K = 0;
  static constexpr int V = K + NS * RAW;
  static constexpr int CV = V + NS * RAW;            // E4M3: decoded V tiles
  static constexpr int Q = CV + (F8 ? NCV * TILE : 0);
  static constexpr bool QS = F8 || HD == 128;        // part of Q is in shared memory
  static constexpr int QB = QS ? 128 * 128 : 0;      // bytes of it per row tile
  static constexpr int BARS = Q + 2 * QB;
  static constexpr size_t SMEM = (size_t)BARS + sizeof(Bars);
  static_assert(!F8 || HD == 128, "E4M3 rows of one head are one 128-byte swizzle row");
  static_assert(SMEM <= 227 * 1024, "dynamic shared memory above the per-CTA limit");
  static constexpr int THREADS = NTHREADS + (F8 ? NCONV : 0);
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

// Four scaled Q elements as hi + lo E4M3 terms (attn_tc.cu, split_q_e4m3).
__device__ __forceinline__ void split_q(const float* x, uint32_t& whi, uint32_t& wlo) {
  const uint32_t h01 = f32x2_to_e4m3x2(x[0], x[1]), h23 = f32x2_to_e4m3x2(x[2], x[3]);
  const float2 d01 = e4m3x2_to_f32x2(h01), d23 = e4m3x2_to_f32x2(h23);
  const uint32_t l01 = f32x2_to_e4m3x2(x[0] - d01.x, x[1] - d01.y);
  const uint32_t l23 = f32x2_to_e4m3x2(x[2] - d23.x, x[3] - d23.y);
  whi = h01 | (h23 << 16);
  wlo = l01 | (l23 << 16);
}

// One unit's share of a CTA's range: tiles [j0, j1) of part v, KV head g, row pair mt.
struct Seg {
  int u, v, g, mt, j0, j1;
  int nkeys, rows, table_row;  // of the part; rows: live query rows of the pair
  int64_t q_off;
};

__device__ __forceinline__ bool seg_next(const AttnParams& p, int num_units, int& t, int t_end,
                                         int& u, Seg& s) {
  if (t >= t_end || u >= num_units) return false;
  const int4 info = p.units[u];
  const int ub = p.ubeg[u], ue = p.ubeg[u + 1];
  const SharedSeq part = p.parts[info.x];
  s.u = u;
  s.v = info.x;
  s.g = info.y;
  s.mt = info.z;
  s.j0 = t - ub;
  s.j1 = min(t_end, ue) - ub;
  s.nkeys = part.nkeys;
  s.rows = min(2 * MT, p.G * part.rows - info.z * 2 * MT);
  s.table_row = part.table_row;
  s.q_off = part.q_off;
  if (s.j1 <= s.j0) return false;
  t = ub + s.j1;
  ++u;
  return true;
}
// Row tiles of a segment, and steps of its tile j.
__device__ __forceinline__ int tiles_of(const Seg& s) { return s.rows > MT ? 2 : 1; }
__device__ __forceinline__ int steps_of(const Seg& s, int j) {
  return s.nkeys - j * KT > HK ? 2 : 1;
}

template <int HD, bool F8>
__global__ void __launch_bounds__(F8 ? NTHREADS + NCONV : NTHREADS, 1)
    attn_prefix_kernel(const AttnParams p, const __grid_constant__ CUtensorMap tmk,
                       const __grid_constant__ CUtensorMap tmv) {
  using L = Layout<HD, F8>;
  extern __shared__ __align__(1024) uint8_t smem[];  // 128-byte swizzled tiles: 1 KiB aligned
  Bars* bars = (Bars*)(smem + L::BARS);
  volatile int* abort = &bars->abort;
  const Waiter wt{abort, p.flags, p.wait_limit > 0 ? p.wait_limit : TIMEOUT_CYCLES};
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform: the roles' branches too
  pdl_wait();     // the plan of this call is complete
  pdl_trigger();  // the sequences' kernel, which needs the plan only, may fill SMs as they empty

  const int num_units = p.hdr->num_units;
  const int2 rb = p.cta_tab[blockIdx.x], re = p.cta_tab[blockIdx.x + 1];
  const int t_begin = rb.x, t_end = re.x, u_first = rb.y;
  if (t_begin >= t_end) return;  // uniform across the CTA
  if (saddr(smem) & 1023) {      // the swizzle phases below assume a 1 KiB-aligned base
    if (tid == 0) atomicOr(p.flags, FLAG_ATTN_SHAPE);
    return;
  }
  if (tid == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->k_empty[s], 1);  // the commit after the tile's last score MMA
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->v_empty[s], F8 ? NCONV : 1);  // decoded, or the last P V's commit
    }
    for (int s = 0; s < NCV; ++s) {
      mbar_init(&bars->vc_full[s], NCONV);
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

  if (warp == 0 || warp == 2) {
    // ------------------------------------------------------------ TMA producers
    // A tile is KT / box boxes of box = min(block_size, KT) rows, lane n loading box n from
    // the page its table entry names. Entries are requested a group of tiles ahead (one per
    // lane); boxes past the prefix load from a negative row, which fills them with zeros.
    const bool is_k = warp == 0;
    const CUtensorMap* tm = is_k ? &tmk : &tmv;
    uint64_t* full = is_k ? bars->k_full : bars->v_full;
    uint64_t* empty = is_k ? bars->k_empty : bars->v_empty;
    const uint32_t ring = saddr(smem + (is_k ? L::K : L::V));
    if (lane == 0) asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)tm) : "memory");
    const int box = min(p.block_size, KT), nbox = KT / box, tg = 32 / nbox;
    const bool mine = lane < nbox;
    // test hook: the first tile of the range is never loaded, so every wait for it runs out
    const bool withhold = p.stall_first_tile != 0;
    int t = t_begin, u = u_first;
    Seg s;
    uint32_t it = 0;
    bool ok = true;
    while (ok && seg_next(p, num_units, t, t_end, u, s)) {
      const int32_t* tab = p.block_table + (size_t)s.table_row * p.bt_stride;
      auto box_pos = [&](int j, int n) { return j * KT + n * box; };
      auto fetch = [&](int jg) -> int {  // this lane's entry of the group starting at tile jg
        const int j = jg + lane / nbox, pos = box_pos(j, lane % nbox);
        return j < s.j1 && pos < s.nkeys ? __ldg(tab + (pos >> p.bs_log2)) : 0;
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
        if (mine && pos < s.nkeys) {
          if (blk < 0 || blk >= p.num_blocks) {  // a table entry outside the pool
            atomicOr(p.flags, FLAG_ATTN_SHAPE);
          } else {
            grow = blk * p.block_size + (pos & (p.block_size - 1));
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
            tma_load_3d(dst, tm, &full[st], 0, s.g, grow);
          } else {
#pragma unroll
            for (int c = 0; c < HD / 64; ++c)
              tma_load_3d(dst + c * L::BLK, tm, &full[st], c * 64, s.g, grow);
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
      int t = t_begin, u = u_first;
      Seg s;
      uint32_t it = 0, n[2] = {0, 0}, units[2] = {0, 0};
      bool ok = true;
      while (ok && seg_next(p, num_units, t, t_end, u, s)) {
        const int nr = tiles_of(s);
        for (int j = s.j0; ok && j < s.j1; ++j, ++it) {
          const uint32_t st = it % L::NS;
          if (!(ok = wwait(&bars->k_full[st], (it / L::NS) & 1))) break;
          const int steps = steps_of(s, j);
          for (int h = 0; ok && h < steps; ++h) {
            const uint64_t kd = kdesc0 + ((st * L::RAW + h * HK * 128) >> 4);
            for (int r = 0; r < nr; ++r) {
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
        for (int r = 0; r < nr; ++r) ++units[r];
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
      int t = t_begin, u = u_first;
      Seg s;
      uint32_t it = 0, n[2] = {0, 0};
      bool ok = true;
      while (ok && seg_next(p, num_units, t, t_end, u, s)) {
        const int nr = tiles_of(s);
        for (int j = s.j0; ok && j < s.j1; ++j, ++it) {
          constexpr uint32_t NV = F8 ? NCV : L::NS;
          const uint32_t st = it % NV;
          if (!(ok = wwait(F8 ? &bars->vc_full[st] : &bars->v_full[st], (it / NV) & 1))) break;
          const int steps = steps_of(s, j);
          for (int h = 0; ok && h < steps; ++h) {
            const uint64_t vd = vdesc0 + ((st * L::TILE + h * HK * 128) >> 4);
            for (int r = 0; r < nr; ++r) {
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
  } else if (warp < CONV_WARP0) {
    // ------------------------------------------------------------ softmax of row tile r
    const int r = (warp - SOFTMAX_WARP0) >> 2;
    const int rr = (warp & 3) * 32 + lane;  // the thread's row in its tile = TMEM lane
    const uint32_t tq = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    int t = t_begin, u = u_first;
    Seg s;
    uint32_t it = 0, n = 0;  // tiles of the range; steps of this row tile
    bool ok = true;
    while (ok && seg_next(p, num_units, t, t_end, u, s)) {
      if (r >= tiles_of(s)) {
        it += s.j1 - s.j0;
        continue;
      }
      const int row = r * MT + rr;
      const bool live = row < s.rows;
      const int rg = s.mt * 2 * MT + (live ? row : r * MT);  // a dead row repeats a live one
      const uint4* qsrc = reinterpret_cast<const uint4*>(
          (const __nv_bfloat16*)p.q +
          ((s.q_off + rg / p.G) * p.Hq + (int64_t)s.g * p.G + rg % p.G) * HD);
      float sc = p.scale_log2;  // score scale in log2 units
      uint8_t* qrow = smem + L::Q + r * L::QB + rr * 128;
      if constexpr (F8) {
        // Q row x 2^e, its largest magnitude in [128, 256), as hi + lo (attn_tc.cu)
        uint32_t rq[HD / 2];
        uint32_t amax = 0;
#pragma unroll
        for (int e = 0; e < HD / 8; ++e) {
          const uint4 v = __ldg(qsrc + e);
          rq[4 * e] = v.x;
          rq[4 * e + 1] = v.y;
          rq[4 * e + 2] = v.z;
          rq[4 * e + 3] = v.w;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            amax = max(amax, max(rq[4 * e + k] & 0x7fffu, (rq[4 * e + k] >> 16) & 0x7fffu));
        }
        const int eb = max((int)(amax >> 7), 1);
        const int e2 = amax == 0 ? 0 : min(max(134 - eb, -120), 120);
        const float f = __int_as_float((e2 + 127) << 23);
#pragma unroll
        for (int c = 0; c < 4; ++c) {  // 32 elements: 8 TMEM columns, two 16-byte chunks
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int w = 0; w < 8; ++w) {
            const uint32_t a = rq[16 * c + 2 * w], b = rq[16 * c + 2 * w + 1];
            const float x[4] = {__uint_as_float(a << 16) * f, __uint_as_float(a & 0xffff0000u) * f,
                                __uint_as_float(b << 16) * f, __uint_as_float(b & 0xffff0000u) * f};
            split_q(x, hi[w], lo[w]);
          }
          tmem_st8(tq + COL_Q + r * 32 + 8 * c, hi);
          *reinterpret_cast<uint4*>(qrow + (((2 * c) ^ (rr & 7)) << 4)) =
              make_uint4(lo[0], lo[1], lo[2], lo[3]);
          *reinterpret_cast<uint4*>(qrow + (((2 * c + 1) ^ (rr & 7)) << 4)) =
              make_uint4(lo[4], lo[5], lo[6], lo[7]);
        }
        sc = p.scale_log2 * p.kv_scale[s.g] * __int_as_float((127 - e2) << 23);
      } else {
        uint32_t rq[32];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint4 v = __ldg(qsrc + e);
          rq[4 * e] = v.x;
          rq[4 * e + 1] = v.y;
          rq[4 * e + 2] = v.z;
          rq[4 * e + 3] = v.w;
        }
        tmem_st32(tq + COL_Q + r * 32, rq);
        if constexpr (L::QS) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<uint4*>(qrow + ((e ^ (rr & 7)) << 4)) = __ldg(qsrc + 8 + e);
        }
      }
      tmem_wait_st();
      if constexpr (L::QS) fence_proxy_async();
      fence_before();
      mbar_arrive(&bars->q_full[r]);

      float m_ref = -INFINITY, lh = 0.f;
      bool good = true;
      for (int j = s.j0; good && j < s.j1; ++j, ++it) {
        const int steps = steps_of(s, j);
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
          const int left = s.nkeys - (j * KT + h * HK);  // keys of the prefix in this step
          if (left < HK) {
#pragma unroll
            for (int c = 0; c < HK; ++c)
              if (c >= left) x[c] = -INFINITY;
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
          if (!F8 && r == 0 && left < HK) {
            // V rows past the prefix (another page's bits): zeros, so that P = 0 never meets
            // non-finite data
            const uint32_t st = it % L::NS;
            if (!(good = wwait(&bars->v_full[st], (it / L::NS) & 1))) break;
            uint8_t* vt = smem + L::V + st * L::RAW;
            const int chunks = (HK - left) * 8;  // 16-byte chunks per column block
            for (int q = rr; q < chunks * (HD / 64); q += 128) {
              const int blk = q / chunks, rem = q % chunks;
              *reinterpret_cast<uint4*>(vt + blk * L::BLK + (h * HK + left + rem / 8) * 128 +
                                        (rem % 8) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async();
          }
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
        break;
      }
      const size_t at = ((size_t)blockIdx.x + s.u) * (2 * MT) + row;
#pragma unroll 1
      for (int c = 0; c < HD / 32; ++c) {
        uint32_t ro[32];
        tmem_ld32(tq + COL_O + r * 128 + c * 32, ro);
        tmem_wait_ld();
        reg_fence32(ro);
        if (live) {
          uint4* dst = reinterpret_cast<uint4*>(p.part_o + at * HD + c * 32);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            dst[e] = make_uint4(ro[4 * e], ro[4 * e + 1], ro[4 * e + 2], ro[4 * e + 3]);
        }
      }
      if (live) p.part_ml[at] = make_float2(m_ref, lh);
      fence_before();  // TMEM reads above complete before the next unit's MMAs
    }
  }

  if constexpr (F8) {
    if (warp >= CONV_WARP0) {
      // ---------------------------------------------------------- E4M3 -> f16 V decoding
      // As in attn_tc.cu: raw 128-byte swizzled rows in, the 16-bit MN-major operand layout
      // out; rows past the prefix become zeros.
      const int ct = (warp - CONV_WARP0) * 32 + lane;
      const int c = ct & 7;
      const int rw = (ct >> 3) ^ (c >> 2);
      const int ph = rw & 7;
      const uint32_t src_off = rw * 128 + ((c ^ ph) << 4);
      const uint32_t dst_off = (c >> 2) * L::BLK + rw * 128;
      const uint32_t w0 = ((2 * (c & 3)) ^ ph) << 4, w1 = ((2 * (c & 3) + 1) ^ ph) << 4;
      constexpr int RSTEP = 16 * 128;
      int t = t_begin, u = u_first;
      Seg s;
      uint32_t it = 0;
      bool ok = true;
      while (ok && seg_next(p, num_units, t, t_end, u, s)) {
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
          uint4 w[KT / 16];
#pragma unroll
          for (int k = 0; k < KT / 16; ++k)
            w[k] = *reinterpret_cast<const uint4*>(rsrc + k * RSTEP);
          mbar_arrive(&bars->v_empty[rs]);
          const int lim = s.nkeys - j * KT;  // rows >= lim lie past the prefix
#pragma unroll
          for (int k = 0; k < KT / 16; ++k) {
            uint32_t h[8];
            e4m3x4_to_f16x4(w[k].x, h[0], h[1]);
            e4m3x4_to_f16x4(w[k].y, h[2], h[3]);
            e4m3x4_to_f16x4(w[k].z, h[4], h[5]);
            e4m3x4_to_f16x4(w[k].w, h[6], h[7]);
            if (rw + 16 * k >= lim) {
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
  if (warp == 1) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(TMEM_COLS)
                 : "memory");
  }
}

template <int HD, bool F8>
cudaError_t launch_hd(const AttnParams& p, cudaStream_t s) {
  using L = Layout<HD, F8>;
  CUtensorMap mk, mv;
  const int box = p.block_size < KT ? p.block_size : KT;
  if (!kv_tensor_map(&mk, p.k, p.kv_rows, p.Hkv, HD, F8, box) ||
      !kv_tensor_map(&mv, p.v, p.kv_rows, p.Hkv, HD, F8, box))
    return cudaErrorInvalidValue;
  auto kernel = attn_prefix_kernel<HD, F8>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(p.n_ctas), dim3(L::THREADS), L::SMEM, s, p, mk, mv);
}

}  // namespace

cudaError_t launch_attn_prefix(const AttnParams& p, bool fp8, cudaStream_t s) {
  if (!attn_tc_supports(p.d, fp8) || p.block_size == 0) return cudaErrorNotSupported;
  if (fp8) return launch_hd<128, true>(p, s);
  return p.d == 128 ? launch_hd<128, false>(p, s) : launch_hd<64, false>(p, s);
}

}  // namespace sv
