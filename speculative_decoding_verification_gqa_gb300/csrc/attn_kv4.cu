// attn_kv4.cu -- verify attention over a 4-bit paged cache (format: kv4.cuh) for few query rows
// a KV head, or short sequences, on warp-level MMAs with the keys as the M dimension.
//
// The transposed products S^T = K Q^T and O^T = V^T P^T put the 16 keys (or 16 elements of d)
// of an m16n8k16 step in M and up to 8 query rows in N, so that a single token's G rows fill
// N = 8 instead of an eighth of M = 128, and K and V are the A operands, whose fragments each
// lane decodes from the codes in its own registers: nothing of the 16-bit K or V is ever
// written to shared memory. What makes the fragments fall in place:
//   * the order of d within S^T is free as long as Q has the same: lane t of a key's four takes
//     a quarter of the key's codes, contiguous (d 128: 16 bytes), four elements a k-step;
//   * the order of d in O^T is free (a permutation of output rows): the lanes of row r of a
//     fragment take the elements 16 r .. 16 r + 15 (d 128), which share one block scale;
//   * an A fragment of V^T pairs two keys at one element, the codes pair two elements of one
//     key: masks exchange the nibbles of two keys' words before the conversion, 4 operations
//     for 16 codes;
//   * P^T's fragments are the 8x8 transposes (movmatrix) of S^T's packed accumulators.
// Row statistics: rows are columns of S^T, so a row's scores are spread over the lanes; the
// reference maximum is the same in all lanes of a column and moves only when some lane of the
// warp sees a score far above it, so the usual tile needs one vote and no exchange.
//
// A warp takes chunks of 32 keys of one KV head, its own ring of cp.async stages, its own (O, m,
// l). The CTA's four warps are spread over the unit's neighbouring heads, then over its keys;
// they meet only at the end of a unit, where a head's parts are joined by the rule of the
// online softmax. Units, their line and the join across CTAs (kv4_join, below): line.cuh.
//
// Rounding: Q is held in f16 after a power of two that puts its row's largest element in [128,
// 256), P in f16 (2^-11 of a weight; SHIFT, below); O is accumulated from these, while the row's
// sum, and with it the log-sum, is that of the unrounded fp32 weights. Scores, sums and O are fp32.
//
// Measured (d 128): 64 single tokens over up to 8192 positions, 32 query and 8 KV heads, 78 us
// with the join, 308 MB at 3.9 TB/s. With half of the issue slots taken (decoding, MMAs and
// exponentials for 8 rows a head of which 4 are live) and less than 60% of HBM it is bound by
// latency, which 12 warps an SM do not cover. More than 8 rows a head (16 held) spill 46 words of
// a thread at the 168 registers that three CTAs leave.
#include <cuda_bf16.h>

#include <algorithm>

#include "kv4.cuh"
#include "line.cuh"

namespace sv {
namespace {

constexpr int KT = KV4_KT;         // keys per tile of the line
constexpr int CK = 32;             // keys of a chunk
constexpr int NW = 4;              // warps
constexpr int NTHREADS = NW * 32;
constexpr int ST = 3;              // ring stages of a warp
constexpr int SM_CTAS = 3;         // CTAs of an SM: 168 registers a thread. (64 sequences of up to
                                   // 8192 positions, single tokens, with 3 CTAs 76.8 us, 4: 81.2,
                                   // 5: 92)
// Reference of a row: its largest score less SHIFT (log2 units), raised when a score is more
// than RESCALE above that score. P = 2^(s - reference) then lies below 2^15 and the largest at
// 2^7 or more, so that f16 (largest 65504, least step 2^-24) drops only weights below 2^-32 of
// it: at the reference itself it would drop those below 2^-25, 3% of a row of a million keys.
constexpr float SHIFT = 7.f, RESCALE = 8.f;

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
template <int N>  // bytes; not valid: zeros, nothing is read
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? N : 0;
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;\n" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

template <int HD>
struct L4 {
  static constexpr int KS = HD / 16;        // k-steps of S^T, m-tiles of O^T
  static constexpr int RB = HD / 2;         // bytes of a row's codes
  static constexpr int SB = HD / 8;         // bytes of a row's scales (K, then V)
  static constexpr int NB = HD / 16;        // blocks of a row
  static constexpr int CODES = CK * RB;     // one tensor's codes of a stage
  static constexpr int STAGE = 2 * CODES + CK * SB;
  static constexpr int OSTRIDE = HD + 4;    // floats of an output row in shared memory
  static constexpr int RING = ST * STAGE;
};
// The bytes a warp owns: its ring, which holds its output part at the end of a unit.
template <int HD, int NT>
constexpr int warp_bytes() {
  return L4<HD>::RING > 8 * NT * L4<HD>::OSTRIDE * 4 ? L4<HD>::RING : 8 * NT * L4<HD>::OSTRIDE * 4;
}

// Where key kk of a chunk has its V codes: keys 2t, 2t + 1 of eight lie 4 rows apart, and d 128
// exchanges the halves of the rows of t = 2, 3, so that a warp's loads, four keys (one of each
// t) by eight elements' bytes, meet every bank once.
__device__ __forceinline__ int v_place(int kk) { return (kk & ~7) | ((kk & 1) << 2) | ((kk >> 1) & 3); }

// Four columns of an output row from O (unnormalised) and the row's (reference, sum).
template <int HD>
__device__ __forceinline__ void store_row(const Kv4Attn& p, int64_t row, int g, int c, const float4& o,
                                          float m, float l) {
  const float inv = p.kv_scale[p.Hkv + g] / l;
  const __nv_bfloat162 x = __floats2bfloat162_rn(o.x * inv, o.y * inv);
  const __nv_bfloat162 y = __floats2bfloat162_rn(o.z * inv, o.w * inv);
  *reinterpret_cast<uint2*>((uint16_t*)p.out + row * HD + c * 4) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  if (p.lse && c == 0) p.lse[row] = (m + log2f(l)) * 0.6931471805599453f;
}

// NT: n-tiles of 8 query rows, of which a unit has as many for each of its heads. HG: heads of a
// unit; warp w takes head w % HG and every (NW / HG)-th chunk of its keys.
template <int HD, int NT, int HG>
__global__ void __launch_bounds__(NTHREADS, SM_CTAS) attn_kv4_kernel(const Kv4Attn p) {
  using L = L4<HD>;
  constexpr int KS = L::KS, ROWS = 8 * NT, NK = NW / HG;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_m[NW][ROWS], s_l[NW][ROWS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r8 = lane >> 2, t4 = lane & 3;
  const int hg = warp % HG, kw = warp / HG;
  uint8_t* ring = smem + warp * warp_bytes<HD, NT>();
  pdl_wait();
  pdl_trigger();
  LineWalk walk;
  if (!line_begin<NTHREADS>(p, blockIdx.x, walk)) return;

  LineSeg seg;
  while (walk.next(p, seg)) {
    {
      const int b = seg.b, g = seg.g * HG + hg;
      const int T = seg.T, D = seg.D;
      const int row0 = seg.mt * ROWS;                 // of the (sequence, head)'s rows
      const int rows = min(ROWS, p.G * (D + 1) - row0);
      const int nkeys = T + D + 1;
      const int kvis = first_visible_key(T, p.window);
      const int64_t qo = seg.q_off;
      const float sck = p.scale_log2 * p.kv_scale[g];
      const int key_first = seg.kbase + seg.j0 * KT;
      // chunks with a key of the sequence; this warp takes kw, kw + NK, ...
      const int chunks = min((seg.j1 - seg.j0) * (KT / CK), (nkeys - key_first + CK - 1) / CK);
      const int mine = chunks > kw ? (chunks - kw + NK - 1) / NK : 0;
      const int32_t* tab = p.block_table + (size_t)b * p.bt_stride;

      // ---- the ring. Eight consecutive keys lie in one block: a chunk has four table entries,
      // read a chunk ahead by the lanes, and from each lane's first address on everything is
      // the entry's row times the bytes of a cache position
      constexpr int CH = L::RB / 16;  // 16-byte pieces of a row's codes
      const int code_bytes = p.Hkv * L::RB, scale_bytes = p.Hkv * L::SB;  // of a position
      const int64_t lane_at = (int64_t)(lane / CH % 8) * code_bytes + g * L::RB + lane % CH * 16;
      const uint8_t *kp = (const uint8_t*)p.k + lane_at, *vp = (const uint8_t*)p.v + lane_at;
      const uint8_t* sp = (const uint8_t*)p.scales + (int64_t)(lane & 7) * scale_bytes + g * L::SB;
      const uint32_t ring_at = smem_u32(ring);
      // this lane's V place within the 32 / CH keys that a step covers
      const uint32_t v_at = L::CODES + v_place(lane / CH) * L::RB +
                            (CH == 4 ? (lane % CH) ^ (((lane / CH >> 2) & 1) << 1) : lane % CH) * 16;
      constexpr int UNSEEN = -2;
      auto entry = [&](int i) -> int {  // this lane's entry of the warp's i-th chunk
        const int pos = key_first + (kw + i * NK) * CK + 8 * t4;
        if (i >= mine || pos >= nkeys || pos + 8 <= kvis) return UNSEEN;
        return __ldg(tab + (pos >> p.bs_log2));
      };
      int ent = entry(0);
      auto issue = [&](int i) {
        if (i < mine) {
          const uint32_t st = ring_at + (i % ST) * L::STAGE;
          const int key0 = key_first + (kw + i * NK) * CK;
          const bool full = key0 >= kvis && key0 + CK <= nkeys;
          int base = -1;  // cache row of the first of this lane's eight keys
          if (ent >= 0 && ent < p.num_blocks)
            base = (ent << p.bs_log2) + ((key0 + 8 * t4) & (p.block_size - 1));
          else if (ent != UNSEEN)
            atomicOr(p.flags, FLAG_ATTN_SHAPE);  // an entry outside the pool
          auto step = [&](bool all) {
#pragma unroll
            for (int j = 0; j < CH; ++j) {
              const int kk = (j * 32 + lane) / CH;
              const int row = __shfl_sync(0xffffffffu, base, kk >> 3);
              const bool ok = row >= 0 && (all || (key0 + kk < nkeys && key0 + kk >= kvis));
              const int64_t off = ok ? (int64_t)row * code_bytes : 0;
              cp_async<16>(st + (j * 32 + lane) * 16, kp + off, ok);
              cp_async<16>(st + v_at + j * (32 / CH) * L::RB, vp + off, ok);
            }
            const int row = __shfl_sync(0xffffffffu, base, lane >> 3);
            const bool ok = row >= 0 && (all || (key0 + lane < nkeys && key0 + lane >= kvis));
            cp_async<L::SB>(st + 2 * L::CODES + lane * L::SB, sp + (ok ? (int64_t)row * scale_bytes : 0), ok);
          };
          if (full) step(true);
          else step(false);
          ent = entry(i + 1);
        }
        cp_async_commit();
      };
#pragma unroll
      for (int i = 0; i < ST - 1; ++i) issue(i);

      // ---- Q: column n = lane / 4 of each n-tile, the elements (HD / 4) t .. of its row
      uint32_t qf[NT][KS][2];
      float sc[NT][2];  // score scale (log2 units) of columns 2 t, 2 t + 1
      int i_col[NT][2];  // window row of those columns
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int r = n * 8 + r8;
        const bool live = r < rows;
        const int rg = row0 + (live ? r : 0);
        const uint4* src = reinterpret_cast<const uint4*>(
            (const uint16_t*)p.q + ((qo + rg / p.G) * p.Hq + (int64_t)g * p.G + rg % p.G) * HD +
            t4 * (HD / 4));
        uint32_t w[HD / 8], amax = 0;
#pragma unroll
        for (int e = 0; e < HD / 32; ++e) {
          const uint4 v = live ? __ldg(src + e) : make_uint4(0, 0, 0, 0);
          w[4 * e] = v.x;
          w[4 * e + 1] = v.y;
          w[4 * e + 2] = v.z;
          w[4 * e + 3] = v.w;
        }
#pragma unroll
        for (int e = 0; e < HD / 8; ++e) amax = max(amax, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const float f = exp2_of(q_exponent(amax));  // f16's range: see q_exponent
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t x = w[2 * s + e];
            qf[n][s][e] = pack_f16(__uint_as_float(x << 16) * f, __uint_as_float(x & 0xffff0000u) * f);
          }
        const float mysc = q_row_scale(sck, amax);
        const int myi = live ? rg / p.G : D;  // rows past the unit's see every key
        const int from = (2 * t4) * 4;        // a lane that holds column 2 t
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sc[n][e] = __shfl_sync(0xffffffffu, mysc, from + 4 * e);
          i_col[n][e] = __shfl_sync(0xffffffffu, myi, from + 4 * e);
        }
      }
      float o[KS][NT][4], m[NT][2], l[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
#pragma unroll
        for (int s = 0; s < KS; ++s) o[s][n][0] = o[s][n][1] = o[s][n][2] = o[s][n][3] = 0.f;
      }
      const int lo_max = p.window > 0 ? max(T + D + 1 - p.window, 0) : 0;

      for (int i = 0; i < mine; ++i) {
        cp_async_wait<ST - 2>();
        __syncwarp();  // the chunk's bytes of every lane are here; the last chunk's are read
        issue(i + ST - 1);
        const uint8_t* st = ring + (i % ST) * L::STAGE;
        const uint8_t* sS = st + 2 * L::CODES;
        const int key0 = key_first + (kw + i * NK) * CK;

        // ---- S^T = K Q^T
        float s[2][NT][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int n = 0; n < NT; ++n) s[h][n][0] = s[h][n][1] = s[h][n][2] = s[h][n][3] = 0.f;
          float s2[NT][4] = {};  // the odd k-steps: two chains of MMAs
          uint32_t w[2][HD / 32], u[2][HD / 64];  // codes and scale pairs of keys r8, r8 + 8
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int kk = h * 16 + e * 8 + r8;
            const uint8_t* row = st + kk * L::RB + t4 * (L::RB / 4);
            if constexpr (HD == 128) {
              const uint4 v = *reinterpret_cast<const uint4*>(row);
              w[e][0] = v.x;
              w[e][1] = v.y;
              w[e][2] = v.z;
              w[e][3] = v.w;
              const uint32_t c = *reinterpret_cast<const uint16_t*>(sS + kk * L::SB + 2 * t4);
              const uint32_t f = e4m3x2_to_f16x2(c);
              u[e][0] = lo_twice(f);
              u[e][1] = hi_twice(f);
            } else {
              const uint2 v = *reinterpret_cast<const uint2*>(row);
              w[e][0] = v.x;
              w[e][1] = v.y;
              u[e][0] = lo_twice(e4m3x2_to_f16x2(sS[kk * L::SB + t4]));
            }
          }
#pragma unroll
          for (int q = 0; q < HD / 32; ++q) {  // a word of codes: two k-steps
            uint32_t x[4], y[4];
            e2m1x8_to_f16(w[0][q], x);
            e2m1x8_to_f16(w[1][q], y);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              x[e] = hmul2(x[e], u[0][q >> 1]);
              y[e] = hmul2(y[e], u[1][q >> 1]);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t a[4] = {x[2 * e], y[2 * e], x[2 * e + 1], y[2 * e + 1]};
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma_f16(e ? s2[n] : s[h][n], a, qf[n][2 * q + e][0], qf[n][2 * q + e][1]);
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[h][n][e] += s2[n][e];
        }
        // ---- mask, exponents above the reference, raised where one is far above
        if (key0 + CK > T || key0 < lo_max) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int key = key0 + h * 16 + r8 + (e >> 1) * 8;
                const int hi = T + i_col[n][e & 1];
                if (key > hi || (p.window > 0 && key <= hi - p.window)) s[h][n][e] = -INFINITY;
              }
        }
        float x[2][NT][4];
        bool above = false;
        auto exponents = [&](int n, int e) {  // of column e of n-tile n
          const float nm = m[n][e] == -INFINITY ? 0.f : -m[n][e];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            x[h][n][e] = fmaf(s[h][n][e], sc[n][e], nm);
            x[h][n][e + 2] = fmaf(s[h][n][e + 2], sc[n][e], nm);
          }
          return fmaxf(fmaxf(x[0][n][e], x[0][n][e + 2]), fmaxf(x[1][n][e], x[1][n][e + 2]));
        };
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            above |= exponents(n, e) > (m[n][e] == -INFINITY ? -INFINITY : SHIFT + RESCALE);
        if (__any_sync(0xffffffffu, above)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float y = fmaxf(fmaxf(s[0][n][e], s[0][n][e + 2]), fmaxf(s[1][n][e], s[1][n][e + 2])) * sc[n][e];
#pragma unroll
              for (int o2 = 4; o2 < 32; o2 <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, o2));
              const float mn = fmaxf(m[n][e], y - SHIFT);
              const float al = mn == -INFINITY ? 1.f : ex2(m[n][e] - mn);
              m[n][e] = mn;
              l[n][e] *= al;
#pragma unroll
              for (int k = 0; k < KS; ++k) {
                o[k][n][e] *= al;
                o[k][n][e + 2] *= al;
              }
              exponents(n, e);
            }
        }
        // ---- P = 2^x, its fragments
        uint32_t pf[2][NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float a[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) a[e] = ex2(x[h][n][e]);
            l[n][0] += a[0] + a[2];
            l[n][1] += a[1] + a[3];
            pf[h][n][0] = transpose8x8(pack_f16(a[0], a[1]));
            pf[h][n][1] = transpose8x8(pack_f16(a[2], a[3]));
          }
        // ---- O^T += V^T P^T
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          constexpr int VW = HD / 64;  // words of codes a lane takes of each key
          uint32_t w[4][VW], u[2];
#pragma unroll
          for (int e = 0; e < 4; ++e) {  // keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9
            const int kk = h * 16 + (e >> 1) * 8 + 2 * t4 + (e & 1);
            const uint8_t* row = st + L::CODES + v_place(kk) * L::RB;
            if constexpr (HD == 128) {
              const int c = (r8 >> 1) ^ (((kk >> 2) & 1) << 1);
              const uint2 v = *reinterpret_cast<const uint2*>(row + c * 16 + (r8 & 1) * 8);
              w[e][0] = v.x;
              w[e][1] = v.y;
            } else {
              w[e][0] = *reinterpret_cast<const uint32_t*>(row + r8 * 4);
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint8_t* sv = sS + (h * 16 + e * 8 + 2 * t4) * L::SB + L::NB + (HD == 128 ? r8 : r8 >> 1);
            u[e] = e4m3x2_to_f16x2((uint32_t)sv[0] | ((uint32_t)sv[L::SB] << 8));
          }
#pragma unroll
          for (int q = 0; q < VW; ++q) {  // a word of each key: 4 m-tiles
            uint32_t f[2][2][4];          // [keys 2 t, + 8][element 2 i, 2 i + 1][i]
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t k0 = w[2 * e][q], k1 = w[2 * e + 1][q];
              e2m1x8_to_f16((k0 & 0x0f0f0f0fu) | ((k1 << 4) & 0xf0f0f0f0u), f[e][0]);
              e2m1x8_to_f16(((k0 >> 4) & 0x0f0f0f0fu) | (k1 & 0xf0f0f0f0u), f[e][1]);
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                f[e][0][x] = hmul2(f[e][0][x], u[e]);
                f[e][1][x] = hmul2(f[e][1][x], u[e]);
              }
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint32_t a[4] = {f[0][0][x], f[0][1][x], f[1][0][x], f[1][1][x]};
#pragma unroll
              for (int n = 0; n < NT; ++n) mma_f16(o[4 * q + x][n], a, pf[h][n][0], pf[h][n][1]);
            }
          }
        }
      }
      cp_async_wait<0>();

      // ---- join of the CTA's warps
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], x);
          if (r8 == 0) {
            s_m[warp][n * 8 + 2 * t4 + e] = m[n][e];
            s_l[warp][n * 8 + 2 * t4 + e] = l[n][e];
          }
        }
      __syncthreads();  // every warp is done with its ring, its (m, l) are written
      float* part = reinterpret_cast<float*>(ring);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = n * 8 + 2 * t4 + e;
          float M = s_m[hg][r];
#pragma unroll
          for (int w = 1; w < NK; ++w) M = fmaxf(M, s_m[hg + w * HG][r]);
          const float f = m[n][e] == -INFINITY ? 0.f : ex2(m[n][e] - M);
          // elements: m-tile i, fragment rows r8 and r8 + 8 are (HD / 8) r8 + 2 i and + 1
          float* dst = part + r * L::OSTRIDE + r8 * (HD / 8);
#pragma unroll
          for (int k = 0; k < KS; k += 2)
            *reinterpret_cast<float4*>(dst + 2 * k) =
                make_float4(o[k][n][e] * f, o[k][n][e + 2] * f, o[k + 1][n][e] * f, o[k + 1][n][e + 2] * f);
        }
      __syncthreads();
      // (a warp without chunks: m = -inf, O = 0; a NaN in l or O stays)
      for (int idx = tid; idx < HG * ROWS * (HD / 4); idx += NTHREADS) {
        const int c = idx % (HD / 4), r = idx / (HD / 4) % ROWS, h = idx / (HD / 4) / ROWS;
        if (r >= rows) continue;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float M = s_m[h][r], lsum = 0.f;
#pragma unroll
        for (int w = 1; w < NK; ++w) M = fmaxf(M, s_m[h + w * HG][r]);
#pragma unroll
        for (int w = 0; w < NK; ++w) {
          const int ww = h + w * HG;
          const float4 v = *reinterpret_cast<const float4*>(
              reinterpret_cast<const float*>(smem + ww * warp_bytes<HD, NT>()) + r * L::OSTRIDE + c * 4);
          acc.x += v.x;
          acc.y += v.y;
          acc.z += v.z;
          acc.w += v.w;
          lsum += s_m[ww][r] == -INFINITY ? s_l[ww][r] : s_l[ww][r] * ex2(s_m[ww][r] - M);
        }
        if (seg.whole) {
          const int rg = row0 + r, gh = seg.g * HG + h;
          store_row<HD>(p, (qo + rg / p.G) * p.Hq + (int64_t)gh * p.G + rg % p.G, gh, c, acc, M, lsum);
        } else {
          const size_t at = ((size_t)(2 * blockIdx.x + seg.begins) * HG + h) * ROWS + r;
          *reinterpret_cast<float4*>(p.part_o + at * HD + c * 4) = acc;
          if (c == 0) p.part_ml[at] = make_float2(M, lsum);
        }
      }
      __syncthreads();  // the parts are read before the rings are filled again
    }
  }
}

// ------------------------------------------------------------------------------ join

constexpr int JT = 256;  // threads
constexpr int SPREAD_PARTS = 8;

// The units that several CTAs share: their parts, in the CTAs' order, by the rule of the online
// softmax. An item is JROWS rows of one head of a unit, RW for each warp, whose parts are asked
// for together; or (RW = 0), where units have many parts, one row, of which each warp takes every
// eighth part, added up through shared memory, so that a long sequence's hundred parts are not
// read one after another. Items in contiguous ranges of the grid's CTAs, as the lines are walked.
template <int HD, int RWS>
__global__ void __launch_bounds__(JT) kv4_join_kernel(const Kv4Attn p) {
  constexpr bool SPREAD = RWS == 0;
  constexpr int RW = SPREAD ? 1 : RWS, JROWS = SPREAD ? 1 : RW * (JT / 32);
  __shared__ float4 s_o[JT / 32][HD / 4];
  __shared__ float2 s_ml[JT / 32];
  pdl_trigger();
  pdl_wait();  // before the lengths too: only this grid's own wait makes what wrote them visible
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = p.heads * ((p.mr + JROWS - 1) / JROWS);  // items of a unit
  Line total = {};
  LineAt at;
  int64_t it = 0, end = 0;
  const bool any = line_scan<JT>(p, total, &at, [&](bool& by_unit) -> int64_t {
    const int64_t items = total.whole ? 0 : total.units * per;
    it = (int64_t)blockIdx.x * items / gridDim.x;
    end = (int64_t)(blockIdx.x + 1) * items / gridDim.x;
    by_unit = true;
    return it < end ? it / per : -1;
  });
  if (!any) return;
  LineWalk walk = line_enter(p, at, it / per - at.units, true);
  walk.v0 = 0;
  walk.v1 = total.virt;
  constexpr int LN = HD / 4;  // lanes of a row
  while (it < end) {
    const int64_t us = walk.us;
    LineSeg s;
    walk.next(p, s);  // the whole unit
    const int64_t first = us + p.switch_tiles;
    const int c0 = cta_of_tile(first, total.virt, total.ctas);
    const int c1 = cta_of_tile(first + s.nt - 1, total.virt, total.ctas);
    const int64_t next = min(end, (it / per + 1) * per);
    if (c0 == c1) {  // one CTA's: written already
      it = next;
      continue;
    }
    const int rows = min(p.mr, p.G * (s.D + 1) - s.mt * p.mr);
    for (; it < next; ++it) {
      const int i = (int)(it % per), h = i % p.heads, r0 = i / p.heads * JROWS;
      const int gh = s.g * p.heads + h;
      // parts c0 + w, c0 + w + step, ... of rows r, r + JT / 32, ...
      float4 acc[RW];
      float m[RW], l[RW];
      auto gather = [&](int r, int w, int step) {
        constexpr int U = 8 / RW;
#pragma unroll
        for (int e = 0; e < RW; ++e) {
          acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
          m[e] = -INFINITY;
          l[e] = 0.f;
        }
        for (int c = c0 + w; c <= c1; c += U * step) {
          float2 ml[RW][U];
          float4 v[RW][U];
#pragma unroll
          for (int e = 0; e < RW; ++e)
#pragma unroll
            for (int k = 0; k < U; ++k) {
              const int cc = c + k * step, rr = r + e * (JT / 32);
              const bool have = cc <= c1 && rr < rows;
              const size_t at2 = ((size_t)(2 * cc + (cc == c0)) * p.heads + h) * p.mr + rr;
              ml[e][k] = have ? __ldcg(p.part_ml + at2) : make_float2(-INFINITY, 0.f);
              v[e][k] = have && lane < LN ? __ldcg(reinterpret_cast<const float4*>(p.part_o + at2 * HD) + lane)
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
          for (int e = 0; e < RW; ++e) {
            float mn = m[e];
#pragma unroll
            for (int k = 0; k < U; ++k) mn = fmaxf(mn, ml[e][k].x);
            const float mu = mn == -INFINITY ? 0.f : mn;
            const float f0 = ex2(m[e] - mu);
            float4 o = acc[e];
            m[e] = mn;
            l[e] *= f0;
            o = make_float4(o.x * f0, o.y * f0, o.z * f0, o.w * f0);
#pragma unroll
            for (int k = 0; k < U; ++k) {
              // (a part without a reference: O = 0 and l = 0, or NaN, which stays)
              const float f = ml[e][k].x == -INFINITY ? 1.f : ex2(ml[e][k].x - mu);
              l[e] += ml[e][k].y * f;
              o = make_float4(o.x + v[e][k].x * f, o.y + v[e][k].y * f, o.z + v[e][k].z * f, o.w + v[e][k].w * f);
            }
            acc[e] = o;
          }
        }
      };
      auto out_row = [&](int r) {
        const int rg = s.mt * p.mr + r;
        return (s.q_off + rg / p.G) * p.Hq + (int64_t)gh * p.G + rg % p.G;
      };
      if (!SPREAD) {
        gather(r0 + warp, 0, 1);
#pragma unroll
        for (int e = 0; e < RW; ++e) {
          const int r = r0 + warp + e * (JT / 32);
          if (r < rows && lane < LN) store_row<HD>(p, out_row(r), gh, lane, acc[e], m[e], l[e]);
        }
      } else if (r0 < rows) {
        gather(r0, warp, JT / 32);
        if (lane < LN) s_o[warp][lane] = acc[0];
        if (lane == 0) s_ml[warp] = make_float2(m[0], l[0]);
        __syncthreads();
        if (warp == 0 && lane < LN) {
          float M = -INFINITY, ls = 0.f;
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < JT / 32; ++w) M = fmaxf(M, s_ml[w].x);
#pragma unroll
          for (int w = 0; w < JT / 32; ++w) {
            const float f = s_ml[w].x == -INFINITY ? 1.f : ex2(s_ml[w].x - M);
            const float4 v = s_o[w][lane];
            ls += s_ml[w].y * f;
            o = make_float4(o.x + v.x * f, o.y + v.y * f, o.z + v.z * f, o.w + v.w * f);
          }
          store_row<HD>(p, out_row(r0), gh, lane, o, M, ls);
        }
        __syncthreads();
      }
    }
  }
}

template <int HD, int NT, int HG>
cudaError_t launch_nt(const Kv4Attn& p, cudaStream_t s) {
  const size_t smem = (size_t)NW * warp_bytes<HD, NT>();
  auto kernel = attn_kv4_kernel<HD, NT, HG>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(p.n_ctas), dim3(NTHREADS), smem, s, p);
}
template <int HD, int NT>
cudaError_t launch_nt(const Kv4Attn& p, cudaStream_t s) {
  return p.heads == 2 ? launch_nt<HD, NT, 2>(p, s) : launch_nt<HD, NT, 1>(p, s);
}

}  // namespace

// CTAs of a call on `sms` SMs: what an SM holds at once; query rows of a unit and head.
int attn_kv4_ctas(int sms) { return sms * SM_CTAS; }
int attn_kv4_rows(int rows_per_kv) { return rows_per_kv <= 8 ? 8 : 16; }

cudaError_t launch_attn_kv4(const Kv4Attn& p, cudaStream_t s) {
  if (p.d == 128) return p.mr == 8 ? launch_nt<128, 1>(p, s) : launch_nt<128, 2>(p, s);
  return p.mr == 8 ? launch_nt<64, 1>(p, s) : launch_nt<64, 2>(p, s);
}

cudaError_t launch_kv4_join(const Kv4Attn& p, int sms, cudaStream_t s) {
  const int64_t rows = (int64_t)p.G * (1 + p.max_draft);
  const int64_t units = (int64_t)p.B * (p.Hkv / p.heads) * ((rows + p.mr - 1) / p.mr);
  // (4 rows a warp where a unit has 128)
  const int rw = p.n_ctas >= SPREAD_PARTS * units ? 0 : p.mr > 16 ? 4 : 1;
  const int jrows = rw ? rw * (JT / 32) : 1;
  const int64_t items = units * p.heads * ((p.mr + jrows - 1) / jrows);
  const dim3 grid((unsigned)std::min<int64_t>(items, 4 * (int64_t)sms));
  auto kernel = p.d == 128 ? (rw == 0   ? kv4_join_kernel<128, 0>
                              : rw == 1 ? kv4_join_kernel<128, 1>
                                        : kv4_join_kernel<128, 4>)
                           : (rw == 0   ? kv4_join_kernel<64, 0>
                              : rw == 1 ? kv4_join_kernel<64, 1>
                                        : kv4_join_kernel<64, 4>);
  return launch_pdl(kernel, grid, dim3(JT), 0, s, p);
}

}  // namespace sv
