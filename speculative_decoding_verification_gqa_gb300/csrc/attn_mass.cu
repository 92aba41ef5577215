// attn_mass.cu -- attention weight added up by cached position (spec_attn_mass): what the rows
// of a verify step gave to every key of a KV head, summed over the group's query heads and the
// window's counted rows,
//   mass[b, g, j] += sum_{h, i} 2^(s_{h,i,j} - L_{h,i}),  s scores in log2 units, L their
// row's log-sum. Every key is one thread quartet's and the rows are added in one order, so the
// sums have the same bits every time, without atomics.
//
// Keys are the M dimension (S^T = K Q^T, m16n8k16): the sum over rows then runs along a
// thread's own accumulators, and only at the end over the four lanes of a key. K fragments are
// built in registers straight from the cache's rows: the order of d is free as long as Q has
// the same, so lane t of a key's four takes whole 16-byte pieces (every fourth) of its row.
// Q lies in shared memory in fragment order.
//
// Without given log-sums a first pass over the keys reduces (max, sum) for every row, each
// CTA for its own tiles, and a second kernel joins those into L.
//
// Work: tiles of 256 keys (8 warps x 32) of each (sequence, KV head), end to end on one line,
// an equal range of it for each CTA, which finds its place by scanning the lengths itself.
#include <cuda_bf16.h>

#include "kv4.cuh"

namespace sv {
namespace {

constexpr int NW = 8;
constexpr int NTHREADS = NW * 32;
constexpr int KT = NW * 32;      // keys of a tile
constexpr int RB = 128;          // query rows held at once
constexpr float LN2 = 0.6931471805599453f, LOG2E = 1.4426950408889634f;

struct MassArgs {
  const uint16_t* q;
  const uint8_t* k;          // rows of the cache: bf16, E4M3 or E2M1 codes
  const uint8_t* scales;     // 4 bits: [.., Hkv, 2, d / 16]
  const float* kv_scale;
  const int32_t *table, *seq_lens, *draft_len, *row_count;
  const float* lse;          // [rows, Hq] natural, or null
  float* lse_ws;             // [rows, Hq], written by the joining kernel
  float2* part;              // [n_ctas + B * Hkv][max_rows] (max, sum) in log2 units
  float* mass;
  uint32_t* flags;
  int64_t mass_stride, q_rows, num_blocks;
  int B, Hq, Hkv, G, max_draft, max_seq, bt_stride, block_size, bs_log2;
  int max_rows;              // G * (1 + max_draft)
  int n_ctas;
  float scale_log2;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <bool F16>
__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

enum { BF16 = 0, E4M3 = 1, KV4 = 2 };
template <int HD, int TY>
struct LM {
  static constexpr int KS = HD / 16;
  static constexpr int ROWB = TY == BF16 ? HD * 2 : TY == E4M3 ? HD : HD / 2;  // bytes of a row
  static constexpr int LANEB = ROWB / 4 < 16 ? ROWB / 4 : 16;  // bytes of a lane's piece
  static constexpr int PIECES = ROWB / 4 / LANEB;
  static constexpr int PE = TY == BF16 ? LANEB / 2 : TY == E4M3 ? LANEB : LANEB * 2;  // elements
  // first of the 8 elements of lane t in k-steps 2 j, 2 j + 1
  __device__ static __forceinline__ int elem(int j, int t) {
    return PE * (4 * (8 * j / PE) + t) + 8 * j % PE;
  }
};

// The lengths of sequence b, checked; false if the call must do nothing.
__device__ __forceinline__ bool lengths(const MassArgs& a, int b, int& T, int& D, int& n) {
  T = a.seq_lens[b];
  D = a.draft_len[b];
  n = a.row_count ? a.row_count[b] : 1 + D;  // counted rows
  return T >= 0 && T <= a.max_seq && D >= 0 && D <= a.max_draft && n >= 0 && n <= 1 + D &&
         (((int64_t)T + D + a.block_size) >> a.bs_log2) <= a.bt_stride &&
         (int64_t)T + 1 + D <= a.mass_stride;
}
// Tiles of a KV head: keys that a counted row sees.
__device__ __forceinline__ int tiles_of(int T, int n) {
  return n == 0 ? 0 : (int)(((int64_t)T + n + KT - 1) / KT);
}

// A CTA's place on the line.
struct Place {
  int64_t total, t, end, q_off;
  int b;        // sequence of tile t
  int64_t in_b; // tiles of it before t
};
// Scan of the lengths: totals, and the sequence that holds tile c * total / n_ctas. One CTA's
// threads together; false (flag set) if a length is out of range.
__device__ bool find_place(const MassArgs& a, Place& pl) {
  __shared__ int64_t s_warp[NW][2];
  __shared__ int64_t s_place[3];
  __shared__ int64_t s_total;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  bool bad = false;
  int64_t begin = 0;
  for (int pass = 0; pass < 2; ++pass) {
    int64_t carry_t = 0, carry_q = 0;
    for (int base = 0; base < a.B; base += NTHREADS) {
      const int b = base + tid;
      int64_t v[2] = {0, 0};
      if (b < a.B) {
        int T, D, n;
        if (lengths(a, b, T, D, n)) {
          v[0] = (int64_t)a.Hkv * tiles_of(T, n);
          v[1] = 1 + D;
        } else {
          bad = true;
        }
      }
      int64_t x[2] = {v[0], v[1]};
#pragma unroll
      for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int64_t y = __shfl_up_sync(0xffffffffu, x[k], o);
          if (lane >= o) x[k] += y;
        }
      if (lane == 31) {
        s_warp[wid][0] = x[0];
        s_warp[wid][1] = x[1];
      }
      __syncthreads();
      int64_t before[2] = {0, 0}, all[2] = {0, 0};
#pragma unroll
      for (int w = 0; w < NW; ++w)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          before[k] += w < wid ? s_warp[w][k] : 0;
          all[k] += s_warp[w][k];
        }
      const int64_t tb = carry_t + before[0] + x[0] - v[0];
      if (pass == 1 && begin >= tb && begin < tb + v[0]) {
        s_place[0] = b;
        s_place[1] = begin - tb;
        s_place[2] = carry_q + before[1] + x[1] - v[1];
      }
      carry_t += all[0];
      carry_q += all[1];
      __syncthreads();
    }
    if (pass == 0) {
      bad |= carry_q > a.q_rows;
      if (__syncthreads_or(bad)) {
        if (tid == 0) atomicOr(a.flags, FLAG_ATTN_SHAPE);
        return false;
      }
      pl.total = carry_t;
      begin = blockIdx.x * carry_t / a.n_ctas;
      pl.t = begin;
      pl.end = (blockIdx.x + 1) * carry_t / a.n_ctas;
    }
  }
  if (pl.t >= pl.end) return false;
  __syncthreads();
  pl.b = (int)s_place[0];
  pl.in_b = s_place[1];
  pl.q_off = s_place[2];
  return true;
}

// STATS: the first pass, (max, sum) of each row over the CTA's tiles; else the weights.
template <int HD, int TY, bool STATS>
__global__ void __launch_bounds__(NTHREADS, 2) mass_kernel(const MassArgs a) {
  using L = LM<HD, TY>;
  constexpr int KS = L::KS;
  constexpr bool F16 = TY != BF16;
  extern __shared__ __align__(16) uint8_t smem[];
  uint4* sQ = reinterpret_cast<uint4*>(smem);                 // [RB / 8][KS / 2][32]
  float2* s_row = reinterpret_cast<float2*>(smem + RB * HD * 2);  // [RB] (score scale, log-sum)
  int* s_i = reinterpret_cast<int*>(s_row + RB);              // [RB] window row
  float2* s_ml = reinterpret_cast<float2*>(s_i + RB);         // STATS: [NW][RB]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r8 = lane >> 2, t4 = lane & 3;
  pdl_trigger();
  pdl_wait();
  Place pl;
  if (!find_place(a, pl)) return;
  const float* lse = a.lse ? a.lse : a.lse_ws;

  int64_t t = pl.t;
  for (int b = pl.b; t < pl.end; ++b) {
    int T, D, n;
    lengths(a, b, T, D, n);
    const int nt = tiles_of(T, n);
    const int nkeys = T + n;             // keys that a counted row sees
    const int rows = a.G * n;
    const int32_t* tab = a.table + (size_t)b * a.bt_stride;
    for (int64_t in_b = pl.in_b; in_b < (int64_t)a.Hkv * nt && t < pl.end;) {
      const int g = (int)(in_b / nt), j0 = (int)(in_b - (int64_t)g * nt);
      const int j1 = (int)min((int64_t)nt, j0 + (pl.end - t));
      const float sck = a.scale_log2 * (TY == BF16 ? 1.f : a.kv_scale[g]);
      for (int rb = 0; rb < rows; rb += RB) {
        const int nr = min(RB, rows - rb), ntile = (nr + 7) / 8;
        __syncthreads();  // the last block's readers are done
        // ---- Q rows rb .. of the unit, in fragment order; row = window row i, head of the group
        for (int idx = tid; idx < ntile * 8 * (HD / 8); idx += NTHREADS) {
          const int r = idx / (HD / 8), c = idx % (HD / 8);  // 8 elements; a row's lie in
          const int j = c >> 2, tt = c & 3;                  // neighbouring lanes
          const int rg = rb + r;
          const bool live = r < nr;
          const int64_t row = live ? (pl.q_off + rg / a.G) * a.Hq + (int64_t)g * a.G + rg % a.G : 0;
          uint4 v = make_uint4(0, 0, 0, 0);
          if (live) v = __ldg(reinterpret_cast<const uint4*>(a.q + row * HD + L::elem(j, tt)));
          float sc = sck;
          if constexpr (F16) {
            uint32_t w[4] = {v.x, v.y, v.z, v.w}, amax = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) amax = max(amax, max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
#pragma unroll
            for (int o = 1; o < HD / 8; o <<= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            const float f = exp2_of(q_exponent(amax));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const __half2 h = __floats2half2_rn(__uint_as_float(w[k] << 16) * f,
                                                  __uint_as_float(w[k] & 0xffff0000u) * f);
              w[k] = *reinterpret_cast<const uint32_t*>(&h);
            }
            v = make_uint4(w[0], w[1], w[2], w[3]);
            sc = q_row_scale(sck, amax);
          }
          sQ[((r >> 3) * (KS / 2) + j) * 32 + (r & 7) * 4 + tt] = v;
          if (c == 0) {
            // rows past the block's: weight 2^-inf
            s_row[r] = make_float2(sc, !live ? INFINITY : STATS ? 0.f : lse[row] * LOG2E);
            s_i[r] = live ? rg / a.G : n - 1;
          }
        }
        if constexpr (STATS)
          for (int i = tid; i < NW * RB; i += NTHREADS) s_ml[i] = make_float2(-INFINITY, 0.f);
        __syncthreads();
        for (int j = j0; j < j1; ++j) {
          const int key0 = j * KT + warp * 32;
          if (key0 >= nkeys) continue;
          // ---- K fragments of 32 keys (two m-tiles)
          uint32_t kf[2][KS][4];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int key = key0 + h * 16 + e * 8 + r8;
              bool ok = key < nkeys;
              int64_t row = 0;
              if (ok) {
                const int blk = __ldg(tab + (key >> a.bs_log2));
                ok = blk >= 0 && blk < a.num_blocks;
                if (!ok) atomicOr(a.flags, FLAG_ATTN_SHAPE);
                row = ok ? ((int64_t)blk << a.bs_log2) + (key & (a.block_size - 1)) : 0;
              }
              const int64_t at = row * a.Hkv + g;
              const uint8_t* src = a.k + at * L::ROWB + t4 * L::LANEB;
#pragma unroll
              for (int i = 0; i < L::PIECES; ++i) {
                uint32_t w[L::LANEB / 4];
                if constexpr (L::LANEB == 16) {
                  const uint4 v = ok ? __ldg(reinterpret_cast<const uint4*>(src + i * 64)) : make_uint4(0, 0, 0, 0);
                  w[0] = v.x;
                  w[1] = v.y;
                  w[2] = v.z;
                  w[3] = v.w;
                } else {
                  const uint2 v = ok ? __ldg(reinterpret_cast<const uint2*>(src + i * 32)) : make_uint2(0, 0);
                  w[0] = v.x;
                  w[1] = v.y;
                }
                constexpr int PS = KS / L::PIECES;  // k-steps of a piece
                if constexpr (TY == BF16) {
#pragma unroll
                  for (int x = 0; x < PS; ++x) {
                    kf[h][i * PS + x][e] = w[2 * x];
                    kf[h][i * PS + x][e + 2] = w[2 * x + 1];
                  }
                } else if constexpr (TY == E4M3) {
#pragma unroll
                  for (int x = 0; x < PS; ++x) {
                    kf[h][i * PS + x][e] = e4m3x2_to_f16x2(w[x] & 0xffffu);
                    kf[h][i * PS + x][e + 2] = e4m3x2_to_f16x2(w[x] >> 16);
                  }
                } else {
                  const uint8_t* sp = a.scales + at * (HD / 8) + t4 * (HD / 64);
                  uint32_t f = 0;
                  if (ok) f = HD == 128 ? *reinterpret_cast<const uint16_t*>(sp) : *sp;
                  f = e4m3x2_to_f16x2(f);
                  const uint32_t u[2] = {lo_twice(f), hi_twice(f)};
#pragma unroll
                  for (int x = 0; x < PS / 2; ++x) {  // a word: two k-steps
                    uint32_t d[4];
                    e2m1x8_to_f16(w[x], d);
                    const uint32_t s = u[x >> 1];
                    kf[h][2 * x][e] = hmul2(d[0], s);
                    kf[h][2 * x][e + 2] = hmul2(d[1], s);
                    kf[h][2 * x + 1][e] = hmul2(d[2], s);
                    kf[h][2 * x + 1][e + 2] = hmul2(d[3], s);
                  }
                }
              }
            }
          const bool edge = key0 + 32 > T;  // a key that some counted row does not see
          float acc[2][2] = {};  // keys r8, r8 + 8 of each m-tile
          for (int q = 0; q < ntile; ++q) {
            float s[2][4] = {};
#pragma unroll
            for (int jj = 0; jj < KS / 2; ++jj) {
              const uint4 v = sQ[(q * (KS / 2) + jj) * 32 + lane];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                mma<F16>(s[h], kf[h][2 * jj], v.x, v.y);
                mma<F16>(s[h], kf[h][2 * jj + 1], v.z, v.w);
              }
            }
            const float4 rr = *reinterpret_cast<const float4*>(s_row + q * 8 + 2 * t4);
            if constexpr (STATS) {
              const int2 ii = *reinterpret_cast<const int2*>(s_i + q * 8 + 2 * t4);
#pragma unroll
              for (int e = 0; e < 2; ++e) {  // rows 2 t, 2 t + 1
                float x[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  x[k] = s[k >> 1][(k & 1) * 2 + e] * (e ? rr.z : rr.x);
                  const int key = key0 + (k >> 1) * 16 + (k & 1) * 8 + r8;
                  if (edge && (key > T + (e ? ii.y : ii.x) || key >= nkeys)) x[k] = -INFINITY;
                }
                float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const float mu = mx == -INFINITY ? 0.f : mx;
                float sum = (ex2(x[0] - mu) + ex2(x[1] - mu)) + (ex2(x[2] - mu) + ex2(x[3] - mu));
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                if (r8 == 0) {
                  float2* ml = s_ml + warp * RB + q * 8 + 2 * t4 + e;
                  const float2 o = *ml;
                  const float m = fmaxf(o.x, mx), mm = m == -INFINITY ? 0.f : m;
                  *ml = make_float2(m, o.y * ex2(o.x - mm) + sum * ex2(mx - mm));
                }
              }
            } else {
              float w[2][4];
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  w[h][e] = ex2(fmaf(s[h][e], e & 1 ? rr.z : rr.x, e & 1 ? -rr.w : -rr.y));
              if (edge) {
                const int2 ii = *reinterpret_cast<const int2*>(s_i + q * 8 + 2 * t4);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    const int key = key0 + h * 16 + (e >> 1) * 8 + r8;
                    if (key > T + (e & 1 ? ii.y : ii.x)) w[h][e] = 0.f;
                  }
              }
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                acc[h][0] += w[h][0] + w[h][1];
                acc[h][1] += w[h][2] + w[h][3];
              }
            }
          }
          if constexpr (!STATS) {
            float* dst = a.mass + ((int64_t)b * a.Hkv + g) * a.mass_stride;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float v = acc[h][e];
                v += __shfl_xor_sync(0xffffffffu, v, 1);
                v += __shfl_xor_sync(0xffffffffu, v, 2);
                const int key = key0 + h * 16 + e * 8 + r8;
                if (t4 == 0 && key < nkeys) dst[key] += v;
              }
          }
        }
        if constexpr (STATS) {
          __syncthreads();
          const int64_t slot = blockIdx.x + (int64_t)b * a.Hkv + g;
          for (int r = tid; r < nr; r += NTHREADS) {
            float m = -INFINITY, l = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) m = fmaxf(m, s_ml[w * RB + r].x);
            const float mm = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int w = 0; w < NW; ++w) l += s_ml[w * RB + r].y * ex2(s_ml[w * RB + r].x - mm);
            a.part[slot * a.max_rows + rb + r] = make_float2(m, l);
          }
        }
      }
      t += j1 - j0;
      in_b += j1 - j0;
    }
    pl.in_b = 0;
    pl.q_off += 1 + D;
  }
}

// L of every counted row: the parts of the CTAs whose ranges hold its (sequence, KV head)'s
// tiles, joined in order. The CTAs walk the line as the pass before did; a CTA takes the units
// whose first tile is in its range.
__global__ void __launch_bounds__(NTHREADS) mass_join_kernel(const MassArgs a) {
  pdl_trigger();
  pdl_wait();
  Place pl;
  if (!find_place(a, pl)) return;
  int64_t t = pl.t;
  for (int b = pl.b; t < pl.end; ++b) {
    int T, D, n;
    lengths(a, b, T, D, n);
    const int nt = tiles_of(T, n);
    const int rows = a.G * n;
    for (int64_t in_b = pl.in_b; in_b < (int64_t)a.Hkv * nt && t < pl.end;) {
      const int g = (int)(in_b / nt), j0 = (int)(in_b - (int64_t)g * nt);
      if (j0 == 0) {
        // the line's ranges: tile x is CTA ((x + 1) n_ctas - 1) / total's
        const int c0 = cta_of_tile(t, pl.total, a.n_ctas), c1 = cta_of_tile(t + nt - 1, pl.total, a.n_ctas);
        const int64_t unit = (int64_t)b * a.Hkv + g;
        for (int r = threadIdx.x; r < rows; r += NTHREADS) {
          float m = -INFINITY, l = 0.f;
          for (int c = c0; c <= c1; ++c) {
            if (!cta_has_tiles(c, pl.total, a.n_ctas)) continue;
            const float2 v = a.part[(unit + c) * a.max_rows + r];
            const float mn = fmaxf(m, v.x), mm = mn == -INFINITY ? 0.f : mn;
            l = l * ex2(m - mm) + v.y * ex2(v.x - mm);
            m = mn;
          }
          a.lse_ws[(pl.q_off + r / a.G) * a.Hq + (int64_t)g * a.G + r % a.G] = (m + log2f(l)) * LN2;
        }
      }
      const int64_t step = min((int64_t)nt - j0, pl.end - t);
      t += step;
      in_b += step;
    }
    pl.in_b = 0;
    pl.q_off += 1 + D;
  }
}

struct MassWs {
  size_t lse, part, total;
};
int mass_ctas(int sms) { return 2 * sms; }
MassWs mass_ws(const sv_attn_desc* d, int sms) {
  MassWs w;
  const size_t max_rows = (size_t)(d->num_q_heads / d->num_kv_heads) * (1 + d->max_draft_len);
  const size_t slots = (size_t)mass_ctas(sms) + (size_t)d->batch * d->num_kv_heads;
  w.lse = 256;
  w.part = align_up(w.lse + 4 * (size_t)d->q_rows * d->num_q_heads, 256);
  w.total = align_up(w.part + 8 * slots * max_rows, 256);
  return w;
}

template <int HD, int TY, bool STATS>
cudaError_t launch_pass(const MassArgs& a, cudaStream_t s) {
  const size_t smem = RB * HD * 2 + RB * (sizeof(float2) + sizeof(int)) + (STATS ? NW * RB * sizeof(float2) : 0);
  auto kernel = mass_kernel<HD, TY, STATS>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(a.n_ctas), dim3(NTHREADS), smem, s, a);
}
template <int HD, int TY>
cudaError_t launch_all(const MassArgs& a, cudaStream_t s) {
  if (!a.lse) {
    cudaError_t e = launch_pass<HD, TY, true>(a, s);
    if (e == cudaSuccess) e = launch_pdl(mass_join_kernel, dim3(a.n_ctas), dim3(NTHREADS), 0, s, a);
    if (e != cudaSuccess) return e;
  }
  return launch_pass<HD, TY, false>(a, s);
}

}  // namespace

size_t mass_ws_bytes(const sv_attn_desc* d, int sms) { return mass_ws(d, sms).total; }

cudaError_t launch_mass(const sv_attn_desc* d, float scale_log2, const void* q, const void* k_pages,
                        const void* scales, const float* kv_scale, int64_t num_blocks, int block_size,
                        const int32_t* table, int max_blocks, const int32_t* seq_lens,
                        const int32_t* draft_len, const int32_t* row_count, const float* lse,
                        float* mass, int64_t mass_stride, void* ws, int sms, cudaStream_t s) {
  const MassWs w = mass_ws(d, sms);
  MassArgs a = {};
  a.q = (const uint16_t*)q;
  a.k = (const uint8_t*)k_pages;
  a.scales = (const uint8_t*)scales;
  a.kv_scale = kv_scale;
  a.table = table;
  a.seq_lens = seq_lens;
  a.draft_len = draft_len;
  a.row_count = row_count;
  a.lse = lse;
  a.lse_ws = (float*)((uint8_t*)ws + w.lse);
  a.part = (float2*)((uint8_t*)ws + w.part);
  a.mass = mass;
  a.flags = (uint32_t*)ws;
  a.mass_stride = mass_stride;
  a.q_rows = d->q_rows;
  a.num_blocks = num_blocks;
  a.B = d->batch;
  a.Hq = d->num_q_heads;
  a.Hkv = d->num_kv_heads;
  a.G = a.Hq / a.Hkv;
  a.max_draft = d->max_draft_len;
  a.max_seq = d->max_seq_len;
  a.bt_stride = max_blocks;
  a.block_size = block_size;
  while ((1 << a.bs_log2) < block_size) ++a.bs_log2;
  a.max_rows = a.G * (1 + d->max_draft_len);
  a.n_ctas = mass_ctas(sms);
  a.scale_log2 = scale_log2;
  if (d->head_dim == 128)
    return d->kv_dtype == SV_BF16 ? launch_all<128, BF16>(a, s)
           : d->kv_dtype == SV_FP8_E4M3 ? launch_all<128, E4M3>(a, s)
                                        : launch_all<128, KV4>(a, s);
  return d->kv_dtype == SV_BF16 ? launch_all<64, BF16>(a, s)
         : d->kv_dtype == SV_FP8_E4M3 ? launch_all<64, E4M3>(a, s)
                                      : launch_all<64, KV4>(a, s);
}

}  // namespace sv
