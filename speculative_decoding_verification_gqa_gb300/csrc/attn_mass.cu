// attn_mass.cu -- attention weight added up by cached position (spec_attn_mass): what the rows
// of a verify step gave to every key of a KV head, summed over the group's query heads and the
// window's counted rows,
//   mass[b, g, j] += sum_{h, i} 2^(s_{h,i,j} - L_{h,i}),  s scores in log2 units, L their
// row's log-sum. Every key is one thread quartet's and the rows are added in one order, so the
// sums have the same bits every time, without atomics.
//
// Keys are the M dimension (S^T = K Q^T, m16n8k16): the sum over rows then runs along a
// thread's own accumulators, and only at the end over the four lanes of a key. A warp takes
// chunks of 32 keys through a ring of cp.async stages of its own and builds the K fragments from
// the raw rows: the order of d is free as long as Q has the same, so lane t of a key's four takes
// whole 16-byte pieces (every fourth) of its row. Q lies in shared memory in fragment order.
//
// Without given log-sums a first pass over the keys reduces (max, sum) for every row, 64 rows at
// a time in registers, each lane for its own keys, and each CTA for its own tiles; the second
// pass begins every unit by joining those.
//
// Work: a unit is a sequence and one or two neighbouring KV heads, whose rows share 128-byte
// lines of a 4-bit cache; its 12 warps take the heads in turn and 32 keys each, a tile. Units lie
// end to end on one line, a unit's start and every tile as long as their work: a tile's fixed
// part and one for every 8 rows. Each CTA (one an SM) takes the tiles that begin in its equal
// share of the line, and finds its place by scanning the lengths itself.
//
// Measured (d 128): 32 sequences of up to 16384 positions, 8 tokens, 32 query and 4 KV heads,
// bf16: the first pass 61 us, the second 70, of 278 MB each (4.0 to 4.5 TB/s; 62 us with log-sums
// given); 16 of up to 8192, 9 tokens, 8 KV heads, 4 bits, log-sums given: 23.4-25 us for 43 MB, a
// chain of short phases (scan, Q, ten chunks a warp). With 40 to 52% of the issue slots taken both
// are bound by latency: 12 warps of up to 168 registers, 64 of which hold two tiles of decoded
// keys, are all that an SM has. (The first pass spills up to 24 words a thread with bf16, 14 with
// E4M3, 9 with 4 bits.) Q is held in f16 next to E4M3 and 4-bit keys. On tcgen05 with K by TMA (a key
// in a TMEM lane, a row's sum in a register) they took 122 to 131 and 28 us: a page of 16 rows
// makes 2 KB boxes, about 100 clocks each.
#include <cuda_bf16.h>

#include "kv4.cuh"

namespace sv {
namespace {

constexpr int NW = 12;
constexpr int NTHREADS = NW * 32;
constexpr int CK = 32;           // keys of a chunk
constexpr int RB = 128;          // query rows held at once
constexpr int RS = 64;           // in the pass for the log-sums
constexpr float LOG2E = 1.4426950408889634f;

struct MassArgs {
  const uint16_t* q;
  const uint8_t* k;          // rows of the cache: bf16, E4M3 or E2M1 codes
  const uint8_t* scales;     // 4 bits: [.., Hkv, 2, d / 16]
  const float* kv_scale;
  const int32_t *table, *seq_lens, *draft_len, *row_count;
  const float* lse;          // [rows, Hq] natural, or null
  float2* part;              // [n_ctas + B * Hkv][max_rows] (max, sum) in log2 units
  float* mass;
  uint32_t* flags;
  int64_t mass_stride, q_rows, num_blocks;
  int B, Hq, Hkv, G, max_draft, max_seq, bt_stride, block_size, bs_log2;
  int max_rows;              // G * (1 + max_draft)
  int n_ctas;
  int heads;                 // of a unit
  int fixed;                 // a tile's loads and decoding, in 8 rows' time
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
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm(
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
  static constexpr int SB = TY == KV4 ? HD / 8 : 0;   // bytes of a row's block scales
  static constexpr int STAGE = CK * (ROWB + SB);
  static constexpr int ST = TY == BF16 ? 2 : 4;       // ring stages of a warp
  static constexpr int CH = ROWB / 16;                // 16-byte pieces of a row
  // where piece c of row kk of a stage lies: rows of 128 bytes and more exchange places so that
  // eight lanes, four pieces of two rows, meet every bank once
  __device__ static __forceinline__ int place(int kk, int c) {
    return kk * CH + (ROWB == 256 ? c ^ ((kk & 1) << 2) : ROWB == 128 ? c ^ ((kk & 1) << 2) : c);
  }
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
// A sequence's units: their tiles (up to the keys that a counted row sees), the length of a tile
// on the line (its rows' MMAs and exponentials by 8 rows, `fixed` of that for its loads and
// decoding) and of a unit with its START (all 0 without a counted row).
constexpr int START = 16;
struct SeqLine {
  int tiles, tile;
};
__device__ __forceinline__ SeqLine line_of(const MassArgs& a, int T, int n) {
  if (n == 0) return SeqLine{0, 1};
  const int keys = NW / a.heads * CK;  // of a tile
  SeqLine s;
  s.tiles = (int)(((int64_t)T + n + keys - 1) / keys);
  s.tile = a.fixed + (a.G * n + 15) / 16 * 2;
  return s;
}
__device__ __forceinline__ int64_t unit_length(const SeqLine& s) {
  return s.tiles == 0 ? 0 : START + (int64_t)s.tiles * s.tile;
}

// A CTA's place on the line, whose range is [v0, v1).
struct Place {
  int64_t total, v0, v1;
  int b;                // sequence that holds v0
  int64_t base, q_off;  // where that begins on the line, and its first packed row
};
__device__ __forceinline__ int64_t ceil_div(int64_t x, int y) { return x <= 0 ? 0 : (x + y - 1) / y; }
__device__ __forceinline__ int64_t range_begin(const MassArgs& a, int64_t total, int c) {
  return c * total / a.n_ctas;
}
// Scan of the lengths: totals, and the sequence that holds the range's beginning. One CTA's
// threads together; false (flag set) if a length is out of range. One pass for up to NTHREADS
// sequences, whose shares stay in registers, else two.
__device__ bool find_place(const MassArgs& a, Place& pl) {
  __shared__ int64_t s_warp[NW][2];
  __shared__ int64_t s_place[3];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  bool bad = false;
  int64_t carry[2] = {0, 0}, v[2], x[2];  // line and rows; of this thread's sequence; before it
  auto shares = [&](int base) {
    const int b = base + tid;
    v[0] = v[1] = 0;
    if (b < a.B) {
      int T, D, n;
      if (lengths(a, b, T, D, n)) {
        v[0] = a.Hkv / a.heads * unit_length(line_of(a, T, n));
        v[1] = 1 + D;
      } else {
        bad = true;
      }
    }
    x[0] = v[0];
    x[1] = v[1];
    const int nw = min(NW, (a.B - base + 31) / 32);
    if (wid < nw) {
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
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      int64_t before = carry[k];
      for (int w = 0; w < nw; ++w) {
        const int64_t y = s_warp[w][k];
        if (w < wid) before += y;
        carry[k] += y;
      }
      x[k] += before - v[k];  // exclusive
    }
  };
  for (int base = 0; base < a.B; base += NTHREADS) {
    if (base > 0) __syncthreads();
    shares(base);
  }
  if (__syncthreads_or(bad || carry[1] > a.q_rows)) {
    if (tid == 0) atomicOr(a.flags, FLAG_ATTN_SHAPE);
    return false;
  }
  pl.total = carry[0];
  pl.v0 = range_begin(a, pl.total, blockIdx.x);
  pl.v1 = range_begin(a, pl.total, blockIdx.x + 1);
  if (pl.v0 >= pl.v1) return false;
  auto look = [&](int base) {
    if (pl.v0 >= x[0] && pl.v0 < x[0] + v[0]) {
      s_place[0] = base + tid;
      s_place[1] = x[0];
      s_place[2] = x[1];
    }
  };
  if (a.B <= NTHREADS) {
    look(0);
  } else {
    carry[0] = carry[1] = 0;
    for (int base = 0; base < a.B; base += NTHREADS) {
      __syncthreads();
      shares(base);
      look(base);
    }
  }
  __syncthreads();
  pl.b = (int)s_place[0];
  pl.base = s_place[1];
  pl.q_off = s_place[2];
  return true;
}

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

// STATS: the first pass, (max, sum) of each row over the CTA's tiles; else the weights.
template <int HD, int TY, bool STATS, int HG>
__global__ void __launch_bounds__(NTHREADS, 1) mass_kernel(const MassArgs a) {
  using L = LM<HD, TY>;
  constexpr int NK = NW / HG, KT = NK * CK;          // chunks and keys of a tile, each head
  constexpr int KS = L::KS, ST = L::ST, ROWS = STATS ? RS : RB / HG;  // rows held of each head
  constexpr bool F16 = TY != BF16;
  extern __shared__ __align__(128) uint8_t smem[];
  uint4* sQ0 = reinterpret_cast<uint4*>(smem);                           // [HG][ROWS / 8][KS / 2][32]
  float2* s_row0 = reinterpret_cast<float2*>(smem + HG * ROWS * HD * 2); // [HG][ROWS] (score scale, log-sum)
  int* s_i = reinterpret_cast<int*>(s_row0 + HG * ROWS);                 // [ROWS] window row
  float2* s_ml = reinterpret_cast<float2*>(smem);  // STATS, in Q's place: [NW][ROWS]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r8 = lane >> 2, t4 = lane & 3;
  const int hg = warp % HG, kw = warp / HG;
  const uint4* sQ = sQ0 + hg * ROWS / 8 * (KS / 2) * 32;
  const float2* s_row = s_row0 + hg * ROWS;
  uint8_t* ring = smem + HG * ROWS * (HD * 2 + 8) + ROWS * 4 + warp * ST * L::STAGE;
  pdl_trigger();
  pdl_wait();
  Place pl;
  if (!find_place(a, pl)) return;
  const int code_bytes = a.Hkv * L::ROWB, scale_bytes = a.Hkv * L::SB;  // of a cache position

  for (int b = pl.b; b < a.B && pl.base < pl.v1; ++b) {
    int T, D, n;
    lengths(a, b, T, D, n);
    const SeqLine sl = line_of(a, T, n);
    const int nt = sl.tiles, W = sl.tile;
    const int64_t length = unit_length(sl);
    const int nkeys = T + n;             // keys that a counted row sees
    const int rows = a.G * n;
    const int32_t* tab = a.table + (size_t)b * a.bt_stride;
    const int groups = a.Hkv / HG;
    // units with tiles that begin in the range
    for (int gg = length == 0 || pl.v0 <= pl.base ? 0 : (int)min((int64_t)groups, (pl.v0 - pl.base) / length);
         length > 0 && gg < groups && pl.base + gg * length < pl.v1; ++gg) {
      const int64_t first = pl.base + gg * length + START;  // where the unit's first tile begins
      const int j0 = (int)min((int64_t)nt, ceil_div(pl.v0 - first, W));
      const int j1 = (int)min((int64_t)nt, ceil_div(pl.v1 - first, W));
      if (j0 >= j1) continue;
      const int g = gg * HG + hg;
      // this warp's chunks of the tiles: 32 keys of each
      const int key_first = j0 * KT + kw * CK;
      const int mine = key_first < nkeys ? min(j1 - j0, (nkeys - key_first + KT - 1) / KT) : 0;
      const int64_t lane_at = (int64_t)(lane / L::CH % 8) * code_bytes + g * L::ROWB + lane % L::CH * 16;
      const uint8_t* kp = a.k + lane_at;
      const uint8_t* sp = TY == KV4 ? a.scales + (int64_t)(lane & 7) * scale_bytes + g * L::SB : nullptr;
      float* dst = a.mass + ((int64_t)b * a.Hkv + g) * a.mass_stride;
      for (int rb = 0; rb < rows; rb += ROWS) {
        const int nr = min(ROWS, rows - rb), ntile = (nr + 15) / 16 * 2;  // (two at a time)
        // ---- the ring. Eight consecutive keys lie in one block: a chunk has four table entries,
        // read a chunk ahead by the lanes
        constexpr int UNSEEN = -2;
        auto entry = [&](int i) -> int {
          const int pos = key_first + i * KT + 8 * t4;
          return i < mine && pos < nkeys ? __ldg(tab + (pos >> a.bs_log2)) : UNSEEN;
        };
        int ent = entry(0);
        auto issue = [&](int i) {
          if (i < mine) {
            const uint32_t st = smem_u32(ring + (i % ST) * L::STAGE);
            const int key0 = key_first + i * KT;
            int base = -1;  // cache row of the first of this lane's eight keys
            if (ent >= 0 && ent < a.num_blocks)
              base = (ent << a.bs_log2) + ((key0 + 8 * t4) & (a.block_size - 1));
            else if (ent != UNSEEN)
              atomicOr(a.flags, FLAG_ATTN_SHAPE);  // an entry outside the pool
            constexpr int PER = 32 / L::CH;  // keys of a step (2: within eight, 4, 8, 16)
#pragma unroll
            for (int j = 0; j < L::CH; ++j) {
              const int kk = j * PER + lane / L::CH;
              const int row = __shfl_sync(0xffffffffu, base, kk >> 3);
              const bool ok = row >= 0 && key0 + kk < nkeys;
              // (the lane's address holds its key of a step; steps shorter than eight keys walk on)
              const int64_t at = (int64_t)(row + (PER < 8 ? (j * PER & 7) : 0)) * code_bytes;
              cp_async<16>(st + L::place(kk, lane % L::CH) * 16, kp + (ok ? at : 0), ok);
            }
            if constexpr (TY == KV4) {
              const int row = __shfl_sync(0xffffffffu, base, lane >> 3);
              const bool ok = row >= 0 && key0 + lane < nkeys;
              cp_async<L::SB>(st + CK * L::ROWB + lane * L::SB, sp + (ok ? (int64_t)row * scale_bytes : 0), ok);
            }
            ent = entry(i + 1);
          }
          cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < ST - 1; ++i) issue(i);

        __syncthreads();  // the last block's readers are done
        // ---- Q rows rb .. of the unit, in fragment order; row = window row i, head of the group
        for (int idx = tid; idx < HG * ntile * 8 * (HD / 8); idx += NTHREADS) {
          const int rr = idx / (HD / 8), c = idx % (HD / 8);  // 8 elements; a row's lie in
          const int j = c >> 2, tt = c & 3;                   // neighbouring lanes
          const int h = rr / (ntile * 8), r = rr - h * ntile * 8;
          const int rg = rb + r;
          const bool live = r < nr;
          const int64_t row = live ? (pl.q_off + rg / a.G) * a.Hq + (int64_t)(gg * HG + h) * a.G + rg % a.G : 0;
          const float sck = a.scale_log2 * (TY == BF16 ? 1.f : a.kv_scale[gg * HG + h]);
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
          sQ0[((h * ROWS / 8 + (r >> 3)) * (KS / 2) + j) * 32 + (r & 7) * 4 + tt] = v;
          if (c == 0) {
            // rows past the block's: weight 2^-inf
            s_row0[h * ROWS + r] = make_float2(sc, !live ? INFINITY : STATS || !a.lse ? 0.f : a.lse[row] * LOG2E);
            s_i[r] = live ? rg / a.G : n - 1;
          }
        }
        __syncthreads();
        if (!STATS && !a.lse) {
          // L from the parts of the first pass: of the CTAs in whose ranges tiles of the unit
          // begin, four lanes a row
          const int c0 = cta_of_tile(first, pl.total, a.n_ctas);
          const int c1 = cta_of_tile(first + (int64_t)(nt - 1) * W, pl.total, a.n_ctas);
          const int64_t unit = (int64_t)b * groups + gg;
          for (int idx = tid; idx < (HG * nr * 4 + 31) / 32 * 32; idx += NTHREADS) {
            const int e = min(idx >> 2, HG * nr - 1), h = e / nr, r = e - h * nr;
            float m = -INFINITY, l = 0.f;
#pragma unroll 4
            for (int c = c0 + t4; c <= c1; c += 4) {
              if (c > c0 && c < c1 && ceil_div(range_begin(a, pl.total, c) - first, W) >=
                                          ceil_div(range_begin(a, pl.total, c + 1) - first, W))
                continue;  // no tile begins there
              const float2 v = __ldcg(a.part + ((unit + c) * HG + h) * a.max_rows + rb + r);
              const float mn = fmaxf(m, v.x), mm = mn == -INFINITY ? 0.f : mn;
              l = l * ex2(m - mm) + (v.x == -INFINITY ? v.y : v.y * ex2(v.x - mm));
              m = mn;
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
              const float m2 = __shfl_xor_sync(0xffffffffu, m, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
              const float mn = fmaxf(m, m2), mm = mn == -INFINITY ? 0.f : mn;
              l = (m == -INFINITY ? l : l * ex2(m - mm)) + (m2 == -INFINITY ? l2 : l2 * ex2(m2 - mm));
              m = mn;
            }
            if (t4 == 0 && (idx >> 2) < HG * nr) s_row0[h * ROWS + r].y = m + log2f(l);
          }
          __syncthreads();
        }
        float ml[STATS ? ROWS / 8 : 1][4];  // rows 2 t, 2 t + 1 of each n-tile: this lane's (max,
                                            // sum) over its own keys
        if constexpr (STATS)
#pragma unroll
          for (int q = 0; q < ROWS / 8; ++q) {
            ml[q][0] = ml[q][1] = -INFINITY;
            ml[q][2] = ml[q][3] = 0.f;
          }
        for (int i = 0; i < mine; ++i) {
          cp_async_wait<ST - 2>();
          __syncwarp();  // the chunk's bytes of every lane are here; the last chunk's are read
          issue(i + ST - 1);
          const uint8_t* st = ring + (i % ST) * L::STAGE;
          const int key0 = key_first + i * KT;
          float old[2][2];  // what the chunk's keys have had so far
          if constexpr (!STATS)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int key = key0 + h * 16 + e * 8 + r8;
                old[h][e] = t4 == 0 && key < nkeys ? dst[key] : 0.f;
              }
          // ---- K fragments of 32 keys (two m-tiles)
          uint32_t kf[2][KS][4];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int kk = h * 16 + e * 8 + r8;
#pragma unroll
              for (int x0 = 0; x0 < L::PIECES; ++x0) {
                uint32_t w[L::LANEB / 4];
                if constexpr (L::LANEB == 16) {
                  const uint4 v = *reinterpret_cast<const uint4*>(st + L::place(kk, x0 * 4 + t4) * 16);
                  w[0] = v.x;
                  w[1] = v.y;
                  w[2] = v.z;
                  w[3] = v.w;
                } else {
                  const uint2 v = *reinterpret_cast<const uint2*>(st + kk * L::ROWB + t4 * 8);
                  w[0] = v.x;
                  w[1] = v.y;
                }
                constexpr int PS = KS / L::PIECES;  // k-steps of a piece
                if constexpr (TY == BF16) {
#pragma unroll
                  for (int x = 0; x < PS; ++x) {
                    kf[h][x0 * PS + x][e] = w[2 * x];
                    kf[h][x0 * PS + x][e + 2] = w[2 * x + 1];
                  }
                } else if constexpr (TY == E4M3) {
#pragma unroll
                  for (int x = 0; x < PS; ++x) {
                    kf[h][x0 * PS + x][e] = e4m3x2_to_f16x2(w[x] & 0xffffu);
                    kf[h][x0 * PS + x][e + 2] = e4m3x2_to_f16x2(w[x] >> 16);
                  }
                } else {
                  const uint8_t* ss = st + CK * L::ROWB + kk * L::SB + t4 * (HD / 64);
                  uint32_t f = HD == 128 ? *reinterpret_cast<const uint16_t*>(ss) : *ss;
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
          const bool edge = key0 + CK > T;  // a key that some counted row does not see
          float acc[2][2] = {};  // keys r8, r8 + 8 of each m-tile
          // of n-tiles q, q + 1: four chains of MMAs
          auto scores = [&](int q, float (&s)[2][2][4]) {
#pragma unroll
            for (int jj = 0; jj < KS / 2; ++jj)
#pragma unroll
              for (int w = 0; w < 2; ++w) {
                const uint4 v = sQ[((q + w) * (KS / 2) + jj) * 32 + lane];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  mma<F16>(s[w][h], kf[h][2 * jj], v.x, v.y);
                  mma<F16>(s[w][h], kf[h][2 * jj + 1], v.z, v.w);
                }
              }
            if (edge) {
#pragma unroll
              for (int w = 0; w < 2; ++w) {
                const int2 ii = *reinterpret_cast<const int2*>(s_i + (q + w) * 8 + 2 * t4);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    const int key = key0 + h * 16 + (e >> 1) * 8 + r8;
                    if (key > T + (e & 1 ? ii.y : ii.x)) s[w][h][e] = -INFINITY;
                  }
              }
            }
          };
          if constexpr (STATS) {
#pragma unroll
            for (int q = 0; q < ROWS / 8; q += 2) {
              if (q >= ntile) break;
              float s[2][2][4] = {};
              scores(q, s);
#pragma unroll
              for (int w = 0; w < 2; ++w) {
                const float4 rr = *reinterpret_cast<const float4*>(s_row + (q + w) * 8 + 2 * t4);
                float(&o)[4] = ml[q + w];
#pragma unroll
                for (int e = 0; e < 2; ++e) {  // rows 2 t, 2 t + 1
                  const float sc = e ? rr.z : rr.x;
                  const float a0 = s[w][0][e], a1 = s[w][0][e + 2], a2 = s[w][1][e], a3 = s[w][1][e + 2];
                  const float mx = fmaxf(fmaxf(a0, a1), fmaxf(a2, a3)) * sc;
                  const float m = fmaxf(o[e], mx), nm = m == -INFINITY ? 0.f : -m;
                  const float sum = (ex2(fmaf(a0, sc, nm)) + ex2(fmaf(a1, sc, nm))) +
                                    (ex2(fmaf(a2, sc, nm)) + ex2(fmaf(a3, sc, nm)));
                  o[2 + e] = fmaf(o[2 + e], ex2(o[e] + nm), sum);
                  o[e] = m;
                }
              }
            }
          } else {
            for (int q = 0; q < ntile; q += 2) {
              float s[2][2][4] = {};
              scores(q, s);
#pragma unroll
              for (int w = 0; w < 2; ++w) {
                const float4 rr = *reinterpret_cast<const float4*>(s_row + (q + w) * 8 + 2 * t4);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  float x[4];
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    x[e] = ex2(fmaf(s[w][h][e], e & 1 ? rr.z : rr.x, e & 1 ? -rr.w : -rr.y));
                  if (edge) {  // (a row without numbers has NaN for the keys that it does not see too)
                    const int2 ii = *reinterpret_cast<const int2*>(s_i + (q + w) * 8 + 2 * t4);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                      if (key0 + h * 16 + (e >> 1) * 8 + r8 > T + (e & 1 ? ii.y : ii.x)) x[e] = 0.f;
                  }
                  acc[h][0] += x[0] + x[1];
                  acc[h][1] += x[2] + x[3];
                }
              }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float v = acc[h][e];
                v += __shfl_xor_sync(0xffffffffu, v, 1);
                v += __shfl_xor_sync(0xffffffffu, v, 2);
                const int key = key0 + h * 16 + e * 8 + r8;
                if (t4 == 0 && key < nkeys) dst[key] = old[h][e] + v;
              }
          }
        }
        cp_async_wait<0>();
        if constexpr (STATS) {
          // lanes of a column, then the head's warps
          __syncthreads();  // Q is read
#pragma unroll
          for (int q = 0; q < ROWS / 8; ++q)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float m = ml[q][e];
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
              // (a lane without a maximum has the sum 0, or NaN, which stays)
              float l = ml[q][e] == -INFINITY ? ml[q][2 + e] : ml[q][2 + e] * ex2(ml[q][e] - m);
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
              if (r8 == 0) s_ml[warp * ROWS + q * 8 + 2 * t4 + e] = make_float2(m, l);
            }
          __syncthreads();
          const int64_t slot = blockIdx.x + (int64_t)b * groups + gg;
          for (int e = tid; e < HG * nr; e += NTHREADS) {
            const int h = e / nr, r = e - h * nr;
            float m = -INFINITY, l = 0.f;
#pragma unroll
            for (int w = 0; w < NK; ++w) m = fmaxf(m, s_ml[(w * HG + h) * ROWS + r].x);
            const float mm = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int w = 0; w < NK; ++w) {
              const float2 v = s_ml[(w * HG + h) * ROWS + r];
              l += v.x == -INFINITY ? v.y : v.y * ex2(v.x - mm);
            }
            a.part[(slot * HG + h) * a.max_rows + rb + r] = make_float2(m, l);
          }
        }
      }
    }
    pl.base += groups * length;
    pl.q_off += 1 + D;
  }
}

struct MassWs {
  size_t part, total;
};
int mass_ctas(int sms) { return sms; }
MassWs mass_ws(const sv_attn_desc* d, int sms) {
  MassWs w;
  const size_t max_rows = (size_t)(d->num_q_heads / d->num_kv_heads) * (1 + d->max_draft_len);
  const size_t slots = 2 * (size_t)mass_ctas(sms) + (size_t)d->batch * d->num_kv_heads;
  w.part = 256;
  w.total = align_up(w.part + 8 * slots * max_rows, 256);
  return w;
}

template <int HD, int TY, bool STATS, int HG>
cudaError_t launch_pass(const MassArgs& a, cudaStream_t s) {
  using L = LM<HD, TY>;
  constexpr int ROWS = STATS ? RS : RB / HG;
  constexpr size_t smem = HG * ROWS * (HD * 2 + 8) + ROWS * 4 + NW * L::ST * L::STAGE;
  static_assert(smem <= 226 * 1024 && NW * ROWS * 8 <= HG * ROWS * HD * 2, "shared memory of an SM");
  auto kernel = mass_kernel<HD, TY, STATS, HG>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(a.n_ctas), dim3(NTHREADS), smem, s, a);
}
template <int HD, int TY, bool STATS>
cudaError_t launch_pass(const MassArgs& a, cudaStream_t s) {
  return a.heads == 2 ? launch_pass<HD, TY, STATS, 2>(a, s) : launch_pass<HD, TY, STATS, 1>(a, s);
}
template <int HD, int TY>
cudaError_t launch_all(const MassArgs& a, cudaStream_t s) {
  if (!a.lse) {
    const cudaError_t e = launch_pass<HD, TY, true>(a, s);
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
  // (swept: bf16 1, 2, 3, 8 of the largest case 134, 128, 134, 146 us; 4 bits 1, 3, 4, 8: 26.0,
  // 24.3, 24.5, 25.5)
  a.fixed = d->kv_dtype == SV_BF16 ? 2 : 3;
  // two heads while their rows fit where one's would: half as many units to start
  a.heads = a.Hkv % 2 == 0 && a.max_rows <= RB / 2 ? 2 : 1;
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
