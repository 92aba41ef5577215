// shared_prefix.cu -- verify attention over a prefix that a group of sequences shares: the
// plan and the join around the attention kernels.
//
// A softmax over keys A u B is the join of those over A and over B: with (m, l, O) the
// maximum, the sum of 2^(s - m) and the unnormalised output of each, m* = max(m_A, m_B) and
//   out = (2^(m_A - m*) O_A + 2^(m_B - m*) O_B) / (2^(m_A - m*) l_A + 2^(m_B - m*) l_B).
// So the prefix of a group is one part, attended by the rows of all its sequences at once
// (G * sum W rows: full tensor-core tiles, and one read of the prefix per unit's rows instead
// of one per sequence), and what is behind it one part per sequence (internal.cuh,
// SharedSeq). Units lie on a tile line split over the CTAs like that of spec_verify_attn
// (internal.cuh). tcgen05 kernels (attn_parts.cu): the prefixes' units, of 256 rows, on a
// line of their own, the sequences' on another. mma.sync kernel: all units, of 128 rows, on
// one line. A row's partial results are joined by combine_shared.
#include <cuda_bf16.h>

#include <algorithm>

#include "internal.cuh"

namespace sv {

namespace {

// Threads of the plan. It is a chain of barriers and short steps that each warp goes through,
// 4 to 5 us (7 to 9 with the window rows and the units' CTAs in the same chain). Captured calls
// with 256, 512, 768 threads: 2 sequences 10.1, 10.5, 11.5 us; 32 sequences 22.4, 22.9, 23.6;
// 64 over a prefix of 8192 65.4, 65.4, 66.1; 100 in 8 groups 46.3, 44.7, 45.1.
constexpr int PLAN_T = 512;
static_assert(PLAN_T % 32 == 0 && PLAN_T <= 1024, "whole warps, whose sums one warp scans");

// Exclusive scans of N values per thread over the block (PLAN_T threads).
template <int N>
__device__ void scan_block(const int64_t (&v)[N], int64_t (&ex)[N], int64_t (&total)[N]) {
  __shared__ int64_t s_warp[N][PLAN_T / 32];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  int64_t x[N], w[N];
#pragma unroll
  for (int k = 0; k < N; ++k) x[k] = v[k];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x[k], o);
      if (lane >= o) x[k] += y;
    }
  }
  if (lane == 31)
#pragma unroll
    for (int k = 0; k < N; ++k) s_warp[k][wid] = x[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) w[k] = lane < PLAN_T / 32 ? s_warp[k][lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int64_t y = __shfl_up_sync(0xffffffffu, w[k], o);
      if (lane >= o) w[k] += y;
    }
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    total[k] = __shfl_sync(0xffffffffu, w[k], 31);
    const int64_t before = __shfl_sync(0xffffffffu, w[k], wid > 0 ? wid - 1 : 0);
    ex[k] = x[k] - v[k] + (wid > 0 ? before : 0);
  }
  __syncthreads();  // s_warp is reused by the next scan
}

constexpr int MAJOR_ENTRIES = 16384;

// The place of a prefix's first row tile among those of all prefixes: with q_off window rows
// and n prefixes before it there are at most this many row tiles before it.
// (32 bits: a call has at most 2^22 units, api.cu.)
__device__ __forceinline__ int32_t tile_base(int q_off, int G, int row_log2, int n) {
  return ((q_off * G) >> row_log2) + n;
}

// The last index in [0, n) whose key is at most x (keys not decreasing, key(0) <= x).
template <class T, class F>
__device__ __forceinline__ int last_at_most(int n, T x, F key) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (key(mid) <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Unit u: row tile mt and KV head g of part v = s, from cache position kbase on, its first
// tile `tile` of the line. `both`: for the mma.sync kernel, which reads parts and units.
__device__ __forceinline__ void put_unit(const AttnParams& p, bool both, int u, int v,
                                         const SharedSeq& s, int g, int mt, int kbase, int tile) {
  p.ubeg[u] = tile;
  if (both) {
    p.units[u] = make_int4(v, g, mt, kbase);
    return;
  }
  const int rt = v < p.num_groups ? 1 << p.row_log2 : MT;
  const int rows = min(rt, p.G * s.rows - mt * rt);
  p.sunits[u] = SharedUnit{s.q_off, g, mt, kbase, s.start - kbase, s.nkeys - kbase,
                           s.last0 - kbase, rows, s.table_row, tile, s.nt};
}

constexpr int CACHED = 1024;        // sequences, and groups, kept in shared memory
constexpr int CACHED_UNITS = 1024;  // unit starts kept in shared memory
constexpr int MIN_PART = 4;         // tiles that are worth a CTA of the prefixes

struct PlanShared {
  int32_t gb[CACHED + 1], len[CACHED];                      // groups
  int32_t q[CACHED], T[CACHED], ub[CACHED], tb[CACHED];  // sequences
  uint16_t n[CACHED];
  uint8_t D[CACHED];
  int32_t ubeg[CACHED_UNITS + 1];
  int4 entry[PLAN_T];
  uint32_t prefix_units, prefix_tiles;  // (of a valid call)
  int maxmt;
};

// Three CTAs check the call and describe its parts; the first writes the prefixes' line (pa),
// the second the sequences' (pb), the third the window rows. (A single line: one CTA for all.)
// All make the same checks, so a call is skipped as a whole. All of it is latency, a chain of dependent
// steps, hence the tables in shared memory and arithmetic in 32 bits where it suffices.
__global__ void __launch_bounds__(PLAN_T) plan_shared_kernel(AttnParams pa, AttnParams pb) {
  const bool both = gridDim.x == 1;  // one line for all parts
  const bool prefixes = both || blockIdx.x == 0, sequences = both || blockIdx.x == 1;
  const bool window_rows = both || blockIdx.x == 2;
  const AttnParams& p = prefixes && !both ? pa : pb;
  const int tid = threadIdx.x, NG = p.num_groups, B = p.B, G = p.G;
  const int seq_box = min(p.block_size, pb.kt), row_log2 = p.row_log2;
  const int prefix_log2 = __ffs(pa.kt) - 1, seq_log2 = __ffs(pb.kt) - 1;
  __shared__ PlanShared sm;
  pdl_trigger();
  pdl_wait();
  // the first lengths are asked for before the groups are looked at
  const HandOver was = *p.handover;
  int T0 = 0, D0 = 0;
  if (tid < B) {
    T0 = p.seq_lens[tid];
    D0 = p.draft_len[tid];
  }
  if (tid == 0) {
    sm.maxmt = 0;
    sm.prefix_units = sm.prefix_tiles = 0;
  }
  bool bad = false;
  // the groups: consecutive ranges of the batch
  for (int n = tid; n < NG; n += PLAN_T) {
    const int g0 = p.group_begin[n], g1 = p.group_begin[n + 1], P = p.prefix_len[n];
    if (g0 < 0 || g1 < g0 || g1 > B || (n == 0 && g0 != 0) || (n == NG - 1 && g1 != B) || P < 0 ||
        P > p.max_seq)
      bad = true;
    if (n < CACHED) {
      sm.gb[n] = g0;
      sm.len[n] = P;
      if (n == NG - 1 || n == CACHED - 1) sm.gb[n + 1] = g1;
    }
  }
  bad = __syncthreads_or(bad);
  auto group_at = [&](int n) -> int { return NG <= CACHED ? sm.gb[n] : p.group_begin[n]; };
  auto prefix_at = [&](int n) -> int { return NG <= CACHED ? sm.len[n] : p.prefix_len[n]; };
  // the sequences, and their units and tiles, which come first on a line for both
  SharedSeq* seq = p.parts + NG;
  auto describe = [&](int b, int T, int D, int n) {
    const int P = prefix_at(n);
    SharedSeq s = {};
    s.rows = 1 + D;
    s.start = P;
    s.nkeys = T + 1 + D;
    s.last0 = T;
    s.table_row = b;
    s.alone = P == 0;
    s.group = n;
    s.nmt = (G * s.rows + MT - 1) / MT;
    s.nt = (s.nkeys - (P & ~(seq_box - 1)) + pb.kt - 1) >> seq_log2;
    return s;
  };
  int64_t q_total = 0, U = 0, TT = 0;
  for (int base = 0; base < B && !bad; base += PLAN_T) {
    const int b = base + tid;
    SharedSeq s = {};
    if (b < B) {
      const int T = base == 0 ? T0 : p.seq_lens[b], D = base == 0 ? D0 : p.draft_len[b];
      const int n = last_at_most(NG, b, group_at);
      if (T < prefix_at(n) || T > p.max_seq || D < 0 || D > p.max_draft ||
          (((int64_t)T + D + p.block_size) >> p.bs_log2) > p.bt_stride)
        bad = true;
      else
        s = describe(b, T, D, n);
    }
    const int64_t c[2] = {(int64_t)s.rows << 32 | (uint32_t)(p.Hkv * s.nmt),  // two sums in one
                          (int64_t)p.Hkv * s.nmt * s.nt};
    int64_t ex[2], tot[2];
    scan_block<2>(c, ex, tot);
    if (b < B) {
      s.q_off = q_total + (ex[0] >> 32);
      s.ubase = (int32_t)(U + (int64_t)(uint32_t)ex[0]);
      s.tbase = (int32_t)(TT + ex[1]);
      if (B <= CACHED) {
        sm.q[b] = (int32_t)s.q_off;
        sm.T[b] = s.last0;
        sm.D[b] = (uint8_t)(s.rows - 1);
        sm.n[b] = (uint16_t)s.group;  // (below B)
        sm.ub[b] = s.ubase;
        sm.tb[b] = s.tbase;
      } else {
        p.row_begin[b] = (int32_t)s.q_off;
      }
      // (of two CTAs that write and read a long batch here, both write the same)
      if (both || (B > CACHED && !prefixes)) seq[b] = s;
    }
    q_total += tot[0] >> 32;
    U += (uint32_t)tot[0];
    TT += tot[1];
    bad = __syncthreads_or(bad);
  }
  // (every CTA knows the sequences' work, for the shares of the SMs)
  const int64_t U_seq = U, TT_seq = TT;
  if (!sequences) U = TT = 0;
  bad = bad || q_total > p.q_rows || U > p.max_units || TT >= 0x7fffffffll;
  auto seq_at = [&](int b) {
    if (B > CACHED) return seq[b];
    SharedSeq s = describe(b, sm.T[b], sm.D[b], sm.n[b]);
    s.q_off = sm.q[b];
    s.ubase = sm.ub[b];
    s.tbase = sm.tb[b];
    return s;
  };
  auto first_row = [&](int b) -> int {
    return b >= B ? (int)q_total : B <= CACHED ? sm.q[b] : p.row_begin[b];
  };
  // the prefixes
  auto prefix_part = [&](int n) {
    const int g0 = group_at(n), P = prefix_at(n), q0 = first_row(g0);
    SharedSeq s = {};
    s.q_off = q0;
    s.rows = P > 0 ? first_row(group_at(n + 1)) - q0 : 0;
    s.nkeys = P;
    s.last0 = P - 1;
    s.table_row = g0;
    s.group = n;
    s.nmt = (G * s.rows + (1 << row_log2) - 1) >> row_log2;
    s.nt = (P + pa.kt - 1) >> prefix_log2;
    s.mbase = tile_base(q0, G, row_log2, n);
    return s;
  };
  if (!bad && sequences) {  // (TT and U are in range: every unit below is)
    for (int u = tid; u < (int)U; u += PLAN_T) {
      const int b = B <= CACHED ? last_at_most(B, u, [&](int i) { return sm.ub[i]; })
                                : last_at_most(B, u, [&](int i) { return seq[i].ubase; });
      const SharedSeq s = seq_at(b);
      const int k = u - s.ubase, g = s.nmt == 1 ? k : k / s.nmt, tile = s.tbase + k * s.nt;
      put_unit(p, both, u, NG + b, s, g, k - g * s.nmt, s.start & ~(seq_box - 1), tile);
      if (u < CACHED_UNITS) sm.ubeg[u] = tile;
    }
  }
  if (!bad && window_rows) {
    for (int w = tid; w < (int)q_total; w += PLAN_T) {
      const int b = last_at_most(B, w, first_row);
      const SharedSeq s = seq_at(b);
      const int q0 = first_row(group_at(s.group));  // the group's first row
      int4* dst = reinterpret_cast<int4*>(p.rows + w);
      dst[0] = make_int4(w - (int)s.q_off, s.ubase, s.nmt,
                         s.alone ? -1 : tile_base(q0, G, row_log2, s.group));
      dst[1] = make_int4(w - q0, 0, 0, 0);
    }
  }
  if (!both && window_rows) return;
  for (int n = tid; n < NG && !bad; n += PLAN_T) {
    const SharedSeq s = prefix_part(n);
    atomicMax(&sm.maxmt, s.nmt);
    atomicAdd(&sm.prefix_units, (uint32_t)(p.Hkv * s.nmt));
    atomicAdd(&sm.prefix_tiles, (uint32_t)(p.Hkv * s.nmt) * s.nt);
    if (both) p.parts[n] = s;
  }
  __syncthreads();
  // Units of the prefixes, entry (row tile mt, part v) by entry, the KV heads of an entry
  // together. Row-tile-major (mt first), so that the slices of the line that read the same
  // prefix are read by their CTAs at about the same time and share it through L2; with very
  // many groups of very different sizes part-major, over the row tiles' places.
  const int maxmt = sm.maxmt;
  const bool major = (int64_t)maxmt * NG <= MAJOR_ENTRIES;
  const int entries =
      prefixes && !bad ? (major ? maxmt * NG : tile_base((int)q_total, G, row_log2, NG)) : 0;
  for (int base = 0; base < entries; base += PLAN_T) {
    const int e = base + tid;
    int v = 0, mt = 0;
    int64_t c[2] = {0, 0}, ex[2], tot[2];
    if (e < entries) {
      if (major) {
        mt = e / NG;
        v = e - mt * NG;
      } else {
        auto place = [&](int i) { return tile_base(first_row(group_at(i)), G, row_log2, i); };
        v = last_at_most(NG, e, place);
        mt = e - place(v);
      }
      const SharedSeq s = prefix_part(v);
      if (mt < s.nmt) {
        c[0] = p.Hkv;
        c[1] = (int64_t)p.Hkv * s.nt;
      }
    }
    scan_block<2>(c, ex, tot);
    const bool fits = U + tot[0] <= p.max_units && TT + tot[1] < 0x7fffffffll;
    sm.entry[tid] = c[0] > 0 ? make_int4(v, mt, (int)(U + ex[0]), (int)(TT + ex[1])) : make_int4(-1, 0, 0, 0);
    __syncthreads();
    const int pairs = min(entries - base, PLAN_T) * p.Hkv;
    for (int k = tid; fits && k < pairs; k += PLAN_T) {
      const int4 en = sm.entry[k / p.Hkv];
      if (en.x < 0) continue;
      const int g = k % p.Hkv, u = en.z + g;
      const SharedSeq s = prefix_part(en.x);
      if (g == 0) p.tile_unit[s.mbase + en.y] = u;
      put_unit(p, both, u, en.x, s, g, en.y, 0, en.w + g * s.nt);
      if (u < CACHED_UNITS) sm.ubeg[u] = en.w + g * s.nt;
    }
    U += tot[0];
    TT += tot[1];
    __syncthreads();
  }
  bad = bad || U > p.max_units || TT >= 0x7fffffffll;
  if (bad) U = TT = 0;  // (every thread: nothing below is then written or run)
  if (tid == 0) {
    if (bad) atomicOr(p.flags, FLAG_ATTN_SHAPE);
    // (a call whose prefixes' kernel was not launched has left permits without tickets)
    if (prefixes && was.tickets != was.permits) p.handover->tickets = was.permits;
    p.hdr->num_units = (int32_t)U;
    p.hdr->total_tiles = (int32_t)TT;
    p.hdr->kt = p.kt;
    p.hdr->sum_w = bad ? 0 : q_total;
    p.ubeg[U] = (int32_t)TT;
    if (U <= CACHED_UNITS) sm.ubeg[U] = (int32_t)TT;
  }
  __syncthreads();
  // CTA c starts at the first tile at or after its position on the virtual line. One line:
  // the CTAs' parts of it are equal. Two lines run at the same time (attn_parts.cu): with W_p
  // and W_s the work of the prefixes and the sequences, in prefix tiles, the sequences get the
  // N SMs that finish theirs in T = (W_p + W_s) / SMs, the prefixes' CTAs on the other SMs
  // get parts of T each, and the last N, which follow the sequences, what is left. No part
  // is shorter than a tile, so every CTA between the first and the last of a unit has tiles
  // of it.
  const int32_t* ubeg = U <= CACHED_UNITS ? sm.ubeg : p.ubeg;
  const int X = p.switch_tiles;
  const int64_t VT = TT + U * X;
  int C1 = (int)min((int64_t)p.n_ctas, max(VT, (int64_t)1)), C2 = 0;
  int64_t V1 = VT;  // C1 CTAs take equal parts of [0, V1), C2 after them of [V1, VT)
  if (!both) {
    const int sms = pa.n_ctas;  // one CTA of prefixes per SM
    const uint32_t VP = sm.prefix_tiles + sm.prefix_units * pa.switch_tiles;
    const float ws = (float)(uint32_t)(TT_seq + U_seq * pb.switch_tiles) * pb.tile_cost;
    const float T = fmaxf(((float)VP + ws) / sms, (float)MIN_PART);
    const int half_n = ((int)ceilf(ws / T) + 1) / 2;  // pairs of SMs
    const int N = VP > 0 ? min(max(2 * half_n, 2), max(sms - 2, 1)) : sms;
    if (sequences) {
      C1 = min(C1, 2 * N);
    } else {
      C1 = (int)min((int64_t)max(sms - N, 1), max(VT, (int64_t)1));
      const int64_t early = (uint32_t)(C1 * T);
      if (VT - early >= N * MIN_PART) {
        V1 = early;
        C2 = N;
      }
    }
  }
  const int C = C1 + C2;
  // (VT < 2^31 + 2^24: 32 bits without a sign)
  auto begin_of = [&](int c) -> int64_t {
    const bool one = c <= C1;
    const uint32_t k = one ? c : c - C1, n = one ? C1 : C2, v = (uint32_t)(one ? V1 : VT - V1);
    const uint32_t part = v / n, rest = v - part * n;
    return (one ? 0 : V1) + (int64_t)k * part + k * rest / n;
  };
  for (int c = tid; c <= p.n_ctas; c += PLAN_T) {
    int2 e = make_int2((int32_t)TT, (int32_t)U);
    if (c < C && TT > 0) {
      const int64_t v0 = begin_of(c);
      const int u = last_at_most((int)U, v0, [&](int i) { return ubeg[i] + (int64_t)i * X; });
      const int64_t into = v0 - (ubeg[u] + (int64_t)u * X) - X;  // < 0: before its tiles
      e = make_int2((int32_t)(ubeg[u] + (into > 0 ? into : 0)), u);
    }
    p.cta_tab[c] = e;
  }
}

// One output row (window row, query head) per 16 lanes, HD / 16 columns a lane: joins the
// partials that the row's prefix unit and its sequence's unit left, three at a time (a row has
// two to four). Memory-bound: reads each partial row (4 d + 8 bytes) once and writes 2 d
// bytes; what costs beside that is the chain of dependent reads before the partials (row,
// units, their CTAs), so the tables are small and rows many. 12 us for 10 thousand rows of
// d = 128 (22 MB from HBM), 17 us for 32 thousand (53 MB), each from cold caches.
template <int HD>
__global__ void __launch_bounds__(256, 4) combine_shared_kernel(AttnParams pa, AttnParams pb) {
  constexpr int LANES = 16, PER = HD / LANES, MAXP = 3, ROWS = 256 / LANES;
  pdl_trigger();
  pdl_wait();
  // 0: the call was refused. (32 bits: 2^22 units of 128 rows at most.)
  const int rows = (int)(min(pa.hdr->sum_w, pb.hdr->sum_w) * pb.Hq);
  const int sub = threadIdx.x % LANES;
  for (int o = blockIdx.x * ROWS + threadIdx.x / LANES; o < rows; o += gridDim.x * ROWS) {
    const int w = o / pb.Hq, h = o - w * pb.Hq, g = h / pb.G, hl = h - g * pb.G;
    const int4 r0 = reinterpret_cast<const int4*>(pb.rows + w)[0];  // RowInfo: i, ubase, nmt,
    const int of_group = pb.rows[w].of_group;                       // mbase
    const int rs = r0.x * pb.G + hl, us = r0.y + g * r0.z + rs / MT;
    // (a unit whose CTAs gave up waiting may have left no note of them: any, but in range)
    auto ctas_of = [](const AttnParams& l, int u) {
      const int2 c = l.unit_ctas[u];
      return make_int2((int)min((uint32_t)c.x, (uint32_t)(l.n_ctas - 1)),
                       (int)min((uint32_t)c.y, (uint32_t)(l.n_ctas - 1)));
    };
    const int2 cs = ctas_of(pb, us);
    int ua = 0, ra = 0;
    int2 ca = make_int2(0, -1);
    if (r0.w >= 0) {
      const int pr = of_group * pb.G + hl;
      ua = pa.tile_unit[r0.w + (pr >> pa.row_log2)] + g;
      ra = pr & ((1 << pa.row_log2) - 1);
      ca = ctas_of(pa, ua);
    }
    // the partials' rows, first those of the sequence's unit
    const int ns = cs.y - cs.x + 1, n = ns + ca.y - ca.x + 1;
    const int64_t at_s = ((int64_t)cs.x + us) * MT + rs % MT;
    const int64_t at_a = (((int64_t)ca.x + ua) << pa.row_log2) + ra;
    float m = -INFINITY, l = 0.f, acc[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = 0.f;
    for (int k0 = 0; k0 < n; k0 += MAXP) {
      float2 ml[MAXP];
      float4 ov[MAXP][PER / 4];
#pragma unroll
      for (int k = 0; k < MAXP; ++k) {
        const int i = k0 + k;
        const bool own = i < ns;
        const int64_t at = own ? at_s + (int64_t)i * MT : at_a + ((int64_t)(i - ns) << pa.row_log2);
        const float4* src = reinterpret_cast<const float4*>((own ? pb.part_o : pa.part_o) + at * HD) + sub;
        ml[k] = i < n ? (own ? pb.part_ml : pa.part_ml)[at] : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int e = 0; e < PER / 4; ++e)
          ov[k][e] = i < n ? __ldcs(src + e * LANES) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float bm = m;
#pragma unroll
      for (int k = 0; k < MAXP; ++k) bm = fmaxf(bm, ml[k].x);
      const float mu = bm == -INFINITY ? 0.f : bm;
      const float rescale = exp2f(m - mu);
      l *= rescale;
#pragma unroll
      for (int e = 0; e < PER; ++e) acc[e] *= rescale;
#pragma unroll
      for (int k = 0; k < MAXP; ++k) {
        const float wgt = exp2f(ml[k].x - mu);  // 0 for unused places (m = -inf)
        l += ml[k].y * wgt;
#pragma unroll
        for (int e = 0; e < PER / 4; ++e) {
          acc[4 * e] += wgt * ov[k][e].x;
          acc[4 * e + 1] += wgt * ov[k][e].y;
          acc[4 * e + 2] += wgt * ov[k][e].z;
          acc[4 * e + 3] += wgt * ov[k][e].w;
        }
      }
      m = bm;
    }
    const float inv = (pb.kv_scale ? pb.kv_scale[pb.Hkv + g] : 1.f) / l;
    uint2* dst = reinterpret_cast<uint2*>((__nv_bfloat16*)pb.out + (int64_t)o * HD) + sub;
#pragma unroll
    for (int e = 0; e < PER / 4; ++e) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(acc[4 * e] * inv, acc[4 * e + 1] * inv);
      const __nv_bfloat162 c = __floats2bfloat162_rn(acc[4 * e + 2] * inv, acc[4 * e + 3] * inv);
      dst[e * LANES] = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&c));
    }
  }
}

}  // namespace

SharedWs shared_ws_layout(const sv_attn_desc* d, int num_groups, int sms, bool lines) {
  SharedWs w = {};
  const int64_t G = d->num_q_heads / d->num_kv_heads;
  const int64_t rows = std::min(d->q_rows, (int64_t)d->batch * (1 + d->max_draft_len));
  const int64_t tile = lines ? 2 * MT : MT;
  // a sequence's rows, and a group's, end in one partly filled row tile at most
  const int64_t prefix_tiles = num_groups + G * rows / tile;
  const int64_t seq_units =
      d->num_kv_heads * (int64_t)d->batch * ((G * (1 + d->max_draft_len) + MT - 1) / MT);
  w.max_units[0] = d->num_kv_heads * prefix_tiles;
  w.max_units[1] = seq_units + (lines ? 0 : w.max_units[0]);
  size_t o = 256;  // the flag word, and the sequences' and prefixes' hand-over
  w.handover = 128;
  w.parts = o;     o = align_up(o + sizeof(SharedSeq) * ((size_t)num_groups + d->batch), 256);
  w.row_begin = o; o = align_up(o + sizeof(int32_t) * d->batch, 256);
  w.rows = o;      o = align_up(o + sizeof(RowInfo) * rows, 256);
  w.tile_unit = o; o = align_up(o + sizeof(int32_t) * prefix_tiles, 256);
  for (int k = lines ? 0 : 1; k < 2; ++k) {
    SharedWs::Line& l = w.line[k];
    w.n_ctas[k] = lines && k == 1 ? 4 * ((sms + 1) / 2) : sms;  // (clusters of two CTAs)
    const size_t n_ctas = w.n_ctas[k], U = (size_t)w.max_units[k], slots = U + n_ctas;
    l.hdr = o;       o += 256;
    l.units = l.sunits = o;
    o = align_up(o + (lines ? sizeof(SharedUnit) : sizeof(int4)) * U, 256);
    l.ubeg = o;      o = align_up(o + sizeof(int32_t) * (U + 1), 256);
    l.unit_ctas = o; o = align_up(o + sizeof(int2) * U, 256);
    l.cta_tab = o;   o = align_up(o + sizeof(int2) * ((size_t)n_ctas + 1), 256);
    const size_t slot_rows = slots * (k == 0 ? 2 * MT : MT);
    l.part_o = o;    o = align_up(o + sizeof(float) * slot_rows * d->head_dim, 256);
    l.part_ml = o;   o = align_up(o + sizeof(float2) * slot_rows, 256);
  }
  if (!lines) {
    w.line[0] = w.line[1];
    w.n_ctas[0] = w.n_ctas[1];
  }
  w.total = o;
  return w;
}

cudaError_t launch_plan_shared(const AttnParams& pa, const AttnParams& pb, bool lines,
                               cudaStream_t s) {
  return launch_pdl(plan_shared_kernel, dim3(lines ? 3 : 1), dim3(PLAN_T), 0, s, pa, pb);
}

cudaError_t launch_combine_shared(const AttnParams& pa, const AttnParams& pb, cudaStream_t s) {
  const int64_t ctas = (pb.q_rows * pb.Hq + 15) / 16;
  const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>(ctas, 8 * (int64_t)pa.n_ctas));
  return pb.d == 128 ? launch_pdl(combine_shared_kernel<128>, dim3(grid), dim3(256), 0, s, pa, pb)
                     : launch_pdl(combine_shared_kernel<64>, dim3(grid), dim3(256), 0, s, pa, pb);
}

}  // namespace sv
