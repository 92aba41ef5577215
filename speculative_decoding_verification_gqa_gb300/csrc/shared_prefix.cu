// shared_prefix.cu -- verify attention over a prefix that a group of sequences shares: the
// plan and the join around the attention kernels.
//
// A softmax over keys A u B is the join of those over A and over B: with (m, l, O) the
// maximum, the sum of 2^(s - m) and the unnormalised output of each, m* = max(m_A, m_B) and
//   out = (2^(m_A - m*) O_A + 2^(m_B - m*) O_B) / (2^(m_A - m*) l_A + 2^(m_B - m*) l_B).
// So the prefix of a group is one part, attended by the rows of all its sequences at once
// (G * sum W rows: full tensor-core tiles, and one read of the prefix per 128 rows instead
// of one per sequence), and what is behind it one part per sequence (internal.cuh,
// SharedSeq). The units of all parts lie on one tile line, split over the CTAs like that of
// spec_verify_attn (internal.cuh); a row's partial results are joined by combine_shared.
#include <cuda_bf16.h>

#include <algorithm>

#include "internal.cuh"

namespace sv {

namespace {

constexpr int PLAN_T = 1024;

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
  for (int k = 0; k < N; ++k) w[k] = s_warp[k][lane];
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

// One CTA: checks, parts, units, and each CTA's range of the tile line.
__global__ void __launch_bounds__(PLAN_T) plan_shared_kernel(AttnParams p, int kt) {
  const int tid = threadIdx.x, NG = p.num_groups, B = p.B, V = NG + B;
  pdl_trigger();
  pdl_wait();
  bool bad = false;
  // the groups: consecutive ranges of the batch
  for (int n = tid; n < NG; n += PLAN_T) {
    const int g0 = p.group_begin[n], g1 = p.group_begin[n + 1], P = p.prefix_len[n];
    if (g0 < 0 || g1 < g0 || g1 > B || (n == 0 && g0 != 0) || (n == NG - 1 && g1 != B) || P < 0 ||
        P > p.max_seq)
      bad = true;
  }
  bad = __syncthreads_or(bad);
  // the sequences
  int64_t q_total = 0;
  for (int base = 0; base < B && !bad; base += PLAN_T) {
    const int b = base + tid;
    int T = 0, D = -1, P = 0, n = 0;
    if (b < B) {
      T = p.seq_lens[b];
      D = p.draft_len[b];
      int lo = 0, hi = NG - 1;  // the last group that begins at or before b
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.group_begin[mid] <= b) lo = mid; else hi = mid - 1;
      }
      n = lo;
      P = p.prefix_len[n];
      if (T < P || T > p.max_seq || D < 0 || D > p.max_draft ||
          (((int64_t)T + D + p.block_size) >> p.bs_log2) > p.bt_stride)
        bad = true;
    }
    const int64_t w[1] = {b < B && !bad ? 1 + D : 0};
    int64_t ex[1], tot[1];
    scan_block<1>(w, ex, tot);
    if (b < B && !bad) {
      SharedSeq s;
      s.q_off = q_total + ex[0];
      s.rows = 1 + D;
      s.start = P;
      s.nkeys = T + 1 + D;
      s.last0 = T;
      s.table_row = b;
      s.alone = P == 0;
      s.group = n;
      s.nmt = (int)(((int64_t)p.G * s.rows + MT - 1) / MT);
      const int box = min(p.block_size, kt), k0 = P / box * box;
      s.nt = (int)(((int64_t)s.nkeys - k0 + kt - 1) / kt);
      s.ubase = s.tbase = 0;
      p.parts[NG + b] = s;
    }
    q_total += tot[0];
    bad = __syncthreads_or(bad);
  }
  bad = bad || q_total > p.q_rows;
  // the prefixes
  for (int n = tid; n < NG && !bad; n += PLAN_T) {
    const int g0 = p.group_begin[n], g1 = p.group_begin[n + 1], P = p.prefix_len[n];
    SharedSeq s = {};
    s.q_off = g0 < B ? p.parts[NG + g0].q_off : q_total;
    const int64_t end = g1 < B ? p.parts[NG + g1].q_off : q_total;
    s.rows = P > 0 ? (int)(end - s.q_off) : 0;
    s.nkeys = P;
    s.last0 = P - 1;
    s.table_row = g0;
    s.group = n;
    s.nmt = (int)(((int64_t)p.G * s.rows + MT - 1) / MT);
    s.nt = (P + kt - 1) / kt;
    p.parts[n] = s;
  }
  __syncthreads();
  // units and tiles of the parts
  int64_t U = 0, TT = 0;
  for (int base = 0; base < V && !bad; base += PLAN_T) {
    const int v = base + tid;
    int64_t c[2] = {0, 0}, ex[2], tot[2];
    if (v < V) {
      c[0] = (int64_t)p.Hkv * p.parts[v].nmt;
      c[1] = c[0] * p.parts[v].nt;
    }
    scan_block<2>(c, ex, tot);
    if (v < V) {
      p.parts[v].ubase = (int32_t)(U + ex[0]);
      p.parts[v].tbase = (int32_t)(TT + ex[1]);
    }
    U += tot[0];
    TT += tot[1];
  }
  bad = bad || U > p.max_units || TT >= 0x7fffffffll;
  if (tid == 0) {
    if (bad) {
      atomicOr(p.flags, FLAG_ATTN_SHAPE);
      U = TT = 0;
    }
    p.hdr->num_units = (int32_t)U;
    p.hdr->total_tiles = (int32_t)TT;
    p.hdr->kt = kt;
    p.hdr->unit_ctas = 0;
    p.hdr->sum_w = q_total;
    p.ubeg[U] = (int32_t)TT;
  }
  if (bad) U = TT = 0;  // (every thread: the ranges below are then empty)
  __syncthreads();
  for (int u = tid; u < (int)U; u += PLAN_T) {
    int lo = 0, hi = V - 1;  // the last part whose units begin at or before u
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.parts[mid].ubase <= u) lo = mid; else hi = mid - 1;
    }
    const SharedSeq s = p.parts[lo];
    const int k = u - s.ubase, box = min(p.block_size, kt);
    p.units[u] = make_int4(lo, k / s.nmt, k % s.nmt, s.start / box * box);
    p.ubeg[u] = s.tbase + k * s.nt;
  }
  // CTA c starts at the first tile at or after position c * VT / C of the virtual line
  const int64_t X = p.switch_tiles, VT = TT + U * X;
  for (int c = tid; c <= p.n_ctas; c += PLAN_T) {
    int2 e = make_int2((int32_t)TT, (int32_t)U);
    if (c < p.n_ctas && TT > 0) {
      const int64_t v0 = (int64_t)c * VT / p.n_ctas;
      int lo = 0, hi = V - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.parts[mid].tbase + (int64_t)p.parts[mid].ubase * X <= v0) lo = mid; else hi = mid - 1;
      }
      const SharedSeq s = p.parts[lo];
      const int64_t at = v0 - (s.tbase + (int64_t)s.ubase * X);
      const int k = (int)(at / (s.nt + X));
      const int64_t into = at - k * (s.nt + X) - X;  // < 0: before the unit's first tile
      e = make_int2((int32_t)(s.tbase + (int64_t)k * s.nt + (into > 0 ? into : 0)), s.ubase + k);
    }
    p.cta_tab[c] = e;
  }
}

constexpr int COMBINE_ROWS = 8;

// (m, l, O) of one row, a warp's lanes PER columns each.
template <int PER>
struct Row {
  float m, l, o[PER];
};

// Joins the partials that the CTAs left of row r of unit u.
template <int HD>
__device__ __forceinline__ void join_unit(const AttnParams& p, int u, int r, int lane, int64_t VT,
                                          Row<HD / 32>& acc) {
  constexpr int PER = HD / 32, MAXP = 4;
  const int64_t ub = p.ubeg[u], ue = p.ubeg[u + 1];
  const int c_lo = cta_of_tile(vpos_of_tile(ub, u, p.switch_tiles), VT, p.n_ctas);
  const int c_hi = cta_of_tile(vpos_of_tile(ue - 1, u, p.switch_tiles), VT, p.n_ctas);
  for (int c0 = c_lo; c0 <= c_hi; c0 += MAXP) {
    // every load of the batch before any use (one L2 round trip per batch)
    float2 ml[MAXP];
    float ov[MAXP][PER];
#pragma unroll
    for (int k = 0; k < MAXP; ++k) {
      const int c = c0 + k;
      const bool use = c <= c_hi && cta_has_tiles(c, VT, p.n_ctas);
      const size_t at = ((size_t)(c + u) * MT + r);
      ml[k] = use ? p.part_ml[at] : make_float2(-INFINITY, 0.f);
      const float* src = p.part_o + at * HD + lane * PER;
      if constexpr (PER == 4) {
        const float4 v = use ? __ldcs(reinterpret_cast<const float4*>(src)) : make_float4(0, 0, 0, 0);
        ov[k][0] = v.x;
        ov[k][1] = v.y;
        ov[k][2] = v.z;
        ov[k][3] = v.w;
      } else {
        const float2 v = use ? __ldcs(reinterpret_cast<const float2*>(src)) : make_float2(0, 0);
        ov[k][0] = v.x;
        ov[k][1] = v.y;
      }
    }
    float bm = acc.m;
#pragma unroll
    for (int k = 0; k < MAXP; ++k) bm = fmaxf(bm, ml[k].x);
    const float mu = bm == -INFINITY ? 0.f : bm;
    const float rs = exp2f(acc.m - mu);
    acc.l *= rs;
#pragma unroll
    for (int e = 0; e < PER; ++e) acc.o[e] *= rs;
#pragma unroll
    for (int k = 0; k < MAXP; ++k) {
      const float w = exp2f(ml[k].x - mu);  // 0 for unused slots (m = -inf)
      acc.l += ml[k].y * w;
#pragma unroll
      for (int e = 0; e < PER; ++e) acc.o[e] += w * ov[k][e];
    }
    acc.m = bm;
  }
}

template <int HD>
__global__ void __launch_bounds__(256) combine_shared_kernel(AttnParams p) {
  constexpr int PER = HD / 32;
  pdl_trigger();
  pdl_wait();
  const int U = p.hdr->num_units;
  if (U == 0) return;
  const int64_t VT = p.hdr->total_tiles + (int64_t)U * p.switch_tiles;
  const int u0 = p.parts[p.num_groups].ubase;  // the first sequence's units
  const int lane = threadIdx.x & 31;
  const int64_t items = (int64_t)(U - u0) * (MT / COMBINE_ROWS);
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int u = u0 + (int)(it / (MT / COMBINE_ROWS));
    const int r = (int)(it % (MT / COMBINE_ROWS)) * COMBINE_ROWS + (threadIdx.x >> 5);
    const int4 info = p.units[u];
    const SharedSeq s = p.parts[info.x];
    const int g = info.y, rg = info.z * MT + r;
    if (rg >= p.G * s.rows) continue;
    if (s.alone) {  // written by the attention kernel if one CTA saw all of the unit
      const int64_t ub = p.ubeg[u], ue = p.ubeg[u + 1];
      if (cta_of_tile(vpos_of_tile(ub, u, p.switch_tiles), VT, p.n_ctas) ==
          cta_of_tile(vpos_of_tile(ue - 1, u, p.switch_tiles), VT, p.n_ctas))
        continue;
    }
    Row<PER> acc;
    acc.m = -INFINITY;
    acc.l = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) acc.o[e] = 0.f;
    join_unit<HD>(p, u, r, lane, VT, acc);
    if (!s.alone) {  // the same row among those of its group
      const SharedSeq pre = p.parts[s.group];
      const int64_t pr = (s.q_off - pre.q_off) * p.G + rg;
      join_unit<HD>(p, pre.ubase + g * pre.nmt + (int)(pr / MT), (int)(pr % MT), lane, VT, acc);
    }
    const float inv = (p.kv_scale ? p.kv_scale[p.Hkv + g] : 1.f) / acc.l;
    __nv_bfloat16* dst = (__nv_bfloat16*)p.out +
                         ((s.q_off + rg / p.G) * p.Hq + (int64_t)g * p.G + rg % p.G) * HD + lane * PER;
    __nv_bfloat162 a = __floats2bfloat162_rn(acc.o[0] * inv, acc.o[1] * inv);
    if constexpr (PER == 4) {
      __nv_bfloat162 c = __floats2bfloat162_rn(acc.o[2] * inv, acc.o[3] * inv);
      uint2 w;
      w.x = *reinterpret_cast<uint32_t*>(&a);
      w.y = *reinterpret_cast<uint32_t*>(&c);
      *reinterpret_cast<uint2*>(dst) = w;
    } else {
      *reinterpret_cast<__nv_bfloat162*>(dst) = a;
    }
  }
}

}  // namespace

SharedWs shared_ws_layout(const sv_attn_desc* d, int num_groups, int n_ctas) {
  SharedWs w;
  const int64_t G = d->num_q_heads / d->num_kv_heads;
  const int64_t rows = std::min(d->q_rows, (int64_t)d->batch * (1 + d->max_draft_len));
  // a sequence's rows, and a group's, end in one partly filled row tile at most
  w.max_units = d->num_kv_heads * ((int64_t)d->batch * ((G * (1 + d->max_draft_len) + MT - 1) / MT) +
                                   num_groups + G * rows / MT);
  const size_t U = (size_t)w.max_units, slots = U + n_ctas;
  size_t o = 0;
  w.ctrl = o;    o += 256;
  w.hdr = o;     o += 256;
  w.parts = o;   o = align_up(o + sizeof(SharedSeq) * ((size_t)num_groups + d->batch), 256);
  w.units = o;   o = align_up(o + sizeof(int4) * U, 256);
  w.ubeg = o;    o = align_up(o + sizeof(int32_t) * (U + 1), 256);
  w.cta_tab = o; o = align_up(o + sizeof(int2) * ((size_t)n_ctas + 1), 256);
  w.part_o = o;  o = align_up(o + sizeof(float) * slots * MT * d->head_dim, 256);
  w.part_ml = o; o = align_up(o + sizeof(float2) * slots * MT, 256);
  w.total = o;
  return w;
}

cudaError_t launch_plan_shared(const AttnParams& p, int kt, cudaStream_t s) {
  return launch_pdl(plan_shared_kernel, dim3(1), dim3(PLAN_T), 0, s, p, kt);
}

cudaError_t launch_combine_shared(const AttnParams& p, cudaStream_t s) {
  // at most 8 CTAs of 256 threads per CTA of the attention grid (about one SM each)
  const unsigned items = (unsigned)p.max_units * (MT / COMBINE_ROWS);
  const unsigned grid = std::min(items, 8u * (unsigned)(p.n_ctas > 0 ? p.n_ctas : 1));
  return p.d == 128 ? launch_pdl(combine_shared_kernel<128>, dim3(grid), dim3(256), 0, s, p)
                    : launch_pdl(combine_shared_kernel<64>, dim3(grid), dim3(256), 0, s, p);
}

}  // namespace sv
