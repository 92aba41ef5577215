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
// (internal.cuh). tcgen05 kernels: the prefixes' units, of 256 rows, on a line of their own
// (attn_prefix.cu), the sequences' on another (attn_tc.cu). mma.sync kernel: all units, of
// 128 rows, on one line. A row's partial results are joined by combine_shared.
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

constexpr int MAJOR_ENTRIES = 16384;

// The last index in [0, n) whose key is at most x (keys not decreasing, key(0) <= x).
template <class F>
__device__ __forceinline__ int last_at_most(int n, int64_t x, F key) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (key(mid) <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// CTA `line` of 2 (or the one CTA of a single line) checks the call, describes its parts and
// writes its line: line 0 the prefixes (pa), line 1 the sequences (pb). Both CTAs make the
// same checks, so a call is skipped as a whole.
__global__ void __launch_bounds__(PLAN_T) plan_shared_kernel(AttnParams pa, AttnParams pb, int kt) {
  const bool both = gridDim.x == 1;  // one line for all parts
  const bool prefixes = both || blockIdx.x == 0, sequences = both || blockIdx.x == 1;
  const AttnParams& p = prefixes && !both ? pa : pb;
  const int tid = threadIdx.x, NG = p.num_groups, B = p.B;
  __shared__ int s_maxmt;
  pdl_trigger();
  pdl_wait();
  if (tid == 0) s_maxmt = 0;
  bool bad = false;
  // the groups: consecutive ranges of the batch
  for (int n = tid; n < NG; n += PLAN_T) {
    const int g0 = p.group_begin[n], g1 = p.group_begin[n + 1], P = p.prefix_len[n];
    if (g0 < 0 || g1 < g0 || g1 > B || (n == 0 && g0 != 0) || (n == NG - 1 && g1 != B) || P < 0 ||
        P > p.max_seq)
      bad = true;
  }
  bad = __syncthreads_or(bad);
  // the sequences; line 0 keeps their row offsets in its own scratch
  SharedSeq* seq = p.parts + NG;
  int64_t q_total = 0;
  for (int base = 0; base < B && !bad; base += PLAN_T) {
    const int b = base + tid;
    int T = 0, D = -1, P = 0, n = 0;
    if (b < B) {
      T = p.seq_lens[b];
      D = p.draft_len[b];
      n = last_at_most(NG, b, [&](int i) { return p.group_begin[i]; });
      P = p.prefix_len[n];
      if (T < P || T > p.max_seq || D < 0 || D > p.max_draft ||
          (((int64_t)T + D + p.block_size) >> p.bs_log2) > p.bt_stride)
        bad = true;
    }
    const int64_t w[1] = {b < B && !bad ? 1 + D : 0};
    int64_t ex[1], tot[1];
    scan_block<1>(w, ex, tot);
    if (b < B && !bad) {
      if (prefixes) p.row_begin[b] = (int32_t)(q_total + ex[0]);
      if (sequences) {
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
        s.ubase = s.tbase = s.mbase = 0;
        seq[b] = s;
      }
    }
    q_total += tot[0];
    bad = __syncthreads_or(bad);
  }
  bad = bad || q_total > p.q_rows;
  // the prefixes: their parts, and the first of each one's row tiles
  const int rows_of_tile = p.row_tile;
  int64_t n_tiles = 0;  // row tiles of all prefixes
  for (int base = 0; base < NG && prefixes && !bad; base += PLAN_T) {
    const int n = base + tid;
    SharedSeq s = {};
    if (n < NG) {
      const int g0 = p.group_begin[n], g1 = p.group_begin[n + 1], P = p.prefix_len[n];
      s.q_off = g0 < B ? p.row_begin[g0] : q_total;
      const int64_t end = g1 < B ? p.row_begin[g1] : q_total;
      s.rows = P > 0 ? (int)(end - s.q_off) : 0;
      s.nkeys = P;
      s.last0 = P - 1;
      s.table_row = g0;
      s.group = n;
      s.nmt = (int)(((int64_t)p.G * s.rows + rows_of_tile - 1) / rows_of_tile);
      s.nt = (P + kt - 1) / kt;
      atomicMax(&s_maxmt, s.nmt);
    }
    const int64_t c[1] = {s.nmt};
    int64_t ex[1], tot[1];
    scan_block<1>(c, ex, tot);
    s.mbase = (int32_t)(n_tiles + ex[0]);
    if (n < NG) p.parts[n] = s;
    n_tiles += tot[0];
  }
  __syncthreads();
  // Units of the prefixes, entry (row tile mt, part v) by entry, the KV heads of an entry
  // together. Row-tile-major (mt first), so that the slices of the line that read the same
  // prefix are read by their CTAs at about the same time and share it through L2; with very
  // many groups of very different sizes part-major, which needs no empty entries.
  const int maxmt = s_maxmt;
  const bool major = (int64_t)maxmt * NG <= MAJOR_ENTRIES;
  const int64_t entries = prefixes && !bad ? (major ? (int64_t)maxmt * NG : n_tiles) : 0;
  int64_t U = 0, TT = 0;
  for (int64_t base = 0; base < entries; base += PLAN_T) {
    const int64_t e = base + tid;
    int v = 0, mt = 0;
    int64_t c[2] = {0, 0}, ex[2], tot[2];
    SharedSeq s = {};
    if (e < entries) {
      if (major) {
        mt = (int)(e / NG);
        v = (int)(e % NG);
      } else {
        v = last_at_most(NG, e, [&](int i) { return p.parts[i].mbase; });
        mt = (int)(e - p.parts[v].mbase);
      }
      s = p.parts[v];
      if (mt < s.nmt) {
        c[0] = p.Hkv;
        c[1] = (int64_t)p.Hkv * s.nt;
      }
    }
    scan_block<2>(c, ex, tot);
    if (c[0] > 0 && TT + ex[1] + c[1] < 0x7fffffffll && U + ex[0] + c[0] <= p.max_units) {
      p.tile_unit[s.mbase + mt] = (int32_t)(U + ex[0]);
      for (int g = 0; g < p.Hkv; ++g) {
        p.units[U + ex[0] + g] = make_int4(v, g, mt, 0);
        p.ubeg[U + ex[0] + g] = (int32_t)(TT + ex[1] + (int64_t)g * s.nt);
      }
    }
    U += tot[0];
    TT += tot[1];
  }
  // units of the sequences
  const int64_t U0 = U;
  for (int base = 0; base < B && sequences && !bad; base += PLAN_T) {
    const int b = base + tid;
    int64_t c[2] = {0, 0}, ex[2], tot[2];
    if (b < B) {
      c[0] = (int64_t)p.Hkv * seq[b].nmt;
      c[1] = c[0] * seq[b].nt;
    }
    scan_block<2>(c, ex, tot);
    if (b < B) {
      seq[b].ubase = (int32_t)(U + ex[0]);
      seq[b].tbase = (int32_t)(TT + ex[1]);
    }
    U += tot[0];
    TT += tot[1];
  }
  bad = bad || U > p.max_units || TT >= 0x7fffffffll;
  if (bad) U = TT = 0;  // (every thread: nothing below is then written or run)
  if (tid == 0) {
    if (bad) atomicOr(p.flags, FLAG_ATTN_SHAPE);
    p.hdr->num_units = (int32_t)U;
    p.hdr->total_tiles = (int32_t)TT;
    p.hdr->kt = kt;
    p.hdr->unit_ctas = 0;
    p.hdr->sum_w = bad ? 0 : q_total;
    p.ubeg[U] = (int32_t)TT;
  }
  __syncthreads();
  const int box = min(p.block_size, kt);
  for (int64_t u = U0 + tid; u < U; u += PLAN_T) {
    const SharedSeq s = seq[last_at_most(B, u, [&](int i) { return seq[i].ubase; })];
    const int k = (int)(u - s.ubase);
    p.units[u] = make_int4(NG + s.table_row, k / s.nmt, k % s.nmt, s.start / box * box);
    p.ubeg[u] = s.tbase + k * s.nt;
  }
  if (sequences && !bad)
    for (int b = tid; b < B; b += PLAN_T)
      for (int i = 0; i < seq[b].rows; ++i) p.row_seq[seq[b].q_off + i] = b;
  __syncthreads();
  // CTA c starts at the first tile at or after position c * VT / C of the virtual line;
  // which CTAs' partials make up a unit
  const int64_t X = p.switch_tiles, VT = TT + U * X;
  for (int c = tid; c <= p.n_ctas; c += PLAN_T) {
    int2 e = make_int2((int32_t)TT, (int32_t)U);
    if (c < p.n_ctas && TT > 0) {
      const int64_t v0 = (int64_t)c * VT / p.n_ctas;
      const int u = last_at_most((int)U, v0, [&](int i) { return p.ubeg[i] + (int64_t)i * X; });
      const int64_t into = v0 - (p.ubeg[u] + (int64_t)u * X) - X;  // < 0: before its tiles
      e = make_int2((int32_t)(p.ubeg[u] + (into > 0 ? into : 0)), u);
    }
    p.cta_tab[c] = e;
  }
  for (int u = tid; u < (int)U; u += PLAN_T)
    p.unit_ctas[u] = make_int2(cta_of_tile(vpos_of_tile(p.ubeg[u], u, (int)X), VT, p.n_ctas),
                               cta_of_tile(vpos_of_tile((int64_t)p.ubeg[u + 1] - 1, u, (int)X), VT, p.n_ctas));
}

// One output row (window row, query head) per group of 8 lanes, PER columns a lane: joins
// the partials that the row's prefix unit and its sequence's unit left, in batches whose
// loads are all issued before any use. A unit's CTAs with no tile of it (an empty range, or
// one that ends in the unit's switch) left none.
template <int HD>
__global__ void __launch_bounds__(256) combine_shared_kernel(AttnParams pa, AttnParams pb) {
  constexpr int PER = HD / 8, MAXP = 4;
  pdl_trigger();
  pdl_wait();
  const int64_t rows = min(pa.hdr->sum_w, pb.hdr->sum_w) * pb.Hq;  // 0: the call was refused
  const int sub = threadIdx.x & 7;
  for (int64_t o = (int64_t)blockIdx.x * 32 + (threadIdx.x >> 3); o < rows;
       o += (int64_t)gridDim.x * 32) {
    const int64_t w = o / pb.Hq;
    const int h = (int)(o % pb.Hq), g = h / pb.G;
    const SharedSeq* sp = pb.parts + pb.num_groups + pb.row_seq[w];
    const int rg = (int)(w - sp->q_off) * pb.G + h % pb.G;
    const int us = sp->ubase + g * sp->nmt + rg / MT;
    const int2 cs = pb.unit_ctas[us];
    const bool alone = sp->alone != 0;
    if (alone && cs.x == cs.y) continue;  // one CTA saw the unit and wrote the output
    int ua = 0, ra = 0;
    int2 ca = make_int2(0, -1);
    if (!alone) {
      const SharedSeq* pre = pa.parts + sp->group;
      const int64_t pr = (w - pre->q_off) * pb.G + h % pb.G;
      ua = pa.tile_unit[pre->mbase + (int)(pr / pa.row_tile)] + g;
      ra = (int)(pr % pa.row_tile);
      ca = pa.unit_ctas[ua];
    }
    const int ns = cs.y - cs.x + 1, n = ns + ca.y - ca.x + 1;
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
        const AttnParams& p = own ? pb : pa;
        const int c = own ? cs.x + i : ca.x + i - ns, u = own ? us : ua;
        bool use = i < n;
        if (use) {  // has CTA c tiles of unit u?
          const int b0 = p.cta_tab[c].x, b1 = p.cta_tab[c + 1].x;
          use = max(b0, p.ubeg[u]) < min(b1, p.ubeg[u + 1]);
        }
        const size_t at = ((size_t)c + u) * (own ? MT : pa.row_tile) + (own ? rg % MT : ra);
        ml[k] = use ? p.part_ml[at] : make_float2(-INFINITY, 0.f);
        const float4* src = reinterpret_cast<const float4*>(p.part_o + at * HD) + sub;
#pragma unroll
        for (int e = 0; e < PER / 4; ++e)
          ov[k][e] = use ? __ldcs(src + e * 8) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float bm = m;
#pragma unroll
      for (int k = 0; k < MAXP; ++k) bm = fmaxf(bm, ml[k].x);
      const float mu = bm == -INFINITY ? 0.f : bm;
      const float rs = exp2f(m - mu);
      l *= rs;
#pragma unroll
      for (int e = 0; e < PER; ++e) acc[e] *= rs;
#pragma unroll
      for (int k = 0; k < MAXP; ++k) {
        const float wgt = exp2f(ml[k].x - mu);  // 0 for unused slots (m = -inf)
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
    uint2* dst = reinterpret_cast<uint2*>((__nv_bfloat16*)pb.out + o * HD) + sub;
#pragma unroll
    for (int e = 0; e < PER / 4; ++e) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(acc[4 * e] * inv, acc[4 * e + 1] * inv);
      const __nv_bfloat162 c = __floats2bfloat162_rn(acc[4 * e + 2] * inv, acc[4 * e + 3] * inv);
      dst[e * 8] = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&c));
    }
  }
}

}  // namespace

SharedWs shared_ws_layout(const sv_attn_desc* d, int num_groups, int n_ctas, bool lines) {
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
  size_t o = 256;  // the flag word
  w.parts = o;     o = align_up(o + sizeof(SharedSeq) * ((size_t)num_groups + d->batch), 256);
  w.row_begin = o; o = align_up(o + sizeof(int32_t) * d->batch, 256);
  w.row_seq = o;   o = align_up(o + sizeof(int32_t) * rows, 256);
  w.tile_unit = o; o = align_up(o + sizeof(int32_t) * prefix_tiles, 256);
  for (int k = lines ? 0 : 1; k < 2; ++k) {
    SharedWs::Line& l = w.line[k];
    const size_t U = (size_t)w.max_units[k], slots = U + n_ctas;
    l.hdr = o;       o += 256;
    l.units = o;     o = align_up(o + sizeof(int4) * U, 256);
    l.ubeg = o;      o = align_up(o + sizeof(int32_t) * (U + 1), 256);
    l.unit_ctas = o; o = align_up(o + sizeof(int2) * U, 256);
    l.cta_tab = o;   o = align_up(o + sizeof(int2) * ((size_t)n_ctas + 1), 256);
    const size_t slot_rows = slots * (k == 0 ? 2 * MT : MT);
    l.part_o = o;    o = align_up(o + sizeof(float) * slot_rows * d->head_dim, 256);
    l.part_ml = o;   o = align_up(o + sizeof(float2) * slot_rows, 256);
  }
  if (!lines) w.line[0] = w.line[1];
  w.total = o;
  return w;
}

cudaError_t launch_plan_shared(const AttnParams& pa, const AttnParams& pb, bool lines, int kt,
                               cudaStream_t s) {
  return launch_pdl(plan_shared_kernel, dim3(lines ? 2 : 1), dim3(PLAN_T), 0, s, pa, pb, kt);
}

cudaError_t launch_combine_shared(const AttnParams& pa, const AttnParams& pb, cudaStream_t s) {
  const int64_t ctas = (pb.q_rows * pb.Hq + 31) / 32;
  const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>(ctas, 8 * (int64_t)pb.n_ctas));
  return pb.d == 128 ? launch_pdl(combine_shared_kernel<128>, dim3(grid), dim3(256), 0, s, pa, pb)
                     : launch_pdl(combine_shared_kernel<64>, dim3(grid), dim3(256), 0, s, pa, pb);
}

}  // namespace sv
