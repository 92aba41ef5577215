// line.cuh -- the work of a 4-bit attention call, laid out by its own kernels: no planning
// kernel runs before them, every CTA works out its place from the lengths.
//
//   unit  = (sequence, group of `heads` neighbouring KV heads, row tile of `mr` query rows a
//           head); neighbouring heads' rows lie side by side in a page, and a line of 128 bytes
//           holds those of two or more: read far apart in time they would come from HBM twice
//   tile  = KV4_KT consecutive cache positions of a unit, from the one holding the first key
//           that its rows see to the one holding T + D
//   line  = all units end to end by sequence, head group, row tile, each with `switch_tiles`
//           virtual tiles before its own (the time its start takes); CTA c of C takes the
//           virtual range [c VT / C, (c + 1) VT / C) and with it the tiles inside.
// With C at most the number of tiles, every CTA between the first and the last of a unit holds
// nothing else, so a CTA shares at most two units: the one that it continues (slot 2 c) and the
// one that it begins and does not end (slot 2 c + 1).
#pragma once

#include "internal.cuh"

namespace sv {
namespace {

struct LineSeq {
  int T, D, nmt;
  int64_t tiles, virt;  // of a head group: tiles, and with the virtual ones
};
__device__ __forceinline__ int line_groups(const Kv4Attn& p) { return p.Hkv / p.heads; }
__device__ __forceinline__ int line_tiles(const Kv4Attn& p, int T, int D, int mt, int& kb) {
  kb = 0;
  if (p.window > 0) {
    const int lo = T + mt * p.mr / p.G + 1 - p.window;  // first key of the tile's first row
    kb = lo > 0 ? lo / KV4_KT : 0;
  }
  return (int)(((int64_t)T + D + KV4_KT) / KV4_KT) - kb;
}
// False if a length is out of range.
__device__ __forceinline__ bool line_seq(const Kv4Attn& p, int b, LineSeq& s) {
  s.T = p.seq_lens[b];
  s.D = p.draft_len[b];
  if (s.T < 0 || s.T > p.max_seq || s.D < 0 || s.D > p.max_draft ||
      (((int64_t)s.T + s.D + p.block_size) >> p.bs_log2) > p.bt_stride)
    return false;
  s.nmt = (p.G * (s.D + 1) + p.mr - 1) / p.mr;
  s.tiles = 0;
  int kb;
  if (p.window > 0)
    for (int mt = 0; mt < s.nmt; ++mt) s.tiles += line_tiles(p, s.T, s.D, mt, kb);
  else
    s.tiles = (int64_t)s.nmt * line_tiles(p, s.T, s.D, 0, kb);
  s.virt = s.tiles + (int64_t)s.nmt * p.switch_tiles;
  return true;
}

struct Line {
  int64_t virt, tiles, units, rows;  // of the whole call
  int ctas;                          // ranges in use
  bool whole;                        // range c is unit c
};
struct LineAt {  // a sequence, and what lies before it
  int b;
  int64_t virt, units, rows;
};

// The totals, by a CTA of NTH threads; then the sequence that holds a virtual position (or, with
// by_unit, a unit) which `target(by_unit)` works out from them (-1: none). False if there is
// none or, with the flag set, if a length is out of range or the rows are more than q's. One
// pass over the lengths for up to NTH sequences, whose shares stay in registers, else two.
template <int NTH, class Target>
__device__ bool line_scan(const Kv4Attn& p, Line& total, LineAt* at, Target target) {
  constexpr int NWARP = NTH / 32;
  __shared__ int64_t s_warp[NWARP][4];
  __shared__ int64_t s_at[4];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int groups = line_groups(p);
  int64_t carry[4] = {0, 0, 0, 0};
  int64_t v[4], x[4];  // of this thread's sequence: virtual tiles, tiles, units, rows; before it
  int longest = 0;     // tiles of the longest unit of this thread's sequences
  bool bad = false;
  auto shares = [&](int base) {
    const int b = base + tid;
    v[0] = v[1] = v[2] = v[3] = 0;
    LineSeq s;
    if (b < p.B) {
      if (line_seq(p, b, s)) {
        int kb;
        longest = max(longest, line_tiles(p, s.T, s.D, 0, kb));
        v[0] = s.virt * groups;
        v[1] = s.tiles * groups;
        v[2] = (int64_t)s.nmt * groups;
        v[3] = 1 + s.D;
      } else {
        bad = true;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = v[k];
    const int nw = min(NWARP, (p.B - base + 31) / 32);  // warps with a sequence
    if (wid < nw) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int64_t y = __shfl_up_sync(0xffffffffu, x[k], o);
          if (lane >= o) x[k] += y;
        }
      if (lane == 31)
#pragma unroll
        for (int k = 0; k < 4; ++k) s_warp[wid][k] = x[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      int64_t before = carry[k];
      for (int w = 0; w < nw; ++w) {
        const int64_t y = s_warp[w][k];
        if (w < wid) before += y;
        carry[k] += y;
      }
      x[k] += before - v[k];  // exclusive
    }
  };
  for (int base = 0; base < p.B; base += NTH) {
    if (base > 0) __syncthreads();  // s_warp is reused
    shares(base);
  }
  total.virt = carry[0];
  total.tiles = carry[1];
  total.units = carry[2];
  total.rows = carry[3];
  total.ctas = (int)(carry[1] < p.n_ctas ? carry[1] : p.n_ctas);
  const int64_t share = total.ctas > 0 ? carry[0] / total.ctas : 0;
  total.whole = !__syncthreads_or(longest > share + p.join_tiles) && carry[2] <= p.n_ctas;
  if (total.whole) total.ctas = (int)carry[2];
  if (__syncthreads_or(bad || carry[3] > p.q_rows)) {
    if (tid == 0) atomicOr(p.flags, FLAG_ATTN_SHAPE);
    return false;
  }
  bool by_unit = false;
  const int64_t t = target(by_unit);
  if (t < 0) return false;
  const int k = by_unit ? 2 : 0;
  auto look = [&](int base) {
    if (t >= x[k] && t < x[k] + v[k]) {
      s_at[0] = base + tid;
      s_at[1] = x[0];
      s_at[2] = x[2];
      s_at[3] = x[3];
    }
  };
  if (p.B <= NTH) {
    look(0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) carry[i] = 0;
    for (int base = 0; base < p.B; base += NTH) {
      __syncthreads();
      shares(base);
      look(base);
    }
  }
  __syncthreads();
  *at = LineAt{(int)s_at[0], s_at[1], s_at[2], s_at[3]};
  return true;
}

// A CTA's share of one unit: tiles [j0, j1) of its nt, tile j at position kbase + j * KV4_KT.
struct LineSeg {
  int b, g, mt, T, D, j0, j1, nt, kbase;
  int64_t q_off;
  bool whole;
  int begins;  // 1: holds the unit's first tile (the part's slot)
};
// The units of a virtual range, one after another.
struct LineWalk {
  int64_t v0, v1, us, q_off;  // the range; the next unit's virtual start, its sequence's first row
  int b, g, mt;
  __device__ __forceinline__ bool next(const Kv4Attn& p, LineSeg& s) {
    const int groups = line_groups(p);
    while (us < v1 && b < p.B) {
      s.T = p.seq_lens[b];
      s.D = p.draft_len[b];
      int kb;
      s.nt = line_tiles(p, s.T, s.D, mt, kb);
      const int64_t first = us + p.switch_tiles;
      const int64_t lo = v0 - first, hi = v1 - first;
      s.j0 = lo > 0 ? (int)(lo < s.nt ? lo : s.nt) : 0;
      s.j1 = hi < s.nt ? (int)hi : s.nt;
      s.b = b;
      s.g = g;
      s.mt = mt;
      s.kbase = kb * KV4_KT;
      s.q_off = q_off;
      us = first + s.nt;
      if (++mt * p.mr >= p.G * (s.D + 1)) {
        mt = 0;
        if (++g == groups) {
          g = 0;
          ++b;
          q_off += 1 + s.D;
        }
      }
      if (s.j0 < s.j1) {
        s.whole = s.j0 == 0 && s.j1 == s.nt;
        s.begins = s.j0 == 0;
        return true;
      }
    }
    return false;
  }
};

// The walk that begins with the unit `off` virtual tiles (by_unit: units) into sequence at.b.
__device__ __forceinline__ LineWalk line_enter(const Kv4Attn& p, const LineAt& at, int64_t off,
                                               bool by_unit) {
  LineSeq s;
  line_seq(p, at.b, s);
  LineWalk w;
  w.b = at.b;
  w.q_off = at.rows;
  const int64_t per = by_unit ? s.nmt : s.virt;
  w.g = (int)(off / per);
  int64_t left = off - w.g * per;
  w.us = at.virt + w.g * s.virt;
  w.mt = 0;
  while (true) {  // the row tile: a sequence has few
    int kb;
    const int64_t n = line_tiles(p, s.T, s.D, w.mt, kb) + p.switch_tiles;
    const int64_t step = by_unit ? 1 : n;
    if (left < step || w.mt == s.nmt - 1) break;
    left -= step;
    w.us += n;
    ++w.mt;
  }
  return w;
}

// This CTA's walk: range `c` of the call's. False if it has nothing to do, or (flag set) a
// length is out of range. By all NTH threads of the CTA.
template <int NTH>
__device__ bool line_begin(const Kv4Attn& p, int c, LineWalk& w) {
  Line total = {};
  LineAt at;
  int64_t v0 = 0, v1 = 0;
  if (!line_scan<NTH>(p, total, &at, [&](bool& by_unit) -> int64_t {
        if (c >= total.ctas) return -1;
        by_unit = total.whole;
        if (total.whole) return c;
        v0 = (int64_t)c * total.virt / total.ctas;
        v1 = (int64_t)(c + 1) * total.virt / total.ctas;
        return v0;
      }))
    return false;
  if (total.whole) {
    w = line_enter(p, at, c - at.units, true);
    int kb;
    v0 = w.us;
    v1 = w.us + p.switch_tiles + line_tiles(p, p.seq_lens[w.b], p.draft_len[w.b], w.mt, kb);
  } else {
    w = line_enter(p, at, v0 - at.virt, false);
  }
  w.v0 = v0;
  w.v1 = v1;
  return true;
}

}  // namespace
}  // namespace sv
