// pages.cu -- the pages of a paged cache: fork, extend (with copy on write), trim, compact.
//
// State (the caller's): ref_count[p], the number of table entries in use that name page p
// (p is free iff it is 0); block_table[r, j], the page of positions j * bs .. of row r;
// cached_len[r], the positions row r holds, so that its entries in use are those with
// j < ceil(cached_len[r] / bs). Every operator checks all rows of the call before it
// changes anything, in a first kernel that ends with one verdict (PagesHdr::ok); the
// kernels after it do nothing when that is 0.
//
// Results do not depend on the order in which threads run: counts change by integer
// additions, free pages are taken lowest first by ranks from a prefix sum over the pool,
// and ties between rows go by their order in the call.
//
// All of it is bound by latency (a few dependent kernels) until tables of a million entries
// or megabytes of page data are touched; the page data then moves at the copy bandwidth.
#include "internal.cuh"

namespace sv {
namespace {

constexpr int PT = 1024;          // threads of the planning kernels
constexpr int CHUNK = 4096;       // pages counted by one CTA (PT threads x 4)
constexpr int AT = 256;           // threads of the applying kernels
constexpr int SEG = 512;          // table entries of one work item
constexpr int FORK_ROWS = 8;      // consecutive children of one work item
constexpr int COPY_BYTES = 16384; // page bytes of one copying work item
constexpr int TABLE_CTAS = 64;    // compact: CTAs that check the tables

// Verdict and totals of a call; every field is written before it is read in each call.
struct PagesHdr {
  int32_t ok;
  int32_t rows_bad;   // a check on the rows failed
  int32_t need;       // extend: pages taken
  int32_t cows;       // extend: rows that part from a shared page
  int32_t live;       // compact: L
  int32_t below;      // compact: live pages among the first L
};

struct Pages {
  sv_page_table t;
  int n;
  const int32_t *rows, *to;  // fork: parents, children; extend, trim: rows (null: row i of
                             // the table), new lengths
  const int32_t* fork_len;
  uint32_t* flags;
  uint32_t* ticket;  // zero between calls
  PagesHdr* hdr;
  int32_t *mark, *row_a, *row_b, *row_c, *row_d;  // [table_rows] each
  int32_t* chunk;                         // [chunks], then [TABLE_CTAS] of compact
  int32_t *blk_a, *blk_b;                 // [num_blocks] each
  int32_t *remap, *num_live;              // compact: outputs or null
  int chunks;
  int bs_log2;
};

// Byte offsets inside a workspace.
struct PagesWs {
  size_t hdr, rows, chunk, blk, total;
};

struct PoolList {
  int n;
  int seg_max;  // copying items of the largest page
  sv_page_data p[SV_MAX_PAGE_POOLS];
};

__device__ __forceinline__ int pages_of(int len, int bs_log2) {
  return (int)(((int64_t)len + (1 << bs_log2) - 1) >> bs_log2);
}
__device__ __forceinline__ bool len_fits(const Pages& a, int64_t len) {
  return len >= 0 && len <= ((int64_t)a.t.max_blocks_per_seq << a.bs_log2);
}

// Exclusive scan of one whole number per thread over a block of PT threads.
template <class T>
__device__ T scan_pt(T v, T& total) {
  __shared__ T s_warp[PT / 32];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[wid] = x;
  __syncthreads();
  T w = s_warp[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const T before = wid > 0 ? __shfl_sync(0xffffffffu, w, wid - 1) : 0;
  __syncthreads();  // s_warp is reused by the next scan
  return x - v + before;
}

// The four pages of this thread in chunk c: their counts (-1 past the pool's end).
__device__ __forceinline__ int4 chunk_counts(const Pages& a, int c) {
  const int64_t p = (int64_t)c * CHUNK + threadIdx.x * 4;
  if (p + 3 < a.t.num_blocks) return *reinterpret_cast<const int4*>(a.t.ref_count + p);
  int4 v = make_int4(-1, -1, -1, -1);
  if (p < a.t.num_blocks) v.x = a.t.ref_count[p];
  if (p + 1 < a.t.num_blocks) v.y = a.t.ref_count[p + 1];
  if (p + 2 < a.t.num_blocks) v.z = a.t.ref_count[p + 2];
  return v;
}

// True in every thread of the CTA that finishes last among the grid's; what the others
// wrote before is then visible to it. Leaves the ticket at zero.
__device__ bool last_cta(const Pages& a) {
  __shared__ bool s_last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    s_last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
    if (s_last) *a.ticket = 0;
  }
  __syncthreads();
  if (s_last) __threadfence();
  return s_last;
}

// Exclusive prefix sums of the chunk counts, in place; returns their total. One CTA.
__device__ int scan_chunks(const Pages& a) {
  int carry = 0;
  for (int base = 0; base < a.chunks; base += PT) {
    const int c = base + threadIdx.x;
    const int v = c < a.chunks ? __ldcg(a.chunk + c) : 0;
    int total;
    const int ex = scan_pt(v, total);
    if (c < a.chunks) a.chunk[c] = carry + ex;
    carry += total;
  }
  return carry;
}

__device__ __forceinline__ int row_at(const Pages& a, int i) { return a.rows ? a.rows[i] : i; }
__device__ __forceinline__ bool row_ok(const Pages& a, int r) {
  return r >= 0 && r < a.t.table_rows;
}

// Marks the rows of `list` (null: row i); true where one stands twice or lies outside the
// table.
__device__ bool mark_rows(const Pages& a, const int32_t* list) {
  bool bad = false;
  for (int i = threadIdx.x; i < a.n; i += PT) {
    const int r = list ? list[i] : i;
    if (row_ok(a, r)) a.mark[r] = 0;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.n; i += PT) {
    const int r = list ? list[i] : i;
    if (!row_ok(a, r) || atomicAdd(a.mark + r, 1) != 0) bad = true;
  }
  return bad;
}

__device__ __forceinline__ void verdict(const Pages& a, bool ok) {
  if (threadIdx.x == 0) {
    a.hdr->ok = ok ? 1 : 0;
    if (!ok) atomicOr(a.flags, FLAG_PAGES_SHAPE);
  }
}

// ---------------------------------------------------------------------------- fork

// One CTA: children distinct, empty and not parents; lengths within the parents'.
// row_a[i]: the child's length.
__global__ void __launch_bounds__(PT) fork_plan(const Pages a) {
  pdl_trigger();
  pdl_wait();
  bool bad = false;
  for (int i = threadIdx.x; i < a.n; i += PT)
    if (row_ok(a, a.rows[i])) a.mark[a.rows[i]] = 0;
  __syncthreads();
  bad |= mark_rows(a, a.to);
  __syncthreads();
  for (int i = threadIdx.x; i < a.n; i += PT) {
    const int p = a.rows[i], c = a.to[i];
    if (!row_ok(a, p) || !row_ok(a, c) || __ldcg(a.mark + p) != 0 || a.t.cached_len[c] != 0) {
      bad = true;
      continue;
    }
    const int have = a.t.cached_len[p], len = a.fork_len ? a.fork_len[i] : have;
    if (!len_fits(a, have) || len < 0 || len > have) bad = true;
    a.row_a[i] = len;
  }
  verdict(a, !__syncthreads_or(bad));
}

// An item: FORK_ROWS consecutive children, SEG entries. A run of children of one parent
// reads each entry once and adds the run's length to its page's count at once.
__global__ void __launch_bounds__(AT) fork_apply(const Pages a, int segs) {
  pdl_trigger();
  pdl_wait();
  if (!a.hdr->ok) return;
  const int64_t stride = a.t.max_blocks_per_seq;
  const int groups = (a.n + FORK_ROWS - 1) / FORK_ROWS;
  const int64_t items = (int64_t)groups * segs;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int i0 = (int)(it / segs) * FORK_ROWS, s = (int)(it % segs);
    const int i1 = min(i0 + FORK_ROWS, a.n);
    if (s == 0 && threadIdx.x < i1 - i0)
      a.t.cached_len[a.to[i0 + threadIdx.x]] = a.row_a[i0 + threadIdx.x];
    int nmax = 0;
    for (int i = i0; i < i1; ++i) nmax = max(nmax, pages_of(a.row_a[i], a.bs_log2));
    for (int j = s * SEG + threadIdx.x; j < min(nmax, (s + 1) * SEG); j += AT) {
      int prev = -1, e = -1, add = 0;
      for (int i = i0; i < i1; ++i) {
        if (j >= pages_of(a.row_a[i], a.bs_log2)) continue;
        const int p = a.rows[i];
        if (p != prev) {
          if (add) atomicAdd(a.t.ref_count + e, add);
          add = 0;
          prev = p;
          e = a.t.block_table[p * stride + j];
          if (e < 0 || e >= a.t.num_blocks) atomicOr(a.flags, FLAG_PAGES_SHAPE);
        }
        if (e >= 0 && e < a.t.num_blocks) ++add;
        a.t.block_table[a.to[i] * stride + j] = e;
      }
      if (add) atomicAdd(a.t.ref_count + e, add);
    }
  }
}

// ---------------------------------------------------------------------------- trim

// One CTA: rows distinct, 0 <= new <= old. row_a[i]: the old length.
__global__ void __launch_bounds__(PT) trim_plan(const Pages a) {
  pdl_trigger();
  pdl_wait();
  bool bad = mark_rows(a, a.rows);
  for (int i = threadIdx.x; i < a.n; i += PT) {
    const int r = row_at(a, i);
    if (!row_ok(a, r)) continue;
    const int old = a.t.cached_len[r], to = a.to[i];
    if (!len_fits(a, old) || to < 0 || to > old) bad = true;
    a.row_a[i] = old;
  }
  verdict(a, !__syncthreads_or(bad));
}

__global__ void __launch_bounds__(AT) trim_apply(const Pages a, int segs) {
  pdl_trigger();
  pdl_wait();
  if (!a.hdr->ok) return;
  const int64_t stride = a.t.max_blocks_per_seq;
  const int64_t items = (int64_t)a.n * segs;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int i = (int)(it / segs), s = (int)(it % segs);
    const int r = row_at(a, i), to = a.to[i];
    const int j0 = pages_of(to, a.bs_log2) + s * SEG;
    const int j1 = min(pages_of(a.row_a[i], a.bs_log2), j0 + SEG);
    if (s == 0 && threadIdx.x == 0) a.t.cached_len[r] = to;
    for (int j = j0 + threadIdx.x; j < j1; j += AT) {
      int32_t* at = a.t.block_table + r * stride + j;
      const int e = *at;
      *at = -1;
      if (e < 0 || e >= a.t.num_blocks) {
        atomicOr(a.flags, FLAG_PAGES_SHAPE);
      } else if (atomicSub(a.t.ref_count + e, 1) <= 0) {  // was free: a count stays >= 0
        atomicAdd(a.t.ref_count + e, 1);
        atomicOr(a.flags, FLAG_PAGES_SHAPE);
      }
    }
  }
}

// -------------------------------------------------------------------------- extend

// CTA 0 plans the rows: row_a[i] the first fresh page's rank, row_b[i] the shared page that
// row i parts from (-1: none), row_c the rows that do, in call order, row_d[i] the old
// length. A row parts from its
// partial last page when another holder of it remains: some holder is not in the call, or
// a later row of the call is one. The other CTAs count the free pages of a chunk each; the
// last to finish turns the counts into ranks and compares the free pages with the need.
__global__ void __launch_bounds__(PT) extend_plan(const Pages a) {
  pdl_trigger();
  pdl_wait();
  const int64_t stride = a.t.max_blocks_per_seq;
  if (blockIdx.x == 0) {
    bool bad = mark_rows(a, a.rows);
    auto partial_page = [&](int i) -> int {  // the page row i would write into, or -1
      const int r = row_at(a, i);
      if (!row_ok(a, r)) return -1;
      const int old = a.t.cached_len[r];
      if (!len_fits(a, old) || a.to[i] <= old || (old & ((1 << a.bs_log2) - 1)) == 0) return -1;
      const int e = a.t.block_table[r * stride + (old >> a.bs_log2)];
      return e >= 0 && e < a.t.num_blocks ? e : -2;
    };
    for (int i = threadIdx.x; i < a.n; i += PT) {
      const int r = row_at(a, i);
      if (!row_ok(a, r)) continue;
      const int old = a.t.cached_len[r];
      const int e = partial_page(i);
      if (!len_fits(a, old) || !len_fits(a, a.to[i]) || a.to[i] < old || e == -2 ||
          (e >= 0 && a.t.ref_count[e] < 1))
        bad = true;
      if (e >= 0) {
        a.blk_a[e] = 0;   // rows of the call that hold page e
        a.blk_b[e] = -1;  // the last of them
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.n; i += PT) {
      const int e = partial_page(i);
      if (e >= 0) {
        atomicAdd(a.blk_a + e, 1);
        atomicMax(a.blk_b + e, i);
      }
    }
    bad = __syncthreads_or(bad);
    long long need = 0;
    int cows = 0;
    for (int base = 0; base < a.n && !bad; base += PT) {
      const int i = base + threadIdx.x;
      int cow = 0, e = -1;
      long long want = 0;
      if (i < a.n) {
        e = partial_page(i);
        if (e >= 0 && a.t.ref_count[e] > 1)
          cow = !(__ldcg(a.blk_a + e) == a.t.ref_count[e] && __ldcg(a.blk_b + e) == i);
        want = cow + pages_of(a.to[i], a.bs_log2) - pages_of(a.t.cached_len[row_at(a, i)], a.bs_log2);
      }
      long long total;
      int nc;
      const long long ex = scan_pt(want, total);
      const int exc = scan_pt(cow, nc);
      if (i < a.n) {
        a.row_a[i] = (int32_t)(need + ex);
        a.row_b[i] = cow ? e : -1;
        a.row_d[i] = a.t.cached_len[row_at(a, i)];
        if (cow) a.row_c[cows + exc] = i;
      }
      need += total;
      cows += nc;
      if (need > a.t.num_blocks) break;  // more than the pool has: no rank is used
    }
    if (threadIdx.x == 0) {
      a.hdr->rows_bad = bad ? 1 : 0;
      a.hdr->need = (int32_t)min(need, 0x7fffffffll);
      a.hdr->cows = cows;
    }
  } else {
    const int c = blockIdx.x - 1;
    const int4 v = chunk_counts(a, c);
    const int mine = (v.x == 0) + (v.y == 0) + (v.z == 0) + (v.w == 0);
    int total;
    scan_pt(mine, total);
    if (threadIdx.x == 0) a.chunk[c] = total;
  }
  if (!last_cta(a)) return;
  const int free_pages = scan_chunks(a);
  if (threadIdx.x == 0) {
    const bool bad = __ldcg(&a.hdr->rows_bad) != 0, few = __ldcg(&a.hdr->need) > free_pages;
    a.hdr->ok = !bad && !few;
    if (bad) atomicOr(a.flags, FLAG_PAGES_SHAPE);
    else if (few) atomicOr(a.flags, FLAG_NO_PAGES);
  }
}

// blk_a[k]: the k-th free page, k < need.
__global__ void __launch_bounds__(PT) extend_fresh(const Pages a) {
  pdl_trigger();
  pdl_wait();
  const int need = a.hdr->need, base = a.chunk[blockIdx.x];
  if (!a.hdr->ok || base >= need) return;
  const int4 v = chunk_counts(a, blockIdx.x);
  int total;
  int k = base + scan_pt((v.x == 0) + (v.y == 0) + (v.z == 0) + (v.w == 0), total);
  const int p = blockIdx.x * CHUNK + threadIdx.x * 4;
  if (v.x == 0 && k < need) a.blk_a[k] = p;
  k += v.x == 0;
  if (v.y == 0 && k < need) a.blk_a[k] = p + 1;
  k += v.y == 0;
  if (v.z == 0 && k < need) a.blk_a[k] = p + 2;
  k += v.z == 0;
  if (v.w == 0 && k < need) a.blk_a[k] = p + 3;
}

// bytes (a multiple of 16) from src to dst by the CTA's threads, eight loads in flight each.
__device__ __forceinline__ void copy_bytes(uint8_t* dst, const uint8_t* src, int bytes) {
  const uint4* s = reinterpret_cast<const uint4*>(src);
  uint4* d = reinterpret_cast<uint4*>(dst);
  const int n = bytes >> 4;
  constexpr int U = COPY_BYTES / 16 / AT;
  for (int base = threadIdx.x; base < n; base += U * AT) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (base + u * AT < n) v[u] = __ldcs(s + base + u * AT);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (base + u * AT < n) __stcs(d + base + u * AT, v[u]);
  }
}

// Items 0 .. n - 1 (a warp each): a row's table entries, counts and length. After them, for
// each row that parts from a shared page, its filled positions in every pool.
__global__ void __launch_bounds__(AT) extend_apply(const Pages a, const __grid_constant__ PoolList pl) {
  pdl_trigger();
  pdl_wait();
  if (!a.hdr->ok) return;
  const int64_t stride = a.t.max_blocks_per_seq;
  const int lane = threadIdx.x & 31;
  for (int i = blockIdx.x * (AT / 32) + (threadIdx.x >> 5); i < a.n; i += gridDim.x * (AT / 32)) {
    const int r = row_at(a, i), to = a.to[i], old = a.row_d[i], shared = a.row_b[i];
    const int cow = shared >= 0 ? 1 : 0;
    const int j0 = pages_of(old, a.bs_log2) - cow, j1 = pages_of(to, a.bs_log2);
    for (int j = j0 + lane; j < j1; j += 32) {
      const int p = a.blk_a[a.row_a[i] + j - j0];
      a.t.block_table[r * stride + j] = p;
      a.t.ref_count[p] = 1;
    }
    __syncwarp();
    if (lane == 0) {
      if (cow) atomicSub(a.t.ref_count + shared, 1);
      a.t.cached_len[r] = to;
    }
  }
  const int64_t per_row = (int64_t)pl.n * pl.seg_max, items = (int64_t)a.hdr->cows * per_row;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int i = a.row_c[it / per_row];
    const int q = (int)(it % per_row), pool = q / pl.seg_max, s = q % pl.seg_max;
    const int64_t row_bytes = pl.p[pool].page_bytes >> a.bs_log2;
    const int64_t filled = (a.row_d[i] & ((1 << a.bs_log2) - 1)) * row_bytes;
    const int64_t b0 = (int64_t)s * COPY_BYTES;
    if (b0 >= filled) continue;
    uint8_t* base = (uint8_t*)pl.p[pool].base;
    const int dst = a.blk_a[a.row_a[i]], src = a.row_b[i];
    copy_bytes(base + dst * pl.p[pool].page_bytes + b0, base + src * pl.p[pool].page_bytes + b0,
               (int)min(filled - b0, (int64_t)COPY_BYTES));
  }
}

// ------------------------------------------------------------------------- compact

// CTAs 0 .. table CTAs - 1 check the tables (lengths in range, entries naming pages in
// use); the others count the live pages of a chunk each. The last CTA: L = live pages, the
// live pages before each chunk, and those among the first L.
__global__ void __launch_bounds__(PT) compact_plan(const Pages a, int table_ctas, int segs) {
  pdl_trigger();
  pdl_wait();
  if ((int)blockIdx.x < table_ctas) {
    const int64_t items = (int64_t)a.t.table_rows * segs;
    bool bad = false;
    for (int64_t it = blockIdx.x * (int64_t)(PT / 32) + (threadIdx.x >> 5); it < items;
         it += (int64_t)table_ctas * (PT / 32)) {
      const int64_t r = it / segs;
      const int s = (int)(it % segs), len = a.t.cached_len[r];
      if (!len_fits(a, len)) {
        bad = true;
        continue;
      }
      const int j1 = min(pages_of(len, a.bs_log2), (s + 1) * SEG);
      for (int j = s * SEG + (threadIdx.x & 31); j < j1; j += 32) {
        const int e = a.t.block_table[r * a.t.max_blocks_per_seq + j];
        if (e < 0 || e >= a.t.num_blocks || a.t.ref_count[e] < 1) bad = true;
      }
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) a.chunk[a.chunks + blockIdx.x] = bad ? 1 : 0;
  } else {
    const int c = blockIdx.x - table_ctas;
    const int4 v = chunk_counts(a, c);
    int total;
    scan_pt((v.x > 0) + (v.y > 0) + (v.z > 0) + (v.w > 0), total);
    if (threadIdx.x == 0) a.chunk[c] = total;
  }
  if (!last_cta(a)) return;
  bool bad = false;
  for (int i = threadIdx.x; i < table_ctas; i += PT) bad |= __ldcg(a.chunk + a.chunks + i) != 0;
  bad = __syncthreads_or(bad);
  const int live = scan_chunks(a);
  __syncthreads();
  // live pages before page L: those before its chunk, and the chunk's own before it
  int below = live;
  if (live < a.t.num_blocks) {
    const int c = live / CHUNK, p = c * CHUNK + threadIdx.x * 4;
    const int4 v = chunk_counts(a, c);
    int total;
    scan_pt((v.x > 0 && p < live) + (v.y > 0 && p + 1 < live) + (v.z > 0 && p + 2 < live) +
                (v.w > 0 && p + 3 < live),
            total);
    below = __ldcg(a.chunk + c) + total;
  }
  if (threadIdx.x == 0) {
    a.hdr->live = live;
    a.hdr->below = below;
  }
  verdict(a, !bad);
}

// Ranks: the k-th live page p at or above L moves to the k-th free page below L. blk_b[p] =
// k, blk_a[k] = the free page, blk_a[num_blocks - 1 - k] = p. (There are at most min(L,
// num_blocks - L) moves, so the two parts of blk_a do not meet.) The map of the other pages.
__global__ void __launch_bounds__(PT) compact_rank(const Pages a) {
  pdl_trigger();
  pdl_wait();
  if (!a.hdr->ok) return;
  const int live = a.hdr->live, below = a.hdr->below;
  const int4 v = chunk_counts(a, blockIdx.x);
  int total;
  int before = a.chunk[blockIdx.x] + scan_pt((v.x > 0) + (v.y > 0) + (v.z > 0) + (v.w > 0), total);
  const int p0 = blockIdx.x * CHUNK + threadIdx.x * 4;
  const int w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int p = p0 + e;
    if (p >= a.t.num_blocks) break;
    if (w[e] > 0) {
      if (p >= live) {
        a.blk_b[p] = before - below;
        a.blk_a[a.t.num_blocks - 1 - (before - below)] = p;
      } else if (a.remap) {
        a.remap[p] = p;
      }
      ++before;
    } else {
      if (p < live) a.blk_a[p - before] = p;
      if (a.remap) a.remap[p] = -1;
    }
  }
}

// Grid-stride over: the page data (move x pool x COPY_BYTES), the table entries, and the
// counts of the pages that move.
__global__ void __launch_bounds__(AT) compact_apply(const Pages a, int segs,
                                                    const __grid_constant__ PoolList pl) {
  pdl_trigger();
  pdl_wait();
  if (!a.hdr->ok) return;
  const int live = a.hdr->live, moves = live - a.hdr->below, nb = a.t.num_blocks;
  const int64_t per_move = (int64_t)pl.n * pl.seg_max, items = moves * per_move;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int k = (int)(it / per_move);
    const int q = (int)(it % per_move), pool = q / pl.seg_max, s = q % pl.seg_max;
    const int64_t bytes = pl.p[pool].page_bytes, b0 = (int64_t)s * COPY_BYTES;
    if (b0 >= bytes) continue;
    uint8_t* base = (uint8_t*)pl.p[pool].base;
    copy_bytes(base + a.blk_a[k] * bytes + b0, base + a.blk_a[nb - 1 - k] * bytes + b0,
               (int)min(bytes - b0, (int64_t)COPY_BYTES));
  }
  const int64_t ents = (int64_t)a.t.table_rows * segs;
  for (int64_t it = blockIdx.x; it < ents; it += gridDim.x) {
    const int64_t r = it / segs;
    const int s = (int)(it % segs);
    const int j1 = min(pages_of(a.t.cached_len[r], a.bs_log2), (s + 1) * SEG);
    for (int j = s * SEG + threadIdx.x; j < j1; j += AT) {
      int32_t* at = a.t.block_table + r * a.t.max_blocks_per_seq + j;
      const int e = *at;
      if (e >= live) *at = a.blk_a[a.blk_b[e]];
    }
  }
  for (int64_t k = blockIdx.x * (int64_t)AT + threadIdx.x; k < moves; k += (int64_t)gridDim.x * AT) {
    const int dst = a.blk_a[k], src = a.blk_a[nb - 1 - k];
    a.t.ref_count[dst] = a.t.ref_count[src];
    a.t.ref_count[src] = 0;
    if (a.remap) a.remap[src] = dst;
  }
  if (a.num_live && blockIdx.x == 0 && threadIdx.x == 0) *a.num_live = live;
}

PagesWs pages_layout(int32_t num_blocks, int32_t table_rows) {
  PagesWs w;
  const size_t R = (size_t)table_rows * 4, N = (size_t)num_blocks * 4;
  size_t o = 256;  // the flag word and the ticket
  w.hdr = o;   o += 256;
  w.rows = o;  o = align_up(o + 5 * R, 256);
  w.chunk = o; o = align_up(o + 4 * ((size_t)(num_blocks + CHUNK - 1) / CHUNK + TABLE_CTAS), 256);
  w.blk = o;   o = align_up(o + 2 * N, 256);
  w.total = o;
  return w;
}

Pages make(const sv_page_table& t, void* ws) {
  const PagesWs w = pages_layout(t.num_blocks, t.table_rows);
  uint8_t* base = (uint8_t*)ws;
  Pages a = {};
  a.t = t;
  a.flags = (uint32_t*)base;
  a.ticket = (uint32_t*)base + 1;
  a.hdr = (PagesHdr*)(base + w.hdr);
  a.mark = (int32_t*)(base + w.rows);
  a.row_a = a.mark + t.table_rows;
  a.row_b = a.row_a + t.table_rows;
  a.row_c = a.row_b + t.table_rows;
  a.row_d = a.row_c + t.table_rows;
  a.chunk = (int32_t*)(base + w.chunk);
  a.blk_a = (int32_t*)(base + w.blk);
  a.blk_b = a.blk_a + t.num_blocks;
  a.chunks = (t.num_blocks + CHUNK - 1) / CHUNK;
  while ((1 << a.bs_log2) < t.block_size) ++a.bs_log2;
  return a;
}

PoolList pool_list(int n, const sv_page_data* p) {
  PoolList l = {};
  l.n = n;
  int64_t most = 0;
  for (int i = 0; i < n; ++i) {
    l.p[i] = p[i];
    most = p[i].page_bytes > most ? p[i].page_bytes : most;
  }
  l.seg_max = (int)((most + COPY_BYTES - 1) / COPY_BYTES);
  return l;
}

unsigned grid_for(int64_t items, int sms) {  // resident at once: 8 CTAs of AT threads an SM
  const int64_t most = (int64_t)sms * (2048 / AT);
  return (unsigned)(items < 1 ? 1 : items < most ? items : most);
}

}  // namespace

size_t pages_ws_bytes(int32_t num_blocks, int32_t table_rows) {
  return pages_layout(num_blocks, table_rows).total;
}

cudaError_t launch_pages_fork(const sv_page_table& t, int n, const int32_t* parents,
                              const int32_t* children, const int32_t* fork_len, void* ws, int sms,
                              cudaStream_t s) {
  Pages a = make(t, ws);
  a.n = n;
  a.rows = parents;
  a.to = children;
  a.fork_len = fork_len;
  cudaError_t e = launch_pdl(fork_plan, dim3(1), dim3(PT), 0, s, a);
  if (e != cudaSuccess) return e;
  const int segs = (t.max_blocks_per_seq + SEG - 1) / SEG;
  const int64_t items = (int64_t)((n + FORK_ROWS - 1) / FORK_ROWS) * segs;
  return launch_pdl(fork_apply, dim3(grid_for(items, sms)), dim3(AT), 0, s, a, segs);
}

cudaError_t launch_pages_trim(const sv_page_table& t, int n, const int32_t* rows,
                              const int32_t* new_len, void* ws, int sms, cudaStream_t s) {
  Pages a = make(t, ws);
  a.n = n;
  a.rows = rows;
  a.to = new_len;
  cudaError_t e = launch_pdl(trim_plan, dim3(1), dim3(PT), 0, s, a);
  if (e != cudaSuccess) return e;
  const int segs = (t.max_blocks_per_seq + SEG - 1) / SEG;
  return launch_pdl(trim_apply, dim3(grid_for((int64_t)n * segs, sms)), dim3(AT), 0, s, a, segs);
}

cudaError_t launch_pages_extend(const sv_page_table& t, int n, const int32_t* rows,
                                const int32_t* new_len, int num_pools, const sv_page_data* pools,
                                void* ws, int sms, cudaStream_t s) {
  Pages a = make(t, ws);
  a.n = n;
  a.rows = rows;
  a.to = new_len;
  cudaError_t e = launch_pdl(extend_plan, dim3(1 + a.chunks), dim3(PT), 0, s, a);
  if (e != cudaSuccess) return e;
  e = launch_pdl(extend_fresh, dim3(a.chunks), dim3(PT), 0, s, a);
  if (e != cudaSuccess) return e;
  const PoolList l = pool_list(num_pools, pools);
  const int64_t copies = (int64_t)n * l.n * l.seg_max, rows_items = (n + AT / 32 - 1) / (AT / 32);
  return launch_pdl(extend_apply, dim3(grid_for(copies > rows_items ? copies : rows_items, sms)),
                    dim3(AT), 0, s, a, l);
}

cudaError_t launch_pages_compact(const sv_page_table& t, int num_pools, const sv_page_data* pools,
                                 int32_t* remap, int32_t* num_live, void* ws, int sms,
                                 cudaStream_t s) {
  Pages a = make(t, ws);
  a.remap = remap;
  a.num_live = num_live;
  const int segs = (t.max_blocks_per_seq + SEG - 1) / SEG;
  const int64_t warps = (int64_t)t.table_rows * segs;
  const int table_ctas = (int)(warps > TABLE_CTAS * (PT / 32) ? TABLE_CTAS
                                                              : (warps + PT / 32 - 1) / (PT / 32));
  cudaError_t e =
      launch_pdl(compact_plan, dim3(table_ctas + a.chunks), dim3(PT), 0, s, a, table_ctas, segs);
  if (e != cudaSuccess) return e;
  e = launch_pdl(compact_rank, dim3(a.chunks), dim3(PT), 0, s, a);
  if (e != cudaSuccess) return e;
  const PoolList l = pool_list(num_pools, pools);
  const int64_t copies = (int64_t)t.num_blocks * l.n * l.seg_max;  // at least the moves'
  return launch_pdl(compact_apply, dim3(grid_for(copies > warps ? copies : warps, sms)), dim3(AT),
                    0, s, a, segs, l);
}

}  // namespace sv
