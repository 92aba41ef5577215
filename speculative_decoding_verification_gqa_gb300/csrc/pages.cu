// pages.cu -- the pages of a paged cache: fork, extend (with copy on write), trim, compact.
//
// State (the caller's): ref_count[p], the number of table entries in use that name page p
// (p is free iff it is 0); block_table[r, j], the page of positions j * bs .. of row r;
// cached_len[r], the positions row r holds, so that its entries in use are those with
// j < ceil(cached_len[r] / bs). Every operator checks all rows of the call before it changes
// anything. fork and trim are one kernel, whose CTAs each make the same checks and whose
// last CTA writes the lengths, which the checks read; extend and compact begin with a kernel
// that ends with one verdict (PagesHdr::ok), and the kernels after it do nothing when that
// is 0.
//
// Results do not depend on the order in which threads run: counts change by integer
// additions, free pages are taken lowest first by ranks from a prefix sum over the pool,
// and ties between rows go by their order in the call.
//
// All of it is bound by latency (launches, and a chain of dependent reads) until tables of a
// million entries or megabytes of page data are touched; the page data then moves at the
// copy bandwidth.
#include <climits>

#include "internal.cuh"

namespace sv {
namespace {

constexpr int PT = 1024;          // threads of the planning kernels
constexpr int CHUNK = 4096;       // pages counted by one CTA (PT threads x 4)
constexpr int AT = 256;           // threads of the other kernels
constexpr int SEG = 512;          // table entries of one work item
constexpr int NR = 4;             // rows of a thread whose reads run together
constexpr int FORK_ROWS = 8;      // consecutive children of one work item
constexpr int COPY_BYTES = 16384; // page bytes of one copying work item
constexpr int TABLE_CTAS = 64;    // compact: CTAs that check the tables

// Verdict and totals of a call; every field is written before it is read in each call.
struct PagesHdr {
  int32_t ok;
  int32_t rows_bad;   // extend: a check on the rows failed
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
  int32_t *row_a, *row_b, *row_c, *row_d, *row_e;  // [table_rows] each
  int32_t* chunk;                         // [chunks + 1], then [TABLE_CTAS] of compact
  int32_t *blk_a, *blk_b, *blk_c;         // [num_blocks] each
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

static_assert(PT == 1024, "the scan below has 32 warps' sums");

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

// A set of table rows in shared memory, a bit each.
extern __shared__ uint32_t s_rows[];
__device__ __forceinline__ void clear_rows(const Pages& a) {
  for (int i = threadIdx.x; i < (a.t.table_rows + 31) / 32; i += blockDim.x) s_rows[i] = 0;
}
__device__ __forceinline__ bool add_row(int r) {  // false if it was there
  return (atomicOr(s_rows + (r >> 5), 1u << (r & 31)) >> (r & 31) & 1) == 0;
}
__device__ __forceinline__ bool has_row(int r) { return (s_rows[r >> 5] >> (r & 31) & 1) != 0; }

__device__ __forceinline__ void verdict(const Pages& a, bool ok) {
  if (threadIdx.x == 0) {
    a.hdr->ok = ok ? 1 : 0;
    if (!ok) atomicOr(a.flags, FLAG_PAGES_SHAPE);
  }
}

// ---------------------------------------------------------------------------- fork

// Checks: children distinct, empty and not parents; lengths within the parents'. An item:
// FORK_ROWS consecutive children, SEG entries. A run of children of one parent reads each
// entry once and adds the run's length to its page's count at once. (992 children of up to
// 2048 entries: 16.5 us captured; 17.2 with a row at a time in the checks. 6 children of 63
// entries: 6.3.)
__global__ void __launch_bounds__(AT) fork_kernel(const Pages a, int segs) {
  pdl_trigger();
  pdl_wait();
  clear_rows(a);
  __syncthreads();
  bool bad = false;
  for (int i0 = threadIdx.x; i0 < a.n; i0 += NR * AT) {
    int c[NR];
#pragma unroll
    for (int k = 0; k < NR; ++k) c[k] = i0 + k * AT < a.n ? a.to[i0 + k * AT] : 0;
#pragma unroll
    for (int k = 0; k < NR; ++k)
      if (i0 + k * AT < a.n && (!row_ok(a, c[k]) || !add_row(c[k]))) bad = true;
  }
  __syncthreads();
  for (int i0 = threadIdx.x; i0 < a.n; i0 += NR * AT) {
    int p[NR], c[NR], have[NR], len[NR], used[NR];
#pragma unroll
    for (int k = 0; k < NR; ++k) {
      const int i = i0 + k * AT;
      p[k] = i < a.n ? a.rows[i] : -1;
      c[k] = i < a.n ? a.to[i] : -1;
      len[k] = i < a.n && a.fork_len ? a.fork_len[i] : 0;
    }
#pragma unroll
    for (int k = 0; k < NR; ++k) {
      const bool ok = row_ok(a, p[k]) && row_ok(a, c[k]);
      have[k] = ok ? a.t.cached_len[p[k]] : 0;
      used[k] = ok ? a.t.cached_len[c[k]] : 1;
    }
#pragma unroll
    for (int k = 0; k < NR; ++k)
      if (i0 + k * AT < a.n && (used[k] != 0 || has_row(p[k]) || !len_fits(a, have[k]) ||
                                len[k] < 0 || len[k] > have[k]))
        bad = true;
  }
  bad = __syncthreads_or(bad);
  auto length = [&](int i) { return a.fork_len ? a.fork_len[i] : a.t.cached_len[a.rows[i]]; };
  const int64_t stride = a.t.max_blocks_per_seq;
  const int groups = (a.n + FORK_ROWS - 1) / FORK_ROWS;
  const int64_t items = bad ? 0 : (int64_t)groups * segs;
  int least = 1;  // the least count met: whoever adds to a free page first finds 0
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int i0 = (int)(it / segs) * FORK_ROWS, s = (int)(it % segs);
    const int cnt = min(FORK_ROWS, a.n - i0);
    // the item's rows, read at once
    int par[FORK_ROWS], child[FORK_ROWS], pages[FORK_ROWS], nmax = 0;
#pragma unroll
    for (int k = 0; k < FORK_ROWS; ++k) {
      par[k] = k < cnt ? a.rows[i0 + k] : -1;
      child[k] = k < cnt ? a.to[i0 + k] : -1;
      pages[k] = k < cnt ? pages_of(length(i0 + k), a.bs_log2) : 0;
      nmax = max(nmax, pages[k]);
    }
    for (int j = s * SEG + threadIdx.x; j < min(nmax, (s + 1) * SEG); j += AT) {
      int prev = -1, e = -1, add = 0;
#pragma unroll
      for (int k = 0; k < FORK_ROWS; ++k) {
        if (j >= pages[k]) continue;
        if (par[k] != prev) {
          if (add) least = min(least, atomicAdd(a.t.ref_count + e, add));
          add = 0;
          prev = par[k];
          e = a.t.block_table[prev * stride + j];
          if (e < 0 || e >= a.t.num_blocks) atomicOr(a.flags, FLAG_PAGES_SHAPE);
        }
        if (e >= 0 && e < a.t.num_blocks) ++add;
        a.t.block_table[child[k] * stride + j] = e;
      }
      if (add) least = min(least, atomicAdd(a.t.ref_count + e, add));
    }
  }
  if (least < 1) atomicOr(a.flags, FLAG_PAGES_SHAPE);
  if (!last_cta(a)) return;  // every CTA has read the lengths
  if (bad) {
    if (threadIdx.x == 0) atomicOr(a.flags, FLAG_PAGES_SHAPE);
    return;
  }
  for (int i = threadIdx.x; i < a.n; i += AT) a.t.cached_len[a.to[i]] = length(i);
}

// ---------------------------------------------------------------------------- trim

// Checks: rows distinct, 0 <= new <= old. An item: TRIM_ROWS consecutive rows of the call, AT
// entries, a thread each. Rows of the run that drop the same page (samples that finish
// together) take its count down at once: bound by those atomics, 20 to 26 a ns at L2, and the
// reads before them. 1024 rows in families of 8 that drop 0.5 million entries: 14.6 us
// captured, 20.0 with an atomic for each entry; 64 rows that drop one or none 5.2.
constexpr int TRIM_ROWS = 8;
__global__ void __launch_bounds__(AT) trim_kernel(const Pages a, int segs) {
  pdl_trigger();
  pdl_wait();
  clear_rows(a);
  __syncthreads();
  bool bad = false;
  for (int i0 = threadIdx.x; i0 < a.n; i0 += NR * AT) {
    int r[NR], to[NR], old[NR];
#pragma unroll
    for (int k = 0; k < NR; ++k) {
      const int i = i0 + k * AT;
      r[k] = i < a.n ? row_at(a, i) : -1;
      to[k] = i < a.n ? a.to[i] : 0;
    }
#pragma unroll
    for (int k = 0; k < NR; ++k) old[k] = row_ok(a, r[k]) ? a.t.cached_len[r[k]] : 0;
#pragma unroll
    for (int k = 0; k < NR; ++k)
      if (i0 + k * AT < a.n && (!row_ok(a, r[k]) || !add_row(r[k]) || !len_fits(a, old[k]) ||
                                to[k] < 0 || to[k] > old[k]))
        bad = true;
  }
  bad = __syncthreads_or(bad);
  const int64_t stride = a.t.max_blocks_per_seq;
  const int groups = (a.n + TRIM_ROWS - 1) / TRIM_ROWS;
  const int64_t items = bad ? 0 : (int64_t)groups * segs;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int s = (int)(it / groups), i0 = (int)(it - (int64_t)s * groups) * TRIM_ROWS;
    int row[TRIM_ROWS], from[TRIM_ROWS], end[TRIM_ROWS], lo = INT_MAX, hi = 0;
#pragma unroll
    for (int k = 0; k < TRIM_ROWS; ++k) {
      const int i = i0 + k;
      row[k] = i < a.n ? row_at(a, i) : 0;
      from[k] = i < a.n ? pages_of(a.to[i], a.bs_log2) : 0;
    }
#pragma unroll
    for (int k = 0; k < TRIM_ROWS; ++k) {
      end[k] = i0 + k < a.n ? pages_of(a.t.cached_len[row[k]], a.bs_log2) : 0;
      if (from[k] < end[k]) {
        lo = min(lo, from[k]);
        hi = max(hi, end[k]);
      }
    }
    if (lo >= hi || hi - lo <= s * AT) continue;
    const int j = lo + s * AT + (int)threadIdx.x;
    int e[TRIM_ROWS], run[TRIM_ROWS], was[TRIM_ROWS];
#pragma unroll
    for (int k = 0; k < TRIM_ROWS; ++k) {
      const bool drops = j >= from[k] && j < end[k];
      int32_t* at = a.t.block_table + row[k] * stride + j;
      e[k] = drops ? *at : -1;
      if (drops) {
        *at = -1;
        if (e[k] < 0 || e[k] >= a.t.num_blocks) {
          atomicOr(a.flags, FLAG_PAGES_SHAPE);
          e[k] = -1;
        }
      }
    }
#pragma unroll
    for (int k = TRIM_ROWS - 1; k >= 0; --k)  // how many from row k on drop its page
      run[k] = k < TRIM_ROWS - 1 && e[k] == e[k + 1] ? run[k + 1] + 1 : 1;
#pragma unroll
    for (int k = 0; k < TRIM_ROWS; ++k) {
      const bool first = e[k] >= 0 && (k == 0 || e[k] != e[k - 1]);
      was[k] = first ? atomicSub(a.t.ref_count + e[k], run[k]) : run[k];
    }
#pragma unroll
    for (int k = 0; k < TRIM_ROWS; ++k)
      if (was[k] < run[k]) {  // more entries than the page's count: that stays >= 0
        atomicAdd(a.t.ref_count + e[k], run[k] - max(was[k], 0));
        atomicOr(a.flags, FLAG_PAGES_SHAPE);
      }
  }
  if (!last_cta(a)) return;  // every CTA has read the lengths
  if (bad) {
    if (threadIdx.x == 0) atomicOr(a.flags, FLAG_PAGES_SHAPE);
    return;
  }
  for (int i = threadIdx.x; i < a.n; i += AT) a.t.cached_len[row_at(a, i)] = a.to[i];
}

// -------------------------------------------------------------------------- extend

// The last chunk c with chunk[c] <= k (the chunk that holds the page of rank k).
__device__ __forceinline__ int chunk_of(const Pages& a, int k) {
  int lo = 0, hi = a.chunks - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldcg(a.chunk + mid) <= k) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// CTA 0 plans the rows: row_a[i] the first fresh page's rank, row_b[i] the shared page that
// row i parts from (-1: none), row_c the rows that do, in call order, row_d[i] the old
// length. A row parts from its partial last page when another holder of it remains: some
// holder is not in the call, or a later row of the call is one. The other CTAs list the free
// pages of a chunk each in blk_a; the last to finish turns their numbers into ranks, finds
// the chunk of each row's first page (row_e) and compares the free pages with the need.
// Up to PT rows what a row needs stays in its thread, and the holders of a page are counted
// in a table in shared memory; beyond, by page in blk_b and blk_c.
// (256 rows, of which 224 part from shared pages, 8 pools: 14.5 us captured with extend_apply,
// of which this is the longer half; 8 rows 10.6.)
constexpr int SLOTS = 2 * PT;
__global__ void __launch_bounds__(PT) extend_plan(const Pages a) {
  __shared__ int s_page[SLOTS], s_cnt[SLOTS], s_last[SLOTS];
  pdl_trigger();
  pdl_wait();
  const int64_t stride = a.t.max_blocks_per_seq;
  const bool small = a.n <= PT;
  if (blockIdx.x == 0) {
    bool bad = false;
    clear_rows(a);
    for (int i = threadIdx.x; i < SLOTS; i += PT) {
      s_page[i] = -1;
      s_cnt[i] = 0;
      s_last[i] = -1;
    }
    __syncthreads();
    struct Row {
      int old, to, page, ref;  // page: what the row would write into, -1 none, -2 damaged
    };
    auto look = [&](int i) {
      Row w = {0, 0, -1, 0};
      const int r = row_at(a, i);
      w.to = a.to[i];
      if (!row_ok(a, r)) return w;
      w.old = a.t.cached_len[r];
      if (len_fits(a, w.old) && w.to > w.old && (w.old & ((1 << a.bs_log2) - 1)) != 0) {
        const int e = a.t.block_table[r * stride + (w.old >> a.bs_log2)];
        w.page = e >= 0 && e < a.t.num_blocks ? e : -2;
        if (w.page >= 0) w.ref = a.t.ref_count[e];
        if (w.page >= 0 && w.ref < 1) w.page = -2;
      }
      return w;
    };
    auto slot_of = [&](int page) {  // open addressing: at most PT pages in SLOTS places
      int h = (int)((uint32_t)page * 2654435761u >> (32 - 11));
      while (true) {
        const int was = atomicCAS(s_page + h, -1, page);
        if (was == -1 || was == page) return h;
        h = (h + 1) & (SLOTS - 1);
      }
    };
    static_assert(SLOTS == 1 << 11, "the hash keeps 11 bits");
    int32_t *count = small ? s_cnt : a.blk_b, *last = small ? s_last : a.blk_c;
    Row mine = {0, 0, -1, 0};
    int slot = 0;
    for (int i = threadIdx.x; i < a.n; i += PT) {
      const int r = row_at(a, i);
      mine = look(i);
      if (!row_ok(a, r) || !add_row(r) || !len_fits(a, mine.old) || !len_fits(a, mine.to) ||
          mine.to < mine.old || mine.page == -2)
        bad = true;
      if (mine.page >= 0) {
        if (small) {
          slot = slot_of(mine.page);
        } else {
          count[mine.page] = 0;
          last[mine.page] = -1;
        }
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.n; i += PT) {
      const Row w = small ? mine : look(i);
      if (w.page >= 0) {
        atomicAdd(count + (small ? slot : w.page), 1);
        atomicMax(last + (small ? slot : w.page), i);
      }
    }
    bad = __syncthreads_or(bad);
    long long need = 0;
    int cows = 0;
    for (int base = 0; base < a.n && !bad; base += PT) {
      const int i = base + threadIdx.x;
      int cow = 0;
      long long want = 0;
      Row w = {0, 0, -1, 0};
      if (i < a.n) {
        w = small ? mine : look(i);
        if (w.page >= 0 && w.ref > 1) {
          const int at = small ? slot : w.page;
          const int cnt = small ? s_cnt[at] : __ldcg(count + at);
          const int lst = small ? s_last[at] : __ldcg(last + at);
          cow = !(cnt == w.ref && lst == i);
        }
        want = cow + pages_of(w.to, a.bs_log2) - pages_of(w.old, a.bs_log2);
      }
      long long total;
      int nc;
      const long long ex = scan_pt(want, total);
      const int exc = scan_pt(cow, nc);
      if (i < a.n) {
        a.row_a[i] = (int32_t)(need + ex);
        a.row_b[i] = cow ? w.page : -1;
        a.row_d[i] = w.old;
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
    int32_t* dst = a.blk_a + (int64_t)c * CHUNK + scan_pt(mine, total);
    const int p = c * CHUNK + threadIdx.x * 4;
    if (v.x == 0) *dst++ = p;
    if (v.y == 0) *dst++ = p + 1;
    if (v.z == 0) *dst++ = p + 2;
    if (v.w == 0) *dst++ = p + 3;
    if (threadIdx.x == 0) a.chunk[c] = total;
  }
  if (!last_cta(a)) return;
  const int free_pages = scan_chunks(a);
  const bool bad = __ldcg(&a.hdr->rows_bad) != 0, few = __ldcg(&a.hdr->need) > free_pages;
  if (threadIdx.x == 0) {
    a.chunk[a.chunks] = free_pages;
    a.hdr->ok = !bad && !few;
    if (bad) atomicOr(a.flags, FLAG_PAGES_SHAPE);
    else if (few) atomicOr(a.flags, FLAG_NO_PAGES);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.n && !bad && !few; i += PT)
    a.row_e[i] = chunk_of(a, __ldcg(a.row_a + i));
}

// The page of rank k, from chunk c on.
__device__ __forceinline__ int page_of_rank(const Pages& a, int k, int c) {
  while (k >= a.chunk[c + 1]) ++c;
  return a.blk_a[(int64_t)c * CHUNK + k - a.chunk[c]];
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
      const int p = page_of_rank(a, a.row_a[i] + j - j0, a.row_e[i]);
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
    const int dst = page_of_rank(a, a.row_a[i], a.row_e[i]), src = a.row_b[i];
    copy_bytes(base + dst * pl.p[pool].page_bytes + b0, base + src * pl.p[pool].page_bytes + b0,
               (int)min(filled - b0, (int64_t)COPY_BYTES));
  }
}

// ------------------------------------------------------------------------- compact

// Ranks of chunk c: the k-th live page p at or above L moves to the k-th free page below L.
// blk_b[p] = k, blk_a[k] = the free page, blk_a[num_blocks - 1 - k] = p. (There are at most
// min(L, num_blocks - L) moves, so the two parts of blk_a do not meet.) The map of the other
// pages. Called by PT threads.
__device__ void rank_chunk(const Pages& a, int c, int live, int below) {
  const int4 v = chunk_counts(a, c);
  int total;
  int before = __ldcg(a.chunk + c) + scan_pt((v.x > 0) + (v.y > 0) + (v.z > 0) + (v.w > 0), total);
  const int p0 = c * CHUNK + threadIdx.x * 4;
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

// A pool of one chunk is ranked by the last CTA of compact_plan, for one launch less (512
// pages: 19 us a call instead of 22). With three chunks that CTA takes longer than the launch
// (12288 pages: 79 us against 75).
constexpr int RANK_INLINE = 1;
__global__ void __launch_bounds__(PT) compact_rank(const Pages a) {
  pdl_trigger();
  pdl_wait();
  if (a.hdr->ok) rank_chunk(a, blockIdx.x, a.hdr->live, a.hdr->below);
}

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
    if (threadIdx.x == 0) a.chunk[a.chunks + 1 + blockIdx.x] = bad ? 1 : 0;
  } else {
    const int c = blockIdx.x - table_ctas;
    const int4 v = chunk_counts(a, c);
    int total;
    scan_pt((v.x > 0) + (v.y > 0) + (v.z > 0) + (v.w > 0), total);
    if (threadIdx.x == 0) a.chunk[c] = total;
  }
  if (!last_cta(a)) return;
  bool bad = false;
  for (int i = threadIdx.x; i < table_ctas; i += PT) bad |= __ldcg(a.chunk + a.chunks + 1 + i) != 0;
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
  for (int c = 0; c < a.chunks && a.chunks <= RANK_INLINE && !bad; ++c) rank_chunk(a, c, live, below);
}

// Grid-stride over: the page data (move x pool x COPY_BYTES), the table entries, and the
// counts of the pages that move. Memory-bound: 343 MB in 60 us (5.7 TB/s) when 2.9 thousand
// pages of 2 pools, 32 KB each, move.
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
  w.chunk = o; o = align_up(o + 4 * ((size_t)(num_blocks + CHUNK - 1) / CHUNK + 1 + TABLE_CTAS), 256);
  w.blk = o;   o = align_up(o + 3 * N, 256);
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
  a.row_a = (int32_t*)(base + w.rows);
  a.row_b = a.row_a + t.table_rows;
  a.row_c = a.row_b + t.table_rows;
  a.row_d = a.row_c + t.table_rows;
  a.row_e = a.row_d + t.table_rows;
  a.chunk = (int32_t*)(base + w.chunk);
  a.blk_a = (int32_t*)(base + w.blk);
  a.blk_b = a.blk_a + t.num_blocks;
  a.blk_c = a.blk_b + t.num_blocks;
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

// Items of a row. A row has fewer than 2^31 positions, so at most 2^28 entries are in use,
// however long it is.
int segs_of(const sv_page_table& t, int seg = SEG) {
  const int most = t.max_blocks_per_seq < (1 << 28) ? t.max_blocks_per_seq : 1 << 28;
  return (most + seg - 1) / seg;
}

constexpr size_t set_bytes(int32_t rows) { return ((size_t)rows + 31) / 32 * 4; }
size_t row_set_bytes(const sv_page_table& t) { return set_bytes(t.table_rows); }
// Sets beyond what a launch may ask for unasked. The limit belongs to the kernel, not to the
// call: it is the same for every size, so that no call lowers it between another one's setting
// and launch.
template <class F>
cudaError_t allow_set(F kernel, size_t bytes) {
  return bytes <= 16 * 1024 ? cudaSuccess
                            : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)set_bytes(SV_MAX_TABLE_ROWS));
}

// Up to 8 CTAs of AT threads for each SM; an odd number, so that what repeats along the items
// (every other row dropped, say) falls to all CTAs. Not all of them are resident at once: the
// registers of the copying kernels let 6 onto an SM and those of fork and trim 5, a table of
// 2^20 rows one.
unsigned grid_for(int64_t items, int sms) {
  const int64_t most = ((int64_t)sms * (2048 / AT) - 1) | 1;
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
  const size_t set = row_set_bytes(t);
  cudaError_t e = allow_set(fork_kernel, set);
  if (e != cudaSuccess) return e;
  const int segs = segs_of(t);
  const int64_t items = (int64_t)((n + FORK_ROWS - 1) / FORK_ROWS) * segs;
  return launch_pdl(fork_kernel, dim3(grid_for(items, sms)), dim3(AT), set, s, a, segs);
}

cudaError_t launch_pages_trim(const sv_page_table& t, int n, const int32_t* rows,
                              const int32_t* new_len, void* ws, int sms, cudaStream_t s) {
  Pages a = make(t, ws);
  a.n = n;
  a.rows = rows;
  a.to = new_len;
  const size_t set = row_set_bytes(t);
  cudaError_t e = allow_set(trim_kernel, set);
  if (e != cudaSuccess) return e;
  const int segs = segs_of(t, AT);
  const int64_t items = (int64_t)((n + TRIM_ROWS - 1) / TRIM_ROWS) * segs;
  return launch_pdl(trim_kernel, dim3(grid_for(items, sms)), dim3(AT), set, s, a, segs);
}

cudaError_t launch_pages_extend(const sv_page_table& t, int n, const int32_t* rows,
                                const int32_t* new_len, int num_pools, const sv_page_data* pools,
                                void* ws, int sms, cudaStream_t s) {
  Pages a = make(t, ws);
  a.n = n;
  a.rows = rows;
  a.to = new_len;
  const size_t set = row_set_bytes(t);
  cudaError_t e = allow_set(extend_plan, set);
  if (e != cudaSuccess) return e;
  e = launch_pdl(extend_plan, dim3(1 + a.chunks), dim3(PT), set, s, a);
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
  const int segs = segs_of(t);
  const int64_t warps = (int64_t)t.table_rows * segs;
  const int table_ctas = (int)(warps > TABLE_CTAS * (PT / 32) ? TABLE_CTAS
                                                              : (warps + PT / 32 - 1) / (PT / 32));
  cudaError_t e =
      launch_pdl(compact_plan, dim3(table_ctas + a.chunks), dim3(PT), 0, s, a, table_ctas, segs);
  if (e != cudaSuccess) return e;
  if (a.chunks > RANK_INLINE) e = launch_pdl(compact_rank, dim3(a.chunks), dim3(PT), 0, s, a);
  if (e != cudaSuccess) return e;
  const PoolList l = pool_list(num_pools, pools);
  const int64_t copies = (int64_t)t.num_blocks * l.n * l.seg_max;  // at least the moves'
  return launch_pdl(compact_apply, dim3(grid_for(copies > warps ? copies : warps, sms)), dim3(AT),
                    0, s, a, segs, l);
}

}  // namespace sv
