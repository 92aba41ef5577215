// evict.cu -- eviction from a paged cache by accumulated attention weight (spec_kv_evict).
//
// For a table row with n positions and a budget m < n, every KV head keeps the row's first f
// and last l positions and, of those between, the m - f - l of largest weight, ties going to
// the lowest position; in ascending order src[0] < src[1] < ... they become positions 0 .. m - 1
// of the row's pages, in every pool. Two kernels:
//   select  a CTA per (row of the call, KV head) finds the weight of the last position kept by
//           a radix select over order-preserving 32-bit keys (11, 11 and 10 bits, histograms
//           in shared memory), then writes src in one ordered pass. CTA 0 of a row also makes
//           the row's checks and leaves a verdict in the workspace.
//   move    after every verdict is in: each CTA takes a column slice (SLICE bytes) of one
//           pool's rows of one (row, KV head), or its weights, and gathers forwards in place:
//           src[k] >= k, so what a batch of destinations overwrites has been read by the
//           batches before it or by itself, whose loads end before its stores begin. Slices
//           never touch each other's bytes, so nothing else orders them. A batch is a chain of
//           dependent reads (src, table, data), so many narrow slices in flight pay.
// Select reads the weights (4 bytes a position) four times, from L2 after the first; move is
// bound by memory. Measured: 32 rows of 16384 positions to 4096, 4 heads of 128 bytes, two pools:
// select 17 us, move 46 us for 277 MB (6.0 TB/s).
#include "internal.cuh"

namespace sv {
namespace {

constexpr int ST = 1024;        // threads of select
constexpr int BINS = 2048;
constexpr int MTH = 256;        // threads of move
// Bytes of a column slice, and pieces of 32 of a thread in flight. (32 rows of 16384 positions cut
// to 4096, 4 heads of 128 bytes, two pools, with the copy of the weights: 73 us; slices of 32 and
// 128 bytes 89 and 90; 1, 3, 4 and 8 pieces 88, 74, 76 and 95; 128 and 512 threads 100 and 85;
// pieces of 16 bytes 82.)
constexpr int SLICE = 64, MOVES = 2;

struct EvictArgs {
  sv_page_table t;
  int n, Hkv, bs_log2;
  const int32_t *rows, *new_len, *keep_first;
  int keep_last;
  float* mass;
  int64_t mass_stride;
  int32_t* kept;        // [n, Hkv, kept_stride]: src, the caller's or the workspace's
  int64_t kept_stride;
  int32_t* verdict;     // [n] 1: the row's checks hold
  uint32_t* flags;
  int num_pools, slices;  // slices of a (row, head): the pools' and one for the weights
};
struct EvictPools {
  int n;
  sv_page_data p[SV_MAX_PAGE_POOLS];
};

// Larger weight, larger key; NaN below everything, -0 as +0.
__device__ __forceinline__ uint32_t key_of(float w) {
  if (w != w) return 0;
  const uint32_t b = __float_as_uint(w + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ int row_at(const EvictArgs& a, int i) { return a.rows ? a.rows[i] : i; }

struct RowPlan {
  int r, n, m, first, mid;  // table row, positions, budget, kept first, candidates: [first, mid)
};
__device__ __forceinline__ RowPlan plan_of(const EvictArgs& a, int i, int r) {
  RowPlan p;
  p.r = r;
  p.n = a.t.cached_len[r];
  p.m = a.new_len[i];
  p.first = a.keep_first ? a.keep_first[i] : 0;
  p.mid = p.n - a.keep_last;
  return p;
}

// The row's checks, by one CTA's threads together.
__device__ bool row_good(const EvictArgs& a, int i) {
  const int r = row_at(a, i);
  bool bad = r < 0 || r >= a.t.table_rows;
  if (!bad) {
    if (a.rows)
      for (int k = threadIdx.x; k < i; k += ST) bad |= a.rows[k] == r;  // the same row twice
    const RowPlan p = plan_of(a, i, r);
    const int64_t cap = (int64_t)a.t.max_blocks_per_seq << a.bs_log2;
    bool lens = p.n >= 0 && p.n <= cap && p.n <= a.mass_stride && p.m >= 0 && p.m <= p.n;
    if (lens && p.m < p.n)
      lens = p.m <= a.kept_stride && p.first >= 0 && (int64_t)p.first + a.keep_last <= p.m;
    if (!lens) {
      bad = true;
    } else if (p.m < p.n) {
      // pages in use name pages of the pool; those that are written are no other row's
      const int last = (p.n - 1) >> a.bs_log2;
      for (int j = threadIdx.x; j <= last; j += ST) {
        const int e = a.t.block_table[(int64_t)r * a.t.max_blocks_per_seq + j];
        if (e < 0 || e >= a.t.num_blocks) bad = true;
        else if (((int64_t)j << a.bs_log2) < p.m && ((int64_t)(j + 1) << a.bs_log2) > p.first &&
                 a.t.ref_count[e] != 1)
          bad = true;
      }
    } else if (p.m > a.kept_stride) {
      bad = true;
    }
  }
  return !__syncthreads_or(bad);
}

// Exclusive scan over the block of one 32-bit value a thread.
__device__ uint32_t scan_st(uint32_t v, uint32_t& total) {
  __shared__ uint32_t s_warp[ST / 32];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[wid] = x;
  __syncthreads();
  uint32_t w = s_warp[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const uint32_t before = wid > 0 ? __shfl_sync(0xffffffffu, w, wid - 1) : 0;
  __syncthreads();
  return x - v + before;
}

__global__ void __launch_bounds__(ST) select_kernel(const EvictArgs a) {
  __shared__ uint32_t s_hist[BINS];
  __shared__ uint32_t s_digit, s_above;
  const int i = blockIdx.x / a.Hkv, g = blockIdx.x % a.Hkv, tid = threadIdx.x;
  pdl_trigger();
  pdl_wait();
  const int r = row_at(a, i);
  if (g == 0) {
    const bool good = row_good(a, i);
    if (tid == 0) a.verdict[i] = good;
    if (!good) {
      if (tid == 0) atomicOr(a.flags, FLAG_PAGES_SHAPE);
      return;
    }
  }
  if (r < 0 || r >= a.t.table_rows) return;
  const RowPlan p = plan_of(a, i, r);
  // (the other heads' CTAs go by what their own accesses need)
  if (p.n < 0 || p.n > a.mass_stride || p.m < 0 || p.m > p.n || p.m > a.kept_stride) return;
  int32_t* src = a.kept + ((int64_t)i * a.Hkv + g) * a.kept_stride;
  if (p.m == p.n) {
    for (int k = tid; k < p.m; k += ST) src[k] = k;
    return;
  }
  if (p.first < 0 || (int64_t)p.first + a.keep_last > p.m) return;
  const float* w = a.mass + ((int64_t)r * a.Hkv + g) * a.mass_stride;
  int want = p.m - p.first - a.keep_last;  // of the candidates [first, mid), >= 0 and < mid - first
  // the key of the want-th largest candidate, digit by digit
  uint32_t prefix = 0, known = 0;
  int left = want;
  if (want > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t mask = pass == 2 ? 1023u : 2047u;
      for (int x = tid; x < BINS; x += ST) s_hist[x] = 0;
      __syncthreads();
      for (int j0 = p.first + tid; j0 < p.mid; j0 += 8 * ST) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = j0 + e * ST < p.mid ? w[j0 + e * ST] : 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t k = key_of(x[e]);
          if (j0 + e * ST < p.mid && (k & known) == prefix) atomicAdd(&s_hist[(k >> shift) & mask], 1u);
        }
      }
      __syncthreads();
      // thread x has bins 2 x and 2 x + 1 counted from the top
      const uint32_t h0 = s_hist[BINS - 1 - 2 * tid], h1 = s_hist[BINS - 2 - 2 * tid];
      uint32_t total;
      const uint32_t above = scan_st(h0 + h1, total);
      if (above < (uint32_t)left && above + h0 >= (uint32_t)left) {
        s_digit = BINS - 1 - 2 * tid;
        s_above = above;
      } else if (above + h0 < (uint32_t)left && above + h0 + h1 >= (uint32_t)left) {
        s_digit = BINS - 2 - 2 * tid;
        s_above = above + h0;
      }
      __syncthreads();
      prefix |= s_digit << shift;
      known |= mask << shift;
      left -= (int)s_above;
      __syncthreads();
    }
  }
  // ---- in order: larger keys, and the first `left` of the equal ones
  for (int k = tid; k < p.first; k += ST) src[k] = k;
  uint32_t n_above = 0, n_equal = 0;  // before the chunk
  for (int base = p.first; base < p.mid && want > 0; base += 4 * ST) {
    uint32_t cls[4], mine = 0;  // (above, equal) counts packed in 16 bits each
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = base + 4 * tid + e;
      cls[e] = 0;
      if (j < p.mid) {
        const uint32_t k = key_of(w[j]);
        cls[e] = k > prefix ? 1u : k == prefix ? 0x10000u : 0u;
      }
      mine += cls[e];
    }
    uint32_t total;
    uint32_t before = scan_st(mine, total);
    uint32_t up = n_above + (before & 0xffffu), eq = n_equal + (before >> 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool keep = cls[e] == 1u || (cls[e] != 0 && eq < (uint32_t)left);
      if (keep) src[p.first + up + min(eq, (uint32_t)left)] = base + 4 * tid + e;
      up += cls[e] & 0xffffu;
      eq += cls[e] >> 16;
    }
    n_above += total & 0xffffu;
    n_equal += total >> 16;
  }
  for (int k = tid; k < a.keep_last; k += ST) src[p.m - a.keep_last + k] = p.mid + k;
}

template <int V>
struct VecOf;
template <>
struct VecOf<16> {
  using type = uint4;
};
template <>
struct VecOf<8> {
  using type = uint2;
};
struct Vec32 {
  uint4 x[2];
};
template <>
struct VecOf<32> {
  using type = Vec32;
};
template <class T>
__device__ __forceinline__ void load_piece(const uint8_t* p, T& v) {
  v = *reinterpret_cast<const T*>(p);
}
template <class T>
__device__ __forceinline__ void store_piece(uint8_t* p, const T& v) {
  *reinterpret_cast<T*>(p) = v;
}
__device__ __forceinline__ void load_piece(const uint8_t* p, Vec32& v) {  // (a whole sector at once)
  uint4 &a = v.x[0], &b = v.x[1];
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void store_piece(uint8_t* p, const Vec32& v) {
  const uint4 &a = v.x[0], &b = v.x[1];
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
               "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// One slice: `cols` pieces of V bytes at `base`, positions `pos_bytes` apart in a page, through
// the table's row. The next batch's places (src, then the table) are looked up while this one's
// data is on its way.
template <int V>
__device__ __forceinline__ void move_slice(const EvictArgs& a, const RowPlan& p, const int32_t* src,
                                           uint8_t* base, int64_t pos_bytes, int cols) {
  using T = typename VecOf<V>::type;
  constexpr int U = MOVES;
  const int32_t* tab = a.t.block_table + (int64_t)p.r * a.t.max_blocks_per_seq;
  const int per = MTH / cols;  // destinations of an unroll step
  const int lr = threadIdx.x / cols, lc = threadIdx.x % cols;
  base += lc * V;
  auto row_of = [&](int pos) { return (tab[pos >> a.bs_log2] << a.bs_log2) + (pos & ((1 << a.bs_log2) - 1)); };
  int from[U], to[U];  // cache rows; from -1: nothing to move
  auto look = [&](int k0) {
#pragma unroll
    for (int e = 0; e < U; ++e) {
      const int k = k0 + e * per + lr;
      from[e] = lr < per && k < p.m ? src[k] : -1;
    }
#pragma unroll
    for (int e = 0; e < U; ++e) {
      const int k = k0 + e * per + lr;
      if (from[e] == k) from[e] = -1;  // stays where it is
      to[e] = from[e] >= 0 ? row_of(k) : 0;
      if (from[e] >= 0) from[e] = row_of(from[e]);
    }
  };
  look(p.first);
  for (int k0 = p.first; k0 < p.m; k0 += per * U) {
    T v[U];
    int dst[U];
#pragma unroll
    for (int e = 0; e < U; ++e) {
      dst[e] = from[e] >= 0 ? to[e] : -1;
      if (from[e] >= 0) load_piece(base + from[e] * pos_bytes, v[e]);
    }
    look(k0 + per * U);
    __syncthreads();  // the batch is read
#pragma unroll
    for (int e = 0; e < U; ++e)
      if (dst[e] >= 0) store_piece(base + dst[e] * pos_bytes, v[e]);
  }
}

__device__ void move_mass(const EvictArgs& a, const RowPlan& p, const int32_t* src, float* w) {
  constexpr int U = 8;
  for (int k0 = p.first; k0 < p.m; k0 += MTH * U) {
    float v[U];
#pragma unroll
    for (int e = 0; e < U; ++e) {
      const int k = k0 + e * MTH + threadIdx.x;
      if (k < p.m) v[e] = w[src[k]];
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < U; ++e) {
      const int k = k0 + e * MTH + threadIdx.x;
      if (k < p.m) w[k] = v[e];
    }
  }
  __syncthreads();
  for (int k = p.m + threadIdx.x; k < p.n; k += MTH) w[k] = 0.f;
}

__global__ void __launch_bounds__(MTH) move_kernel(const EvictArgs a, const __grid_constant__ EvictPools pools) {
  pdl_trigger();
  pdl_wait();
  bool bad = false;
  for (int i = threadIdx.x; i < a.n; i += MTH) bad |= __ldcg(a.verdict + i) == 0;
  if (__syncthreads_or(bad)) return;
  int s = blockIdx.x % a.slices;
  const int e = blockIdx.x / a.slices, g = e % a.Hkv, i = e / a.Hkv;
  const RowPlan p = plan_of(a, i, row_at(a, i));
  if (p.m == p.n) return;
  const int32_t* src = a.kept + (int64_t)e * a.kept_stride;
  if (s == 0) {
    move_mass(a, p, src, a.mass + ((int64_t)p.r * a.Hkv + g) * a.mass_stride);
    return;
  }
  --s;
  for (int k = 0; k < pools.n; ++k) {
    const int64_t pos_bytes = pools.p[k].page_bytes >> a.bs_log2, row_bytes = pos_bytes / a.Hkv;
    const int n = (int)((row_bytes + SLICE - 1) / SLICE);
    if (s < n) {
      uint8_t* base = (uint8_t*)pools.p[k].base + g * row_bytes + s * SLICE;
      const int bytes = (int)min((int64_t)SLICE, row_bytes - s * SLICE);
      if (((uintptr_t)pools.p[k].base | row_bytes | bytes) % 32 == 0)
        move_slice<32>(a, p, src, base, pos_bytes, bytes / 32);
      else if (bytes % 16 == 0 && row_bytes % 16 == 0)
        move_slice<16>(a, p, src, base, pos_bytes, bytes / 16);
      else
        move_slice<8>(a, p, src, base, pos_bytes, bytes / 8);
      return;
    }
    s -= n;
  }
}

}  // namespace

size_t evict_ws_bytes(int n, int Hkv, int64_t max_positions) {
  return 256 + align_up(4 * (size_t)n, 256) + 4 * (size_t)n * Hkv * max_positions;
}

cudaError_t launch_evict(const sv_page_table& t, int n, const int32_t* rows, const int32_t* new_len,
                         const int32_t* keep_first, int keep_last, int Hkv, float* mass,
                         int64_t mass_stride, int32_t* kept, int64_t kept_stride, int num_pools,
                         const sv_page_data* pools, void* ws, cudaStream_t s) {
  EvictArgs a = {};
  a.t = t;
  a.n = n;
  a.Hkv = Hkv;
  while ((1 << a.bs_log2) < t.block_size) ++a.bs_log2;
  a.rows = rows;
  a.new_len = new_len;
  a.keep_first = keep_first;
  a.keep_last = keep_last;
  a.mass = mass;
  a.mass_stride = mass_stride;
  a.flags = (uint32_t*)ws;
  a.verdict = (int32_t*)((uint8_t*)ws + 256);
  a.kept = kept ? kept : (int32_t*)((uint8_t*)ws + 256 + align_up(4 * (size_t)n, 256));
  a.kept_stride = kept ? kept_stride : mass_stride;
  EvictPools pl;
  pl.n = num_pools;
  a.slices = 1;
  for (int k = 0; k < num_pools; ++k) {
    pl.p[k] = pools[k];
    a.slices += (int)((pools[k].page_bytes / t.block_size / Hkv + SLICE - 1) / SLICE);
  }
  const cudaError_t e = launch_pdl(select_kernel, dim3((unsigned)(n * Hkv)), dim3(ST), 0, s, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(move_kernel, dim3((unsigned)((int64_t)n * Hkv * a.slices)), dim3(MTH), 0, s, a, pl);
}

}  // namespace sv
