// kv4.cu -- rows of a 4-bit paged cache: bf16 rows rounded into the pages, and read back.
//
// For a block x of 16 elements of a row and the head's scale s (format: kv4.cuh)
//   c = E4M3(max |x| / (6 s)),  code_k = E2M1(x_k / (s c))  (0 where c = 0),
// each the nearest value of its type to the REAL quotient, ties to the even code, saturating.
// The quotients are formed in fp32 as products with a reciprocal, whose error is below 2^-21
// of them (the reciprocal's 2^-23 and three roundings of 2^-24): the product is formed twice,
// a little smaller and a little larger (2^-20), and where the two codes differ, about one
// block in 2^12, the choice is made in 64 bits, where x and the middle of
// two codes times s c are exact (8 and 31 significant bits). So the codes do not depend on
// how the quotient is computed, and a reference in 64 bits gives the same.
// A block with an infinity or a NaN gets the scale NaN: it reads as NaN, all 16 elements. A head
// scale of 0, which a head of zeros gets from its largest magnitude, makes other blocks zeros.
//
// Both calls move bytes and nothing else bounds them: a thread takes a block (32 bytes of bf16,
// 8 bytes of codes, a scale). The scan that finds each row's sequence and position runs in
// every CTA (counts of a batch are a few KB in L2) while a write's loads are in flight.
//
// Measured: 197 thousand rows of 8 heads, d 128, read back in 157 us (1.03 GB, 6.6 TB/s: 0.97 of a
// copy; 191 us with two stores of 16 bytes); 49 thousand written and read back in 108 us (133;
// 117 with 3 CTAs of the write on an SM), where the write is bound by issue: two products, two
// conversions and a comparison for each element.
#include <cuda_bf16.h>

#include "kv4.cuh"

namespace sv {
namespace {

constexpr int NTH = 256;

struct Kv4Args {
  uint8_t *kc, *vc, *sc;    // [num_blocks * block_size, Hkv, d / 2] twice, [.., Hkv, 2, d / 16]
  const float* head_scale;  // [2, Hkv]
  int64_t num_blocks;
  int bs_log2, Hkv, d;
  int B, max_blocks;
  const int32_t *table, *start, *count;
  int64_t rows;             // rows of the packed arrays
  const uint16_t *k, *v;    // write: bf16 [rows, Hkv, d], rows k_stride elements apart
  int64_t k_stride, v_stride;
  uint16_t *k_out, *v_out;  // read
  uint32_t* flags;
  int row_items;            // blocks of a row: 2 (K, V) x Hkv x d / 16
  int cta_rows;
  int lanes, rows_at_once;  // threads of a row, and rows that the CTA's threads take at once
};

constexpr int MAX_CTA_ROWS = 64;

// The cache row of each packed row [r0, r0 + a.cta_rows) in s_row: -1 for rows past the
// sequences' total, -2 where the table names no page of the pool. False, with the flag set,
// if a start or count of the call is out of range or the total beyond the arrays.
__device__ bool locate(const Kv4Args& a, int64_t r0, int64_t* s_row) {
  __shared__ int64_t s_warp[NTH / 32];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  if (tid < a.cta_rows) s_row[tid] = -1;
  __syncthreads();
  int64_t carry = 0;
  bool bad = false;
  for (int base = 0; base < a.B; base += NTH) {
    const int b = base + tid;
    int64_t st = 0, n = 0;
    if (b < a.B) {
      st = a.start[b];
      n = a.count[b];
      if (st < 0 || n < 0 || st + n > ((int64_t)a.max_blocks << a.bs_log2)) {
        bad = true;
        n = 0;
      }
    }
    int64_t x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[wid] = x;
    __syncthreads();
    int64_t before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < NTH / 32; ++w) {
      before += w < wid ? s_warp[w] : 0;
      total += s_warp[w];
    }
    const int64_t off = carry + before + x - n;  // the sequence's first packed row
    const int64_t lo = off > r0 ? off : r0, hi = min(off + n, r0 + a.cta_rows);
    for (int64_t r = lo; r < hi; ++r) {
      const int64_t pos = st + (r - off);
      const int blk = a.table[(int64_t)b * a.max_blocks + (pos >> a.bs_log2)];
      const bool ok = blk >= 0 && blk < a.num_blocks;
      if (!ok) atomicOr(a.flags, FLAG_ATTN_SHAPE);
      s_row[r - r0] = ok ? ((int64_t)blk << a.bs_log2) + (pos & ((1 << a.bs_log2) - 1)) : -2;
    }
    carry += total;
    __syncthreads();  // s_warp is reused
  }
  if (__syncthreads_or(bad || carry > a.rows)) {
    if (tid == 0) atomicOr(a.flags, FLAG_ATTN_SHAPE);
    return false;
  }
  return true;
}

// Block `blk` of head h of K (which 0) or V (1): a thread's place in a row, for every row that
// it takes.
struct Item {
  int which, h, blk;
};
__device__ __forceinline__ Item item_of(const Kv4Args& a, int i) {  // item i of a row
  const int nb = a.d >> 4;  // 4 or 8
  Item t;
  t.blk = i & (nb - 1);
  const int e = i / nb;  // which, head
  t.which = e >= a.Hkv;
  t.h = e - (t.which ? a.Hkv : 0);
  return t;
}

__device__ __forceinline__ uint32_t to_e4m3(float x) {  // one value, in the low byte
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xffu;
}
__device__ __forceinline__ float e4m3_value(uint32_t c) {
  const uint32_t h = e4m3x2_to_f16x2(c);
  return __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
}
__device__ __forceinline__ double e2m1_magnitude(uint32_t c) {  // of its low 3 bits
  c &= 7;
  return c < 5 ? 0.5 * c : c == 5 ? 3.0 : c == 6 ? 4.0 : 6.0;
}

// Whether the real quotient a / unit lies above the middle of lower and upper neighbour, or
// on it with the upper code even: a takes the upper code. All in exact products.
__device__ __forceinline__ bool takes_upper(double a, double unit, double lower, double upper,
                                            uint32_t upper_code) {
  const double mid = 0.5 * (lower + upper) * unit;
  return a > mid || (a == mid && (upper_code & 1) == 0);
}

constexpr float LESS = 1.f - 0x1p-20f, MORE = 1.f + 0x1p-20f;

__device__ __forceinline__ float reciprocal(float x) {  // to 2^-23
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// (a, b) * (s, s)
__device__ __forceinline__ float2 mul2(float a, float b, float s) {
  float2 r;
  asm("{\n .reg .b64 v, w;\n mov.b64 v, {%2, %3};\n mov.b64 w, {%4, %4};\n mul.rn.f32x2 v, v, w;\n"
      " mov.b64 {%0, %1}, v;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a), "f"(b), "f"(s));
  return r;
}
// Eight values -> eight E2M1 codes, the first in the lowest nibble; nearest even, saturating.
__device__ __forceinline__ uint32_t to_e2m1x8(const float2 (&y)[4]) {
  uint32_t r;
  asm("{\n .reg .b8 a, b, c, d;\n cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(r)
      : "f"(y[0].x), "f"(y[0].y), "f"(y[1].x), "f"(y[1].y), "f"(y[2].x), "f"(y[2].y), "f"(y[3].x), "f"(y[3].y));
  return r;
}

__device__ __noinline__ uint32_t scale_code_exact(float amax, float head, uint32_t lo, uint32_t hi) {
  return takes_upper(amax, 6.0 * (double)head, e4m3_value(lo), e4m3_value(hi), hi) ? hi : lo;
}
// Eight codes again, in 64 bits where the two candidate words differ.
__device__ __noinline__ uint32_t codes_exact(const uint4 v, double unit, uint32_t lo, uint32_t hi) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t out = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t a = (lo >> (4 * e)) & 15u, b = (hi >> (4 * e)) & 15u;
    const uint32_t bits = e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16;
    const double x = fabs((double)__uint_as_float(bits));
    const bool up = a != b && takes_upper(x, unit, e2m1_magnitude(a), e2m1_magnitude(b), b);
    out |= (up ? b : a) << (4 * e);
  }
  return out;
}

// 8 elements -> 8 codes; less and more: the reciprocal of the unit a little smaller and larger.
__device__ __forceinline__ uint32_t encode8(const uint4 v, float less, float more, float head, float c) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float2 lo[4], hi[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float x0 = __uint_as_float(w[e] << 16), x1 = __uint_as_float(w[e] & 0xffff0000u);
    lo[e] = mul2(x0, x1, less);
    hi[e] = mul2(x0, x1, more);
  }
  const uint32_t a = to_e2m1x8(lo), b = to_e2m1x8(hi);
  return a == b ? a : codes_exact(v, (double)head * (double)c, a, b);
}

__device__ __forceinline__ uint32_t abs_max2(uint32_t a, uint32_t b) {  // of bf16 pairs, NaN kept
  const __nv_bfloat162 x = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&a));
  const __nv_bfloat162 y = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&b));
  const __nv_bfloat162 m = __hmax2_nan(x, y);
  return *reinterpret_cast<const uint32_t*>(&m);
}

// 32 bytes of a thread, in one access where they are aligned (W32), so that no 32-byte sector is
// touched twice. Volatile and with a clobber: what it reads the grid before may have written, so
// the compiler must leave it behind pdl_wait.
template <bool W32>
__device__ __forceinline__ void load32(const void* p, uint4 (&x)[2]) {
  if constexpr (W32) {
    asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(x[0].x), "=r"(x[0].y), "=r"(x[0].z), "=r"(x[0].w), "=r"(x[1].x), "=r"(x[1].y), "=r"(x[1].z),
                   "=r"(x[1].w)
                 : "l"(p)
                 : "memory");
  } else {
    x[0] = *reinterpret_cast<const uint4*>(p);
    x[1] = *(reinterpret_cast<const uint4*>(p) + 1);
  }
}
template <bool W32>
__device__ __forceinline__ void store32(void* p, const uint32_t (&x)[8]) {
  if constexpr (W32) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]), "r"(x[1]), "r"(x[2]),
                 "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(x[4], x[5], x[6], x[7]);
  }
}

// N: rows of a thread whose loads run together.
template <int N, bool W32>
__global__ void __launch_bounds__(NTH, 4) kv4_write_kernel(const Kv4Args a) {
  __shared__ int64_t s_row[MAX_CTA_ROWS];
  const int64_t r0 = (int64_t)blockIdx.x * a.cta_rows;
  const int rows = (int)min((int64_t)a.cta_rows, a.rows - r0);
  const int lr = threadIdx.x / a.lanes, li = threadIdx.x - lr * a.lanes;
  pdl_trigger();
  pdl_wait();
  bool located = false;
  for (int i = li; i < a.row_items + li; i += a.lanes) {  // (one pass but for very many heads)
    const bool in = i < a.row_items && lr < a.rows_at_once;
    const Item t = item_of(a, in ? i : 0);
    const uint16_t* src = (t.which ? a.v : a.k) + t.h * a.d + t.blk * 16;
    const int64_t stride = t.which ? a.v_stride : a.k_stride;
    const float head = __ldg(a.head_scale + t.which * a.Hkv + t.h);
    const float inv6 = reciprocal(6.f * head);
    for (int rr = 0; rr < rows; rr += N * a.rows_at_once) {
      uint4 x[N][2];
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int r = rr + n * a.rows_at_once + lr;
        x[n][0] = x[n][1] = make_uint4(0, 0, 0, 0);
        if (in && r < rows) load32<W32>(src + (r0 + r) * stride, x[n]);
      }
      if (!located) {
        if (!locate(a, r0, s_row)) return;
        located = true;
      }
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int r = rr + n * a.rows_at_once + lr;
        const int64_t row = in && r < rows ? s_row[r] : -1;
        if (row < 0) continue;
        uint32_t m = abs_max2(abs_max2(abs_max2(x[n][0].x, x[n][0].y), abs_max2(x[n][0].z, x[n][0].w)),
                              abs_max2(abs_max2(x[n][1].x, x[n][1].y), abs_max2(x[n][1].z, x[n][1].w)));
        m = abs_max2(m, m >> 16) & 0xffffu;
        uint32_t c = 0;
        uint2 code = make_uint2(0, 0);
        if (m >= 0x7f80u) {  // an infinity or a NaN
          c = 0x7fu;
        } else if (m != 0 && head != 0.f) {  // (a head scale of 0 has no quotients)
          const float amax = __uint_as_float(m << 16);
          const float q = amax * inv6;
          const uint32_t lo = to_e4m3(q * LESS), hi = to_e4m3(q * MORE);
          c = lo == hi ? lo : scale_code_exact(amax, head, lo, hi);
          if (c != 0) {
            const float cv = e4m3_value(c);
            const float inv = reciprocal(head * cv);
            code.x = encode8(x[n][0], inv * LESS, inv * MORE, head, cv);
            code.y = encode8(x[n][1], inv * LESS, inv * MORE, head, cv);
          }
        }
        const int64_t at = row * a.Hkv + t.h;
        *reinterpret_cast<uint2*>((t.which ? a.vc : a.kc) + at * (a.d >> 1) + t.blk * 8) = code;
        a.sc[at * (a.d >> 3) + t.which * (a.d >> 4) + t.blk] = (uint8_t)c;
      }
    }
  }
}

template <int N, bool W32>
__global__ void __launch_bounds__(NTH) kv4_read_kernel(const Kv4Args a) {
  __shared__ int64_t s_row[MAX_CTA_ROWS];
  const int64_t r0 = (int64_t)blockIdx.x * a.cta_rows;
  const int rows = (int)min((int64_t)a.cta_rows, a.rows - r0);
  const int lr = threadIdx.x / a.lanes, li = threadIdx.x - lr * a.lanes;
  pdl_trigger();
  pdl_wait();
  if (!locate(a, r0, s_row)) return;
  if (lr >= a.rows_at_once) return;
  for (int i = li; i < a.row_items; i += a.lanes) {
    const Item t = item_of(a, i);
    const uint8_t* src = (t.which ? a.vc : a.kc) + (int64_t)t.h * (a.d >> 1) + t.blk * 8;
    const uint8_t* ssc = a.sc + (int64_t)t.h * (a.d >> 3) + t.which * (a.d >> 4) + t.blk;
    uint16_t* dst = (t.which ? a.v_out : a.k_out) + (r0 * a.Hkv + t.h) * a.d + t.blk * 16;
    const int code_bytes = a.Hkv * (a.d >> 1), scale_bytes = a.Hkv * (a.d >> 3), out_elems = a.Hkv * a.d;
    const float head = __ldg(a.head_scale + t.which * a.Hkv + t.h);
    for (int rr = lr; rr < rows; rr += N * a.rows_at_once) {
      uint2 code[N];
      uint32_t c[N];
      int64_t row[N];
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int r = rr + n * a.rows_at_once;
        row[n] = r < rows ? s_row[r] : -1;
        code[n] = make_uint2(0, 0);
        c[n] = 0;
        if (row[n] >= 0) {
          code[n] = __ldg(reinterpret_cast<const uint2*>(src + row[n] * code_bytes));
          c[n] = __ldg(ssc + row[n] * scale_bytes);
        }
      }
#pragma unroll
      for (int n = 0; n < N; ++n) {
        if (row[n] == -1) continue;  // past the sequences' total: left as it was
        const uint32_t u = lo_twice(e4m3x2_to_f16x2(c[n]));
        uint32_t out[8];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          uint32_t h[4];
          e2m1x8_to_f16(w ? code[n].y : code[n].x, h);
#pragma unroll
          for (int e = 0; e < 4; ++e) {  // exact in f16, then two roundings: to fp32, to bf16
            const uint32_t p = hmul2(h[e], u);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p));
            const float2 y = mul2(f.x, f.y, head);
            const __nv_bfloat162 o = __floats2bfloat162_rn(y.x, y.y);
            out[4 * w + e] = *reinterpret_cast<const uint32_t*>(&o);
          }
        }
        store32<W32>(dst + (int64_t)(rr + n * a.rows_at_once) * out_elems, out);
      }
    }
  }
}

template <class K1, class KN>
cudaError_t launch_rows(K1 one, KN some, int thread_rows, Kv4Args a, int sms, cudaStream_t s) {
  a.row_items = 2 * a.Hkv * (a.d / 16);
  a.lanes = a.row_items < NTH ? a.row_items : NTH;
  a.rows_at_once = NTH / a.lanes;
  // An item a thread while that leaves no SM with more than two CTAs; else `thread_rows`, some of
  // them at a time, so that the scan for the rows' places costs little next to them. (49 thousand
  // rows of 8 heads written and read back: 16 and 8 rows 108.5 us, 8 and 8 109.3, 8 and 16 110.9, 4
  // and 16 114.6.)
  const bool few = a.rows * a.row_items <= 2 * (int64_t)sms * NTH;
  const int want = few ? a.rows_at_once : thread_rows * a.rows_at_once;
  a.cta_rows = want > MAX_CTA_ROWS ? MAX_CTA_ROWS : want;
  const unsigned grid = (unsigned)((a.rows + a.cta_rows - 1) / a.cta_rows);
  return launch_pdl(few ? one : some, dim3(grid), dim3(NTH), 0, s, a);
}

// Whether rows of bf16, `stride` elements apart, begin on 32 bytes.
bool aligned32(const void* p, int64_t stride) { return ((uintptr_t)p & 31) == 0 && stride % 16 == 0; }

Kv4Args args_of(const sv_kv4_pages& p, int B, const int32_t* table, int max_blocks,
                const int32_t* start, const int32_t* count, int64_t rows, void* ws) {
  Kv4Args a = {};
  a.kc = (uint8_t*)p.k_codes;
  a.vc = (uint8_t*)p.v_codes;
  a.sc = (uint8_t*)p.scales;
  a.head_scale = p.kv_scale;
  a.num_blocks = p.num_blocks;
  while ((1 << a.bs_log2) < p.block_size) ++a.bs_log2;
  a.Hkv = p.num_kv_heads;
  a.d = p.head_dim;
  a.B = B;
  a.max_blocks = max_blocks;
  a.table = table;
  a.start = start;
  a.count = count;
  a.rows = rows;
  a.flags = (uint32_t*)ws;
  return a;
}

}  // namespace

cudaError_t launch_kv4_write(const sv_kv4_pages& p, int B, const int32_t* table, int max_blocks,
                             const int32_t* start, const int32_t* count, int64_t rows,
                             const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                             void* ws, int sms, cudaStream_t s) {
  Kv4Args a = args_of(p, B, table, max_blocks, start, count, rows, ws);
  a.k = (const uint16_t*)k;
  a.v = (const uint16_t*)v;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  if (aligned32(k, k_stride) && aligned32(v, v_stride))
    return launch_rows(kv4_write_kernel<1, true>, kv4_write_kernel<2, true>, 16, a, sms, s);
  return launch_rows(kv4_write_kernel<1, false>, kv4_write_kernel<2, false>, 16, a, sms, s);
}

cudaError_t launch_kv4_read(const sv_kv4_pages& p, int B, const int32_t* table, int max_blocks,
                            const int32_t* start, const int32_t* count, int64_t rows, void* k_out,
                            void* v_out, void* ws, int sms, cudaStream_t s) {
  Kv4Args a = args_of(p, B, table, max_blocks, start, count, rows, ws);
  a.k_out = (uint16_t*)k_out;
  a.v_out = (uint16_t*)v_out;
  if (aligned32(k_out, 16) && aligned32(v_out, 16))
    return launch_rows(kv4_read_kernel<1, true>, kv4_read_kernel<4, true>, 8, a, sms, s);
  return launch_rows(kv4_read_kernel<1, false>, kv4_read_kernel<4, false>, 8, a, sms, s);
}

}  // namespace sv
