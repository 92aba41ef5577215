// kv4.cu -- rows of a 4-bit paged cache: bf16 rows rounded into the pages, and read back.
//
// For a block x of 16 elements of a row and the head's scale s (format: kv4.cuh)
//   c = E4M3(max |x| / (6 s)),  code_k = E2M1(x_k / (s c))  (0 where c = 0),
// each the nearest value of its type to the REAL quotient, ties to the even code, saturating.
// The quotients are formed in fp32 as products with a reciprocal, whose error is below 2^-22
// of them (three roundings of 2^-24, and less than one more for the division): the product is
// converted twice, a little smaller and a little larger (2^-21), and where the two codes
// differ, about one block in 2^13, the choice is made in 64 bits, where x and the middle of
// two codes times s c are exact (8 and 31 significant bits). So the codes do not depend on
// how the quotient is computed, and a reference in 64 bits gives the same.
// A block with an infinity or a NaN gets the scale NaN: it reads as NaN, all 16 elements.
//
// Both calls move bytes and nothing else bounds them: a thread takes a block (32 bytes of bf16,
// 8 bytes of codes, a scale). The scan that finds each row's sequence and position runs in
// every CTA (counts of a batch are a few KB in L2) while a write's loads are in flight.
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
};

constexpr int MAX_CTA_ROWS = 32;

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

// A CTA's item i: block `blk` of head h of K (which 0) or V (1) of its row r.
struct Item {
  int r, which, h, blk;
};
__device__ __forceinline__ Item item_of(const Kv4Args& a, int i) {
  const int nb = a.d >> 4;  // 4 or 8
  Item t;
  t.blk = i & (nb - 1);
  const int e = i / nb;  // (row, which, head)
  const int w = e / a.Hkv;
  t.h = e - w * a.Hkv;
  t.which = w & 1;
  t.r = w >> 1;
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
// Two values -> a byte of two E2M1 codes, the first in the low nibble; nearest even, saturating.
__device__ __forceinline__ uint32_t to_e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n .reg .b8 b;\n cvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n mov.b32 %0, {b, b, b, b};\n}\n"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r & 0xffu;
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

constexpr float LESS = 1.f - 0x1p-21f, MORE = 1.f + 0x1p-21f;

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

// 8 elements -> 8 codes.
__device__ __forceinline__ uint32_t encode8(const uint4 v, float inv, double unit) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t lo = 0, hi = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float y0 = __uint_as_float(w[e] << 16) * inv;
    const float y1 = __uint_as_float(w[e] & 0xffff0000u) * inv;
    lo |= to_e2m1x2(y0 * LESS, y1 * LESS) << (8 * e);
    hi |= to_e2m1x2(y0 * MORE, y1 * MORE) << (8 * e);
  }
  return lo == hi ? lo : codes_exact(v, unit, lo, hi);
}

__device__ __forceinline__ uint32_t abs_max2(uint32_t a, uint32_t b) {  // of bf16 pairs, NaN kept
  const __nv_bfloat162 x = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&a));
  const __nv_bfloat162 y = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&b));
  const __nv_bfloat162 m = __hmax2_nan(x, y);
  return *reinterpret_cast<const uint32_t*>(&m);
}

// N: items of a thread whose loads run together.
template <int N>
__global__ void __launch_bounds__(NTH) kv4_write_kernel(const Kv4Args a) {
  __shared__ int64_t s_row[MAX_CTA_ROWS];
  const int64_t r0 = (int64_t)blockIdx.x * a.cta_rows;
  const int items = (int)min((int64_t)a.cta_rows, a.rows - r0) * a.row_items;
  pdl_trigger();
  pdl_wait();
  bool located = false;
  for (int i0 = threadIdx.x; i0 < items + (int)threadIdx.x; i0 += N * NTH) {
    uint4 x[N][2];
    float head[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      x[n][0] = x[n][1] = make_uint4(0, 0, 0, 0);
      head[n] = 1.f;
      if (i0 + n * NTH < items) {
        const Item t = item_of(a, i0 + n * NTH);
        const uint16_t* src = t.which ? a.v + (r0 + t.r) * a.v_stride : a.k + (r0 + t.r) * a.k_stride;
        const uint4* s4 = reinterpret_cast<const uint4*>(src + t.h * a.d + t.blk * 16);
        x[n][0] = __ldg(s4);
        x[n][1] = __ldg(s4 + 1);
        head[n] = __ldg(a.head_scale + t.which * a.Hkv + t.h);
      }
    }
    if (!located) {
      if (!locate(a, r0, s_row)) return;
      located = true;
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      if (i0 + n * NTH >= items) continue;
      const Item t = item_of(a, i0 + n * NTH);
      const int64_t row = s_row[t.r];
      if (row < 0) continue;
      uint32_t m = abs_max2(abs_max2(abs_max2(x[n][0].x, x[n][0].y), abs_max2(x[n][0].z, x[n][0].w)),
                            abs_max2(abs_max2(x[n][1].x, x[n][1].y), abs_max2(x[n][1].z, x[n][1].w)));
      m = abs_max2(m, m >> 16) & 0xffffu;
      uint32_t c;
      uint2 code = make_uint2(0, 0);
      if (m >= 0x7f80u) {  // an infinity or a NaN
        c = 0x7fu;
      } else {
        const float amax = __uint_as_float(m << 16);
        const float q = amax * (1.f / (6.f * head[n]));
        const uint32_t lo = to_e4m3(q * LESS), hi = to_e4m3(q * MORE);
        c = lo == hi ? lo : scale_code_exact(amax, head[n], lo, hi);
        if (c != 0) {
          const float cv = e4m3_value(c);
          const float inv = 1.f / (head[n] * cv);
          const double unit = (double)head[n] * (double)cv;
          code.x = encode8(x[n][0], inv, unit);
          code.y = encode8(x[n][1], inv, unit);
        }
      }
      const int64_t at = row * a.Hkv + t.h;
      uint8_t* dst = (t.which ? a.vc : a.kc) + at * (a.d >> 1) + t.blk * 8;
      *reinterpret_cast<uint2*>(dst) = code;
      a.sc[at * (a.d >> 3) + t.which * (a.d >> 4) + t.blk] = (uint8_t)c;
    }
  }
}

template <int N>
__global__ void __launch_bounds__(NTH) kv4_read_kernel(const Kv4Args a) {
  __shared__ int64_t s_row[MAX_CTA_ROWS];
  const int64_t r0 = (int64_t)blockIdx.x * a.cta_rows;
  const int items = (int)min((int64_t)a.cta_rows, a.rows - r0) * a.row_items;
  pdl_trigger();
  pdl_wait();
  if (!locate(a, r0, s_row)) return;
  for (int i0 = threadIdx.x; i0 < items; i0 += N * NTH) {
    uint2 code[N];
    uint32_t c[N];
    float head[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      code[n] = make_uint2(0, 0);
      c[n] = 0;
      head[n] = 0.f;
      if (i0 + n * NTH < items) {
        const Item t = item_of(a, i0 + n * NTH);
        const int64_t row = s_row[t.r];
        if (row >= 0) {
          const int64_t at = row * a.Hkv + t.h;
          code[n] = __ldg(reinterpret_cast<const uint2*>((t.which ? a.vc : a.kc) + at * (a.d >> 1)) + t.blk);
          c[n] = __ldg(a.sc + at * (a.d >> 3) + t.which * (a.d >> 4) + t.blk);
          head[n] = __ldg(a.head_scale + t.which * a.Hkv + t.h);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      if (i0 + n * NTH >= items) continue;
      const Item t = item_of(a, i0 + n * NTH);
      if (s_row[t.r] == -1) continue;  // past the sequences' total: left as it was
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
          const __nv_bfloat162 o = __floats2bfloat162_rn(f.x * head[n], f.y * head[n]);
          out[4 * w + e] = *reinterpret_cast<const uint32_t*>(&o);
        }
      }
      uint16_t* dst = (t.which ? a.v_out : a.k_out) + ((r0 + t.r) * a.Hkv + t.h) * a.d + t.blk * 16;
      uint4* d4 = reinterpret_cast<uint4*>(dst);
      d4[0] = make_uint4(out[0], out[1], out[2], out[3]);
      d4[1] = make_uint4(out[4], out[5], out[6], out[7]);
    }
  }
}

template <class K1, class K4>
cudaError_t launch_rows(K1 one, K4 four, Kv4Args a, int sms, cudaStream_t s) {
  a.row_items = 2 * a.Hkv * (a.d / 16);
  // rows of a CTA: an item a thread while that leaves no SM with more than a CTA, else four
  const bool few = a.rows * a.row_items <= (int64_t)sms * NTH;
  const int want = (few ? 1 : 4) * NTH / a.row_items;
  a.cta_rows = want < 1 ? 1 : want > MAX_CTA_ROWS ? MAX_CTA_ROWS : want;
  const unsigned grid = (unsigned)((a.rows + a.cta_rows - 1) / a.cta_rows);
  return launch_pdl(few ? one : four, dim3(grid), dim3(NTH), 0, s, a);
}

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
  return launch_rows(kv4_write_kernel<1>, kv4_write_kernel<4>, a, sms, s);
}

cudaError_t launch_kv4_read(const sv_kv4_pages& p, int B, const int32_t* table, int max_blocks,
                            const int32_t* start, const int32_t* count, int64_t rows, void* k_out,
                            void* v_out, void* ws, int sms, cudaStream_t s) {
  Kv4Args a = args_of(p, B, table, max_blocks, start, count, rows, ws);
  a.k_out = (uint16_t*)k_out;
  a.v_out = (uint16_t*)v_out;
  return launch_rows(kv4_read_kernel<1>, kv4_read_kernel<4>, a, sms, s);
}

}  // namespace sv
