// api.cu -- the C ABI of libspecverify: argument checks, workspace layout, launches.
// Every entry point is declared and documented in include/specverify.h.
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <initializer_list>

#include "internal.cuh"

using namespace sv;

namespace {

#ifndef SV_SWITCH_F8
#define SV_SWITCH_F8 9
#endif
#ifndef SV_SWITCH_BF16
#define SV_SWITCH_BF16 5
#endif
// Virtual tiles charged for starting a unit (see internal.cuh), per attention kernel.
constexpr int SWITCH_TILES_TC_FP8 = SV_SWITCH_F8;
constexpr int SWITCH_TILES_TC_BF16 = SV_SWITCH_BF16;
constexpr int SWITCH_TILES_MMA = 2;
// Shared prefixes. A unit's start in 128-key tiles of 256 rows and in 64-key tiles of 128 rows,
// and the SM time of the latter (two at a time on an SM) in the former. Measured around them at
// d = 128 (short runs of calls back to back, below the power limit; 64 sequences over a prefix
// of 8192, 128 over four of 16385, bf16; 32 over two of 32768, E4M3): 68.8, 254, 369 us; a
// sequence's start of 4: 69.6, 261, 372; costs of 0.31 and 0.50: 68.9, 257, 371; a prefix's
// start of 2: 69.3, 254, 368. They also divide the SMs at d = 64, where nothing was swept.
constexpr int SWITCH_TILES_PREFIX = 3;
constexpr int SWITCH_TILES_SEQUENCE = 3;
constexpr float SEQUENCE_COST_BF16 = 0.28f;
constexpr float SEQUENCE_COST_FP8 = 0.45f;
// Per-tile compute floor of each kernel, in CTAs streaming at once (a 128-key tile's
// compute time x HBM bandwidth / the tile's bytes: bf16 about 0.9 us x 6.8 TB/s / 64 KB,
// E4M3 about 0.89 us x 6.8 TB/s / 32 KB). The cost model is not applied to the mma.sync
// kernel (it keeps the split line unless a policy is forced).
#ifndef SV_TILE_FLOOR_BF16
#define SV_TILE_FLOOR_BF16 93
#endif
#ifndef SV_TILE_FLOOR_F8
#define SV_TILE_FLOOR_F8 185
#endif
#ifndef SV_UNIT_CTAS
#define SV_UNIT_CTAS -1
#endif

// Positions and cache rows are 32-bit on the device (tile arithmetic, TMA coordinates).
constexpr int32_t MAX_SEQ_LEN = 0x7fffffff - 1024;
constexpr int64_t MAX_KV_ROWS = 0x7fffffff - 1024;

// Launches until the armed failure, plus one (0: nothing armed). Tests only.
std::atomic<int> g_fail_countdown{0};
// Wait limit of the next tcgen05 attention launch that withholds a tile (0: none). Tests.
std::atomic<long long> g_stall_limit{0};
int g_attn_kernel = 0;  // 0 automatic, 1 mma.sync, 2 tcgen05
int g_unit_ctas = SV_UNIT_CTAS;  // -1 cost model, 0 split tile line, k > 0 k CTAs per unit
int g_row_pairs = 0;  // 1: the row-pair kernel whenever it applies; 0: never (default)
// bf16 K/V on the tcgen05 kernel: -1 by the call's shape (default), 0 paired K + V stages,
// 1 separate K and V rings.
int g_kv_rings = -1;
// Split rings let the K loads run further ahead of the score MMAs. Measured attention time
// (us, paired / split): c2 92.2 / 89.3; c4 (T = 16384, G = 8) with D = 0, 1, 3, 7, 15:
// 166.5 / 162.0, 167.8 / 161.3, 168.0 / 162.7, 168.2 / 162.2, 169.3 / 164.0; D = 31
// 257.0 / 247.8. Paired stages measured faster where a KV head's second row tile is partial
// (D = 16: 247.1 / 259.3, D = 23: 250.7 / 255.8, although their whole steps ran faster
// split) and on the ragged c5 batch, whose CTAs each stream about 900 tiles (1286 / 1315).
constexpr int64_t KV_RINGS_MAX_TILES_PER_CTA = 1024;
cudaEvent_t g_ev_start = nullptr;
cudaEvent_t g_ev_stop = nullptr;

int current_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

sv_status check_desc(const sv_attn_desc* d) {
  if (!d) return SV_ERR_NULL;
  if (d->batch < 0 || d->num_kv_heads < 1 || d->num_q_heads < 1 ||
      d->num_q_heads % d->num_kv_heads != 0 || d->num_q_heads > 4096 ||
      d->max_draft_len < 0 || d->max_draft_len > 255 || d->max_seq_len < 0 ||
      d->max_seq_len > MAX_SEQ_LEN || d->q_rows < 0 || d->kv_rows < 0 ||
      d->kv_rows > MAX_KV_ROWS || d->sliding_window < 0)
    return SV_ERR_SHAPE;
  if (d->head_dim != 64 && d->head_dim != 128) return SV_ERR_SHAPE;
  if (!(d->softmax_scale >= 0.f) || isinf(d->softmax_scale)) return SV_ERR_SHAPE;
  if (d->kv_dtype != SV_BF16 && d->kv_dtype != SV_FP8_E4M3) return SV_ERR_DTYPE;
  return SV_OK;
}

AttnWs layout_for(const sv_attn_desc* d, int sms) {
  return attn_ws_layout(d->batch, d->num_kv_heads, d->num_q_heads / d->num_kv_heads,
                        d->head_dim, d->max_draft_len, sms);
}

// 1 = mma.sync, 2 = tcgen05
int pick_kernel(const sv_attn_desc* d) {
  const bool tc_ok =
      attn_tc_available() && attn_tc_supports(d->head_dim, d->kv_dtype == SV_FP8_E4M3);
  if (g_attn_kernel == 1) return 1;
  if (g_attn_kernel == 2) return tc_ok ? 2 : 1;
  return tc_ok ? 2 : 1;
}

}  // namespace

bool sv::take_injected_launch_failure() {
  int n = g_fail_countdown.load(std::memory_order_relaxed);
  while (n > 0)
    if (g_fail_countdown.compare_exchange_weak(n, n - 1, std::memory_order_relaxed))
      return n == 1;
  return false;
}

extern "C" {

SV_API int sv_inject_launch_failure(int after) {
  const int prev = g_fail_countdown.exchange(after >= 0 && after < (1 << 30) ? after + 1 : 0);
  return prev - 1;
}

SV_API int sv_inject_wait_timeout(int64_t limit_cycles) {
  return g_stall_limit.exchange(limit_cycles > 0 ? (long long)limit_cycles : 0) > 0 ? 1 : 0;
}

SV_API int sv_version(void) { return 600; }  // 0.6.0: 4-bit caches, attention mass, eviction

SV_API const char* sv_status_string(sv_status s) {
  switch (s) {
    case SV_OK: return "ok";
    case SV_ERR_NULL: return "null pointer";
    case SV_ERR_SHAPE: return "invalid shape";
    case SV_ERR_DTYPE: return "unsupported dtype";
    case SV_ERR_ALIGN: return "misaligned pointer";
    case SV_ERR_WORKSPACE: return "workspace too small";
    case SV_ERR_CUDA: return "CUDA error";
    case SV_ERR_TIMEOUT: return "device-side wait timed out";
    case SV_ERR_DEVICE_SHAPE: return "device-side length check failed";
    case SV_ERR_NO_PAGES: return "too few free pages";
  }
  return "unknown status";
}

SV_API int sv_set_attn_kernel(int which) {
  if (which < 0 || which > 2) return -1;
  if (which == 2 && !attn_tc_available()) return -1;
  const int prev = g_attn_kernel;
  g_attn_kernel = which;
  return prev;
}

SV_API int sv_set_unit_ctas(int mode) {
  if (mode < -1 || mode > 1024) return -2;
  const int prev = g_unit_ctas;
  g_unit_ctas = mode;
  return prev;
}

SV_API int sv_set_row_pairs(int mode) {
  if (mode < 0 || mode > 1) return -2;
  const int prev = g_row_pairs;
  g_row_pairs = mode;
  return prev;
}

SV_API int sv_set_kv_rings(int mode) {
  if (mode < -1 || mode > 1) return -2;
  const int prev = g_kv_rings;
  g_kv_rings = mode;
  return prev;
}

SV_API void sv_set_profile_events(void* start_event, void* stop_event) {
  if (start_event && stop_event) {
    g_ev_start = (cudaEvent_t)start_event;
    g_ev_stop = (cudaEvent_t)stop_event;
  } else {
    g_ev_start = g_ev_stop = nullptr;
  }
}

SV_API size_t spec_verify_attn_workspace_size(const sv_attn_desc* desc) {
  if (check_desc(desc) != SV_OK) return 0;
  const int sms = current_sms();
  if (sms <= 0) return 0;
  return layout_for(desc, sms).total;
}

}  // extern "C"

namespace {

// A paged cache (block_size 0: the packed layout).
struct PagedArgs {
  const int32_t* table;
  int32_t stride;
  int32_t block_size;
  int64_t num_blocks;
};

// The sizes, limits and work-distribution policy of one attention call on `sms` SMs with
// kernel `which` (1 mma.sync, 2 tcgen05); every pointer is left null.
AttnParams shape_params(const sv_attn_desc* desc, const PagedArgs& pg, int which, int sms) {
  const bool fp8 = desc->kv_dtype == SV_FP8_E4M3;
  const int kt = which == 2 ? attn_tc_kt() : attn_mma_kt();
  const int G = desc->num_q_heads / desc->num_kv_heads;
  const int64_t rows_per_kv = (int64_t)G * (1 + desc->max_draft_len);
  const int64_t max_tiles = (int64_t)desc->batch * desc->num_kv_heads * ((rows_per_kv + MT - 1) / MT) *
                            ((desc->max_seq_len + 1 + desc->max_draft_len + kt - 1) / kt);
  AttnParams p = {};
  p.B = desc->batch;
  p.Hq = desc->num_q_heads;
  p.Hkv = desc->num_kv_heads;
  p.G = G;
  p.d = desc->head_dim;
  p.max_draft = desc->max_draft_len;
  p.max_seq = desc->max_seq_len;
  // a window covering every position of the longest sequence is no window
  p.window = (int64_t)desc->sliding_window > (int64_t)desc->max_seq_len + desc->max_draft_len
                 ? 0
                 : desc->sliding_window;
  p.q_rows = desc->q_rows;
  p.kv_rows = pg.block_size > 0 ? pg.num_blocks * pg.block_size : desc->kv_rows;
  p.bt_stride = pg.stride;
  p.block_size = pg.block_size;
  p.bs_log2 = 0;
  while (pg.block_size > 0 && (1 << p.bs_log2) < pg.block_size) ++p.bs_log2;
  p.num_blocks = pg.num_blocks;
  p.max_units = max_units_for(p.B, p.Hkv, G, p.max_draft);
  p.n_ctas = (int)(max_tiles < sms ? (max_tiles > 0 ? max_tiles : 1) : sms);
  // measured cost of starting a unit inside a CTA's range, in tiles of that kernel
  p.switch_tiles = which == 2 ? (fp8 ? SWITCH_TILES_TC_FP8 : SWITCH_TILES_TC_BF16) : SWITCH_TILES_MMA;
  // The same model for a paged cache: with its block-table entries read a group of tiles
  // ahead, a CTA streams 16-position blocks at nearly the packed rate (c2: 97.5 us with
  // one CTA per unit against 115.3 us on the split tile line, packed 95.1 us).
  p.tile_floor = which == 2 ? (fp8 ? SV_TILE_FLOOR_F8 : SV_TILE_FLOOR_BF16) : 0;
  p.unit_ctas_mode = g_unit_ctas;
  const bool partial_row_tile = rows_per_kv > MT && rows_per_kv % MT != 0;
  const bool long_stream = max_tiles > KV_RINGS_MAX_TILES_PER_CTA * p.n_ctas;
  p.kv_rings = g_kv_rings >= 0 ? g_kv_rings : (partial_row_tile || long_stream ? 0 : 1);
  const float scale = desc->softmax_scale > 0.f ? desc->softmax_scale
                                                : 1.f / sqrtf((float)desc->head_dim);
  p.scale_log2 = scale * 1.4426950408889634f;
  return p;
}

// Whether a call of kernel `which` with these parameters runs the row-pair kernel: it is
// switched on and applies (see attn_pair_applies). Off by default: on every workload
// measured, the unit plan (each row tile streaming the keys, the second from L2) is faster.
bool use_row_pairs(const AttnParams& p, bool fp8, int which, int sms) {
  return which == 2 && g_row_pairs == 1 && attn_pair_applies(p, fp8, sms);
}

sv_status verify_impl(const sv_attn_desc* desc, const void* q, const void* k_cache,
                      const void* v_cache, const PagedArgs& pg, const int32_t* seq_lens,
                      const int32_t* draft_len, const float* kv_scale, void* out,
                      void* workspace, size_t workspace_bytes, void* stream,
                      const int32_t* seq_lens_host = nullptr,
                      const int32_t* draft_len_host = nullptr) {
  sv_status st = check_desc(desc);
  if (st != SV_OK) return st;
  if (desc->batch == 0) return SV_OK;
  if (!q || !k_cache || !v_cache || !seq_lens || !draft_len || !out || !workspace)
    return SV_ERR_NULL;
  if (pg.block_size > 0 && !pg.table) return SV_ERR_NULL;
  if (pg.block_size > 0 && !aligned(pg.table, 4)) return SV_ERR_ALIGN;
  if (seq_lens_host && draft_len_host)  // host copies of the lengths: checked here, at once
    for (int b = 0; b < desc->batch; ++b)
      if (seq_lens_host[b] < 0 || seq_lens_host[b] > desc->max_seq_len || draft_len_host[b] < 0 ||
          draft_len_host[b] > desc->max_draft_len)
        return SV_ERR_SHAPE;
  const bool fp8 = desc->kv_dtype == SV_FP8_E4M3;
  if (fp8 && !kv_scale) return SV_ERR_NULL;
  if (!fp8 && kv_scale) return SV_ERR_SHAPE;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(workspace, 256) || !aligned(seq_lens, 4) || !aligned(draft_len, 4) ||
      (kv_scale && !aligned(kv_scale, 4)))
    return SV_ERR_ALIGN;
  const int sms = current_sms();
  if (sms <= 0) return SV_ERR_CUDA;
  const AttnWs lay = layout_for(desc, sms);
  if (workspace_bytes < lay.total) return SV_ERR_WORKSPACE;

  const int which = pick_kernel(desc);
  const int kt = which == 2 ? attn_tc_kt() : attn_mma_kt();
  AttnParams p = shape_params(desc, pg, which, sms);
  if (which == 2) {  // a pending wait-timeout injection applies to this launch
    const long long lim = g_stall_limit.exchange(0);
    if (lim > 0) {
      p.wait_limit = lim;
      p.stall_first_tile = 1;
    }
  }
  uint8_t* ws = (uint8_t*)workspace;
  p.q = q;
  p.k = k_cache;
  p.v = v_cache;
  p.out = out;
  p.kv_scale = kv_scale;
  p.seq_lens = seq_lens;
  p.draft_len = draft_len;
  p.flags = (uint32_t*)(ws + lay.ctrl);
  p.hdr = (PlanHdr*)(ws + lay.hdr);
  p.q_off = (int64_t*)(ws + lay.q_off);
  p.kv_off = (int64_t*)(ws + lay.kv_off);
  p.units = (int4*)(ws + lay.units);
  p.ubeg = (int32_t*)(ws + lay.ubeg);
  p.cta_tab = (int2*)(ws + lay.cta_tab);
  p.part_o = (float*)(ws + lay.part_o);
  p.part_ml = (float2*)(ws + lay.part_ml);
  p.block_table = pg.table;

  cudaStream_t s = (cudaStream_t)stream;
  if (use_row_pairs(p, fp8, which, sms)) {  // one launch: no plan, nothing to combine
    if (g_ev_start && cudaEventRecord(g_ev_start, s) != cudaSuccess) return SV_ERR_CUDA;
    if (launch_attn_pair(p, s) != cudaSuccess) return SV_ERR_CUDA;
    if (g_ev_stop && cudaEventRecord(g_ev_stop, s) != cudaSuccess) return SV_ERR_CUDA;
    return SV_OK;
  }
  // Host lengths: plan on the host and pass the plan with the attention launch (tcgen05
  // kernel, packed cache), unless it does not fit a HostPlan.
  static thread_local HostPlan hp;
  bool host_planned = false;
  if (seq_lens_host && draft_len_host && which == 2 && pg.block_size == 0) {
    const sv_status hs = host_plan(p, kt, seq_lens_host, draft_len_host, &hp);
    if (hs == SV_ERR_SHAPE) return SV_ERR_SHAPE;
    host_planned = hs == SV_OK;
  }
  if (!host_planned && launch_plan(p, kt, s) != cudaSuccess) return SV_ERR_CUDA;
  if (g_ev_start && cudaEventRecord(g_ev_start, s) != cudaSuccess) return SV_ERR_CUDA;
  const cudaError_t e = host_planned ? launch_attn_tc_hp(p, fp8, hp, s)
                        : which == 2 ? launch_attn_tc(p, fp8, s)
                                     : launch_attn_mma(p, fp8, s);
  if (e != cudaSuccess) return SV_ERR_CUDA;
  if (g_ev_stop && cudaEventRecord(g_ev_stop, s) != cudaSuccess) return SV_ERR_CUDA;
  if (launch_combine(p, s) != cudaSuccess) return SV_ERR_CUDA;
  return SV_OK;
}

}  // namespace

extern "C" {

SV_API sv_status spec_verify_attn(const sv_attn_desc* desc, const void* q, const void* k_cache,
                                  const void* v_cache, const int32_t* seq_lens,
                                  const int32_t* draft_len, const float* kv_scale, void* out,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  const PagedArgs packed = {nullptr, 0, 0, 0};
  return verify_impl(desc, q, k_cache, v_cache, packed, seq_lens, draft_len, kv_scale, out,
                     workspace, workspace_bytes, stream);
}

SV_API sv_status spec_verify_attn_host_lengths(const sv_attn_desc* desc, const void* q,
                                               const void* k_cache, const void* v_cache,
                                               const int32_t* seq_lens,
                                               const int32_t* draft_len,
                                               const int32_t* seq_lens_host,
                                               const int32_t* draft_len_host,
                                               const float* kv_scale, void* out,
                                               void* workspace, size_t workspace_bytes,
                                               void* stream) {
  if (desc && desc->batch > 0 && (!seq_lens_host || !draft_len_host)) return SV_ERR_NULL;
  const PagedArgs packed = {nullptr, 0, 0, 0};
  return verify_impl(desc, q, k_cache, v_cache, packed, seq_lens, draft_len, kv_scale, out,
                     workspace, workspace_bytes, stream, seq_lens_host, draft_len_host);
}

SV_API sv_status spec_verify_attn_paged(const sv_attn_desc* desc, const void* q,
                                        const void* k_pages, const void* v_pages,
                                        int64_t num_blocks, int32_t block_size,
                                        const int32_t* block_table, int32_t max_blocks_per_seq,
                                        const int32_t* seq_lens, const int32_t* draft_len,
                                        const float* kv_scale, void* out, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  if (block_size < 8 || block_size > (1 << 16) || (block_size & (block_size - 1)) != 0 ||
      num_blocks < 1 || num_blocks > MAX_KV_ROWS / block_size || max_blocks_per_seq < 1)
    return SV_ERR_SHAPE;
  const PagedArgs pg = {block_table, max_blocks_per_seq, block_size, num_blocks};
  return verify_impl(desc, q, k_pages, v_pages, pg, seq_lens, draft_len, kv_scale, out,
                     workspace, workspace_bytes, stream);
}

}  // extern "C"

namespace {

// Units of 128 query rows that a shared-prefix call may have: the tables of the plan and
// the partials' slots are indexed with 32 bits.
constexpr int64_t MAX_SHARED_UNITS = 1 << 22;

// Small calls take the mma.sync kernel: three launches instead of four, no TMEM, no tensor
// maps. The rule goes by what the host knows, the sequences' units and the longest sequence.
// Calls back to back from Python, mma.sync against tcgen05, d 128, bf16 (E4M3; d 64 not swept):
//     8 units of 512, 960 positions       18.9, 20.7 us against 20.3, 19.7 (18.1, 21.1: 22.8, 23.0)
//    16 units of 80, 320, 1088            15.4, 16.2, 21.2 against 19.9, 20.2, 22.4
//    64 units of 80, 320, 960             18.9, 22.5, 27.6 against 21.2, 22.9, 23.6
//   128 units of 80, 320                  18.8, 26.4 against 20.9, 21.8 (19.1, 27.4: 26.1, 26.3)
constexpr int64_t SMALL_WORK = 20480;  // units x positions
constexpr int SMALL_SEQ = 1024;
int pick_shared(const sv_attn_desc* d) {
  const int64_t rows = (int64_t)(d->num_q_heads / d->num_kv_heads) * (1 + d->max_draft_len);
  const int64_t units = d->num_kv_heads * (int64_t)d->batch * ((rows + MT - 1) / MT);
  const bool small = d->max_seq_len <= SMALL_SEQ && units * d->max_seq_len <= SMALL_WORK;
  return g_attn_kernel == 0 && small ? 1 : pick_kernel(d);
}

sv_status check_shared(const sv_attn_desc* desc, int32_t num_groups) {
  const sv_status st = check_desc(desc);
  if (st != SV_OK) return st;
  if (desc->sliding_window != 0 || num_groups < 0 || num_groups > std::max(desc->batch, 1) ||
      (num_groups == 0 && desc->batch > 0))
    return SV_ERR_SHAPE;
  const SharedWs lay = shared_ws_layout(desc, num_groups, 0, false);
  return lay.max_units[1] > MAX_SHARED_UNITS ? SV_ERR_SHAPE : SV_OK;
}

}  // namespace

extern "C" {

SV_API size_t spec_verify_attn_shared_workspace_size(const sv_attn_desc* desc, int32_t num_groups) {
  if (check_shared(desc, num_groups) != SV_OK) return 0;
  const int sms = current_sms();
  if (sms <= 0) return 0;
  // whichever attention kernel a call will take
  return std::max(shared_ws_layout(desc, num_groups, sms, true).total,
                  shared_ws_layout(desc, num_groups, sms, false).total);
}

SV_API sv_status spec_verify_attn_shared(const sv_attn_desc* desc, const void* q,
                                         const void* k_pages, const void* v_pages,
                                         int64_t num_blocks, int32_t block_size,
                                         const int32_t* block_table, int32_t max_blocks_per_seq,
                                         const int32_t* seq_lens, const int32_t* draft_len,
                                         int32_t num_groups, const int32_t* group_begin,
                                         const int32_t* prefix_len, const float* kv_scale,
                                         void* out, void* workspace, size_t workspace_bytes,
                                         void* stream) {
  if (block_size < 8 || block_size > (1 << 16) || (block_size & (block_size - 1)) != 0 ||
      num_blocks < 1 || num_blocks > MAX_KV_ROWS / block_size || max_blocks_per_seq < 1)
    return SV_ERR_SHAPE;
  const sv_status st = check_shared(desc, num_groups);
  if (st != SV_OK || desc->batch == 0) return st;
  if (!q || !k_pages || !v_pages || !block_table || !seq_lens || !draft_len || !group_begin ||
      !prefix_len || !out || !workspace)
    return SV_ERR_NULL;
  const bool fp8 = desc->kv_dtype == SV_FP8_E4M3;
  if (fp8 && !kv_scale) return SV_ERR_NULL;
  if (!fp8 && kv_scale) return SV_ERR_SHAPE;
  if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(out, 16) ||
      !aligned(workspace, 256) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(draft_len, 4) || !aligned(group_begin, 4) || !aligned(prefix_len, 4) ||
      !aligned(kv_scale, 4))
    return SV_ERR_ALIGN;
  const int sms = current_sms();
  if (sms <= 0) return SV_ERR_CUDA;
  if (workspace_bytes < std::max(shared_ws_layout(desc, num_groups, sms, true).total,
                                 shared_ws_layout(desc, num_groups, sms, false).total))
    return SV_ERR_WORKSPACE;

  const int which = pick_shared(desc);
  const bool lines = which == 2;
  const SharedWs lay = shared_ws_layout(desc, num_groups, sms, lines);
  const PagedArgs pg = {block_table, max_blocks_per_seq, block_size, num_blocks};
  AttnParams p = shape_params(desc, pg, which, sms);
  if (which == 2) {  // a pending wait-timeout injection applies to this launch
    const long long lim = g_stall_limit.exchange(0);
    if (lim > 0) {
      p.wait_limit = lim;
      p.stall_first_tile = 1;
    }
  }
  uint8_t* ws = (uint8_t*)workspace;
  p.q = q;
  p.k = k_pages;
  p.v = v_pages;
  p.out = out;
  p.kv_scale = kv_scale;
  p.seq_lens = seq_lens;
  p.draft_len = draft_len;
  p.block_table = block_table;
  p.num_groups = num_groups;
  p.group_begin = group_begin;
  p.prefix_len = prefix_len;
  p.flags = (uint32_t*)ws;
  p.handover = (HandOver*)(ws + lay.handover);
  p.prefix_ctas = lay.n_ctas[0];
  p.parts = (SharedSeq*)(ws + lay.parts);
  p.row_begin = (int32_t*)(ws + lay.row_begin);
  p.rows = (RowInfo*)(ws + lay.rows);
  p.tile_unit = (int32_t*)(ws + lay.tile_unit);
  p.row_log2 = lines ? 8 : 7;  // 2 * MT or MT rows
  AttnParams line[2] = {p, p};
  for (int k = 0; k < 2; ++k) {
    AttnParams& l = line[k];
    l.max_units = (int)lay.max_units[k];
    l.n_ctas = lay.n_ctas[k];
    l.kt = !lines ? attn_mma_kt() : k == 0 ? 128 : 64;
    l.tile_cost = fp8 ? SEQUENCE_COST_FP8 : SEQUENCE_COST_BF16;
    if (lines) l.switch_tiles = k == 0 ? SWITCH_TILES_PREFIX : SWITCH_TILES_SEQUENCE;
    l.hdr = (PlanHdr*)(ws + lay.line[k].hdr);
    l.units = (int4*)(ws + lay.line[k].units);
    l.sunits = (SharedUnit*)(ws + lay.line[k].sunits);
    l.ubeg = (int32_t*)(ws + lay.line[k].ubeg);
    l.unit_ctas = (int2*)(ws + lay.line[k].unit_ctas);
    l.cta_tab = (int2*)(ws + lay.line[k].cta_tab);
    l.part_o = (float*)(ws + lay.line[k].part_o);
    l.part_ml = (float2*)(ws + lay.line[k].part_ml);
  }

  cudaStream_t s = (cudaStream_t)stream;
  if (launch_plan_shared(line[0], line[1], lines, s) != cudaSuccess) return SV_ERR_CUDA;
  if (g_ev_start && cudaEventRecord(g_ev_start, s) != cudaSuccess) return SV_ERR_CUDA;
  if (lines) {
    if (launch_attn_sequences(line[1], fp8, s) != cudaSuccess) return SV_ERR_CUDA;
    if (launch_attn_prefixes(line[0], fp8, s) != cudaSuccess) return SV_ERR_CUDA;
  } else if (launch_attn_mma_shared(line[1], fp8, s) != cudaSuccess) {
    return SV_ERR_CUDA;
  }
  if (g_ev_stop && cudaEventRecord(g_ev_stop, s) != cudaSuccess) return SV_ERR_CUDA;
  return launch_combine_shared(lines ? line[0] : line[1], line[1], s) == cudaSuccess ? SV_OK
                                                                                  : SV_ERR_CUDA;
}

SV_API sv_status sv_plan_preview(const sv_attn_desc* desc, int32_t block_size,
                                 const int32_t* seq_lens_host, const int32_t* draft_len_host,
                                 int32_t num_sms, int32_t attn_kernel, sv_plan_info* info,
                                 int32_t* units, int32_t* unit_begin, int32_t* cta_begin,
                                 int32_t capacity_units) {
  sv_status st = check_desc(desc);
  if (st != SV_OK) return st;
  if (!info) return SV_ERR_NULL;
  if (desc->batch > 0 && (!seq_lens_host || !draft_len_host)) return SV_ERR_NULL;
  if (num_sms < 1 || capacity_units < 0 || (attn_kernel != 1 && attn_kernel != 2) ||
      (block_size != 0 &&
       (block_size < 8 || block_size > (1 << 16) || (block_size & (block_size - 1)) != 0)))
    return SV_ERR_SHAPE;
  if (attn_kernel == 2 && !attn_tc_supports(desc->head_dim, desc->kv_dtype == SV_FP8_E4M3))
    return SV_ERR_SHAPE;
  // a paged pool's size does not enter the plan: the largest pool the limits allow
  const PagedArgs pg = {nullptr, 1 << 30, block_size,
                        block_size > 0 ? MAX_KV_ROWS / block_size : 0};
  const AttnParams p = shape_params(desc, pg, attn_kernel, num_sms);
  const int kt = attn_kernel == 2 ? attn_tc_kt() : attn_mma_kt();
  *info = sv_plan_info{0, 0, kt, p.n_ctas, 0, p.switch_tiles};
  if (desc->batch == 0) return SV_OK;
  static thread_local HostPlan hp;
  st = host_plan(p, kt, seq_lens_host, draft_len_host, &hp);
  if (st != SV_OK) return st;
  info->num_units = hp.num_units;
  info->total_tiles = hp.total_tiles;
  info->unit_ctas = hp.unit_ctas;
  if ((units || unit_begin) && hp.num_units > capacity_units) return SV_ERR_WORKSPACE;
  for (int u = 0; units && u < hp.num_units; ++u) {
    units[4 * u] = hp.units[u].x;
    units[4 * u + 1] = hp.units[u].y;
    units[4 * u + 2] = hp.units[u].z;
    units[4 * u + 3] = hp.units[u].w;
  }
  for (int u = 0; unit_begin && u <= hp.num_units; ++u) unit_begin[u] = hp.ubeg[u];
  for (int c = 0; cta_begin && c <= p.n_ctas; ++c) {
    cta_begin[2 * c] = hp.cta_tab[c].x;
    cta_begin[2 * c + 1] = hp.cta_tab[c].y;
  }
  return SV_OK;
}

SV_API int sv_row_pair_mode(const sv_attn_desc* desc, int32_t block_size, int32_t num_sms,
                           int32_t attn_kernel) {
  if (check_desc(desc) != SV_OK || num_sms < 1 || (attn_kernel != 1 && attn_kernel != 2) ||
      block_size < 0)
    return -1;
  const PagedArgs pg = {nullptr, 1 << 30, block_size,
                        block_size > 0 ? MAX_KV_ROWS / block_size : 0};
  const AttnParams p = shape_params(desc, pg, attn_kernel, num_sms);
  return use_row_pairs(p, desc->kv_dtype == SV_FP8_E4M3, attn_kernel, num_sms) ? 1 : 0;
}

}  // extern "C"

namespace {

bool pool_sizes_ok(int32_t num_blocks, int32_t block_size) {
  return block_size >= 8 && block_size <= (1 << 16) && (block_size & (block_size - 1)) == 0 &&
         num_blocks >= 1 && num_blocks <= MAX_KV_ROWS / block_size;
}

// The checks that the spec_pages_ calls share. `n`: rows of the call (null lists allowed
// where they have a meaning are checked by the caller).
sv_status check_pages(const sv_page_table* t, int32_t n, const void* ws, size_t ws_bytes) {
  if (!t) return SV_ERR_NULL;
  if (!pool_sizes_ok(t->num_blocks, t->block_size) || t->table_rows < 0 ||
      t->table_rows > SV_MAX_TABLE_ROWS || t->max_blocks_per_seq < 1 || n < 0 || n > t->table_rows)
    return SV_ERR_SHAPE;
  if (!t->ref_count || (t->table_rows > 0 && (!t->block_table || !t->cached_len)) || !ws)
    return SV_ERR_NULL;
  if (!aligned(t->ref_count, 16) || !aligned(t->block_table, 4) || !aligned(t->cached_len, 4) ||
      !aligned(ws, 256))
    return SV_ERR_ALIGN;
  return ws_bytes < pages_ws_bytes(t->num_blocks, t->table_rows) ? SV_ERR_WORKSPACE : SV_OK;
}

// Whether the arrays that a spec_pages_ call changes (the state, the workspace and `out`) and
// the lists that it reads are apart. The kernels read a list more than once, so one that the
// call itself changes would not be the one that was checked. Null arrays are none.
struct Span {
  const void* at;
  size_t bytes;
};
bool arrays_apart(const sv_page_table* t, const void* ws, std::initializer_list<Span> out,
                  std::initializer_list<Span> lists, int num_pools = 0,
                  const sv_page_data* pools = nullptr) {
  Span a[12] = {{t->ref_count, 4 * (size_t)t->num_blocks},
                {t->block_table, 4 * (size_t)t->table_rows * t->max_blocks_per_seq},
                {t->cached_len, 4 * (size_t)t->table_rows},
                {ws, pages_ws_bytes(t->num_blocks, t->table_rows)}};
  int n = 4;
  for (const Span& s : out) a[n++] = s;
  const int changed = n;
  for (const Span& s : lists) a[n++] = s;
  auto meet = [](const Span& x, const Span& y) {
    const uintptr_t b = (uintptr_t)x.at, c = (uintptr_t)y.at;
    return x.at && y.at && b < c + y.bytes && c < b + x.bytes;
  };
  for (int i = 0; i < changed; ++i)
    for (int j = i + 1; j < n; ++j)
      if (meet(a[i], a[j])) return false;
  for (int k = 0; k < num_pools; ++k)
    for (int i = 0; i < n; ++i)
      if (meet(a[i], {pools[k].base, (size_t)pools[k].page_bytes * t->num_blocks})) return false;
  return true;
}

sv_status check_pools(const sv_page_table* t, int32_t num_pools, const sv_page_data* pools) {
  if (num_pools < 0 || num_pools > SV_MAX_PAGE_POOLS) return SV_ERR_SHAPE;
  if (num_pools > 0 && !pools) return SV_ERR_NULL;
  for (int i = 0; i < num_pools; ++i) {
    if (!pools[i].base) return SV_ERR_NULL;
    if (pools[i].page_bytes < 1 || pools[i].page_bytes > (1 << 30) ||
        pools[i].page_bytes % (16 * (int64_t)t->block_size) != 0)
      return SV_ERR_SHAPE;
    if (!aligned(pools[i].base, 16)) return SV_ERR_ALIGN;
  }
  return SV_OK;
}

}  // namespace

extern "C" {

SV_API size_t spec_pages_workspace_size(int32_t num_blocks, int32_t table_rows) {
  if (!pool_sizes_ok(num_blocks, 8) || table_rows < 0 || table_rows > SV_MAX_TABLE_ROWS) return 0;
  return pages_ws_bytes(num_blocks, table_rows);
}

SV_API sv_status spec_pages_fork(const sv_page_table* table, int32_t n, const int32_t* parents,
                                 const int32_t* children, const int32_t* fork_len,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  const sv_status st = check_pages(table, n, workspace, workspace_bytes);
  if (st != SV_OK || n == 0) return st;
  if (!parents || !children) return SV_ERR_NULL;
  if (!aligned(parents, 4) || !aligned(children, 4) || !aligned(fork_len, 4)) return SV_ERR_ALIGN;
  const size_t list = 4 * (size_t)n;
  if (!arrays_apart(table, workspace, {}, {{parents, list}, {children, list}, {fork_len, list}}))
    return SV_ERR_SHAPE;
  const int sms = current_sms();
  if (sms <= 0) return SV_ERR_CUDA;
  return launch_pages_fork(*table, n, parents, children, fork_len, workspace, sms,
                           (cudaStream_t)stream) == cudaSuccess
             ? SV_OK
             : SV_ERR_CUDA;
}

SV_API sv_status spec_pages_extend(const sv_page_table* table, int32_t n, const int32_t* rows,
                                   const int32_t* new_len, int32_t num_pools,
                                   const sv_page_data* pools, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  sv_status st = check_pages(table, n, workspace, workspace_bytes);
  if (st == SV_OK) st = check_pools(table, num_pools, pools);
  if (st != SV_OK || n == 0) return st;
  if (!new_len) return SV_ERR_NULL;
  if (!aligned(rows, 4) || !aligned(new_len, 4)) return SV_ERR_ALIGN;
  const size_t list = 4 * (size_t)n;
  if (!arrays_apart(table, workspace, {}, {{rows, list}, {new_len, list}}, num_pools, pools))
    return SV_ERR_SHAPE;
  const int sms = current_sms();
  if (sms <= 0) return SV_ERR_CUDA;
  return launch_pages_extend(*table, n, rows, new_len, num_pools, pools, workspace, sms,
                             (cudaStream_t)stream) == cudaSuccess
             ? SV_OK
             : SV_ERR_CUDA;
}

SV_API sv_status spec_pages_trim(const sv_page_table* table, int32_t n, const int32_t* rows,
                                 const int32_t* new_len, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  const sv_status st = check_pages(table, n, workspace, workspace_bytes);
  if (st != SV_OK || n == 0) return st;
  if (!new_len) return SV_ERR_NULL;
  if (!aligned(rows, 4) || !aligned(new_len, 4)) return SV_ERR_ALIGN;
  const size_t list = 4 * (size_t)n;
  if (!arrays_apart(table, workspace, {}, {{rows, list}, {new_len, list}})) return SV_ERR_SHAPE;
  const int sms = current_sms();
  if (sms <= 0) return SV_ERR_CUDA;
  return launch_pages_trim(*table, n, rows, new_len, workspace, sms, (cudaStream_t)stream) ==
                 cudaSuccess
             ? SV_OK
             : SV_ERR_CUDA;
}

SV_API sv_status spec_pages_compact(const sv_page_table* table, int32_t num_pools,
                                    const sv_page_data* pools, int32_t* remap, int32_t* num_live,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  sv_status st = check_pages(table, 0, workspace, workspace_bytes);
  if (st == SV_OK) st = check_pools(table, num_pools, pools);
  if (st != SV_OK) return st;
  if (!aligned(remap, 4) || !aligned(num_live, 4)) return SV_ERR_ALIGN;
  if (!arrays_apart(table, workspace, {{remap, 4 * (size_t)table->num_blocks}, {num_live, 4}}, {},
                    num_pools, pools))
    return SV_ERR_SHAPE;
  const int sms = current_sms();
  if (sms <= 0) return SV_ERR_CUDA;
  return launch_pages_compact(*table, num_pools, pools, remap, num_live, workspace, sms,
                              (cudaStream_t)stream) == cudaSuccess
             ? SV_OK
             : SV_ERR_CUDA;
}

}  // extern "C"

namespace {

// Whether [a, a + na) and [b, b + nb) share a byte (null arrays share none).
bool meet(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return a && b && x < y + nb && y < x + na;
}

sv_status check_kv4(const sv_kv4_pages* p) {
  if (!p) return SV_ERR_NULL;
  if (p->num_blocks < 1 || p->num_blocks > 0x7fffffff ||
      !pool_sizes_ok((int32_t)p->num_blocks, p->block_size) || p->num_kv_heads < 1 ||
      p->num_kv_heads > 4096 || (p->head_dim != 64 && p->head_dim != 128))
    return SV_ERR_SHAPE;
  if (!p->k_codes || !p->v_codes || !p->scales || !p->kv_scale) return SV_ERR_NULL;
  if (!aligned(p->k_codes, 16) || !aligned(p->v_codes, 16) || !aligned(p->scales, 16) ||
      !aligned(p->kv_scale, 4))
    return SV_ERR_ALIGN;
  return SV_OK;
}

sv_status check_kv4_rows(const sv_kv4_pages* p, int32_t batch, const int32_t* table,
                         int32_t max_blocks, const int32_t* start, const int32_t* count,
                         int64_t rows, const void* k, const void* v, void* ws, size_t ws_bytes) {
  const sv_status st = check_kv4(p);
  if (st != SV_OK) return st;
  // (a CTA takes a row or more: the grid's limit, with room to spare)
  if (batch < 0 || max_blocks < 1 || rows < 0 || rows > 0x7fffffff) return SV_ERR_SHAPE;
  if (batch == 0) return SV_OK;
  if (!table || !start || !count || !ws || (rows > 0 && (!k || !v))) return SV_ERR_NULL;
  if (!aligned(table, 4) || !aligned(start, 4) || !aligned(count, 4) || !aligned(k, 16) ||
      !aligned(v, 16) || !aligned(ws, 256))
    return SV_ERR_ALIGN;
  return ws_bytes < spec_kv4_workspace_size(batch) ? SV_ERR_WORKSPACE : SV_OK;
}

// The pages' arrays and one that a call reads or writes: apart?
bool kv4_apart(const sv_kv4_pages* p, const void* at, size_t bytes) {
  const size_t rows = (size_t)p->num_blocks * p->block_size * p->num_kv_heads;
  return !meet(p->k_codes, rows * (p->head_dim / 2), at, bytes) &&
         !meet(p->v_codes, rows * (p->head_dim / 2), at, bytes) &&
         !meet(p->scales, rows * (p->head_dim / 8), at, bytes);
}

// The descriptor's checks, for a call that takes SV_KV4.
sv_status check_desc_kv4(const sv_attn_desc* d) {
  if (!d) return SV_ERR_NULL;
  sv_attn_desc c = *d;
  if (c.kv_dtype == SV_KV4) c.kv_dtype = SV_BF16;
  return check_desc(&c);
}

float scale_log2_of(const sv_attn_desc* d) {
  const float scale = d->softmax_scale > 0.f ? d->softmax_scale : 1.f / sqrtf((float)d->head_dim);
  return scale * 1.4426950408889634f;
}

int64_t kv4_rows_per_head(const sv_attn_desc* d) {
  return (int64_t)(d->num_q_heads / d->num_kv_heads) * (1 + d->max_draft_len);
}

// The rules of a 4-bit attention call. The times are of calls replayed from a graph, d = 128, by
// sequences x longest of their ragged lengths, 8 KV heads and 4 query heads each if not stated.
//
// Virtual tiles charged for starting a unit. The tcgen05 kernel at 0-8 tiles of 2, 4, 6, 9, 13:
// 32 x 4000, 8 tokens 71.3, 69.5, 70.0, 71.9, 75.4 us; 57 x 457, 16 tokens, 7 query heads 57.4,
// 55.5, 54.7, 54.7, 54.8. The mma kernel at 0, 1, 2, 4, 8, one token: 64 x 8000 84.9, 76.5, 77.6,
// 80.0, 86.4; one of 30000, 4 KV heads 20.7, 20.6, 22.5, 21.3, 22.5.
constexpr int SWITCH_TILES_KV4 = 6;
constexpr int SWITCH_TILES_KV4_MMA = 1;
// What the join costs in tiles: ranges are whole units where the longest is no longer than an
// even share and this. The tcgen05 kernel, 32 tokens, at 0, 3, 8, 16: 16 x 8192 each 94.4, 94.5,
// 90.4, 90.4; 12 x 2000 each 40.0, 33.9, 34.0, 33.9; 8 x 4000 each 39.0, 39.0, 39.0, 49.2. The mma
// kernel, one token, at 0, 3, 6, 24: 100 x 900 33.9, 31.4, 30.9, 30.9; 4 x 1000 14.3, 14.4, 20.5,
// 20.5; 32 of 4096 each 44.4, 44.0, 43.9, 80.8.
constexpr int JOIN_TILES_KV4 = 8;
constexpr int JOIN_TILES_KV4_MMA = 3;
// Short sequences: up to KV4_SHORT_TILES tiles of the longest, a CTA takes a whole unit and no
// join runs; up to twice that where the units fill half of the CTAs. At twice, whole and split:
// 200 x 1000, one token 57.1 and 59.5; 16 x 1000, 8 tokens 22.6 and 26.6; but with 128 units,
// 32 x 1000, one token 20.5 and 18.4, 8 x 1000, 8 tokens 20.5 and 18.5. At four times, with 800
// units, 200 x 2000 87.9 and 82.4.
constexpr int KV4_SHORT_TILES = 4;
// Two neighbouring heads make one unit from this many heads of all sequences on (they share
// lines of HBM, but are half as many units), with short sequences heads times row tiles. Two and
// one: 32 x 8000, one token 44.6 and 46.9; 64 x 8000 76.8 and 105.2; 16 x 8000 30.8 and 28.7;
// short, 8 tokens, 64 x 700 34.8 and 37.5; 32 x 1000 36.7 and 26.7. The tcgen05 kernel's pairs
// are two CTAs side by side, which costs it no units: always. 32 tokens, 8 x 32768 each 147.2 and
// 153.8; 32 x 4000 each 110.4 and 114.0; 8 x 2000 each 37.8 and 37.4; one of 20000 30.8 and 30.8.
constexpr int KV4_PAIR_UNITS = 256;
constexpr int KV4_PAIR_UNITS_SHORT = 1024;
// The mma kernel (row tiles of 16, no start to speak of) up to 16 rows a KV head, and for more
// rows in calls of so many of its tiles of 128 x 128 altogether; else the tcgen05 kernel (row
// tiles of 128). The mma kernel's and the tcgen05 kernel's time with 4 KV heads, at 32, 48, 64,
// 128 rows: 64 x 16000 170 154, 222 154, 276 155, 486 158; 64 x 4000 65.4 67.5, 79.4 67.0,
// 94.2 68.1, 156 74.8; 8 x 4000 24.6 28.7, 26.7 28.7, 26.6 28.7, 37.4 28.7; one of 20000
// 20.7 24.6, 22.4 26.6, 24.6 26.0, 32.5 28.7; short, 64 x 700 22.5 40.6, 30.0 40.8, 34.9 41.1,
// 52.3 43.0. Many rows: 16 x 300 with 2 KV heads at 256, 512 rows 18.0 20.5, 26.3 20.5. With
// d = 64 a tile of the tcgen05 kernel is not much shorter, and "few rows" are more: 64 x 16000
// 103 135, 133 137, 163 137, 281 139; 64 x 4000 45.1 57.4, 53.0 57.5, 61.5 58.2, 96.8 59.4;
// 8 x 4000 20.5 24.6, 20.8 24.6, 20.5 24.6, 28.7 24.7.
constexpr int KV4_SMALL_ROWS = 16;
constexpr int KV4_FEW_ROWS = 32, KV4_FEW_ROWS_64 = 48;
constexpr int KV4_MMA_ROWS = 256;
constexpr int64_t KV4_MMA_TILES = 6144;
constexpr int64_t KV4_MMA_TILES_SHORT = 12288;  // short sequences
constexpr int64_t KV4_MMA_TILES_FEW = 32768, KV4_MMA_TILES_FEW_64 = 65536;  // up to "few" rows

int64_t kv4_max_tiles(const sv_attn_desc* d) {
  return ((int64_t)d->max_seq_len + d->max_draft_len) / KV4_KT + 1;
}

// 1 = warp-level MMAs (attn_kv4.cu), 2 = tcgen05 (attn_kv4_tc.cu)
int pick_kv4(const sv_attn_desc* d) {
  if (!attn_tc_available() || g_attn_kernel == 1) return 1;
  if (g_attn_kernel == 2) return 2;
  const int64_t rows = kv4_rows_per_head(d), tiles = kv4_max_tiles(d);
  const int64_t all = (int64_t)d->batch * d->num_kv_heads * ((rows + 15) / 16) * tiles * d->head_dim / 128;
  const bool d64 = d->head_dim == 64;
  const int64_t most = rows <= (d64 ? KV4_FEW_ROWS_64 : KV4_FEW_ROWS)
                           ? (d64 ? KV4_MMA_TILES_FEW_64 : KV4_MMA_TILES_FEW)
                       : tiles <= 2 * KV4_SHORT_TILES ? KV4_MMA_TILES_SHORT
                                                      : KV4_MMA_TILES;
  return rows <= KV4_SMALL_ROWS || (rows <= KV4_MMA_ROWS && all <= most) ? 1 : 2;
}

// A call's units and ranges (line.cuh) on `sms` SMs with kernel `which`.
void kv4_line(const sv_attn_desc* d, int which, int sms, Kv4Attn* p) {
  const int64_t rows = kv4_rows_per_head(d), max_tiles = kv4_max_tiles(d);
  const int ctas = which == 2 ? sms : attn_kv4_ctas(sms);
  p->mr = which == 2 ? MT : attn_kv4_rows((int)rows);
  p->switch_tiles = which == 2 ? SWITCH_TILES_KV4 : SWITCH_TILES_KV4_MMA;
  p->join_tiles = which == 2 ? JOIN_TILES_KV4 : JOIN_TILES_KV4_MMA;
  const int64_t row_tiles = (rows + p->mr - 1) / p->mr;
  const int64_t heads = (int64_t)d->batch * d->num_kv_heads;
  const bool shrt = which == 1 && max_tiles <= 2 * KV4_SHORT_TILES;
  const bool pair = which == 2 ? true
                    : shrt     ? heads * row_tiles >= KV4_PAIR_UNITS_SHORT
                               : heads >= KV4_PAIR_UNITS;
  p->heads = d->num_kv_heads % 2 == 0 && pair ? 2 : 1;
  const int64_t units = heads / p->heads * row_tiles;
  // (at most 8 units' time a CTA: with more the ranges of several units cost less)
  p->no_join = shrt && units <= 8 * (int64_t)ctas &&
               (max_tiles <= KV4_SHORT_TILES || 2 * units >= ctas);
  if (p->no_join) {
    p->n_ctas = (int)units;
    p->join_tiles = 2 * KV4_SHORT_TILES;  // (no unit is longer)
  } else {
    p->n_ctas = (int)std::min<int64_t>(units * max_tiles, which == 2 ? ctas / p->heads : ctas);
  }
}

struct Kv4Ws {
  size_t part_o, part_ml, total;
};
Kv4Ws kv4_layout(const sv_attn_desc* d, int sms) {
  // The parts of either kernel and any rule on its units, so that the workspace of a larger
  // shape serves a smaller one, under any sv_set_attn_kernel: at most two a range, its heads
  // (two) times rows of each.
  const size_t rows = std::max<size_t>(2 * (size_t)sms * MT, 2 * (size_t)attn_kv4_ctas(sms) * 2 * 16);
  Kv4Ws w;
  w.part_o = 256;
  w.part_ml = w.part_o + rows * d->head_dim * sizeof(float);
  w.total = w.part_ml + rows * sizeof(float2);
  return w;
}

}  // namespace

extern "C" {

SV_API size_t spec_kv4_workspace_size(int32_t batch) { return batch < 0 ? 0 : 256; }

SV_API sv_status spec_kv4_write(const sv_kv4_pages* pages, int32_t batch,
                                const int32_t* block_table, int32_t max_blocks_per_seq,
                                const int32_t* start, const int32_t* count, int64_t rows,
                                const void* k, int64_t k_row_stride, const void* v,
                                int64_t v_row_stride, void* workspace, size_t workspace_bytes,
                                void* stream) {
  const sv_status st = check_kv4_rows(pages, batch, block_table, max_blocks_per_seq, start, count,
                                      rows, k, v, workspace, workspace_bytes);
  if (st != SV_OK || batch == 0 || rows == 0) return st;
  const int64_t width = (int64_t)pages->num_kv_heads * pages->head_dim;
  for (const int64_t s : {k_row_stride, v_row_stride})
    if (s < width || s % 8 != 0 || s > ((int64_t)1 << 30)) return SV_ERR_SHAPE;
  if (!kv4_apart(pages, k, 2 * (size_t)((rows - 1) * k_row_stride + width)) ||
      !kv4_apart(pages, v, 2 * (size_t)((rows - 1) * v_row_stride + width)))
    return SV_ERR_SHAPE;
  const int sms = current_sms();
  if (sms <= 0) return SV_ERR_CUDA;
  return launch_kv4_write(*pages, batch, block_table, max_blocks_per_seq, start, count, rows, k,
                          k_row_stride, v, v_row_stride, workspace, sms,
                          (cudaStream_t)stream) == cudaSuccess
             ? SV_OK
             : SV_ERR_CUDA;
}

SV_API sv_status spec_kv4_read(const sv_kv4_pages* pages, int32_t batch,
                               const int32_t* block_table, int32_t max_blocks_per_seq,
                               const int32_t* start, const int32_t* count, int64_t rows,
                               void* k_out, void* v_out, void* workspace, size_t workspace_bytes,
                               void* stream) {
  const sv_status st = check_kv4_rows(pages, batch, block_table, max_blocks_per_seq, start, count,
                                      rows, k_out, v_out, workspace, workspace_bytes);
  if (st != SV_OK || batch == 0 || rows == 0) return st;
  const size_t bytes = 2 * (size_t)rows * pages->num_kv_heads * pages->head_dim;
  if (!kv4_apart(pages, k_out, bytes) || !kv4_apart(pages, v_out, bytes) ||
      meet(k_out, bytes, v_out, bytes))
    return SV_ERR_SHAPE;
  const int sms = current_sms();
  if (sms <= 0) return SV_ERR_CUDA;
  return launch_kv4_read(*pages, batch, block_table, max_blocks_per_seq, start, count, rows, k_out,
                         v_out, workspace, sms, (cudaStream_t)stream) == cudaSuccess
             ? SV_OK
             : SV_ERR_CUDA;
}

SV_API size_t spec_verify_attn_kv4_workspace_size(const sv_attn_desc* desc) {
  if (check_desc_kv4(desc) != SV_OK || desc->kv_dtype != SV_KV4) return 0;
  const int sms = current_sms();
  return sms <= 0 ? 0 : kv4_layout(desc, sms).total;
}

SV_API sv_status spec_verify_attn_kv4(const sv_attn_desc* desc, const void* q,
                                      const sv_kv4_pages* pages, const int32_t* block_table,
                                      int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                      const int32_t* draft_len, void* out, float* lse,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  sv_status st = check_desc_kv4(desc);
  if (st != SV_OK) return st;
  if (desc->kv_dtype != SV_KV4) return SV_ERR_DTYPE;
  st = check_kv4(pages);
  if (st != SV_OK) return st;
  // (rows of q and heads together are indexed with 32 bits)
  if (pages->num_kv_heads != desc->num_kv_heads || pages->head_dim != desc->head_dim ||
      max_blocks_per_seq < 1 || desc->q_rows > 0x7fffffff / desc->num_q_heads)
    return SV_ERR_SHAPE;
  if (desc->batch == 0) return SV_OK;
  if (!q || !block_table || !seq_lens || !draft_len || !out || !workspace) return SV_ERR_NULL;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(block_table, 4) ||
      !aligned(seq_lens, 4) || !aligned(draft_len, 4) || !aligned(workspace, 256))
    return SV_ERR_ALIGN;
  const int sms = current_sms();
  if (sms <= 0) return SV_ERR_CUDA;
  const Kv4Ws lay = kv4_layout(desc, sms);
  if (workspace_bytes < lay.total) return SV_ERR_WORKSPACE;

  const int which = pick_kv4(desc);
  uint8_t* ws = (uint8_t*)workspace;
  Kv4Attn p = {};
  p.q = q;
  p.k = pages->k_codes;
  p.v = pages->v_codes;
  p.scales = pages->scales;
  p.kv_scale = pages->kv_scale;
  p.seq_lens = seq_lens;
  p.draft_len = draft_len;
  p.block_table = block_table;
  p.out = out;
  p.lse = lse;
  p.flags = (uint32_t*)ws;
  p.part_o = (float*)(ws + lay.part_o);
  p.part_ml = (float2*)(ws + lay.part_ml);
  p.B = desc->batch;
  p.Hq = desc->num_q_heads;
  p.Hkv = desc->num_kv_heads;
  p.G = p.Hq / p.Hkv;
  p.d = desc->head_dim;
  p.max_draft = desc->max_draft_len;
  p.max_seq = desc->max_seq_len;
  // a window covering every position of the longest sequence is no window
  p.window = (int64_t)desc->sliding_window > (int64_t)desc->max_seq_len + desc->max_draft_len
                 ? 0
                 : desc->sliding_window;
  p.bt_stride = max_blocks_per_seq;
  p.block_size = pages->block_size;
  while ((1 << p.bs_log2) < p.block_size) ++p.bs_log2;
  p.num_blocks = pages->num_blocks;
  p.q_rows = desc->q_rows;
  p.scale_log2 = scale_log2_of(desc);
  kv4_line(desc, which, sms, &p);
  if (which == 2) {  // a pending wait-timeout injection applies to this launch
    p.wait_limit = g_stall_limit.exchange(0);
    p.stall_first_tile = p.wait_limit > 0;
  }
  cudaStream_t s = (cudaStream_t)stream;
  if (g_ev_start && cudaEventRecord(g_ev_start, s) != cudaSuccess) return SV_ERR_CUDA;
  if ((which == 2 ? launch_attn_kv4_tc(p, s) : launch_attn_kv4(p, s)) != cudaSuccess)
    return SV_ERR_CUDA;
  if (g_ev_stop && cudaEventRecord(g_ev_stop, s) != cudaSuccess) return SV_ERR_CUDA;
  if (p.no_join) return SV_OK;
  return launch_kv4_join(p, sms, s) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

SV_API size_t spec_attn_mass_workspace_size(const sv_attn_desc* desc) {
  if (check_desc_kv4(desc) != SV_OK) return 0;
  const int sms = current_sms();
  return sms <= 0 ? 0 : mass_ws_bytes(desc, sms);
}

SV_API sv_status spec_attn_mass(const sv_attn_desc* desc, const void* q, const void* k_pages,
                                const void* scales, const float* kv_scale, int64_t num_blocks,
                                int32_t block_size, const int32_t* block_table,
                                int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                const int32_t* draft_len, const int32_t* row_count,
                                const float* lse, float* mass, int64_t mass_stride,
                                void* workspace, size_t workspace_bytes, void* stream) {
  const sv_status st = check_desc_kv4(desc);
  if (st != SV_OK) return st;
  if (num_blocks < 1 || num_blocks > 0x7fffffff || !pool_sizes_ok((int32_t)num_blocks, block_size) ||
      max_blocks_per_seq < 1 || desc->sliding_window != 0 || mass_stride < 1 ||
      mass_stride > ((int64_t)1 << 40))
    return SV_ERR_SHAPE;
  if (desc->batch == 0) return SV_OK;
  if (!q || !k_pages || !block_table || !seq_lens || !draft_len || !mass || !workspace)
    return SV_ERR_NULL;
  if ((desc->kv_dtype == SV_KV4 && !scales) || (desc->kv_dtype != SV_BF16 && !kv_scale))
    return SV_ERR_NULL;
  if ((desc->kv_dtype != SV_KV4 && scales) || (desc->kv_dtype == SV_BF16 && kv_scale))
    return SV_ERR_SHAPE;
  if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(scales, 16) || !aligned(kv_scale, 4) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(draft_len, 4) ||
      !aligned(row_count, 4) || !aligned(lse, 4) || !aligned(mass, 4) || !aligned(workspace, 256))
    return SV_ERR_ALIGN;
  const int sms = current_sms();
  if (sms <= 0) return SV_ERR_CUDA;
  if (workspace_bytes < mass_ws_bytes(desc, sms)) return SV_ERR_WORKSPACE;
  return launch_mass(desc, scale_log2_of(desc), q, k_pages, scales, kv_scale, num_blocks, block_size,
                     block_table, max_blocks_per_seq, seq_lens, draft_len, row_count, lse, mass,
                     mass_stride, workspace, sms, (cudaStream_t)stream) == cudaSuccess
             ? SV_OK
             : SV_ERR_CUDA;
}

SV_API size_t spec_kv_evict_workspace_size(int32_t n, int32_t num_kv_heads, int64_t mass_stride) {
  // (positions and those that a CTA looks ahead to are 32 bits)
  if (n < 0 || n > SV_MAX_EVICT_ROWS || num_kv_heads < 1 || num_kv_heads > 4096 || mass_stride < 1 ||
      mass_stride > (int64_t)1 << 30)
    return 0;
  return evict_ws_bytes(n, num_kv_heads, mass_stride);
}

SV_API sv_status spec_kv_evict(const sv_page_table* table, int32_t n, const int32_t* rows,
                               const int32_t* new_len, const int32_t* keep_first,
                               int32_t keep_last, int32_t num_kv_heads, float* mass,
                               int64_t mass_stride, int32_t* kept, int64_t kept_stride,
                               int32_t num_pools, const sv_page_data* pools, void* workspace,
                               size_t workspace_bytes, void* stream) {
  // (the page operators' checks, whose own workspace size does not apply)
  sv_status st = check_pages(table, n, workspace, ~(size_t)0);
  if (st == SV_OK) st = check_pools(table, num_pools, pools);
  if (st != SV_OK) return st;
  const size_t need = spec_kv_evict_workspace_size(n, num_kv_heads, mass_stride);
  if (need == 0 || keep_last < 0 || (kept && (kept_stride < 0 || kept_stride > (int64_t)1 << 30)))
    return SV_ERR_SHAPE;
  // (the sizes below stay within 63 bits)
  if ((int64_t)table->table_rows * num_kv_heads > ((int64_t)1 << 60) / mass_stride) return SV_ERR_SHAPE;
  int64_t slices = 1;
  for (int k = 0; k < num_pools; ++k) {
    const int64_t pos = pools[k].page_bytes / table->block_size;
    if (pos % (8 * (int64_t)num_kv_heads) != 0) return SV_ERR_SHAPE;
    slices += (pos / num_kv_heads + 31) / 32;  // (at most: evict.cu, SLICE)
  }
  if (n * (int64_t)num_kv_heads * slices > 0x7fffffff) return SV_ERR_SHAPE;
  if (n == 0) return SV_OK;
  if (!new_len || !mass) return SV_ERR_NULL;
  if (!aligned(rows, 4) || !aligned(new_len, 4) || !aligned(keep_first, 4) || !aligned(mass, 4) ||
      !aligned(kept, 4))
    return SV_ERR_ALIGN;
  if (workspace_bytes < need) return SV_ERR_WORKSPACE;
  // what the call changes and what it reads must be apart
  const size_t list = 4 * (size_t)n;
  const Span spans[] = {
      {workspace, need},
      {mass, 4 * (size_t)table->table_rows * num_kv_heads * mass_stride},
      {kept, 4 * (size_t)n * num_kv_heads * kept_stride},
      {rows, list},
      {new_len, list},
      {keep_first, list},
      {table->ref_count, 4 * (size_t)table->num_blocks},
      {table->block_table, 4 * (size_t)table->table_rows * table->max_blocks_per_seq},
      {table->cached_len, 4 * (size_t)table->table_rows}};
  const int ns = (int)(sizeof spans / sizeof spans[0]);
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < ns; ++j)
      if (meet(spans[i].at, spans[i].bytes, spans[j].at, spans[j].bytes)) return SV_ERR_SHAPE;
  for (int k = 0; k < num_pools; ++k) {
    const size_t bytes = (size_t)pools[k].page_bytes * table->num_blocks;
    for (int j = 0; j < ns; ++j)
      if (meet(pools[k].base, bytes, spans[j].at, spans[j].bytes)) return SV_ERR_SHAPE;
    for (int l = 0; l < k; ++l)
      if (meet(pools[k].base, bytes, pools[l].base, (size_t)pools[l].page_bytes * table->num_blocks))
        return SV_ERR_SHAPE;
  }
  return launch_evict(*table, n, rows, new_len, keep_first, keep_last, num_kv_heads, mass,
                      mass_stride, kept, kept_stride, num_pools, pools, workspace,
                      (cudaStream_t)stream) == cudaSuccess
             ? SV_OK
             : SV_ERR_CUDA;
}

}  // extern "C"

extern "C" {

SV_API size_t spec_accept_workspace_size(int32_t batch, int32_t max_draft_len, int32_t vocab) {
  if (batch < 0 || max_draft_len < 0 || max_draft_len > 255 || vocab <= 0) return 0;
  const int sms = current_sms();
  if (sms <= 0) return 0;
  return accept_ws_layout(batch, max_draft_len, vocab, sms).total;
}

SV_API sv_status spec_accept(int32_t batch, int32_t max_draft_len, int32_t vocab,
                             int32_t logits_dtype, const void* logits,
                             const int32_t* draft_tokens, const int32_t* draft_len,
                             int32_t* accept_len, int32_t* next_token, int32_t* target_tokens,
                             void* workspace, size_t workspace_bytes, void* stream) {
  if (batch < 0 || max_draft_len < 0 || max_draft_len > 255 || vocab <= 0) return SV_ERR_SHAPE;
  if (logits_dtype != SV_BF16 && logits_dtype != SV_FP32) return SV_ERR_DTYPE;
  if (batch == 0) return SV_OK;
  if (!logits || !draft_len || !accept_len || !next_token || !workspace) return SV_ERR_NULL;
  if (max_draft_len > 0 && !draft_tokens) return SV_ERR_NULL;
  const uintptr_t es = logits_dtype == SV_BF16 ? 2 : 4;
  if (!aligned(logits, es) || !aligned(draft_len, 4) || !aligned(accept_len, 4) ||
      !aligned(next_token, 4) || (draft_tokens && !aligned(draft_tokens, 4)) ||
      (target_tokens && !aligned(target_tokens, 4)) || !aligned(workspace, 256))
    return SV_ERR_ALIGN;
  const int sms = current_sms();
  if (sms <= 0) return SV_ERR_CUDA;
  const AcceptWs lay = accept_ws_layout(batch, max_draft_len, vocab, sms);
  if (workspace_bytes < lay.total) return SV_ERR_WORKSPACE;
  const cudaError_t e = launch_accept(batch, max_draft_len, vocab, logits_dtype, logits,
                                      draft_tokens, draft_len, accept_len, next_token,
                                      target_tokens, workspace, lay, (cudaStream_t)stream);
  return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

SV_API size_t spec_accept_stochastic_workspace_size(int32_t batch, int32_t max_draft_len,
                                                   int32_t vocab) {
  if (batch < 0 || max_draft_len < 0 || max_draft_len > 255 || vocab <= 0 ||
      vocab > (1 << 30))
    return 0;
  return 256;  // the flag word
}

SV_API sv_status spec_accept_stochastic(int32_t batch, int32_t max_draft_len, int32_t vocab,
                                        int32_t logits_dtype, const void* target_logits,
                                        const void* draft_logits, const int32_t* draft_tokens,
                                        const int32_t* draft_len, const float* u_accept,
                                        const float* u_sample, float temperature,
                                        int32_t* accept_len, int32_t* next_token,
                                        void* workspace, size_t workspace_bytes, void* stream) {
  if (batch < 0 || max_draft_len < 0 || max_draft_len > 255 || vocab <= 0 ||
      vocab > (1 << 30) || !(temperature > 0.f) || isinf(temperature))
    return SV_ERR_SHAPE;
  if (logits_dtype != SV_BF16 && logits_dtype != SV_FP32) return SV_ERR_DTYPE;
  if (batch == 0) return SV_OK;
  if (!target_logits || !draft_len || !u_sample || !accept_len || !next_token || !workspace)
    return SV_ERR_NULL;
  if (max_draft_len > 0 && (!draft_logits || !draft_tokens || !u_accept)) return SV_ERR_NULL;
  const uintptr_t es = logits_dtype == SV_BF16 ? 2 : 4;
  if (!aligned(target_logits, es) || (draft_logits && !aligned(draft_logits, es)) ||
      !aligned(draft_len, 4) || (draft_tokens && !aligned(draft_tokens, 4)) ||
      (u_accept && !aligned(u_accept, 4)) || !aligned(u_sample, 4) ||
      !aligned(accept_len, 4) || !aligned(next_token, 4) || !aligned(workspace, 256))
    return SV_ERR_ALIGN;
  if (workspace_bytes < 256) return SV_ERR_WORKSPACE;
  const cudaError_t e = launch_accept_stochastic(
      batch, max_draft_len, vocab, logits_dtype, target_logits, draft_logits, draft_tokens,
      draft_len, u_accept, u_sample, 1.f / temperature, accept_len, next_token, workspace,
      (cudaStream_t)stream);
  return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

SV_API size_t spec_draft_signals_workspace_size(int32_t rows, int32_t vocab) {
  if (rows < 0 || vocab <= 0) return 0;
  const int sms = current_sms();
  if (sms <= 0) return 0;
  return signals_ws_layout(rows, vocab, sms).total;
}

SV_API sv_status spec_draft_signals(int32_t rows, int32_t vocab, int32_t logits_dtype,
                                    const void* logits, float* confidence, float* entropy,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  if (rows < 0 || vocab <= 0) return SV_ERR_SHAPE;
  if (logits_dtype != SV_BF16 && logits_dtype != SV_FP32) return SV_ERR_DTYPE;
  if (rows == 0) return SV_OK;
  if (!logits || !confidence || !entropy || !workspace) return SV_ERR_NULL;
  const uintptr_t es = logits_dtype == SV_BF16 ? 2 : 4;
  if (!aligned(logits, es) || !aligned(confidence, 4) || !aligned(entropy, 4) ||
      !aligned(workspace, 256))
    return SV_ERR_ALIGN;
  const int sms = current_sms();
  if (sms <= 0) return SV_ERR_CUDA;
  const SigWs lay = signals_ws_layout(rows, vocab, sms);
  if (workspace_bytes < lay.total) return SV_ERR_WORKSPACE;
  const cudaError_t e = launch_signals(rows, vocab, logits_dtype, logits, confidence, entropy,
                                       workspace, lay, (cudaStream_t)stream);
  return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

SV_API sv_status sv_workspace_status(void* workspace, int clear, void* stream) {
  if (!workspace) return SV_ERR_NULL;
  cudaStream_t s = (cudaStream_t)stream;
  uint32_t flags = 0;
  if (cudaMemcpyAsync(&flags, workspace, sizeof flags, cudaMemcpyDeviceToHost, s) != cudaSuccess)
    return SV_ERR_CUDA;
  if (clear && cudaMemsetAsync(workspace, 0, sizeof flags, s) != cudaSuccess) return SV_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return SV_ERR_CUDA;
  if (flags & FLAG_TIMEOUT) return SV_ERR_TIMEOUT;
  if (flags & (FLAG_ATTN_SHAPE | FLAG_ACCEPT_SHAPE | FLAG_PAGES_SHAPE)) return SV_ERR_DEVICE_SHAPE;
  if (flags & FLAG_NO_PAGES) return SV_ERR_NO_PAGES;
  return SV_OK;
}

}  // extern "C"
