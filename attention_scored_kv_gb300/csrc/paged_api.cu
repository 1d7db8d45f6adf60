// The C ABI of the paged cache: argument checks, workspace and scratch plans, dispatch.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <new>
#include <string>

#include "paged.cuh"
#include "paged_cut.h"
#include "trace.cuh"

using namespace kvs;

struct kvs_paged {
  kvs_paged_config cfg;
  PagedDev dev;
  int device = 0, sms = 0;
  bool tensor = false;
  std::string err;
};

namespace {

constexpr int32_t kMaxStride = kMaxTableStride, kMaxReqs = 1 << 20;   // of block tables

void put(char* msg, size_t n, const char* fmt, ...) {
  if (!msg || n == 0) return;
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, n, fmt, ap);
  va_end(ap);
}

kvs_status fail(kvs_paged* pc, kvs_status st, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  try {
    pc->err = buf;
  } catch (...) {
  }
  return st;
}

kvs_status cuda_ok(kvs_paged* pc, cudaError_t e, const char* what) {
  if (e == cudaSuccess) return KVS_OK;
  return fail(pc, KVS_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// The context's device for the length of a call.
struct OnDevice {
  explicit OnDevice(int device) {
    if (cudaGetDevice(&before) != cudaSuccess) { ok = false; return; }
    if (before != device) { ok = cudaSetDevice(device) == cudaSuccess; moved = ok; }
  }
  ~OnDevice() {
    if (moved) cudaSetDevice(before);
  }
  OnDevice(const OnDevice&) = delete;
  OnDevice& operator=(const OnDevice&) = delete;
  int before = 0;
  bool ok = true, moved = false;
};

bool tensor_shape(const kvs_paged_config* c) {
  return c->in_dtype == KVS_BF16 && (c->head_dim == 64 || c->head_dim == 128);
}

kvs_status check_config(const kvs_paged_config* c, char* msg, size_t n) {
  if (!c) { put(msg, n, "config is NULL"); return KVS_ERR_INVALID_ARGUMENT; }
  if (c->num_layers < 1) { put(msg, n, "num_layers must be >= 1"); return KVS_ERR_INVALID_ARGUMENT; }
  if (c->num_q_heads < 1 || c->num_kv_heads < 1 || c->num_q_heads % c->num_kv_heads) {
    put(msg, n, "num_q_heads must be a positive multiple of num_kv_heads");
    return KVS_ERR_INVALID_ARGUMENT;
  }
  if (c->num_kv_heads > 1024 || c->num_q_heads / c->num_kv_heads > kMaxGroup) {
    put(msg, n, "at most 1024 KV heads and %d query heads per KV head", kMaxGroup);
    return KVS_ERR_UNSUPPORTED;
  }
  if (c->head_dim != 16 && c->head_dim != 32 && c->head_dim != 64 && c->head_dim != 128) {
    put(msg, n, "head_dim must be 16, 32, 64 or 128");
    return KVS_ERR_UNSUPPORTED;
  }
  if (c->num_pages < 1) { put(msg, n, "num_pages must be >= 1"); return KVS_ERR_INVALID_ARGUMENT; }
  if (c->num_pages >= (1 << 27)) { put(msg, n, "num_pages must be below 2^27"); return KVS_ERR_UNSUPPORTED; }
  if (c->block_tokens != kBlock) { put(msg, n, "block_tokens must be 16"); return KVS_ERR_UNSUPPORTED; }
  if (c->in_dtype != KVS_F32 && c->in_dtype != KVS_BF16) { put(msg, n, "in_dtype must be F32 or BF16"); return KVS_ERR_INVALID_ARGUMENT; }
  if (c->kernel < KVS_KERNEL_AUTO || c->kernel > KVS_KERNEL_TENSOR) { put(msg, n, "kernel must be a kvs_kernel"); return KVS_ERR_INVALID_ARGUMENT; }
  for (int i = 0; i < 8; ++i)
    if (c->reserved[i]) { put(msg, n, "reserved fields must be 0"); return KVS_ERR_INVALID_ARGUMENT; }
  if (c->kernel == KVS_KERNEL_TENSOR && !tensor_shape(c)) {
    put(msg, n, "the tensor-core attend needs bf16 inputs and head_dim 64 or 128");
    return KVS_ERR_UNSUPPORTED;
  }
  return KVS_OK;
}

size_t up(size_t x) { return (x + 255) & ~(size_t)255; }

struct Workspace {
  size_t codes, scales;            // bytes of one layer's codes of K (and of V), and of its scales
  size_t k, v, s, err, total;
};
Workspace workspace_of(const kvs_paged_config* c) {
  Workspace w;
  w.codes = (size_t)c->num_pages * c->num_kv_heads * 16 * c->head_dim;
  w.scales = (size_t)c->num_pages * c->num_kv_heads * sizeof(float2);
  w.k = 0;
  w.v = w.k + up(w.codes * c->num_layers);
  w.s = w.v + up(w.codes * c->num_layers);
  w.err = w.s + up(w.scales * c->num_layers);
  w.total = w.err + 256;
  return w;
}

// How an attend call runs; a function of host-known sizes only.
PagedAttendPlan plan_attend(const kvs_paged* pc, int n_reqs, int stride, int total_q, int max_q_len, bool mass) {
  PagedAttendPlan p = {};
  const PagedDev& d = pc->dev;
  size_t recs = 0;
  // The decode kernel's cost grows with its query rows, the prompt kernel's does not until 128.  32/4 heads of
  // 128, decode against prompt: 16 rows 29 against 39 us (16 x 4096 tokens) and 24 against 33 (1 x 32768); 32 rows
  // 57 against 39, 253 against 177 (16 x 32768) and 87 against 46 (64 x 1000).  Block masses are the decode kernel's.
  const long long need = (long long)max_q_len * d.G;       // query rows of a unit
  p.splits = 1;
  if (pc->tensor && (need <= 16 || (mass && need <= 32))) {
    p.kernel = PagedAttendPlan::kDecode;
    p.rows = need <= 8 ? 8 : need <= 16 ? 16 : 32;
    p.grid = paged_decode_ctas_per_sm() * pc->sms;
    recs = (size_t)2 * p.grid * p.rows;                    // a CTA leaves at most two partials
  } else if (pc->tensor && !mass) {
    p.kernel = PagedAttendPlan::kPrompt;
    p.grid = pc->sms;
    recs = (size_t)2 * p.grid * paged_prompt_rows();
  } else {
    p.kernel = PagedAttendPlan::kGeneral;
    // a part per idle CTA, four CTAs to an SM, no part under a page a warp
    const long long units = (long long)total_q * d.Hkv;
    long long want = units > 0 ? (long long)pc->sms * 4 / units : 1;
    if (want > 64) want = 64;
    if (want > stride / 4) want = stride / 4;
    p.splits = want < 1 ? 1 : (int)want;
    if (p.splits > 1) recs = (size_t)total_q * d.Hq * p.splits;
  }
  p.part_o = 0;
  p.part_ml = p.part_o + up(recs * d.D * sizeof(float));
  p.blk = p.part_ml + up(recs * sizeof(float2));
  p.lse = p.blk + (mass ? up((size_t)n_reqs * stride * d.Hq * sizeof(float)) : 0);
  p.q_pieces = p.lse + (mass ? up((size_t)n_reqs * d.Hq * sizeof(float)) : 0);
  const size_t tiles = p.kernel == PagedAttendPlan::kPrompt ? (size_t)paged_prompt_tiles(d.G, n_reqs, total_q) * d.Hkv : 0;
  p.q_factors = p.q_pieces + up(tiles * paged_prompt_tile_bytes(d.D));
  p.cuts = p.q_factors + up(tiles * (paged_prompt_rows() / 2) * sizeof(float));
  p.total = p.cuts + up((size_t)p.grid * 32);
  return p;
}

// Whether a CTA's share of the work stays within 32 bits.
bool work_fits(const kvs_paged* pc, int n_reqs, int stride, int total_q, int max_q_len, bool mass) {
  const PagedAttendPlan p = plan_attend(pc, n_reqs, stride, total_q, max_q_len, mass);
  const long long per = paged_prompt_rows() / pc->dev.G;
  return p.kernel == PagedAttendPlan::kGeneral ||
         cut::share_fits(p.kernel == PagedAttendPlan::kDecode ? n_reqs : total_q / per + n_reqs, stride, pc->dev.Hkv, p.grid);
}

kvs_status check_attend(kvs_paged* pc, int32_t n_reqs, int32_t table_stride, int32_t total_q, int32_t max_q_len,
                        bool mass) {
  if (n_reqs < 1 || n_reqs > kMaxReqs)
    return fail(pc, KVS_ERR_INVALID_ARGUMENT, "n_reqs must be in [1, 2^20] (got %d)", n_reqs);
  if (table_stride < 1 || table_stride > kMaxStride)
    return fail(pc, KVS_ERR_INVALID_ARGUMENT, "table_stride must be in [1, 2^22] (got %d)", table_stride);
  if (total_q < 0 || max_q_len < 1 || total_q > (1 << 28))
    return fail(pc, KVS_ERR_INVALID_ARGUMENT, "total_q must be in [0, 2^28] and max_q_len >= 1 (got %d, %d)", total_q,
                max_q_len);
  if (mass && max_q_len != 1)
    return fail(pc, KVS_ERR_UNSUPPORTED, "block masses need single-token queries (max_q_len 1, got %d)", max_q_len);
  if (!work_fits(pc, n_reqs, table_stride, total_q, max_q_len, mass))
    return fail(pc, KVS_ERR_UNSUPPORTED, "%d rows over tables of %d blocks are too much for one call: split the rows", total_q,
                table_stride);
  return KVS_OK;
}

bool unaligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) & (to - 1); }

}  // namespace

#define ENTER(name)                                                                        \
  Trace trace_(name);                                                                      \
  if (!pc) return KVS_ERR_INVALID_ARGUMENT;                                                \
  const OnDevice on_(pc->device);                                                          \
  if (!on_.ok) return fail(pc, KVS_ERR_CUDA, "cannot use device %d", pc->device)

extern "C" {

void kvs_paged_config_init(kvs_paged_config* cfg) {
  Trace trace_("kvs_paged_config_init");
  if (!cfg) return;
  std::memset(cfg, 0, sizeof *cfg);
  cfg->block_tokens = kBlock;
  cfg->in_dtype = KVS_BF16;
}

kvs_status kvs_paged_validate_config(const kvs_paged_config* cfg, char* msg, size_t msg_len) {
  Trace trace_("kvs_paged_validate_config");
  if (msg && msg_len) msg[0] = 0;
  return check_config(cfg, msg, msg_len);
}

size_t kvs_paged_workspace_bytes(const kvs_paged_config* cfg) {
  Trace trace_("kvs_paged_workspace_bytes");
  return check_config(cfg, nullptr, 0) == KVS_OK ? workspace_of(cfg).total : 0;
}

kvs_status kvs_paged_create(const kvs_paged_config* cfg, void* d_workspace, size_t workspace_bytes,
                            kvs_stream_t stream, kvs_paged** out) {
  Trace trace_("kvs_paged_create");
  if (!out) return KVS_ERR_INVALID_ARGUMENT;
  *out = nullptr;
  const kvs_status st = check_config(cfg, nullptr, 0);
  if (st != KVS_OK) return st;
  const Workspace w = workspace_of(cfg);
  if (!d_workspace || unaligned(d_workspace, 256)) return KVS_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < w.total) return KVS_ERR_CAPACITY;
  kvs_paged* pc = new (std::nothrow) kvs_paged();
  if (!pc) return KVS_ERR_CAPACITY;
  pc->cfg = *cfg;
  if (cudaGetDevice(&pc->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&pc->sms, cudaDevAttrMultiProcessorCount, pc->device) != cudaSuccess ||
      cudaMemsetAsync(d_workspace, 0, w.total, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) {
    delete pc;
    return KVS_ERR_CUDA;
  }
  uint8_t* base = static_cast<uint8_t*>(d_workspace);
  PagedDev& d = pc->dev;
  d.L = cfg->num_layers;
  d.Hq = cfg->num_q_heads;
  d.Hkv = cfg->num_kv_heads;
  d.G = cfg->num_q_heads / cfg->num_kv_heads;
  d.D = cfg->head_dim;
  d.num_pages = cfg->num_pages;
  d.in_dtype = cfg->in_dtype;
  d.k = base + w.k;
  d.v = base + w.v;
  d.layer_bytes = w.codes;
  d.scales = reinterpret_cast<float2*>(base + w.s);
  d.layer_scales = w.scales / sizeof(float2);
  d.err = reinterpret_cast<int32_t*>(base + w.err);
  pc->tensor = cfg->kernel != KVS_KERNEL_GENERAL && tensor_shape(cfg);
  *out = pc;
  return KVS_OK;
}

kvs_status kvs_paged_destroy(kvs_paged* pc) {
  Trace trace_("kvs_paged_destroy");
  if (!pc) return KVS_ERR_INVALID_ARGUMENT;
  delete pc;
  return KVS_OK;
}

kvs_status kvs_paged_plan(kvs_paged* pc, int32_t n_reqs, const int32_t* d_ctx_len, const int32_t* d_new_len,
                          int32_t* d_block_table, int32_t table_stride, const int32_t* d_free_pages,
                          int32_t free_capacity, const int32_t* d_free_count_in, int32_t* d_free_count_out,
                          int32_t* d_row_start, int32_t* d_kv_len, int32_t* d_slots, int32_t* d_positions_opt,
                          int32_t row_capacity, int32_t* d_denied_opt, kvs_stream_t stream) {
  ENTER("kvs_paged_plan");
  if (n_reqs < 1 || n_reqs > kMaxReqs) return fail(pc, KVS_ERR_INVALID_ARGUMENT, "n_reqs must be in [1, 2^20] (got %d)", n_reqs);
  if (table_stride < 1 || table_stride > kMaxStride)
    return fail(pc, KVS_ERR_INVALID_ARGUMENT, "table_stride must be in [1, 2^22] (got %d)", table_stride);
  if (free_capacity < 0 || row_capacity < 0 || row_capacity > (1 << 30))
    return fail(pc, KVS_ERR_INVALID_ARGUMENT, "free_capacity and row_capacity must be >= 0, the latter at most 2^30");
  if (!d_ctx_len || !d_new_len || !d_block_table || !d_free_count_in || !d_free_count_out || !d_row_start || !d_kv_len ||
      (free_capacity && !d_free_pages) || (row_capacity && !d_slots))
    return fail(pc, KVS_ERR_INVALID_ARGUMENT, "a required array is NULL");
  if (d_kv_len == d_new_len || (row_capacity && d_slots == d_positions_opt))
    return fail(pc, KVS_ERR_INVALID_ARGUMENT, "kv_len may share memory with ctx_len only, slots with nothing");
  return cuda_ok(pc, launch_paged_plan(pc->dev, n_reqs, d_ctx_len, d_new_len, d_block_table, table_stride, d_free_pages,
                                       free_capacity, d_free_count_in, d_free_count_out, d_row_start, d_kv_len, d_slots,
                                       d_positions_opt, row_capacity, d_denied_opt, pc->sms,
                                       reinterpret_cast<cudaStream_t>(stream)), "plan");
}

kvs_status kvs_paged_slot_map(kvs_paged* pc, int32_t n_reqs, const int32_t* d_first_opt, const int32_t* d_len,
                              const int32_t* d_block_table, int32_t table_stride, int32_t* d_row_start,
                              int32_t* d_slots, int32_t* d_positions_opt, int32_t row_capacity, kvs_stream_t stream) {
  ENTER("kvs_paged_slot_map");
  if (n_reqs < 1 || n_reqs > kMaxReqs) return fail(pc, KVS_ERR_INVALID_ARGUMENT, "n_reqs must be in [1, 2^20] (got %d)", n_reqs);
  if (table_stride < 1 || table_stride > kMaxStride)
    return fail(pc, KVS_ERR_INVALID_ARGUMENT, "table_stride must be in [1, 2^22] (got %d)", table_stride);
  if (row_capacity < 0 || row_capacity > (1 << 30)) return fail(pc, KVS_ERR_INVALID_ARGUMENT, "row_capacity must be in [0, 2^30]");
  if (!d_len || !d_block_table || !d_row_start || (row_capacity && !d_slots) || (row_capacity && d_slots == d_positions_opt))
    return fail(pc, KVS_ERR_INVALID_ARGUMENT, "a required array is NULL, or slots and positions are one array");
  return cuda_ok(pc, launch_paged_slot_map(pc->dev, n_reqs, d_first_opt, d_len, d_block_table, table_stride, d_row_start,
                                           d_slots, d_positions_opt, row_capacity, pc->sms,
                                           reinterpret_cast<cudaStream_t>(stream)), "slot map");
}

kvs_status kvs_paged_release(kvs_paged* pc, int32_t n_reqs, const int32_t* d_kv_len, int32_t* d_block_table,
                             int32_t table_stride, int32_t* d_free_pages, int32_t free_capacity,
                             int32_t* d_free_count, kvs_stream_t stream) {
  ENTER("kvs_paged_release");
  if (n_reqs < 1 || n_reqs > kMaxReqs) return fail(pc, KVS_ERR_INVALID_ARGUMENT, "n_reqs must be in [1, 2^20] (got %d)", n_reqs);
  if (table_stride < 1 || table_stride > kMaxStride)
    return fail(pc, KVS_ERR_INVALID_ARGUMENT, "table_stride must be in [1, 2^22] (got %d)", table_stride);
  if (free_capacity < 0) return fail(pc, KVS_ERR_INVALID_ARGUMENT, "free_capacity must be >= 0");
  if (!d_kv_len || !d_block_table || !d_free_count || (free_capacity && !d_free_pages))
    return fail(pc, KVS_ERR_INVALID_ARGUMENT, "a required array is NULL");
  return cuda_ok(pc, launch_paged_release(pc->dev, n_reqs, d_kv_len, d_block_table, table_stride, d_free_pages,
                                          free_capacity, d_free_count, reinterpret_cast<cudaStream_t>(stream)), "release");
}

kvs_status kvs_paged_append(kvs_paged* pc, int32_t layer, int32_t n_rows, const int32_t* d_slots, const void* d_k,
                            const void* d_v, kvs_stream_t stream) {
  ENTER("kvs_paged_append");
  if (layer < 0 || layer >= pc->cfg.num_layers) return fail(pc, KVS_ERR_INVALID_ARGUMENT, "layer %d out of range", layer);
  if (n_rows < 0 || n_rows > (1 << 30)) return fail(pc, KVS_ERR_INVALID_ARGUMENT, "n_rows must be in [0, 2^30] (got %d)", n_rows);
  if (n_rows == 0) return KVS_OK;
  if (!d_slots || !d_k || !d_v) return fail(pc, KVS_ERR_INVALID_ARGUMENT, "slots, k and v must not be NULL");
  if (unaligned(d_k, 16) || unaligned(d_v, 16)) return fail(pc, KVS_ERR_INVALID_ARGUMENT, "k and v must be 16-byte aligned");
  return cuda_ok(pc, launch_paged_append(pc->dev, layer, n_rows, d_slots, d_k, d_v, reinterpret_cast<cudaStream_t>(stream)),
                 "append");
}

kvs_status kvs_paged_gather(kvs_paged* pc, int32_t layer, int32_t n_rows, const int32_t* d_slots, void* d_k, void* d_v,
                            kvs_stream_t stream) {
  ENTER("kvs_paged_gather");
  if (layer < 0 || layer >= pc->cfg.num_layers) return fail(pc, KVS_ERR_INVALID_ARGUMENT, "layer %d out of range", layer);
  if (n_rows < 0 || n_rows > (1 << 30)) return fail(pc, KVS_ERR_INVALID_ARGUMENT, "n_rows must be in [0, 2^30] (got %d)", n_rows);
  if (n_rows == 0) return KVS_OK;
  if (!d_slots || !d_k || !d_v) return fail(pc, KVS_ERR_INVALID_ARGUMENT, "slots, k and v must not be NULL");
  if (unaligned(d_k, 16) || unaligned(d_v, 16)) return fail(pc, KVS_ERR_INVALID_ARGUMENT, "k and v must be 16-byte aligned");
  return cuda_ok(pc, launch_paged_gather(pc->dev, layer, n_rows, d_slots, d_k, d_v, reinterpret_cast<cudaStream_t>(stream)),
                 "gather");
}

size_t kvs_paged_attend_scratch_bytes(const kvs_paged* pc, int32_t n_reqs, int32_t table_stride, int32_t total_q,
                                      int32_t max_q_len, int32_t block_mass) {
  Trace trace_("kvs_paged_attend_scratch_bytes");
  if (!pc || n_reqs < 1 || n_reqs > kMaxReqs || table_stride < 1 || table_stride > kMaxStride || total_q < 0 || total_q > (1 << 28) ||
      max_q_len < 1 || (block_mass && max_q_len != 1) ||
      !work_fits(pc, n_reqs, table_stride, total_q, max_q_len, block_mass != 0))
    return 0;
  const size_t n = plan_attend(pc, n_reqs, table_stride, total_q, max_q_len, block_mass != 0).total;
  return n ? n : 256;
}

kvs_status kvs_paged_attend(kvs_paged* pc, int32_t layer, int32_t n_reqs, const int32_t* d_block_table,
                            int32_t table_stride, const int32_t* d_kv_len, const int32_t* d_row_start, int32_t total_q,
                            int32_t max_q_len, int32_t window, const void* d_q, void* d_out, float* d_block_mass_opt,
                            void* d_scratch, size_t scratch_bytes, kvs_stream_t stream) {
  ENTER("kvs_paged_attend");
  if (layer < 0 || layer >= pc->cfg.num_layers) return fail(pc, KVS_ERR_INVALID_ARGUMENT, "layer %d out of range", layer);
  const kvs_status st = check_attend(pc, n_reqs, table_stride, total_q, max_q_len, d_block_mass_opt != nullptr);
  if (st != KVS_OK) return st;
  if (window < 0) return fail(pc, KVS_ERR_INVALID_ARGUMENT, "window must be >= 0 (0 = none)");
  if (!d_row_start && (max_q_len != 1 || total_q != n_reqs))
    return fail(pc, KVS_ERR_INVALID_ARGUMENT, "without row_start there is one row per request (total_q %d, n_reqs %d, "
                                              "max_q_len %d)", total_q, n_reqs, max_q_len);
  if (total_q == 0) return KVS_OK;
  if (!d_block_table || !d_kv_len || !d_q || !d_out || !d_scratch)
    return fail(pc, KVS_ERR_INVALID_ARGUMENT, "a required array is NULL");
  if (unaligned(d_q, 16) || unaligned(d_out, 16) || unaligned(d_scratch, 256) || unaligned(d_block_mass_opt, 4))
    return fail(pc, KVS_ERR_INVALID_ARGUMENT, "q and out must be 16-byte aligned, scratch 256-byte aligned");
  if (d_q == d_out) return fail(pc, KVS_ERR_INVALID_ARGUMENT, "q and out must not be the same array");
  const PagedAttendPlan p = plan_attend(pc, n_reqs, table_stride, total_q, max_q_len, d_block_mass_opt != nullptr);
  if (scratch_bytes < p.total)
    return fail(pc, KVS_ERR_CAPACITY, "scratch of %zu bytes, %zu needed", scratch_bytes, p.total);
  uint8_t* s = static_cast<uint8_t*>(d_scratch);
  PagedAttend a = {};
  a.d = pc->dev;
  a.layer = layer;
  a.n_reqs = n_reqs;
  a.table_stride = table_stride;
  a.total_q = total_q;
  a.max_q_len = max_q_len;
  a.window = window < table_stride * kBlock ? window : 0;     // a longer one hides nothing
  a.table = d_block_table;
  a.kv_len = d_kv_len;
  a.row_start = d_row_start;
  a.q = d_q;
  a.out = d_out;
  a.mass = d_block_mass_opt;
  a.part_o = reinterpret_cast<float*>(s + p.part_o);
  a.part_ml = reinterpret_cast<float2*>(s + p.part_ml);
  a.blk = d_block_mass_opt ? reinterpret_cast<float*>(s + p.blk) : nullptr;
  a.lse = d_block_mass_opt ? reinterpret_cast<float*>(s + p.lse) : nullptr;
  a.splits = p.splits;
  a.q_pieces = s + p.q_pieces;
  a.q_factors = reinterpret_cast<float*>(s + p.q_factors);
  a.cuts = reinterpret_cast<int32_t*>(s + p.cuts);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
#ifdef KVS_DEBUG
  // what the kernels read of the scratch they have written: partials start as NaN, cuts as -1
  if (cudaMemsetAsync(d_scratch, 0xFF, p.total, cs) != cudaSuccess) return cuda_ok(pc, cudaGetLastError(), "attend");
#endif
  cudaError_t e = p.kernel == PagedAttendPlan::kDecode   ? launch_paged_decode(a, p.rows, p.grid, cs)
                  : p.kernel == PagedAttendPlan::kPrompt ? launch_paged_prompt(a, p.grid, cs)
                                                         : launch_paged_general(a, cs);
  if (e == cudaSuccess && a.mass) e = launch_paged_mass(a, cs);
  return cuda_ok(pc, e, "attend");
}

kvs_status kvs_paged_get_status(kvs_paged* pc, kvs_stream_t stream) {
  ENTER("kvs_paged_get_status");
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  kvs_status st = cuda_ok(pc, cudaStreamSynchronize(cs), "synchronise");
  if (st != KVS_OK) return st;
  int32_t e = 0;
  st = cuda_ok(pc, cudaMemcpyAsync(&e, pc->dev.err, 4, cudaMemcpyDeviceToHost, cs), "read error word");
  if (st == KVS_OK) st = cuda_ok(pc, cudaStreamSynchronize(cs), "synchronise");
  if (st != KVS_OK) return st;
  if (e & kErrTimeout) return fail(pc, KVS_ERR_TIMEOUT, "a device-side wait ran out (error word 0x%x)", e);
  if (e & kErrCapacity)
    return fail(pc, KVS_ERR_CAPACITY, "pages, rows or positions ran out on the device (error word 0x%x)", e);
  if (e & (kErrState | kErrBounds))
    return fail(pc, KVS_ERR_STATE, "a length, page or value on the device is out of range (error word 0x%x)", e);
  return KVS_OK;
}

kvs_status kvs_paged_clear_error(kvs_paged* pc, kvs_stream_t stream) {
  ENTER("kvs_paged_clear_error");
  return cuda_ok(pc, cudaMemsetAsync(pc->dev.err, 0, 4, reinterpret_cast<cudaStream_t>(stream)), "clear error");
}

const char* kvs_paged_last_error(const kvs_paged* pc) {
  Trace trace_("kvs_paged_last_error");
  return pc ? pc->err.c_str() : "";
}

}  // extern "C"
