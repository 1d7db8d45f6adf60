// Append and gather of the paged cache: tokens to and from the codes at their slots.
//
// Append: for each page, KV head and cache (K or V), with x the run of new tokens of that
// page: scale s = max(old scale, 2^e), 2^e the smallest power of two with max|x| <= 448 2^e
// (old scale dropped when the run starts the page); codes = rn(x / s); the page's other
// codes c become rn(c * old / s) if s grew, 0 if the page starts.  x / s and c * old / s
// are products with powers of two, so each value is rounded once, to its code.
//
// How: a warp owns one (run, KV head, cache): it reads the run's rows once, keeps them in
// registers over the maximum and the conversion, and writes whole 16-byte pieces.  K
// pieces are 16 dimensions of a token; V pieces are 16 tokens of a dimension, so for V a
// lane reads four dimensions of each token (whole rows stay coalesced) and the
// transposition costs no shared memory.  The row that starts a run leads it; others exit,
// so a batch of single tokens is one warp per token and cache, and rows of a long prompt
// are taken sixteen to a warp to spare idle warps.
#include "append_store.cuh"
#include "paged.cuh"

namespace kvs {
namespace {

constexpr int kWarps = 4;

template <int IN>
__device__ __forceinline__ void load4(const void* base, size_t elem, float v[4]) {
  if constexpr (IN == KVS_BF16) {
    const uint2 raw = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(base) + elem);
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw.x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw.y));
    v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
  } else {
    const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + elem);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  }
}

template <int OUT>
__device__ __forceinline__ void store4(void* base, size_t elem, const float v[4]) {
  if constexpr (OUT == KVS_BF16) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    uint2 raw;
    raw.x = *reinterpret_cast<const uint32_t*>(&a);
    raw.y = *reinterpret_cast<const uint32_t*>(&b);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(base) + elem) = raw;
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(base) + elem) = make_float4(v[0], v[1], v[2], v[3]);
  }
}

// A value as it takes part in the scale: NaN becomes 0, an infinity stays out of the maximum.
__device__ __forceinline__ float clean(float x, float& amax, bool& nan) {
  if (x != x) { nan = true; return 0.f; }
  const float a = fabsf(x);
  if (a <= 3.402823466e38f) amax = fmaxf(amax, a);
  return x;
}

__device__ __forceinline__ uint32_t requantise4(uint32_t codes, float ratio) {
  const float2 a = e4m3x2_to_float2(codes & 0xffffu), b = e4m3x2_to_float2(codes >> 16);
  return float2_to_e4m3x2(a.x * ratio, a.y * ratio) | (float2_to_e4m3x2(b.x * ratio, b.y * ratio) << 16);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// A run: rows of one page, at most 16.  Lane t < 16 holds the row of slot t in the page (-1: none).
struct Run {
  int page, row;
  uint32_t have;
};

template <int IN, int D>
__device__ void store_k(const PagedDev& d, int layer, int head, const void* x, const Run& run, int lane) {
  constexpr int CH = D / 16;                       // pieces of a token
  constexpr int NP = (16 * CH + 31) / 32;          // pieces of a lane
  const size_t at = (size_t)run.page * d.Hkv + head;
  uint8_t* base = d.k + layer * d.layer_bytes + at * (16 * D);
  float* scale_at = &d.scales[layer * d.layer_scales + at].x;
  const bool fresh = run.have & 1;
  const float old = fresh ? exp2_int(kScaleMinExp) : fmaxf(*scale_at, exp2_int(kScaleMinExp));
  float v[NP][16];
  float amax = 0.f;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int piece = i * 32 + lane, t = piece / CH, c = piece % CH;
    const int row = __shfl_sync(0xffffffffu, run.row, t & 15);
    if (piece >= 16 * CH || row < 0) continue;
    const size_t e = ((size_t)row * d.Hkv + head) * D + c * 16;
    load8<IN>(x, e, v[i]);
    load8<IN>(x, e + 8, v[i] + 8);
  }
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int piece = i * 32 + lane, t = piece / CH;
    if (piece >= 16 * CH || !(run.have >> t & 1)) continue;
#pragma unroll
    for (int u = 0; u < 16; ++u) v[i][u] = clean(v[i][u], amax, nan);
  }
  amax = warp_max(amax);
  const float scale = fmaxf(old, exp2_int(scale_exp(amax)));
  const float inv = 1.f / scale, ratio = old * inv;      // powers of two: exact
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int piece = i * 32 + lane, t = piece / CH, c = piece % CH;
    if (piece >= 16 * CH) continue;
    uint4* dst = reinterpret_cast<uint4*>(base + k_code(D, t, c * 16));
    uint4 w = make_uint4(0, 0, 0, 0);
    if (run.have >> t & 1) {
      uint32_t* p = &w.x;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        p[u] = float2_to_e4m3x2(v[i][4 * u] * inv, v[i][4 * u + 1] * inv) |
               (float2_to_e4m3x2(v[i][4 * u + 2] * inv, v[i][4 * u + 3] * inv) << 16);
    } else if (!fresh) {
      if (ratio == 1.f) continue;
      w = *dst;
      w.x = requantise4(w.x, ratio); w.y = requantise4(w.y, ratio);
      w.z = requantise4(w.z, ratio); w.w = requantise4(w.w, ratio);
    }
    *dst = w;
  }
  __syncwarp();                                    // every lane has read the old scale
  if (lane == 0) *scale_at = scale;
  if (nan) paged_error(d, kErrState);
}

template <int IN, int D>
__device__ void store_v(const PagedDev& d, int layer, int head, const void* x, const Run& run, int lane) {
  const size_t at = (size_t)run.page * d.Hkv + head;
  uint8_t* base = d.v + layer * d.layer_bytes + at * (16 * D);
  float* scale_at = &d.scales[layer * d.layer_scales + at].y;
  const bool fresh = run.have & 1, mine = lane < D / 4;
  const float old = fresh ? exp2_int(kScaleMinExp) : fmaxf(*scale_at, exp2_int(kScaleMinExp));
  float v[16][4];
  float amax = 0.f;
  bool nan = false;
#pragma unroll
  for (int t = 0; t < 16; ++t) {
    const int row = __shfl_sync(0xffffffffu, run.row, t);
    v[t][0] = v[t][1] = v[t][2] = v[t][3] = 0.f;
    if (row >= 0 && mine) load4<IN>(x, ((size_t)row * d.Hkv + head) * D + lane * 4, v[t]);
  }
#pragma unroll
  for (int t = 0; t < 16; ++t)
#pragma unroll
    for (int u = 0; u < 4; ++u) v[t][u] = clean(v[t][u], amax, nan);
  amax = warp_max(amax);
  const float scale = fmaxf(old, exp2_int(scale_exp(amax)));
  const float inv = 1.f / scale, ratio = old * inv;
  if (mine) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      uint4* dst = reinterpret_cast<uint4*>(base + (lane * 4 + u) * 16);
      uint4 w = make_uint4(0, 0, 0, 0);
      if (!fresh && run.have != 0xffffu) {
        w = *dst;
        if (ratio != 1.f) {
          w.x = requantise4(w.x, ratio); w.y = requantise4(w.y, ratio);
          w.z = requantise4(w.z, ratio); w.w = requantise4(w.w, ratio);
        }
      }
      uint32_t* p = &w.x;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t codes = float2_to_e4m3x2(v[4 * j][u] * inv, v[4 * j + 1][u] * inv) |
                               (float2_to_e4m3x2(v[4 * j + 2][u] * inv, v[4 * j + 3][u] * inv) << 16);
        const uint32_t h = run.have >> (4 * j);
        const uint32_t mask = (h & 1 ? 0xffu : 0) | (h & 2 ? 0xff00u : 0) | (h & 4 ? 0xff0000u : 0) |
                              (h & 8 ? 0xff000000u : 0);
        p[j] = (p[j] & ~mask) | (codes & mask);
      }
      *dst = w;
    }
  }
  __syncwarp();
  if (lane == 0) *scale_at = scale;
  if (nan) paged_error(d, kErrState);
}

// grid: x groups of `per` rows, kWarps to a CTA; y KV heads; z 0 = K, 1 = V.
template <int IN, int D>
__global__ void __launch_bounds__(kWarps * 32) append_kernel(const PagedDev d, int layer, int n_rows, int per,
                                                             const int32_t* __restrict__ slots, const void* k,
                                                             const void* v) {
  const int lane = threadIdx.x & 31, head = blockIdx.y;
  const long long first = ((long long)blockIdx.x * kWarps + (threadIdx.x >> 5)) * per;
  for (int i = (int)first; i < n_rows && i < first + per; ++i) {
    const int lead = __ldg(slots + i);
    if (lead < 0) continue;
    const int page = lead >> 4;
    if (i > 0) {
      const int before = __ldg(slots + i - 1);
      if (before >= 0 && (before >> 4) == page) continue;
    }
    if (page >= d.num_pages) {
      if (lane == 0) paged_error(d, kErrState);
      continue;
    }
    // the run: rows i, i + 1, ... while they stay in the page
    const int s = lane < 16 && i + lane < n_rows ? __ldg(slots + i + lane) : -1;
    const uint32_t in = __ballot_sync(0xffffffffu, s >= 0 && (s >> 4) == page);
    const int len = __ffs(~in) - 1;
    Run run{page, -1, 0};
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int off = __shfl_sync(0xffffffffu, s, j) & 15;
      if (j < len) {
        if (lane == off) run.row = i + j;
        run.have |= 1u << off;
      }
    }
    if (blockIdx.z == 0) store_k<IN, D>(d, layer, head, k, run, lane);
    else store_v<IN, D>(d, layer, head, v, run, lane);
    i += len - 1;
  }
}

// A warp reads the codes of up to 16 rows at a time, run by run.
template <int OUT, int D>
__global__ void __launch_bounds__(kWarps * 32) gather_kernel(const PagedDev d, int layer, int n_rows, int per,
                                                             const int32_t* __restrict__ slots, void* k, void* v) {
  constexpr int CH = D / 16, NP = (16 * CH + 31) / 32;
  const int lane = threadIdx.x & 31, head = blockIdx.y;
  const long long first = ((long long)blockIdx.x * kWarps + (threadIdx.x >> 5)) * per;
  if (first >= n_rows) return;
  const int i0 = (int)first, n = min(per, n_rows - i0);
  int s = lane < n ? __ldg(slots + i0 + lane) : -1;
  if (s >= 0 && (s >> 4) >= d.num_pages) {
    paged_error(d, kErrState);
    s = -1;
  }
  const float2 sc = s >= 0 ? d.scales[layer * d.layer_scales + (size_t)(s >> 4) * d.Hkv + head] : make_float2(0.f, 0.f);
  if (blockIdx.z == 0) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int piece = i * 32 + lane, j = piece / CH, c = piece % CH;
      const int sj = __shfl_sync(0xffffffffu, s, j & 15);
      const float scale = __shfl_sync(0xffffffffu, sc.x, j & 15);
      if (piece >= 16 * CH || j >= n) continue;
      uint4 w = make_uint4(0, 0, 0, 0);
      if (sj >= 0)
        w = __ldg(reinterpret_cast<const uint4*>(d.k + layer * d.layer_bytes + ((size_t)(sj >> 4) * d.Hkv + head) * (16 * D) +
                                                 k_code(D, sj & 15, c * 16)));
      const uint32_t* p = &w.x;
      const size_t e = ((size_t)(i0 + j) * d.Hkv + head) * D + c * 16;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float2 a = e4m3x2_to_float2(p[u] & 0xffffu), b = e4m3x2_to_float2(p[u] >> 16);
        const float f[4] = {a.x * scale, a.y * scale, b.x * scale, b.y * scale};
        store4<OUT>(k, e + 4 * u, f);
      }
    }
    return;
  }
  const bool mine = lane < D / 4;
  int page = -2;
  uint4 w[4];
  for (int j = 0; j < n; ++j) {
    const int sj = __shfl_sync(0xffffffffu, s, j);
    const float scale = __shfl_sync(0xffffffffu, sc.y, j);
    if (!mine) continue;
    const int pj = sj < 0 ? -1 : sj >> 4;
    if (pj != page) {
      page = pj;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        w[u] = page < 0 ? make_uint4(0, 0, 0, 0)
                        : __ldg(reinterpret_cast<const uint4*>(d.v + layer * d.layer_bytes + ((size_t)page * d.Hkv + head) * (16 * D)) +
                                lane * 4 + u);
    }
    const int word = (sj & 15) >> 2, shift = (sj & 3) * 8;
    float f[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t x = word == 0 ? w[u].x : word == 1 ? w[u].y : word == 2 ? w[u].z : w[u].w;
      f[u] = e4m3x2_to_float2((x >> shift) & 0xffu).x * scale;
    }
    store4<OUT>(v, ((size_t)(i0 + j) * d.Hkv + head) * D + lane * 4, f);
  }
}

// Rows of a warp: one while a row a warp still leaves warps idle, else a page's worth.
int rows_per_warp(int n_rows, int Hkv) { return (long long)n_rows * Hkv * 2 <= 16384 ? 1 : 16; }

template <int DT, int D>
cudaError_t append_d(const PagedDev& d, int layer, int n_rows, const int32_t* slots, const void* k, const void* v,
                     cudaStream_t st) {
  const int per = rows_per_warp(n_rows, d.Hkv);
  const dim3 grid((unsigned)cdiv64(n_rows, (long long)per * kWarps), d.Hkv, 2);
  append_kernel<DT, D><<<grid, kWarps * 32, 0, st>>>(d, layer, n_rows, per, slots, k, v);
  return cudaGetLastError();
}

template <int DT, int D>
cudaError_t gather_d(const PagedDev& d, int layer, int n_rows, const int32_t* slots, void* k, void* v,
                     cudaStream_t st) {
  const int per = rows_per_warp(n_rows, d.Hkv);
  const dim3 grid((unsigned)cdiv64(n_rows, (long long)per * kWarps), d.Hkv, 2);
  gather_kernel<DT, D><<<grid, kWarps * 32, 0, st>>>(d, layer, n_rows, per, slots, k, v);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_append(const PagedDev& d, int layer, int n_rows, const int32_t* slots, const void* k,
                                const void* v, cudaStream_t st) {
  const bool b = d.in_dtype == KVS_BF16;
  switch (d.D) {
    case 16: return b ? append_d<KVS_BF16, 16>(d, layer, n_rows, slots, k, v, st) : append_d<KVS_F32, 16>(d, layer, n_rows, slots, k, v, st);
    case 32: return b ? append_d<KVS_BF16, 32>(d, layer, n_rows, slots, k, v, st) : append_d<KVS_F32, 32>(d, layer, n_rows, slots, k, v, st);
    case 64: return b ? append_d<KVS_BF16, 64>(d, layer, n_rows, slots, k, v, st) : append_d<KVS_F32, 64>(d, layer, n_rows, slots, k, v, st);
    default: return b ? append_d<KVS_BF16, 128>(d, layer, n_rows, slots, k, v, st) : append_d<KVS_F32, 128>(d, layer, n_rows, slots, k, v, st);
  }
}

cudaError_t launch_paged_gather(const PagedDev& d, int layer, int n_rows, const int32_t* slots, void* k, void* v,
                                cudaStream_t st) {
  const bool b = d.in_dtype == KVS_BF16;
  switch (d.D) {
    case 16: return b ? gather_d<KVS_BF16, 16>(d, layer, n_rows, slots, k, v, st) : gather_d<KVS_F32, 16>(d, layer, n_rows, slots, k, v, st);
    case 32: return b ? gather_d<KVS_BF16, 32>(d, layer, n_rows, slots, k, v, st) : gather_d<KVS_F32, 32>(d, layer, n_rows, slots, k, v, st);
    case 64: return b ? gather_d<KVS_BF16, 64>(d, layer, n_rows, slots, k, v, st) : gather_d<KVS_F32, 64>(d, layer, n_rows, slots, k, v, st);
    default: return b ? gather_d<KVS_BF16, 128>(d, layer, n_rows, slots, k, v, st) : gather_d<KVS_F32, 128>(d, layer, n_rows, slots, k, v, st);
  }
}

}  // namespace kvs
