// The paged E4M3 cache: shared declarations of its translation units.
//
// Workspace (256-byte aligned regions, zeroed at creation), per layer:
//   K codes  [num_pages][Hkv][2][D/16][8][16]   token t, dimension d at
//            [t / 8][d / 16][t % 8][d % 16]
//   V codes  [num_pages][Hkv][D][16]            token innermost
//   scales   [num_pages][Hkv] float2            (K scale, V scale), powers of two
// and one error word.  Both code layouts are made of 128-byte "core matrices" (8 rows of
// 16 bytes), which is what the tensor core's unswizzled K-major operands are made of: K
// rows are tokens with the contraction over d, V rows are dimensions with the
// contraction over tokens.  A page is one contiguous 16 * D bytes in each, so a plain bulk copy of it
// lands in shared memory as operand rows, and neither K nor V needs to be transposed,
// swizzled or (as the matrix instruction takes E4M3 operands) converted.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kvs_internal.cuh"

namespace kvs {

constexpr int kScaleMinExp = -100;       // exponents a page scale can have
constexpr int kScaleMaxExp = 119;
constexpr float kFloatMax = 3.402823466e38f;
constexpr int kMaxGroup = 64;            // query heads per KV head at most
constexpr int kMaxTableStride = 1 << 22; // blocks of a request: positions and tile counts fit 32 bits

struct PagedDev {
  int32_t L, Hq, Hkv, G, D, num_pages, in_dtype;
  uint8_t* k; uint8_t* v; size_t layer_bytes;      // num_pages * Hkv * 16 * D
  float2* scales; size_t layer_scales;             // num_pages * Hkv
  int32_t* err;
};

// One attend call, as the kernels see it.
struct PagedAttend {
  PagedDev d;
  int32_t layer, n_reqs, table_stride, total_q, max_q_len, window;
  const int32_t* table; const int32_t* kv_len; const int32_t* row_start;   // row_start may be null
  const void* q; void* out;
  float* mass;             // [n_reqs][table_stride] or null
  // scratch
  float* part_o;           // partial output rows
  float2* part_ml;         // their (reference maximum in log2 units, sum)
  float* blk;              // [n_reqs][table_stride][Hq] log2 of the blocks' weight sums (mass only)
  float* lse;              // [n_reqs][Hq] log2 of the rows' sums (mass only)
  int32_t splits;          // general kernel: parts of a row's range
  uint8_t* q_pieces;       // prompt kernel: split queries, and their rows' factors
  float* q_factors;
  int32_t* cuts;           // decode and prompt kernels: 8 words a CTA
};

// How a call runs: a pure function of host-known sizes, so that the scratch size and the
// launch agree.
struct PagedAttendPlan {
  enum Kernel { kGeneral, kDecode, kPrompt } kernel;
  int splits;              // general kernel
  int rows;                // decode kernel: query rows of a unit
  int grid;                // decode and prompt kernels
  size_t part_o, part_ml, blk, lse, q_pieces, q_factors, cuts, total;   // scratch offsets
};

__host__ __device__ inline size_t k_code(int D, int t, int d) {
  return (size_t)(t >> 3) * 8 * D + (size_t)(d >> 4) * 128 + (t & 7) * 16 + (d & 15);
}

__device__ __forceinline__ void paged_error(const PagedDev& d, int32_t bits) { atomicOr(d.err, bits); }
__device__ __forceinline__ void set_error(const PagedDev& d, int32_t bits) { paged_error(d, bits); }   // KVS_DCHECK's

// 2^e for e in [-126, 127].
__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((e + 127) << 23); }

// Exponent of the smallest power of two s with absmax <= 448 * s (448 = 1.75 * 2^8):
// from the bits, so that it is exact; clamped to the exponents a scale can have.
__device__ __forceinline__ int scale_exp(float absmax) {
  const int bits = __float_as_int(absmax);
  const int e = (bits >> 23) - 127 - 8 + ((bits & 0x7fffff) > 0x600000 ? 1 : 0);
  return max(kScaleMinExp, min(kScaleMaxExp, e));
}

// Two E4M3 codes as floats (exact).
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t codes16) {
  uint32_t h;
  const uint16_t c = (uint16_t)codes16;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ __half2 e4m3x2_to_half2(uint32_t codes16) {
  uint32_t h;
  const uint16_t c = (uint16_t)codes16;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  return *reinterpret_cast<const __half2*>(&h);
}
__device__ __forceinline__ uint32_t f16x2_to_e4m3x2(__half2 v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t*>(&v)));
  return r;
}
// Codes of (lo, hi), round to nearest even, saturating.
__device__ __forceinline__ uint32_t float2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// The same in E5M2, whose codes are the upper bytes of f16.
__device__ __forceinline__ uint32_t float2_to_e5m2x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_to_e5m2x2(__half2 v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t*>(&v)));
  return r;
}
__device__ __forceinline__ float2 e5m2x2_to_float2(uint32_t codes16) {
  const uint32_t h = __byte_perm(codes16, 0, 0x1404);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Request of packed row t: the last r with row_start[r] <= t.
__device__ __forceinline__ int request_of(const int32_t* row_start, int n, int t) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(row_start + mid) <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Reports device row counts that pass what the host was told (one block of `threads`).
__device__ __forceinline__ void report_rows(const PagedAttend& a, int threads) {
  if (!a.row_start) return;
  for (int r = threadIdx.x; r < a.n_reqs; r += threads) {
    const int lo = __ldg(a.row_start + r), hi = __ldg(a.row_start + r + 1);
    if (lo < 0 || hi < lo || hi - lo > a.max_q_len || hi > a.total_q) paged_error(a.d, kErrCapacity);
  }
}

cudaError_t launch_paged_plan(const PagedDev& d, int n, const int32_t* ctx, const int32_t* add, int32_t* table,
                              int stride, const int32_t* free_pages, int free_capacity, const int32_t* count_in,
                              int32_t* count_out, int32_t* row_start, int32_t* kv_len, int32_t* slots,
                              int32_t* positions, int capacity, int32_t* denied, int sms, cudaStream_t st);
cudaError_t launch_paged_slot_map(const PagedDev& d, int n, const int32_t* first, const int32_t* len,
                                  const int32_t* table, int stride, int32_t* row_start, int32_t* slots,
                                  int32_t* positions, int capacity, int sms, cudaStream_t st);
cudaError_t launch_paged_release(const PagedDev& d, int n, const int32_t* kv_len, int32_t* table, int stride,
                                 int32_t* free_pages, int free_capacity, int32_t* free_count, cudaStream_t st);
cudaError_t launch_paged_append(const PagedDev& d, int layer, int n_rows, const int32_t* slots, const void* k,
                                const void* v, cudaStream_t st);
cudaError_t launch_paged_gather(const PagedDev& d, int layer, int n_rows, const int32_t* slots, void* k, void* v,
                                cudaStream_t st);
int paged_decode_ctas_per_sm();
cudaError_t launch_paged_decode(const PagedAttend& a, int rows, int grid, cudaStream_t st);
int paged_prompt_rows();
int paged_prompt_tiles(int G, int n_reqs, int total_q);
size_t paged_prompt_tile_bytes(int D);
cudaError_t launch_paged_prompt(const PagedAttend& a, int grid, cudaStream_t st);
cudaError_t launch_paged_general(const PagedAttend& a, cudaStream_t st);
cudaError_t launch_paged_mass(const PagedAttend& a, cudaStream_t st);

}  // namespace kvs
