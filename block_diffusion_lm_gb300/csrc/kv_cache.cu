// Quantised paged K/V cache (csbp_generate.h): bf16 rows to E4M3 codes with
// one power-of-two scale per 32 features, and back.
//
// The scale is a power of two (2^e with the smallest e for which the group's
// largest magnitude fits E4M3's 448), so x 2^-e is exact and code x 2^e is a
// bf16 number: the only rounding of a write and a read is E4M3's own.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "csbp_generate.h"
#include "csbp_internal.h"

namespace csbp {
namespace {

constexpr int kGroup = 32;  // features per scale

struct CacheArgs {
  int64_t pages;
  int32_t page_size, row_values;  // Hkv x d
  uint8_t* codes[2];
  uint8_t* scales[2];
  int32_t batch, rows, table_pages;
  const int32_t *table, *start, *count;
  const __nv_bfloat16* src[2];
  __nv_bfloat16* dst[2];
  int64_t tok[2], bat[2];
};

// Token slot (page x page_size + place) of row i of sequence b, -1 if its
// position or page is out of range.
__device__ __forceinline__ int64_t slot_of(const CacheArgs& a, int b, int i) {
  const int64_t pos = static_cast<int64_t>(__ldg(a.start + b)) + i;
  if (pos < 0) return -1;
  const int64_t entry = pos / a.page_size;
  if (entry >= a.table_pages) return -1;
  const int64_t page = __ldg(a.table + static_cast<int64_t>(b) * a.table_pages + entry);
  if (page < 0 || page >= a.pages) return -1;
  return page * a.page_size + (pos - entry * a.page_size);
}

__device__ __forceinline__ bool takes_part(const CacheArgs& a, int b, int i) {
  return !a.count || i < __ldg(a.count + b);
}

// One thread per 8 consecutive features; 4 lanes hold a group.
__global__ void __launch_bounds__(256) cache_write_kernel(CacheArgs a) {
  const int chunks = a.row_values >> 3;  // a multiple of 4: groups never cross a warp
  const int64_t total = static_cast<int64_t>(a.batch) * a.rows * chunks;
  const int kv = blockIdx.y;
  for (int64_t idx = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; idx < total;
       idx += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t row = idx / chunks;
    const int c = static_cast<int>(idx - row * chunks);
    const int b = static_cast<int>(row / a.rows);
    const int i = static_cast<int>(row - static_cast<int64_t>(b) * a.rows);
    if (!takes_part(a, b, i)) continue;  // the same for the 4 lanes of a group
    const int64_t slot = slot_of(a, b, i);
    if (slot < 0) continue;
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(a.src[kv] + b * a.bat[kv] +
                                                         i * a.tok[kv]) + c);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t top = 0;  // bits of the largest finite magnitude
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t lo = w[k] & 0x7fffu, hi = (w[k] >> 16) & 0x7fffu;
      if (lo < 0x7f80u) top = max(top, lo);
      if (hi < 0x7f80u) top = max(top, hi);
    }
    const unsigned mask = 0xfu << (threadIdx.x & 28);
    top = max(top, __shfl_xor_sync(mask, top, 1));
    top = max(top, __shfl_xor_sync(mask, top, 2));
    // 448 = 1.75 x 2^8: e = exponent - 8, one more above 1.75
    const int byte = max(0, static_cast<int>(top >> 7) - 8 + ((top & 0x7fu) > 0x60u ? 1 : 0));
    const float inv = __uint_as_float(static_cast<uint32_t>(254 - byte) << 23);  // 2^-e
    uint32_t out[2];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float lo = __uint_as_float(w[k] << 16), hi = __uint_as_float(w[k] & 0xffff0000u);
      lo = (w[k] & 0x7fffu) < 0x7f80u ? lo * inv : NAN;
      hi = ((w[k] >> 16) & 0x7fffu) < 0x7f80u ? hi * inv : NAN;
      uint16_t two;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(hi), "f"(lo));
      if (k & 1)
        out[k >> 1] |= static_cast<uint32_t>(two) << 16;
      else
        out[k >> 1] = two;
    }
    *reinterpret_cast<uint2*>(a.codes[kv] + slot * a.row_values + c * 8) =
        make_uint2(out[0], out[1]);
    if ((c & 3) == 0)
      a.scales[kv][slot * (a.row_values / kGroup) + (c >> 2)] = static_cast<uint8_t>(byte);
  }
}

__device__ __forceinline__ uint32_t decode2(uint32_t two, float scale) {
  uint32_t h2;
  const uint16_t v = static_cast<uint16_t>(two & 0xffffu);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(v));
  __half2 h;
  *reinterpret_cast<uint32_t*>(&h) = h2;
  const float2 f = __half22float2(h);
  __nv_bfloat162 r = __floats2bfloat162_rn(f.x * scale, f.y * scale);
  return *reinterpret_cast<uint32_t*>(&r);
}

// 2^(byte - 127) as fp32: byte 0 is the subnormal 2^-127, 255 is NaN.
__device__ __forceinline__ float scale_of(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7fffffffu : byte << 23);
}

// One thread per 8 consecutive features.
__global__ void __launch_bounds__(256) cache_read_kernel(CacheArgs a) {
  const int chunks = a.row_values >> 3;
  const int64_t total = static_cast<int64_t>(a.batch) * a.rows * chunks;
  const int kv = blockIdx.y;
  for (int64_t idx = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; idx < total;
       idx += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t row = idx / chunks;
    const int c = static_cast<int>(idx - row * chunks);
    const int b = static_cast<int>(row / a.rows);
    const int i = static_cast<int>(row - static_cast<int64_t>(b) * a.rows);
    if (!takes_part(a, b, i)) continue;
    const int64_t slot = slot_of(a, b, i);
    uint4 r = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
    if (slot >= 0) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(a.codes[kv] + slot * a.row_values) + c);
      const float s = scale_of(__ldg(a.scales[kv] + slot * (a.row_values / kGroup) + (c >> 2)));
      r.x = decode2(v.x, s);
      r.y = decode2(v.x >> 16, s);
      r.z = decode2(v.y, s);
      r.w = decode2(v.y >> 16, s);
    }
    reinterpret_cast<uint4*>(a.dst[kv] + b * a.bat[kv] + i * a.tok[kv])[c] = r;
  }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Checks shared by both directions; fills everything but src / dst.
csbp_status make_args(const csbp_kv_cache* c, const csbp_cache_rows* r, const void* k,
                      const void* v, CacheArgs& a) {
  if (!c || !r) return CSBP_ERR_INVALID;
  if (c->pages < 1 || c->pages > 0x7fffffff || c->page_size < 1 || c->page_size > 65536 ||
      c->Hkv < 1 || c->Hkv > 65536 || c->d < kGroup || c->d > 1024 || c->d % kGroup != 0)
    return CSBP_ERR_INVALID;
  if (!c->k || !c->v || !c->k_scale || !c->v_scale) return CSBP_ERR_INVALID;
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return CSBP_ERR_INVALID;
  if (r->batch < 0 || r->rows < 0 || r->table_pages < 0) return CSBP_ERR_INVALID;
  if (r->batch == 0 || r->rows == 0) return CSBP_OK;
  if (!r->table || !r->start || !k || !v) return CSBP_ERR_INVALID;
  if (!aligned(r->table, 4) || !aligned(r->start, 4) || (r->count && !aligned(r->count, 4)) ||
      !aligned(k, 16) || !aligned(v, 16))
    return CSBP_ERR_INVALID;
  const int64_t row = static_cast<int64_t>(c->Hkv) * c->d;  // <= 2^26
  // every element count stays below 2^62, tested by division
  constexpr int64_t kMaxElems = int64_t(1) << 39;
  if (static_cast<int64_t>(r->batch) * r->rows > (kMaxElems - 1) / row ||
      c->pages * c->page_size > ((int64_t(1) << 62) - 1) / row)
    return CSBP_ERR_UNSUPPORTED;
  for (int i = 0; i < 2; ++i) {
    const int64_t st = r->stride_tok[i], sb = r->stride_batch[i];
    if (st < 0 || sb < 0) return CSBP_ERR_INVALID;
    a.tok[i] = st != 0 ? st : row;
    if (a.tok[i] < row || a.tok[i] % 8 != 0 || a.tok[i] > (kMaxElems - 1) / r->rows)
      return CSBP_ERR_INVALID;
    const int64_t span = a.tok[i] * r->rows;
    a.bat[i] = (r->batch > 1 && sb != 0) ? sb : span;
    if (a.bat[i] < span || a.bat[i] % 8 != 0 || a.bat[i] >= kMaxElems) return CSBP_ERR_INVALID;
  }
  a.pages = c->pages;
  a.page_size = c->page_size;
  a.row_values = static_cast<int32_t>(row);
  a.codes[0] = static_cast<uint8_t*>(c->k);
  a.codes[1] = static_cast<uint8_t*>(c->v);
  a.scales[0] = static_cast<uint8_t*>(c->k_scale);
  a.scales[1] = static_cast<uint8_t*>(c->v_scale);
  a.batch = r->batch;
  a.rows = r->rows;
  a.table_pages = r->table_pages;
  a.table = r->table;
  a.start = r->start;
  a.count = r->count;
  return CSBP_OK;
}

csbp_status grid_of(const CacheArgs& a, dim3& grid) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return CSBP_ERR_CUDA;
  const int64_t total = static_cast<int64_t>(a.batch) * a.rows * (a.row_values >> 3);
  const int64_t blocks = (total + 255) / 256, cap = static_cast<int64_t>(sms) * 8;
  grid = dim3(static_cast<unsigned>(blocks < cap ? blocks : cap), 2);
  return CSBP_OK;
}

}  // namespace
}  // namespace csbp

using namespace csbp;

extern "C" csbp_status csbp_cache_write(const csbp_kv_cache* cache, const csbp_cache_rows* rows,
                                        const void* k, const void* v, void* stream) {
  CacheArgs a{};
  csbp_status st = make_args(cache, rows, k, v, a);
  if (st != CSBP_OK || a.batch == 0) return st;
  a.src[0] = static_cast<const __nv_bfloat16*>(k);
  a.src[1] = static_cast<const __nv_bfloat16*>(v);
  dim3 grid;
  if ((st = grid_of(a, grid)) != CSBP_OK) return st;
  const int timed = timer_begin(11, stream);
  cache_write_kernel<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  timer_end(timed, stream);
  return e == cudaSuccess ? CSBP_OK : CSBP_ERR_CUDA;
}

extern "C" csbp_status csbp_cache_read(const csbp_kv_cache* cache, const csbp_cache_rows* rows,
                                       void* k, void* v, void* stream) {
  CacheArgs a{};
  csbp_status st = make_args(cache, rows, k, v, a);
  if (st != CSBP_OK || a.batch == 0) return st;
  a.dst[0] = static_cast<__nv_bfloat16*>(k);
  a.dst[1] = static_cast<__nv_bfloat16*>(v);
  dim3 grid;
  if ((st = grid_of(a, grid)) != CSBP_OK) return st;
  const int timed = timer_begin(12, stream);
  cache_read_kernel<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  timer_end(timed, stream);
  return e == cudaSuccess ? CSBP_OK : CSBP_ERR_CUDA;
}
