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

// Row `i` of sequence `b`, and whether it takes part.
struct Row {
  int b, i;
  bool takes_part;
};

// The rows of a CTA are consecutive; `k` is one of them, the same for the
// lanes that share it.
__device__ __forceinline__ Row row_of(const CacheArgs& a, int64_t first, int k) {
  const int64_t b0 = first / a.rows;  // the same in all threads
  const uint32_t i = static_cast<uint32_t>(first - b0 * a.rows) + static_cast<uint32_t>(k);
  const uint32_t more = i / static_cast<uint32_t>(a.rows);
  Row r;
  const int64_t b = b0 + more;
  r.takes_part = b < a.batch;
  r.b = r.takes_part ? static_cast<int>(b) : 0;
  r.i = static_cast<int>(i - more * static_cast<uint32_t>(a.rows));
  if (r.takes_part && a.count) r.takes_part = r.i < __ldg(a.count + r.b);
  return r;
}

// Token slot (page x page_size + place) of a row, -1 if its position or page
// is out of range.
__device__ __forceinline__ int64_t slot_of(const CacheArgs& a, const Row& r) {
  const int64_t pos = static_cast<int64_t>(__ldg(a.start + r.b)) + r.i;
  if (pos < 0) return -1;
  const uint32_t at = static_cast<uint32_t>(pos);  // below 2^32
  const uint32_t entry = at / static_cast<uint32_t>(a.page_size);
  if (entry >= static_cast<uint32_t>(a.table_pages)) return -1;
  const int64_t page = __ldg(a.table + static_cast<int64_t>(r.b) * a.table_pages + entry);
  if (page < 0 || page >= a.pages) return -1;
  return page * a.page_size + (at - entry * static_cast<uint32_t>(a.page_size));
}

// E4M3 codes of 8 bf16 values (two per word) under the scale byte `byte`.
__device__ __forceinline__ uint2 encode8(const uint32_t w[4], int byte) {
  const float inv = __uint_as_float(static_cast<uint32_t>(254 - byte) << 23);  // 2^-e
  uint32_t two[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float lo = __uint_as_float(w[k] << 16) * inv, hi = __uint_as_float(w[k] & 0xffff0000u) * inv;
    // the conversion would make infinities 448
    if ((w[k] & 0x7fffu) == 0x7f80u) lo = NAN;
    if ((w[k] & 0x7fff0000u) == 0x7f800000u) hi = NAN;
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
    two[k] = c;
  }
  return make_uint2(two[0] | two[1] << 16, two[2] | two[3] << 16);
}

// Bits of the largest finite magnitude of 8 bf16 values.
__device__ __forceinline__ uint32_t top8(const uint32_t w[4]) {
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t lo = w[k] & 0x7fffu, hi = (w[k] >> 16) & 0x7fffu;
    if (lo < 0x7f80u) top = max(top, lo);
    if (hi < 0x7f80u) top = max(top, hi);
  }
  return top;
}

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

// `L` lanes per row (4 .. 32, so that a group of 32 features is 4 lanes of one
// row), 8 features a lane and step, K and V of a row in turn with all loads of
// up to kUnroll steps issued before the first is used: 32 lanes x 16 bytes x 8
// loads in flight per warp.
template <int L>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(CacheArgs a) {
  constexpr int kRows = kThreads / L;
  const int lane = threadIdx.x % L;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kRows;
  const Row r = row_of(a, first, threadIdx.x / L);
  const int chunks = a.row_values >> 3;  // a multiple of 4
  const int64_t slot = r.takes_part ? slot_of(a, r) : -1;
  // the lanes of a row decide alike, those of a warp need not: no early return
  // before the shuffles
  const bool on = slot >= 0;
  for (int c0 = 0; c0 < chunks; c0 += L * kUnroll) {
    uint4 v[2][kUnroll];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const uint4* src = reinterpret_cast<const uint4*>(a.src[kv] + r.b * a.bat[kv] +
                                                        r.i * a.tok[kv]);
#pragma unroll
      for (int t = 0; t < kUnroll; ++t) {
        const int c = c0 + t * L + lane;
        v[kv][t] = on && c < chunks ? __ldcs(src + c) : make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      uint8_t* codes = a.codes[kv] + slot * a.row_values;
      uint8_t* scales = a.scales[kv] + slot * (a.row_values / kGroup);
#pragma unroll
      for (int t = 0; t < kUnroll; ++t) {
        const int c = c0 + t * L + lane;
        const uint32_t w[4] = {v[kv][t].x, v[kv][t].y, v[kv][t].z, v[kv][t].w};
        uint32_t top = top8(w);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 448 = 1.75 x 2^8: e = exponent - 8, one more above 1.75
        const int byte = max(0, static_cast<int>(top >> 7) - 8 + ((top & 0x7fu) > 0x60u ? 1 : 0));
        if (on && c < chunks) {
          *reinterpret_cast<uint2*>(codes + c * 8) = encode8(w, byte);
          if ((c & 3) == 0) scales[c >> 2] = static_cast<uint8_t>(byte);
        }
      }
    }
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

// The same lanes and steps as the write.
template <int L>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(CacheArgs a) {
  constexpr int kRows = kThreads / L;
  const int lane = threadIdx.x % L;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kRows;
  const Row r = row_of(a, first, threadIdx.x / L);
  if (!r.takes_part) return;
  const int chunks = a.row_values >> 3;
  const int64_t slot = slot_of(a, r);
  for (int c0 = 0; c0 < chunks; c0 += L * kUnroll) {
    uint2 v[2][kUnroll];
    uint32_t sb[2][kUnroll];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
#pragma unroll
      for (int t = 0; t < kUnroll; ++t) {
        const int c = c0 + t * L + lane;
        v[kv][t] = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);  // NaN
        sb[kv][t] = 127;
        if (slot >= 0 && c < chunks) {
          v[kv][t] = __ldcs(reinterpret_cast<const uint2*>(a.codes[kv] + slot * a.row_values) + c);
          sb[kv][t] = __ldg(a.scales[kv] + slot * (a.row_values / kGroup) + (c >> 2));
        }
      }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      uint4* dst = reinterpret_cast<uint4*>(a.dst[kv] + r.b * a.bat[kv] + r.i * a.tok[kv]);
#pragma unroll
      for (int t = 0; t < kUnroll; ++t) {
        const int c = c0 + t * L + lane;
        const float s = scale_of(sb[kv][t]);
        const uint4 out = make_uint4(decode2(v[kv][t].x, s), decode2(v[kv][t].x >> 16, s),
                                     decode2(v[kv][t].y, s), decode2(v[kv][t].y >> 16, s));
        if (c < chunks) dst[c] = out;
      }
    }
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

// One launch over all rows with the fewest lanes per row that cover it in one
// step (so that short rows share a warp), at most a warp.
template <bool kWrite>
csbp_status launch(const CacheArgs& a, void* stream) {
  const int chunks = a.row_values >> 3;
  const int lanes = chunks <= 4 ? 4 : chunks <= 8 ? 8 : chunks <= 16 ? 16 : 32;
  const int64_t per = kThreads / lanes;
  const int64_t grid = (static_cast<int64_t>(a.batch) * a.rows + per - 1) / per;
  if (grid > 0x7fffffff) return CSBP_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned g = static_cast<unsigned>(grid);
  const int timed = timer_begin(kWrite ? 11 : 12, stream);
  if (lanes == 4)
    kWrite ? cache_write_kernel<4><<<g, kThreads, 0, s>>>(a)
           : cache_read_kernel<4><<<g, kThreads, 0, s>>>(a);
  else if (lanes == 8)
    kWrite ? cache_write_kernel<8><<<g, kThreads, 0, s>>>(a)
           : cache_read_kernel<8><<<g, kThreads, 0, s>>>(a);
  else if (lanes == 16)
    kWrite ? cache_write_kernel<16><<<g, kThreads, 0, s>>>(a)
           : cache_read_kernel<16><<<g, kThreads, 0, s>>>(a);
  else
    kWrite ? cache_write_kernel<32><<<g, kThreads, 0, s>>>(a)
           : cache_read_kernel<32><<<g, kThreads, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  timer_end(timed, stream);
  return e == cudaSuccess ? CSBP_OK : CSBP_ERR_CUDA;
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
  return launch<true>(a, stream);
}

extern "C" csbp_status csbp_cache_read(const csbp_kv_cache* cache, const csbp_cache_rows* rows,
                                       void* k, void* v, void* stream) {
  CacheArgs a{};
  csbp_status st = make_args(cache, rows, k, v, a);
  if (st != CSBP_OK || a.batch == 0) return st;
  a.dst[0] = static_cast<__nv_bfloat16*>(k);
  a.dst[1] = static_cast<__nv_bfloat16*>(v);
  return launch<false>(a, stream);
}
