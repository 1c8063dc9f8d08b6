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

#include "bf16_bits.cuh"
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
  bool wide;  // rows of the bf16 side start on 32 bytes
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

// 16 bf16 values (two per word), or their codes (four per word).
struct Values16 {
  uint32_t w[8];
};
struct Codes16 {
  uint32_t w[4];
};

// 32 bytes: one access, or two of 16 where rows start on 16 only (`wide`, the
// same for all threads).  Streamed: nobody comes back soon.  8 x 25,000 rows of
// 128 features are read back in 28.4 us wide, in 31.4 otherwise (writes: 30.0
// either way).
__device__ __forceinline__ Values16 load16(const void* p, bool wide) {
  Values16 v;
  if (wide) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]),
                   "=r"(v.w[5]), "=r"(v.w[6]), "=r"(v.w[7])
                 : "l"(p));
  } else {
    const uint4 lo = __ldg(static_cast<const uint4*>(p));
    const uint4 hi = __ldg(static_cast<const uint4*>(p) + 1);
    v = Values16{{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w}};
  }
  return v;
}
__device__ __forceinline__ void store16(void* p, const Values16& v, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v.w[0]),
                 "r"(v.w[1]), "r"(v.w[2]), "r"(v.w[3]), "r"(v.w[4]), "r"(v.w[5]), "r"(v.w[6]),
                 "r"(v.w[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
    static_cast<uint4*>(p)[1] = make_uint4(v.w[4], v.w[5], v.w[6], v.w[7]);
  }
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Bits of the largest magnitude (NaN and infinities, the largest bit patterns,
// among them).
__device__ __forceinline__ uint32_t top16(const Values16& v) {
  uint32_t m = v.w[0] & 0x7fff7fffu;
#pragma unroll
  for (int k = 1; k < 8; ++k) m = max_u16x2(m, v.w[k] & 0x7fff7fffu);
  return max(m & 0xffffu, m >> 16);
}

// The values with NaN and infinities replaced by zero.
__device__ __forceinline__ Values16 finite16(Values16 v) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if ((v.w[k] & 0x7f80u) == 0x7f80u) v.w[k] &= 0xffff0000u;
    if ((v.w[k] & 0x7f800000u) == 0x7f800000u) v.w[k] &= 0xffffu;
  }
  return v;
}

// E4M3 of finite values under the scale byte `byte`.  x 2^-e is exact in bf16
// (e is the group's own, so only what rounds to zero anyway can underflow).
__device__ __forceinline__ Codes16 encode16(const Values16& v, int byte) {
  const uint32_t inv = static_cast<uint32_t>(254 - byte) << 7;  // 2^-e
  uint32_t two[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t x = mul_bf16x2(v.w[k], inv | inv << 16);
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(c)
        : "f"(__uint_as_float(x & 0xffff0000u)), "f"(__uint_as_float(x << 16)));
    two[k] = c;
  }
  Codes16 r;
#pragma unroll
  for (int k = 0; k < 4; ++k) r.w[k] = two[2 * k] | two[2 * k + 1] << 16;
  return r;
}

// NaN codes in the place of values that are not finite.
__device__ __forceinline__ Codes16 mark16(const Values16& v, Codes16 r) {
#pragma unroll
  for (int k = 0; k < 16; ++k)
    if ((v.w[k >> 1] >> (k & 1) * 16 & 0x7f80u) == 0x7f80u) r.w[k >> 2] |= 0x7fu << (k & 3) * 8;
  return r;
}

constexpr int kThreads = 256;

// Layout of both kernels.  `L` lanes hold a row (2 .. 32, so that a group of 32
// features is 2 lanes of one row), 16 features a lane and step; K or V by
// blockIdx.y.  N pieces are in flight per lane, each issued before the first is
// used: steps of one row where a row takes several (R = 1), else R = N rows, so
// that short rows do not make short threads.  HBM bounds it: 3 + 1/32 bytes per
// value, at 4 to 5 instructions per value, about half the issue rate (one value
// at a time took 10 and was bound by them).  131,072 rows of 8 x 128 features:
// write 127.6 us, 6.38 TB/s, 0.94 of a plain copy's measured rate; read 122.7
// us, 6.63 TB/s, 0.98.  A token for each of 8 sequences: 2 to 2.8 us.
template <int L, int R>
struct Shape {
  static constexpr int kRows = kThreads / L * R;  // of a CTA
  static constexpr int kPieces = R == 1 ? 2 : R;
};

template <int L, int R>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(CacheArgs a) {
  constexpr int N = Shape<L, R>::kPieces;
  const int lane = threadIdx.x % L, kv = blockIdx.y;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * Shape<L, R>::kRows;
  Row r[R];
#pragma unroll
  for (int t = 0; t < R; ++t) r[t] = row_of(a, first, threadIdx.x / L + t * (kThreads / L));
  const int chunks = a.row_values >> 4;  // a multiple of 2
  const __nv_bfloat16* src = kv ? a.src[1] : a.src[0];
  const int64_t bat = kv ? a.bat[1] : a.bat[0], tok = kv ? a.tok[1] : a.tok[0];
  uint8_t* codes = kv ? a.codes[1] : a.codes[0];
  uint8_t* scales = kv ? a.scales[1] : a.scales[0];
  // the lanes of a row decide alike, those of a warp need not: no early return
  // before the shuffles
  for (int c0 = lane; c0 - lane < chunks; c0 += R == 1 ? L * N : L) {
    Values16 v[N];
#pragma unroll
    for (int t = 0; t < N; ++t) {
      const Row& w = r[R == 1 ? 0 : t];
      const int c = R == 1 ? c0 + t * L : c0;
      v[t] = w.takes_part && c < chunks ? load16(src + w.b * bat + w.i * tok + c * 16, a.wide)
                                        : Values16{};
    }
    int64_t slot[R];
#pragma unroll
    for (int t = 0; t < R; ++t) slot[t] = r[t].takes_part ? slot_of(a, r[t]) : -1;
#pragma unroll
    for (int t = 0; t < N; ++t) {
      const int64_t to = slot[R == 1 ? 0 : t];
      const int c = R == 1 ? c0 + t * L : c0;
      uint32_t top = top16(v[t]);
      const bool bad = __any_sync(0xffffffffu, top >= 0x7f80u);
      const Values16 x = bad ? finite16(v[t]) : v[t];
      if (bad) top = top16(x);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      // 448 = 1.75 x 2^8: e = exponent - 8, one more above 1.75
      const int byte = max(0, static_cast<int>((top + 0x1fu) >> 7) - 8);
      Codes16 out = encode16(x, byte);
      if (bad) out = mark16(v[t], out);
      if (to >= 0 && c < chunks) {
        *reinterpret_cast<uint4*>(codes + to * a.row_values + c * 16) =
            make_uint4(out.w[0], out.w[1], out.w[2], out.w[3]);
        if ((c & 1) == 0)
          scales[to * (a.row_values / kGroup) + (c >> 1)] = static_cast<uint8_t>(byte);
      }
    }
  }
}

// 16 values of codes times 2^(byte - 127).  Codes are exact in bf16, so the one
// rounding is that of a product below bf16's smallest.
__device__ __forceinline__ Values16 decode16(const uint4& codes, uint32_t byte) {
  const uint32_t s = byte == 0 ? 0x0040u : byte == 255 ? 0x7fffu : byte << 7;  // bf16
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
  Values16 r;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    uint32_t h2;
    const uint16_t two = static_cast<uint16_t>(w[k >> 1] >> (k & 1) * 16);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(two));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
    const __nv_bfloat162 x = __floats2bfloat162_rn(f.x, f.y);
    r.w[k] = mul_bf16x2(*reinterpret_cast<const uint32_t*>(&x), s | s << 16);
  }
  return r;
}

template <int L, int R>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(CacheArgs a) {
  constexpr int N = Shape<L, R>::kPieces;
  const int lane = threadIdx.x % L, kv = blockIdx.y;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * Shape<L, R>::kRows;
  Row r[R];
  int64_t slot[R];
#pragma unroll
  for (int t = 0; t < R; ++t) {
    r[t] = row_of(a, first, threadIdx.x / L + t * (kThreads / L));
    slot[t] = r[t].takes_part ? slot_of(a, r[t]) : -1;
  }
  const int chunks = a.row_values >> 4;
  const uint8_t* codes = kv ? a.codes[1] : a.codes[0];
  const uint8_t* scales = kv ? a.scales[1] : a.scales[0];
  __nv_bfloat16* dst = kv ? a.dst[1] : a.dst[0];
  const int64_t bat = kv ? a.bat[1] : a.bat[0], tok = kv ? a.tok[1] : a.tok[0];
  for (int c0 = lane; c0 < chunks; c0 += R == 1 ? L * N : L) {
    uint4 v[N];
    uint32_t sb[N];
#pragma unroll
    for (int t = 0; t < N; ++t) {
      const int64_t from = slot[R == 1 ? 0 : t];
      const int c = R == 1 ? c0 + t * L : c0;
      v[t] = make_uint4(0, 0, 0, 0);
      sb[t] = 255;  // NaN, for a row that has no place
      if (from >= 0 && c < chunks) {
        v[t] = __ldcs(reinterpret_cast<const uint4*>(codes + from * a.row_values) + c);
        sb[t] = __ldg(scales + from * (a.row_values / kGroup) + (c >> 1));
      }
    }
#pragma unroll
    for (int t = 0; t < N; ++t) {
      const Row& w = r[R == 1 ? 0 : t];
      const int c = R == 1 ? c0 + t * L : c0;
      if (w.takes_part && c < chunks)
        store16(dst + w.b * bat + w.i * tok + c * 16, decode16(v[t], sb[t]), a.wide);
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
  a.wide = aligned(k, 32) && aligned(v, 32) &&
           ((a.tok[0] | a.tok[1] | a.bat[0] | a.bat[1]) & 15) == 0;
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

template <int L, int R, bool kWrite>
csbp_status launch(const CacheArgs& a, void* stream) {
  constexpr int64_t per = Shape<L, R>::kRows;
  const int64_t grid = (static_cast<int64_t>(a.batch) * a.rows + per - 1) / per;
  if (grid > 0x7fffffff) return CSBP_ERR_UNSUPPORTED;
  const dim3 g(static_cast<unsigned>(grid), 2);  // K, V
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int timed = timer_begin(kWrite ? 11 : 12, stream);
  if (kWrite)
    cache_write_kernel<L, R><<<g, kThreads, 0, s>>>(a);
  else
    cache_read_kernel<L, R><<<g, kThreads, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  timer_end(timed, stream);
  return e == cudaSuccess ? CSBP_OK : CSBP_ERR_CUDA;
}

// The fewest lanes that hold a row in one step (so that short rows share a
// warp), at most a warp; two rows per lane where one step is all (25,000 rows of
// 128 features, 8 sequences: write 30.0 us, read 27.8; four rows per lane 38.2
// and 28.4, one row and 16 lanes 81.5 and 58.7).  Few rows, up to one CTA of 16
// per SM, take one row per 16 lanes all the same: then latency counts (8 x 100
// rows: write 2.5 us, read 2.4, against 2.7 and 3.0; 8 x 500: 3.3 and 3.0
// against 2.9 and 3.0).
template <bool kWrite>
csbp_status launch(const CacheArgs& a, void* stream) {
  constexpr int kRows = 2;
  const int chunks = a.row_values >> 4;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return CSBP_ERR_CUDA;
  const bool few = static_cast<int64_t>(a.batch) * a.rows <= 16 * sms;
  if (chunks > 32 || (few && chunks > 16)) return launch<32, 1, kWrite>(a, stream);
  if (few) return launch<16, 1, kWrite>(a, stream);
  if (chunks <= 2) return launch<2, kRows, kWrite>(a, stream);
  if (chunks <= 4) return launch<4, kRows, kWrite>(a, stream);
  if (chunks <= 8) return launch<8, kRows, kWrite>(a, stream);
  if (chunks <= 16) return launch<16, kRows, kWrite>(a, stream);
  return launch<32, kRows, kWrite>(a, stream);
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
