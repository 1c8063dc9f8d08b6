// What the kernels that address the quantised paged K/V cache by rows share
// (csbp_generate.h): where a row of a sequence lies, and the checks of a cache
// and of the rows of a call.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "csbp_generate.h"

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

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Most elements that a strided bf16 tensor spans.
constexpr int64_t kMaxElems = int64_t(1) << 39;

inline csbp_status check_cache(const csbp_kv_cache* c) {
  if (!c) return CSBP_ERR_INVALID;
  if (c->pages < 1 || c->pages > 0x7fffffff || c->page_size < 1 || c->page_size > 65536 ||
      c->Hkv < 1 || c->Hkv > 65536 || c->d < kGroup || c->d > 1024 || c->d % kGroup != 0)
    return CSBP_ERR_INVALID;
  if (!c->k || !c->v || !c->k_scale || !c->v_scale) return CSBP_ERR_INVALID;
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return CSBP_ERR_INVALID;
  return CSBP_OK;
}

// Fills everything but src / dst.
inline csbp_status make_args(const csbp_kv_cache* c, const csbp_cache_rows* r, const void* k,
                      const void* v, CacheArgs& a) {
  const csbp_status st = check_cache(c);
  if (st != CSBP_OK) return st;
  if (!r) return CSBP_ERR_INVALID;
  if (r->batch < 0 || r->rows < 0 || r->table_pages < 0) return CSBP_ERR_INVALID;
  if (r->batch == 0 || r->rows == 0) return CSBP_OK;
  if (!r->table || !r->start || !k || !v) return CSBP_ERR_INVALID;
  if (!aligned(r->table, 4) || !aligned(r->start, 4) || (r->count && !aligned(r->count, 4)) ||
      !aligned(k, 16) || !aligned(v, 16))
    return CSBP_ERR_INVALID;
  const int64_t row = static_cast<int64_t>(c->Hkv) * c->d;  // <= 2^26
  // every element count stays below 2^62, tested by division
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

}  // namespace
}  // namespace csbp
