// What the kernels of csbp_attn_paged share: the problem as they see it, the list of
// steps that the CTAs take equal shares of, and operations on codes and scale bytes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "divisor.cuh"

namespace csbp {
namespace paged {

struct PagedParams {
  int32_t pages, page_size, Hkv, table_pages;
  const uint8_t *k, *v, *k_scale, *v_scale;
  int32_t batch, queries, Hq, G, causal, window, sinks;
  float scale_log2;
  const __nv_bfloat16* q;
  int64_t q_tok, q_bat;
  const int32_t *table, *length;
  __nv_bfloat16* o;
  float* lse;
  // how rows and heads are cut up
  int32_t heads, slices, head_blocks;  // KV heads and slices of a CTA, CTAs' worth of heads
  int32_t row_tiles;
  // of the list: CTA c has share c / lanes of lane c % lanes, which takes every
  // lanes-th block of heads
  int32_t lanes, lane_ctas, lane_blocks;
  int32_t step_keys;    // of a CTA
  int32_t wide_scales;  // scale bytes of a token are loaded in 4-byte words
  Divisor by_page, by_G, by_row_tiles, by_lanes, by_step;  // (step_keys)
  float* part_o;  // [2 x CTAs][heads][tile rows][d]
  float* part_z;  // [2 x CTAs][heads][tile rows]
  int2* pieces;   // per sequence, row tile and head block: first CTA, number of them (-1:
                  // one whole tile, `far`)
  int* arrived;   // in their place where the CTAs join them: how many are there, 0
                  // between launches
  // sums put aside: [CTAs x warps][tile rows][d], or [CTAs][tile rows][d] where a CTA
  // works on whole tiles, and their LSE
  float *aside_o, *aside_z;
  // of whole tiles, per partial: scales lie too far apart for f16 operands, the rows are
  // worked out again where the pieces are joined
  int* far;  // [2 x CTAs]
  int* status;
};

// ----------------------------------------------------------- instructions
// Copies of `n` bytes (16 or 4), or as many zeros (n = 0: nothing is read).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, int n) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
// Two E4M3 codes (of the low or the high half of a word) as f16, exact, NaN as NaN.
__device__ __forceinline__ uint32_t f16_low(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n}"
      : "=r"(r)
      : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t f16_high(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n}"
      : "=r"(r)
      : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float lg2_approx(float x) {
  float r;
  asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Sign bits of the bytes of a that are not below those of b.
__device__ __forceinline__ uint32_t at_least_u8x4(uint32_t a, uint32_t b) {
  const uint32_t t = (a | 0x80808080u) - (b & 0x7f7f7f7fu);
  return ((a & ~b) | (~(a ^ b) & t)) & 0x80808080u;
}
__device__ __forceinline__ bool any_byte_255(uint32_t w) {
  return ((~w - 0x01010101u) & w & 0x80808080u) != 0;
}
// Bytes of E4M3 NaN codes in a word, as 0xff.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  const uint32_t m = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
  return (m >> 7) * 0xffu;
}

// Whole row tiles, on the tensor-memory path (attn_paged_tiles.cu); its steps are tiles
// of 128 keys of one KV head.
constexpr int kPairRows = 256;
constexpr int kTileKeys = 128;

// ------------------------------------------------------------ the work list
// The keys that a row tile reads: [0, first) and [lo, hi), in steps.
struct Range {
  int c;           // keys of the sequence
  int first, lo, hi;
  int n_first, n;  // steps: of [0, first), and all (at least one)
  // Where both parts are one list (whole tiles: a step of a few sinks alone cost a tenth
  // of a window of 1,024), the key at place i of it, and its length.
  __device__ __forceinline__ int key(int i) const { return i < first ? i : i - first + lo; }
  __device__ __forceinline__ int keys() const { return first + hi - lo; }
};

// First key of the window of a query at position t.  (No difference of t and the window
// where it would be negative: with both near 2^31 it could pass 32 bits.)
__device__ __forceinline__ int window_begin(const PagedParams& p, int t) {
  return p.window == 0 || t < p.window ? 0 : t - p.window + 1;
}

__device__ __forceinline__ Range range_of(const PagedParams& p, int b, int tile, int tile_rows) {
  Range r;
  r.c = min(max(__ldg(p.length + b), 0), p.table_pages * p.page_size);
  const int i0 = p.by_G(tile * tile_rows);
  const int i1 = p.by_G(min((tile + 1) * tile_rows, p.queries * p.G) - 1);
  const int t0 = r.c - p.queries + i0, t1 = r.c - p.queries + i1;
  r.hi = p.causal ? max(t1 + 1, 0) : r.c;
  r.lo = min(window_begin(p, t0), r.hi);
  r.first = p.window ? min(p.sinks, r.lo) : 0;
  const int more = p.step_keys - 1;
  r.n_first = tile_rows == kPairRows ? 0 : p.by_step(r.first + more);
  const int others = tile_rows == kPairRows ? r.keys() : r.hi - r.lo;
  r.n = max(r.n_first + static_cast<int>(p.by_step(others + more)), 1);
  return r;
}

// A place in the list: entry (sequence, row tile), block of heads, step of it.
struct Cursor {
  int entry, block, step, b;
  Range r;
  __device__ __forceinline__ void load(const PagedParams& p, int tile_rows) {
    b = p.by_row_tiles(entry);
    if (b < p.batch) r = range_of(p, b, entry - b * p.row_tiles, tile_rows);
  }
};

struct Share {
  uint32_t begin, end, per;  // steps of the list (the host keeps it below 2^31)
};

// Adds all steps up and finds the CTA's share, and the cursor of its begin.
// `room`: a number per warp, and at kMostWarps the cursor.
template <int R, int kMostWarps>
__device__ __forceinline__ Share find_share(const PagedParams& p, uint32_t* room, Cursor& cur) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  const int entries = p.batch * p.row_tiles;
  Share s{0, 0, 0};
  uint32_t total = 0;
  // the total, then the begin; both at once where one sweep takes in all entries
  const bool one_sweep = entries <= static_cast<int>(blockDim.x);
#pragma unroll 1
  for (int pass = one_sweep ? 1 : 0; pass < 2; ++pass) {
    uint32_t before = 0;
#pragma unroll 1
    for (int e0 = 0; e0 < entries; e0 += blockDim.x) {
      Cursor here{e0 + tid, 0, 0, 0, {}};
      uint32_t mine = 0;
      if (here.entry < entries) {
        here.load(p, R);
        mine = static_cast<uint32_t>(here.r.n) * p.lane_blocks;
      }
      uint32_t sum = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
      }
      if (!one_sweep) __syncthreads();
      if (lane == 31) room[warp] = sum;
      __syncthreads();
      uint32_t all = 0;
#pragma unroll 1
      for (int w = 0; w < warps; ++w) {
        if (w < warp) sum += room[w];
        all += room[w];
      }
      if (one_sweep) total = all;
      if (pass == 1) {
        s.per = (total - 1) / p.lane_ctas + 1;
        s.begin = min(s.per * p.by_lanes(blockIdx.x), total);
        s.end = min(s.begin + s.per, total);
        const uint32_t from = before + sum - mine;
        if (s.begin >= from && s.begin < from + mine) {
          const int passed = (s.begin - from) / here.r.n;
          here.step = s.begin - from - passed * here.r.n;
          here.block = passed * p.lanes + blockIdx.x - p.by_lanes(blockIdx.x) * p.lanes;
          *reinterpret_cast<Cursor*>(room + kMostWarps) = here;
        }
      }
      before += all;
    }
    total = before;
  }
  __syncthreads();
  if (s.begin < s.end) cur = *reinterpret_cast<const Cursor*>(room + kMostWarps);
  return s;
}

cudaError_t launch_tiles(const PagedParams& p, int d, cudaStream_t stream);

}  // namespace paged
}  // namespace csbp
