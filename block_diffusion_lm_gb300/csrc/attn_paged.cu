// Attention of a few new tokens per sequence over the quantised paged K/V cache
// (csbp_generate.h), for sm_103a: softmax(scale q K^T) V with K and V read where
// they lie, once, in E4M3.
//
// Rows and keys.  The query rows of one KV head of a sequence are (token, head of
// the group), flattened; a row tile is up to 16 of them (8 where that is all: then
// half of the softmax is left out).  A row tile reads the keys that any of its rows
// reads, sinks first, then the window (or all), in steps of 16 keys per warp.  A
// warp takes one KV head and every S-th step of 16 keys; the CTA's warps are H heads
// x S such slices, so that the scale bytes of a token's heads, which share a 32-byte
// sector, are read by one CTA at one time.
//
// Work.  The steps of all sequences and row tiles, end to end, form one list that
// is cut into equal shares, one per SM: every CTA adds the lengths up and finds its
// share itself, so that lengths never come to the host.  A row tile that is cut
// leaves normalised fp32 partials with their LSE in the workspace, which a second
// kernel joins exactly ([Blog] "在线 softmax 合并：为什么分两段算仍是同一个注意力").
//
// Matrix products.  With at most 16 rows the tensor-memory path would write every K
// and V value to shared memory once more, as bf16, and that alone would bound it:
// the products are m16n8k16 warp MMAs, whose operands go from the codes to registers
// with one conversion per two values (E4M3 to f16 is exact).  Which feature or key
// is which k of an MMA is free as long as both operands agree, so a lane takes
// what lies side by side.
//   S = Q K^T  per group of 32 features in its own accumulator, which is then
//              scaled by the key's 2^e in fp32; Q is held in f16 with a power of
//              two per row (8 bits of mantissa, exact for elements down to 2^-23
//              of the row's largest).
//   O = P V    P is held in f16, as p 2^14 2^(e - E), with V's scale 2^e of the
//              key and group and E the largest so far: its rounding is 2^-12 of
//              p, or 2^-39 of the largest p v below f16's normal range.
// Maxima, sums, O and everything that is scaled are fp32.  The tensor cores'
// accumulator drops what is below its last place at every step of 16 keys: after
// 2,048 of them (2^-13) O is added to a second sum in shared memory.
//
// Keys that a row does not read.  Steps at the edge of a row's range are masked;
// there, NaN codes of V are taken out of the product and put back into the rows
// that read them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "csbp_generate.h"
#include "csbp_internal.h"
#include "device_once.h"
#include "divisor.cuh"
#include "kv_cache.cuh"
#include "ptx_sm100.cuh"

namespace csbp {
namespace {

constexpr size_t kStatusBytes = 256;
constexpr int kMaxWarps = 8;  // of a CTA: two per scheduler, for the registers
constexpr int kStages = 4;
constexpr int kKeys = 16;     // of a warp's step
constexpr int kFlush = 2048;  // steps that one accumulator takes in
constexpr float kShift = 14.f;  // p is held as p 2^14; a row's maximum may lag by 2^1

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
  int32_t wide_scales;  // scale bytes of a token are loaded in 4-byte words
  Divisor by_page, by_G, by_row_tiles;
  float* part_o;  // [2 x CTAs][heads][tile rows][d]
  float* part_z;  // [2 x CTAs][heads][tile rows]
  int2* pieces;   // per sequence, row tile and head block: first CTA, number of them
};

// ----------------------------------------------------------- instructions
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  const int n = there ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool there) {
  const int n = there ? 4 : 0;
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
// Two E4M3 codes (the low 16 bits) as f16, exact, NaN as NaN.
__device__ __forceinline__ uint32_t f16_of(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n}"
      : "=r"(r)
      : "r"(two));
  return r;
}
__device__ __forceinline__ uint32_t f16_of_high(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n}"
      : "=r"(r)
      : "r"(two));
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
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ------------------------------------------------------------ the work list
// The keys that a row tile reads: [0, first) and [lo, hi), in steps.
struct Range {
  int c;           // keys of the sequence
  int first, lo, hi;
  int n_first, n;  // steps: of [0, first), and all (at least one)
};

__device__ __forceinline__ Range range_of(const PagedParams& p, int b, int tile, int tile_rows) {
  Range r;
  r.c = min(max(__ldg(p.length + b), 0), p.table_pages * p.page_size);
  const int i0 = p.by_G(tile * tile_rows);
  const int i1 = p.by_G(min((tile + 1) * tile_rows, p.queries * p.G) - 1);
  const int t0 = r.c - p.queries + i0, t1 = r.c - p.queries + i1;
  r.hi = p.causal ? max(t1 + 1, 0) : r.c;
  r.lo = p.window ? max(t0 - p.window + 1, 0) : 0;
  r.lo = min(r.lo, r.hi);
  r.first = p.window ? min(p.sinks, r.lo) : 0;
  const int per = kKeys * p.slices;
  r.n_first = (r.first + per - 1) / per;
  r.n = max(r.n_first + (r.hi - r.lo + per - 1) / per, 1);
  return r;
}

// A place in the list: entry (sequence, row tile), block of heads, step.
struct Cursor {
  int entry, block, step;
  int b, tile;
  Range r;
  __device__ __forceinline__ void load(const PagedParams& p, int tile_rows) {
    b = p.by_row_tiles(entry);
    tile = entry - b * p.row_tiles;
    if (b < p.batch) r = range_of(p, b, tile, tile_rows);
  }
  __device__ __forceinline__ void next(const PagedParams& p, int tile_rows) {
    if (++step < r.n) return;
    step = 0;
    if (++block < p.head_blocks) return;
    block = 0;
    ++entry;
    load(p, tile_rows);
  }
};

struct Share {
  uint64_t total, per, begin, end;  // steps
};

// Adds all steps up and finds the CTA's share: (entry, block, step) of its begin.
__device__ __forceinline__ Share find_share(const PagedParams& p, int tile_rows, uint64_t* room,
                                            Cursor& cur) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  const int entries = p.batch * p.row_tiles;
  Share s{0, 0, 0, 0};
  // pass 0 finds the total; the begin is found in the same pass where one sweep
  // takes in all entries
  for (int pass = 0; pass < 2; ++pass) {
    uint64_t before = 0;
    for (int e0 = 0; e0 < entries; e0 += blockDim.x) {
      const int e = e0 + tid;
      uint64_t mine = 0;
      int n = 0;
      if (e < entries) {
        const int b = p.by_row_tiles(e);
        n = range_of(p, b, e - b * p.row_tiles, tile_rows).n;
        mine = static_cast<uint64_t>(n) * p.head_blocks;
      }
      uint64_t sum = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
      }
      __syncthreads();
      if (lane == 31) room[warp] = sum;
      __syncthreads();
      uint64_t all = 0;
      for (int w = 0; w < warps; ++w) {
        if (w < warp) sum += room[w];
        all += room[w];
      }
      const bool one_sweep = entries <= static_cast<int>(blockDim.x);
      if (pass == 0 && one_sweep) s.total = all;
      if (pass == 1 || one_sweep) {
        s.per = (s.total + gridDim.x - 1) / gridDim.x;
        s.begin = min(s.per * blockIdx.x, s.total);
        s.end = min(s.begin + s.per, s.total);
        const uint64_t from = before + sum - mine;
        if (s.begin >= from && s.begin < from + mine) {
          const uint32_t in = static_cast<uint32_t>(s.begin - from);
          room[kMaxWarps] = static_cast<uint64_t>(e);
          room[kMaxWarps + 1] = static_cast<uint64_t>(in / n) << 32 | in % n;
        }
      }
      before += all;
    }
    if (pass == 0) s.total = before;
    if (entries <= static_cast<int>(blockDim.x)) break;
  }
  __syncthreads();
  if (s.begin < s.end) {
    cur.entry = static_cast<int>(room[kMaxWarps]);
    cur.block = static_cast<int>(room[kMaxWarps + 1] >> 32);
    cur.step = static_cast<int>(room[kMaxWarps + 1]);
    cur.load(p, tile_rows);
  }
  return s;
}

// ------------------------------------------------------------ shared memory
template <int D, bool kHalf>
struct Rows {
  static constexpr int kRows = kHalf ? 8 : 16;  // of a tile
  static constexpr int kGroups = D / 32;
  // a warp's ring stage: K codes, V codes, scale words (K, V), which keys are there
  static constexpr int kCodes = kKeys * D;
  static constexpr int kWords = 2 * kCodes;
  static constexpr int kThere = kWords + 2 * kKeys * 4;
  static constexpr int kStage = kThere + 16;
  // the step's scales: fp32 of K [key][group], f16 of V [key][group]
  static constexpr int kScales = kStages * kStage;
  static constexpr int kScaleBytes = kKeys * kGroups * 6;
  // second sum: normalised O [row][D] and LSE (log2)
  static constexpr int kSum = kScales + kScaleBytes;
  static constexpr int kSumRow = D;
  static constexpr int kSumZ = kSum + kRows * kSumRow * 4;
  static constexpr int kWarpBytes = (kSumZ + kRows * 4 + 127) / 128 * 128;
  static constexpr int kRoom = 128;  // find_share, in front
  static constexpr int smem(int warps) { return kRoom + warps * kWarpBytes; }

  // Place of 32-byte group `g` of key row `r`: rows that are read together lie in
  // different banks (K: a lane quarter reads rows r .. r + 3; V: rows r, r + 2, ..)
  static __device__ __forceinline__ uint32_t k_at(int r, int g) {
    return r * D + (D == 128 ? (g ^ (r & 3)) : (g ^ ((r >> 1) & 1))) * 32;
  }
  static __device__ __forceinline__ uint32_t v_at(int r, int g) {
    const int q = ((r >> 1) & 7) | (r & 1) << 3;
    return q * D + (D == 128 ? (g ^ (q & 3)) : (g ^ ((q >> 1) & 1))) * 32;
  }
};
static_assert(Rows<128, false>::smem(kMaxWarps) <= 232448, "shared memory of a CTA");

// Where key row r of a step stands among the scales: the four that lane quarter t
// works with (2t, 2t + 1, 2t + 8, 2t + 9) side by side.
__device__ __forceinline__ int scale_place(int r) { return (r & 6) << 1 | (r & 1) | (r >> 3) << 1; }

// Byte-wise larger of two words.
__device__ __forceinline__ uint32_t max_u8x4(uint32_t a, uint32_t b) { return __vmaxu4(a, b); }
__device__ __forceinline__ bool any_byte_255(uint32_t w) {
  return ((~w - 0x01010101u) & w & 0x80808080u) != 0;
}
// Bytes of E4M3 NaN codes in a word, as 0xff.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  const uint32_t m = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
  return (m >> 7) * 0xffu;
}

// The keys of one step ahead: what the lane looked up for key row (lane & 15).
struct Ahead {
  int page, place, block;
};

template <int D, bool kHalf>
struct Kernel {
  using L = Rows<D, kHalf>;
  static constexpr int kG = L::kGroups;

  const PagedParams& p;
  const int lane, g, t, slice, head_in;
  const uint32_t mem;  // the warp's shared memory
  float* const sum;    // second sum
  float* const sum_z;

  // rows g and g + 8
  uint32_t q[kG][2][4];
  float acc[D / 8][4];
  float m[2], l[2], row_scale[2];
  int row_lo[2], row_hi[2];  // [lo, hi) of a row, besides the sinks
  int all_lo, all_hi;        // of the rows of the tile alike
  uint32_t top;              // E of each group, a byte each
  bool summed;               // the second sum holds something

  __device__ __forceinline__ Kernel(const PagedParams& p, uint8_t* smem)
      : p(p), lane(threadIdx.x & 31), g(lane >> 2), t(lane & 3),
        slice(static_cast<int>(threadIdx.x >> 5) / p.heads),
        head_in(static_cast<int>(threadIdx.x >> 5) % p.heads),
        mem(smem_u32(smem)), sum(reinterpret_cast<float*>(smem + L::kSum)),
        sum_z(reinterpret_cast<float*>(smem + L::kSumZ)) {}

  __device__ __forceinline__ Ahead look(Cursor& cur) const {
    const bool front = cur.step < cur.r.n_first;
    const int step = front ? cur.step : cur.step - cur.r.n_first;
    const int j = (front ? 0 : cur.r.lo) + (step * p.slices + slice) * kKeys + (lane & 15);
    Ahead a;
    const int entry = p.by_page(j);
    a.place = j - entry * p.page_size;
    a.block = cur.block;
    a.page = -1;
    if (j < (front ? cur.r.first : cur.r.hi))
      a.page = __ldg(p.table + static_cast<int64_t>(cur.b) * p.table_pages + entry);
    cur.next(p, L::kRows);
    return a;
  }

  // Starts the copies of a step into a stage of the ring.
  __device__ __forceinline__ void issue(const Ahead& a, int stage, uint32_t& pending) const {
    const uint32_t at = mem + stage * L::kStage;
    const int head = a.block * p.heads + head_in;
    const bool there = a.page >= 0 && a.page < p.pages && head < p.Hkv;
    const int slot = there ? a.page * p.page_size + a.place : -1;
    constexpr int kChunks = D / 16, kAtOnce = 32 / kChunks;
    const int chunk = lane % kChunks;
#pragma unroll
    for (int i = 0; i < kKeys / kAtOnce; ++i) {
      const int r = i * kAtOnce + lane / kChunks;
      const int from = __shfl_sync(0xffffffffu, slot, r);
      const int64_t row = (static_cast<int64_t>(max(from, 0)) * p.Hkv + head) * D + chunk * 16;
      const bool ok = from >= 0;
      copy16(at + L::k_at(r, chunk >> 1) + (chunk & 1) * 16, p.k + (ok ? row : 0), ok);
      copy16(at + L::kCodes + L::v_at(r, chunk >> 1) + (chunk & 1) * 16, p.v + (ok ? row : 0), ok);
    }
    // scale bytes of K (lanes 0 .. 15) and V; a key that is not there has 0
    const uint8_t* scales = lane < 16 ? p.k_scale : p.v_scale;
    const int64_t place = there ? (static_cast<int64_t>(slot) * p.Hkv + head) * kG : 0;
    if (p.wide_scales) {
      copy4(at + L::kWords + lane * 4, scales + (place & ~int64_t(3)), there);
    } else {
      uint32_t w = 0;
      if (there)
#pragma unroll
        for (int e = 0; e < kG; ++e) w |= static_cast<uint32_t>(__ldg(scales + place + e)) << 8 * e;
      pending = w;  // stored when the next step is issued, so that nobody waits here
    }
    const uint32_t is = __ballot_sync(0xffffffffu, there);
    if (lane == 0) sts32(at + L::kThere, is);
    copies_commit();
  }
  __device__ __forceinline__ void store_pending(int stage, uint32_t pending) const {
    if (!p.wide_scales) sts32(mem + stage * L::kStage + L::kWords + lane * 4, pending);
  }

  // Rows of a tile: queries to registers, and what each row reads.
  __device__ __forceinline__ void begin(const Cursor& cur) {
    const int head = cur.block * p.heads + head_in;
    const int rows = p.queries * p.G, row0 = cur.tile * L::kRows;
#pragma unroll
    for (int x = 0; x < (kHalf ? 1 : 2); ++x) {
      const int r = row0 + g + 8 * x;
      const int i = p.by_G(min(r, rows - 1)), gi = min(r, rows - 1) - i * p.G;
      uint4 raw[kG];
      const __nv_bfloat16* src =
          p.q + cur.b * p.q_bat + i * p.q_tok +
          (static_cast<int64_t>(min(head, p.Hkv - 1)) * p.G + gi) * D + t * 8;
#pragma unroll
      for (int e = 0; e < kG; ++e) raw[e] = __ldg(reinterpret_cast<const uint4*>(src + e * 32));
      uint32_t most = 0;
#pragma unroll
      for (int e = 0; e < kG; ++e) {
        const uint32_t w[4] = {raw[e].x, raw[e].y, raw[e].z, raw[e].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) most = max(most, max(w[k] & 0x7fffu, w[k] >> 16 & 0x7fffu));
      }
      most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
      // the largest element becomes 2^7 .. 2^8
      const int ex = max(static_cast<int>(most >> 7) - 127, -110);
      const float f = __uint_as_float(static_cast<uint32_t>(127 + 7 - ex) << 23);
      row_scale[x] = p.scale_log2 * ldexpf(1.f, ex - 7);
#pragma unroll
      for (int e = 0; e < kG; ++e) {
        const uint32_t w[4] = {raw[e].x, raw[e].y, raw[e].z, raw[e].w};
        uint32_t h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          h[k] = pack_f16(__uint_as_float(w[k] << 16) * f, __uint_as_float(w[k] & 0xffff0000u) * f);
        q[e][0][x] = h[0];
        q[e][0][x + 2] = h[1];
        q[e][1][x] = h[2];
        q[e][1][x + 2] = h[3];
      }
      const int at = cur.r.c - p.queries + i;
      row_hi[x] = p.causal ? at + 1 : cur.r.c;
      row_lo[x] = p.window ? at - p.window + 1 : 0;
    }
    if (kHalf) {
#pragma unroll
      for (int e = 0; e < kG; ++e) q[e][0][1] = q[e][0][3] = q[e][1][1] = q[e][1][3] = 0;
    }
    const int i0 = p.by_G(row0), i1 = p.by_G(min(row0 + L::kRows, rows) - 1);
    all_hi = p.causal ? cur.r.c - p.queries + i0 + 1 : cur.r.c;
    all_lo = p.window ? cur.r.c - p.queries + i1 - p.window + 1 : 0;
#pragma unroll
    for (int e = 0; e < D / 8; ++e)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[e][k] = 0.f;
    // (not -inf: a difference with a masked score has to stay a number)
    m[0] = m[1] = -3e38f;
    l[0] = l[1] = 0.f;
    top = 0;
    summed = false;
  }

  __device__ __forceinline__ bool reads(int x, int j) const {
    return j < row_hi[x] && (j >= row_lo[x] || j < p.sinks);
  }

  // E grows: what was summed under the old one is scaled.
  __device__ __forceinline__ void raise_top(uint32_t w) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) w = max_u8x4(w, __shfl_xor_sync(0xffffffffu, w, o));
    const uint32_t now = max_u8x4(top, w);
#pragma unroll
    for (int e = 0; e < kG; ++e) {
      const int by = static_cast<int>((now >> 8 * e & 255) - (top >> 8 * e & 255));
      const float f = by < 127 ? __uint_as_float(static_cast<uint32_t>(127 - by) << 23) : 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[4 * e + k][c] *= f;
    }
    top = now;
  }

  __device__ __forceinline__ void step(const Cursor& cur, int stage) {
    const uint32_t at = mem + stage * L::kStage;
    const uint32_t scales = mem + L::kScales, v_scales = scales + kKeys * kG * 4;
    // ------- the step's scales
    uint32_t word = lds32(at + L::kWords + lane * 4);
    const uint32_t there = lds32(at + L::kThere) & 0xffffu;
    if (D == 64 && p.wide_scales) {  // its half of the word
      const int head = cur.block * p.heads + head_in;
      word = head & 1 ? word >> 16 : word & 0xffffu;
    }
    const bool odd_scale = any_byte_255(word);
    const uint32_t v_word =
        lane < 16 ? 0 : odd_scale ? word & ~(__vcmpeq4(word, 0xffffffffu)) : word;
    if (__any_sync(0xffffffffu, max_u8x4(top, v_word) != top)) raise_top(v_word);
    const bool is_there = there >> (lane & 15) & 1;
    // byte by byte, nothing is borrowed
    const uint32_t delta = is_there ? top - v_word : 0;
    // f16 holds 2^-delta to delta = 14 (bytes of 4 (15 - delta)); more goes another way
    bool special = lane >= 16 && (odd_scale || ((delta + 0x71717171u) & 0x80808080u) != 0 ||
                                  (delta & 0x80808080u) != 0);
    if (D == 64) special = lane >= 16 && (odd_scale || ((delta + 0x00007171u) & 0x8080u) != 0 ||
                                          (delta & 0x8080u) != 0);
    special = __any_sync(0xffffffffu, special && is_there);
    __syncwarp();  // (the scales of the step before have been read)
    {
      const int place = scale_place(lane & 15);
      if (lane < 16) {
        float f[kG];
#pragma unroll
        for (int e = 0; e < kG; ++e) {
          const uint32_t b = word >> 8 * e & 255;
          f[e] = __uint_as_float(b == 255 ? 0x7fffffffu : max(b << 23, 0x00400000u));
        }
        if constexpr (kG == 4)
          asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(scales + place * 16), "f"(f[0]),
                       "f"(f[1]), "f"(f[2]), "f"(f[3])
                       : "memory");
        else
          asm volatile("st.shared.v2.f32 [%0], {%1,%2};" ::"r"(scales + place * 8), "f"(f[0]),
                       "f"(f[1])
                       : "memory");
      } else {
        // upper bytes of the f16 numbers 2^-delta
        const uint32_t h = 0x3c3c3c3cu - (delta << 2 & 0xfcfcfcfcu);
        if constexpr (kG == 4)
          asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(v_scales + place * 8),
                       "r"(__byte_perm(h, 0, 0x1404)), "r"(__byte_perm(h, 0, 0x3424))
                       : "memory");
        else
          sts32(v_scales + place * 4, __byte_perm(h, 0, 0x1404));
      }
    }
    __syncwarp();

    // ------- S = Q K^T
    float s[2][4];
    {
      float ks[4][kG];  // of keys 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (kG == 4)
          asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                       : "=f"(ks[k][0]), "=f"(ks[k][1]), "=f"(ks[k][2]), "=f"(ks[k][3])
                       : "r"(scales + (4 * t + k) * 16)
                       : "memory");
        else
          asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];"
                       : "=f"(ks[k][0]), "=f"(ks[k][1])
                       : "r"(scales + (4 * t + k) * 8)
                       : "memory");
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int e = 0; e < kG; ++e) {
          const uint2 w = lds64(at + L::k_at(8 * x + g, e) + 8 * t);
          float c[4] = {0.f, 0.f, 0.f, 0.f};
          mma(c, q[e][0], f16_of(w.x), f16_of_high(w.x));
          mma(c, q[e][1], f16_of(w.y), f16_of_high(w.y));
          if (e == 0) {
            s[x][0] = c[0] * ks[2 * x][0];
            s[x][1] = c[1] * ks[2 * x + 1][0];
            s[x][2] = c[2] * ks[2 * x][0];
            s[x][3] = c[3] * ks[2 * x + 1][0];
          } else {
            s[x][0] = fmaf(c[0], ks[2 * x][e], s[x][0]);
            s[x][1] = fmaf(c[1], ks[2 * x + 1][e], s[x][1]);
            s[x][2] = fmaf(c[2], ks[2 * x][e], s[x][2]);
            s[x][3] = fmaf(c[3], ks[2 * x + 1][e], s[x][3]);
          }
        }
      }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int k = 0; k < (kHalf ? 2 : 4); ++k) s[x][k] *= row_scale[k >> 1];

    // ------- mask
    const bool front = cur.step < cur.r.n_first;
    const int j0 = (front ? 0 : cur.r.lo) +
                   ((front ? cur.step : cur.step - cur.r.n_first) * p.slices + slice) * kKeys;
    const bool inside = there == 0xffffu && j0 + kKeys <= all_hi &&
                        (j0 >= all_lo || j0 + kKeys <= p.sinks);
    if (!inside) {
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int k = 0; k < (kHalf ? 2 : 4); ++k) {
          const int r = 8 * x + 2 * t + (k & 1);
          if (!(there >> r & 1) || !reads(k >> 1, j0 + r)) s[x][k] = -INFINITY;
        }
    }

    // ------- softmax
    const float most0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
    const float most1 = kHalf ? 0.f : fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
    if (__any_sync(0xffffffffu, most0 > m[0] + 1.f || (!kHalf && most1 > m[1] + 1.f))) {
#pragma unroll
      for (int x = 0; x < (kHalf ? 1 : 2); ++x) {
        float most = x ? most1 : most0;
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
        const float now = fmaxf(m[x], most), f = ex2_approx(m[x] - now);
        m[x] = now;
        l[x] *= f;
#pragma unroll
        for (int e = 0; e < D / 8; ++e) {
          acc[e][2 * x] *= f;
          acc[e][2 * x + 1] *= f;
        }
      }
    }
    float pr[2][4];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int k = 0; k < (kHalf ? 2 : 4); ++k) pr[x][k] = ex2_approx(s[x][k] - (m[k >> 1] - kShift));
    l[0] += (pr[0][0] + pr[0][1]) + (pr[1][0] + pr[1][1]);
    if (!kHalf) l[1] += (pr[0][2] + pr[0][3]) + (pr[1][2] + pr[1][3]);

    // ------- P under V's scales, a set for each group
    uint32_t a[kG][4];
    if (!special) {
      uint32_t pa[4];
      pa[0] = pack_f16(pr[0][0], pr[0][1]);
      pa[2] = pack_f16(pr[1][0], pr[1][1]);
      if (!kHalf) {
        pa[1] = pack_f16(pr[0][2], pr[0][3]);
        pa[3] = pack_f16(pr[1][2], pr[1][3]);
      }
      uint32_t vs[4][kG / 2];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (kG == 4) {
          const uint2 w = lds64(v_scales + (4 * t + k) * 8);
          vs[k][0] = w.x;
          vs[k][1] = w.y;
        } else {
          vs[k][0] = lds32(v_scales + (4 * t + k) * 4);
        }
      }
#pragma unroll
      for (int e = 0; e < kG; ++e) {
        const int which = e & 1 ? 0x7632 : 0x5410;
        const uint32_t s01 = __byte_perm(vs[0][e >> 1], vs[1][e >> 1], which);
        const uint32_t s23 = __byte_perm(vs[2][e >> 1], vs[3][e >> 1], which);
        a[e][0] = mul_f16x2(pa[0], s01);
        a[e][2] = mul_f16x2(pa[2], s23);
        a[e][1] = kHalf ? 0 : mul_f16x2(pa[1], s01);
        a[e][3] = kHalf ? 0 : mul_f16x2(pa[3], s23);
      }
    } else {
      // in fp32: scales far below the largest, or NaN (in the rows that read the key)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        uint32_t w[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int r = 8 * x + 2 * t + k;
          w[k] = lds32(at + L::kWords + (16 + r) * 4);
          if (D == 64 && p.wide_scales && ((cur.block * p.heads + head_in) & 1)) w[k] >>= 16;
        }
#pragma unroll
        for (int e = 0; e < kG; ++e) {
          float f[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < (kHalf ? 2 : 4); ++k) {
            const int b = static_cast<int>(w[k & 1] >> 8 * e & 255);
            const int by = static_cast<int>(top >> 8 * e & 255) - b;
            const float scale = b == 255 ? NAN : by < 127 ? __uint_as_float((127u - by) << 23) : 0.f;
            if (s[x][k] != -INFINITY) f[k] = pr[x][k] * scale;
          }
          a[e][2 * x] = pack_f16(f[0], f[1]);
          a[e][2 * x + 1] = pack_f16(f[2], f[3]);
        }
      }
    }

    // ------- O += P V
    const uint32_t v = at + L::kCodes + 4 * g;
    bool bad = false;
    if (!inside) {
#pragma unroll
      for (int e = 0; e < kG; ++e)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          bad |= nan_codes(lds32(v + L::v_at(2 * t + (k & 1) + (k >> 1) * 8, e))) != 0;
      bad = __any_sync(0xffffffffu, bad);
    }
    if (!bad) {
#pragma unroll
      for (int e = 0; e < kG; ++e) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = lds32(v + L::v_at(2 * t + (k & 1) + (k >> 1) * 8, e));
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t lo = __byte_perm(w[0], w[1], k ? 0x7362 : 0x5140);
          const uint32_t hi = __byte_perm(w[2], w[3], k ? 0x7362 : 0x5140);
          mma(acc[4 * e + 2 * k], a[e], f16_of(lo), f16_of(hi));
          mma(acc[4 * e + 2 * k + 1], a[e], f16_of_high(lo), f16_of_high(hi));
        }
      }
    } else {
      // NaN codes as 0 in the product, then NaN wherever a row reads one of them
      uint32_t sees[4] = {0, 0, 0, 0};
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        sees[2 * x] = pack_f16(s[x][0] != -INFINITY, s[x][1] != -INFINITY);
        if (!kHalf) sees[2 * x + 1] = pack_f16(s[x][2] != -INFINITY, s[x][3] != -INFINITY);
      }
#pragma unroll 1
      for (int e = 0; e < kG; ++e) {
        uint32_t w[4], is[4], ae[4] = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          w[k] = lds32(v + L::v_at(2 * t + (k & 1) + (k >> 1) * 8, e));
          is[k] = nan_codes(w[k]);
          w[k] &= ~is[k];
          is[k] &= 0x38383838u;  // 1
        }
#pragma unroll
        for (int c = 0; c < kG; ++c)
#pragma unroll
          for (int k = 0; k < 4; ++k) ae[k] = c == e ? a[c][k] : ae[k];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t pick = k & 2 ? 0x7362 : 0x5140;
          const uint32_t lo = __byte_perm(w[0], w[1], pick), hi = __byte_perm(w[2], w[3], pick);
          const uint32_t nlo = __byte_perm(is[0], is[1], pick), nhi = __byte_perm(is[2], is[3], pick);
          float add[4] = {0.f, 0.f, 0.f, 0.f}, n[4] = {0.f, 0.f, 0.f, 0.f};
          mma(add, ae, k & 1 ? f16_of_high(lo) : f16_of(lo), k & 1 ? f16_of_high(hi) : f16_of(hi));
          mma(n, sees, k & 1 ? f16_of_high(nlo) : f16_of(nlo), k & 1 ? f16_of_high(nhi) : f16_of(nhi));
#pragma unroll
          for (int c = 0; c < kG; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (c == e) acc[4 * c + k][i] += n[i] > 0.f ? NAN : add[i];
        }
      }
    }
  }

  // Adds what the registers hold to the second sum (normalised, with its LSE) and
  // starts anew.
  __device__ __forceinline__ void store_sum() {
#pragma unroll
    for (int x = 0; x < (kHalf ? 1 : 2); ++x) {
      float z = l[x];
      z += __shfl_xor_sync(0xffffffffu, z, 1);
      z += __shfl_xor_sync(0xffffffffu, z, 2);
      const int row = g + 8 * x;
      const float inv = z == 0.f ? 0.f : 1.f / z;
      const float lse = z == 0.f ? -INFINITY : m[x] - kShift + log2f(z);
      float mine = 1.f, old = 0.f, all = lse;
      if (summed) {
        const float before = sum_z[row], most = fmaxf(before, lse);
        const float ref = most == -INFINITY ? 0.f : most;
        old = exp2f(before - ref);
        mine = exp2f(lse - ref);
        const float both = old + mine;
        all = both == 0.f ? -INFINITY : ref + log2f(both);
        const float f = both == 0.f ? 0.f : 1.f / both;
        old *= f;
        mine *= f;
      }
      __syncwarp();
      if (t == 0) sum_z[row] = all;
#pragma unroll
      for (int e = 0; e < kG; ++e) {
        // 2^(E - 127), in two steps: the first may lie below fp32's range alone
        const int ex = static_cast<int>(top >> 8 * e & 255);
        const float f0 = __uint_as_float(static_cast<uint32_t>(ex / 2 + 64) << 23);
        const float f1 = __uint_as_float(static_cast<uint32_t>(ex - ex / 2 + 63) << 23);
        float* to = sum + row * L::kSumRow + 32 * e + 8 * t;
        float v[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[k] = acc[4 * e + k][2 * x] * inv * f0 * f1;
          v[4 + k] = acc[4 * e + k][2 * x + 1] * inv * f0 * f1;
        }
        if (summed) {
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = to[k] * old + v[k] * mine;
        }
        reinterpret_cast<float4*>(to)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(to)[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
      l[x] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < D / 8; ++e)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[e][k] = 0.f;
    summed = true;
    __syncwarp();
  }

  // The rows of a piece, joined over the slices: to the outputs where the piece is
  // the whole of a row's keys (`part` < 0), else to a place among the partials.
  __device__ __forceinline__ void finish(const Cursor& cur, int part, const uint8_t* warps) const {
    const int head = cur.block * p.heads + head_in;
    if (head >= p.Hkv) return;
    const int rows = min(L::kRows, p.queries * p.G - cur.tile * L::kRows);
    const uint8_t* first = warps + head_in * L::kWarpBytes;  // slice 0 of the head
    const int64_t stride = static_cast<int64_t>(p.heads) * L::kWarpBytes;
    constexpr int kLanes = D / 4;
    for (int x = slice * 32 + lane; x < rows * kLanes; x += p.slices * 32) {
      const int row = x / kLanes, f = x % kLanes * 4;
      float most = -INFINITY;
      for (int s = 0; s < p.slices; ++s)
        most = fmaxf(most, reinterpret_cast<const float*>(first + s * stride + L::kSumZ)[row]);
      const float ref = most == -INFINITY ? 0.f : most;
      float both = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int s = 0; s < p.slices; ++s) {
        const float z = reinterpret_cast<const float*>(first + s * stride + L::kSumZ)[row];
        if (z == -INFINITY) continue;  // it has read nothing
        const float w = exp2f(z - ref);
        const float4 v = *reinterpret_cast<const float4*>(
            reinterpret_cast<const float*>(first + s * stride + L::kSum) + row * L::kSumRow + f);
        both += w;
        o.x = fmaf(w, v.x, o.x);
        o.y = fmaf(w, v.y, o.y);
        o.z = fmaf(w, v.z, o.z);
        o.w = fmaf(w, v.w, o.w);
      }
      const float inv = both == 0.f ? 0.f : 1.f / both;
      const float z = both == 0.f ? -INFINITY : ref + log2f(both);
      o.x *= inv;
      o.y *= inv;
      o.z *= inv;
      o.w *= inv;
      if (part < 0) {
        const int r = cur.tile * L::kRows + row, i = p.by_G(r), h = head * p.G + r - i * p.G;
        const int64_t token = static_cast<int64_t>(cur.b) * p.queries + i;
        *reinterpret_cast<uint2*>(p.o + (token * p.Hq + h) * D + f) =
            make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
        if (f == 0)
          p.lse[(static_cast<int64_t>(cur.b) * p.Hq + h) * p.queries + i] = z * 0.6931471805599453f;
      } else {
        const int64_t at = (static_cast<int64_t>(part) * p.heads + head_in) * L::kRows + row;
        *reinterpret_cast<float4*>(p.part_o + at * D + f) = o;
        if (f == 0) p.part_z[at] = z;
      }
    }
  }
};

template <int D, bool kHalf>
__global__ void __launch_bounds__(kMaxWarps * 32, 1)
    paged_rows_kernel(const __grid_constant__ PagedParams p) {
  using L = Rows<D, kHalf>;
  extern __shared__ __align__(1024) uint8_t smem[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5;
  Cursor ahead{};
  const Share share = find_share(p, L::kRows, reinterpret_cast<uint64_t*>(smem), ahead);
  if (share.begin >= share.end) return;
  uint8_t* warps = smem + L::kRoom;
  Kernel<D, kHalf> k(p, warps + warp * L::kWarpBytes);
  Cursor cur = ahead;
  const uint32_t steps = static_cast<uint32_t>(share.end - share.begin);
  uint32_t pending = 0;
  uint32_t issued = 0;
  // the first steps' tables are looked up together: one wait for all
  {
    Ahead a[kStages - 1];
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      a[i] = Ahead{-1, 0, 0};
      if (i < static_cast<int>(steps)) a[i] = k.look(ahead);
    }
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      if (i < static_cast<int>(steps)) {
        k.issue(a[i], i, pending);
        k.store_pending(i, pending);
        ++issued;
      } else {
        copies_commit();
      }
    }
  }
  Ahead next{-1, 0, 0};
  if (issued < steps) next = k.look(ahead);
  int pending_stage = -1;
  bool fresh = true;
  int in_sum = 0;
  for (uint32_t i = 0; i < steps; ++i) {
    if (fresh) {
      k.begin(cur);
      fresh = false;
      in_sum = 0;
    }
    copies_wait<kStages - 2>();
    if (pending_stage >= 0) k.store_pending(pending_stage, pending);
    pending_stage = -1;
    __syncwarp();
    if (issued < steps) {
      pending_stage = issued % kStages;
      k.issue(next, pending_stage, pending);
      if (++issued < steps) next = k.look(ahead);
    } else {
      copies_commit();
    }
    k.step(cur, i % kStages);
    const bool ends = cur.step + 1 == cur.r.n || i + 1 == steps;
    if (++in_sum == kFlush || ends) {
      k.store_sum();
      in_sum = 0;
    }
    if (ends) {
      // the item's first and last step in the list, and the CTAs that these are in
      const uint64_t first = share.begin + i - cur.step;
      const uint32_t from = static_cast<uint32_t>(first / share.per);
      const uint32_t pieces = static_cast<uint32_t>((first + cur.r.n - 1) / share.per) - from + 1;
      const bool starts = from == blockIdx.x;
      if (starts && threadIdx.x == 0)
        p.pieces[static_cast<int64_t>(cur.entry) * p.head_blocks + cur.block] =
            make_int2(static_cast<int>(from), static_cast<int>(pieces));
      // a CTA leaves at most two partials: where an item ends or goes through (0)
      // and where one begins (1)
      const int part = pieces == 1 ? -1 : 2 * static_cast<int>(blockIdx.x) + (starts ? 1 : 0);
      if (p.slices > 1) __syncthreads();
      k.finish(cur, part, warps);
      if (p.slices > 1) __syncthreads();
      else __syncwarp();
      fresh = true;
    }
    cur.next(p, L::kRows);
  }
  copies_wait<0>();
}

// Joins the partials of a row tile that was cut; a CTA per head of it.
template <int D, bool kHalf>
__global__ void __launch_bounds__(128) paged_join_kernel(const __grid_constant__ PagedParams p) {
  constexpr int kRows = Rows<D, kHalf>::kRows, kLanes = D / 4;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int item = blockIdx.x, head_in = blockIdx.y;
  const int2 piece = p.pieces[item];
  if (piece.y <= 1) return;
  const int entry = item / p.head_blocks, block = item - entry * p.head_blocks;
  const int b = p.by_row_tiles(entry), tile = entry - b * p.row_tiles;
  const int head = block * p.heads + head_in;
  if (head >= p.Hkv) return;
  const int rows = min(kRows, p.queries * p.G - tile * kRows);
  for (int x = threadIdx.x; x < rows * kLanes; x += 128) {
    const int row = x / kLanes, f = x % kLanes * 4;
    float most = -INFINITY, both = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    // the first piece is where the item begins, the others are their CTAs' first
    const auto place = [&](int k) {
      return (static_cast<int64_t>(2 * (piece.x + k) + (k == 0)) * p.heads + head_in) * kRows + row;
    };
#pragma unroll 4
    for (int k = 0; k < piece.y; ++k) most = fmaxf(most, p.part_z[place(k)]);
    const float ref = most == -INFINITY ? 0.f : most;
#pragma unroll 4
    for (int k = 0; k < piece.y; ++k) {
      const float z = p.part_z[place(k)], w = exp2f(z - ref);
      const float4 v = *reinterpret_cast<const float4*>(p.part_o + place(k) * D + f);
      if (z == -INFINITY) continue;  // it has read nothing
      both += w;
      o.x = fmaf(w, v.x, o.x);
      o.y = fmaf(w, v.y, o.y);
      o.z = fmaf(w, v.z, o.z);
      o.w = fmaf(w, v.w, o.w);
    }
    const float inv = both == 0.f ? 0.f : 1.f / both;
    const float z = both == 0.f ? -INFINITY : ref + log2f(both);
    const int r = tile * kRows + row, i = p.by_G(r), h = head * p.G + r - i * p.G;
    const int64_t token = static_cast<int64_t>(b) * p.queries + i;
    *reinterpret_cast<uint2*>(p.o + (token * p.Hq + h) * D + f) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (f == 0)
      p.lse[(static_cast<int64_t>(b) * p.Hq + h) * p.queries + i] = z * 0.6931471805599453f;
  }
}

// ------------------------------------------------------------------- host
// How the heads and rows of a problem are cut up: H x S warps to a CTA, as many
// as can be with as few heads of the last CTA missing.
struct Cut {
  int heads, slices, head_blocks, row_tiles, tile_rows;
  int64_t items;
};

Cut cut_of(const csbp_paged_problem& p, const csbp_kv_cache& c) {
  Cut r{};
  double best = 0;
  for (int h = 1; h <= std::min(kMaxWarps, c.Hkv); ++h) {
    const int blocks = (c.Hkv + h - 1) / h, s = kMaxWarps / h;
    const double busy = static_cast<double>(h) * s * c.Hkv / (static_cast<double>(blocks) * h);
    if (busy >= best) {
      best = busy;
      r.heads = h;
      r.slices = s;
      r.head_blocks = blocks;
    }
  }
  const int64_t rows = static_cast<int64_t>(p.queries) * (p.Hq / c.Hkv);
  r.tile_rows = rows <= 8 ? 8 : 16;
  r.row_tiles = static_cast<int>((rows + r.tile_rows - 1) / r.tile_rows);
  r.items = static_cast<int64_t>(p.batch) * r.row_tiles * r.head_blocks;
  return r;
}

csbp_status validate(const csbp_paged_problem* p, const csbp_kv_cache* c) {
  if (!p || !c) return CSBP_ERR_INVALID;
  if (p->batch < 1 || p->queries < 1 || p->table_pages < 1 || p->Hq < 1 || p->causal < 0 ||
      p->causal > 1 || p->window < 0 || p->sinks < 0 || !(p->scale > 0.f) ||
      !std::isfinite(p->scale))
    return CSBP_ERR_INVALID;
  if (c->page_size < 1 || c->page_size > 65536 || c->Hkv < 1 || c->Hkv > 65536 ||
      c->d < kGroup || c->d > 1024 || c->d % kGroup != 0 || p->Hq % c->Hkv != 0)
    return CSBP_ERR_INVALID;
  if (c->d != 64 && c->d != 128) return CSBP_ERR_UNSUPPORTED;
  // keys, rows and work items are counted in 32 bits
  if (static_cast<int64_t>(p->table_pages) * c->page_size > 0x7fffffff - 1024)
    return CSBP_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(p->batch) * p->queries > 0x3fffffff / p->Hq)
    return CSBP_ERR_UNSUPPORTED;
  return CSBP_OK;
}

bool device_sms(int& sms) {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess &&
         cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess &&
         sms > 0;
}

size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct Places {
  size_t part_z, pieces, bytes;
};
Places places(const Cut& cut, int d, int sms) {
  const size_t rows = static_cast<size_t>(2) * sms * cut.heads * cut.tile_rows;
  Places r;
  r.part_z = kStatusBytes + round256(rows * d * 4);
  r.pieces = r.part_z + round256(rows * 4);
  r.bytes = r.pieces + round256(static_cast<size_t>(cut.items) * sizeof(int2));
  return r;
}

template <int D, bool kHalf>
cudaError_t launch(const PagedParams& p, const Cut& cut, int sms, cudaStream_t stream) {
  using L = Rows<D, kHalf>;
  static PerDeviceOnce configured;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!configured.run(dev, [&](int) {
        e = cudaFuncSetAttribute(paged_rows_kernel<D, kHalf>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, L::smem(kMaxWarps));
        return e == cudaSuccess;
      }))
    return e != cudaSuccess ? e : cudaErrorInvalidDevice;
  const int warps = cut.heads * cut.slices;
  const int timed = timer_begin(13, stream);
  paged_rows_kernel<D, kHalf><<<sms, warps * 32, L::smem(warps), stream>>>(p);
  e = cudaGetLastError();
  timer_end(timed, stream);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(cut.items), static_cast<unsigned>(cut.heads));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  const int joined = timer_begin(14, stream);
  e = cudaLaunchKernelEx(&cfg, paged_join_kernel<D, kHalf>, p);
  timer_end(joined, stream);
  return e;
}

}  // namespace
}  // namespace csbp

using namespace csbp;

extern "C" size_t csbp_paged_workspace_bytes(const csbp_paged_problem* problem,
                                             const csbp_kv_cache* cache) {
  if (validate(problem, cache) != CSBP_OK) return 0;
  int sms = 0;
  if (!device_sms(sms)) sms = 152;  // no GPU: the GB300's count
  return places(cut_of(*problem, *cache), cache->d, sms).bytes;
}

extern "C" csbp_status csbp_attn_paged(const csbp_paged_problem* problem,
                                       const csbp_kv_cache* cache, const csbp_paged_inputs* in,
                                       void* o, float* lse, void* workspace, size_t ws_bytes,
                                       void* stream) {
  csbp_status st = validate(problem, cache);
  if (st != CSBP_OK) return st;
  if ((st = check_cache(cache)) != CSBP_OK) return st;
  if (!in || !in->q || !in->table || !in->length || !aligned(in->q, 16) ||
      !aligned(in->table, 4) || !aligned(in->length, 4))
    return CSBP_ERR_INVALID;
  if (!o || !lse || !workspace || !aligned(o, 16) || !aligned(lse, 4) || !aligned(workspace, 16))
    return CSBP_ERR_INVALID;
  const csbp_paged_problem& p = *problem;
  const int64_t row = static_cast<int64_t>(p.Hq) * cache->d;
  PagedParams a{};
  if (in->stride_tok < 0 || in->stride_batch < 0) return CSBP_ERR_INVALID;
  a.q_tok = in->stride_tok != 0 ? in->stride_tok : row;
  if (a.q_tok < row || a.q_tok % 8 != 0 || a.q_tok > (kMaxElems - 1) / p.queries)
    return CSBP_ERR_INVALID;
  const int64_t span = a.q_tok * p.queries;
  a.q_bat = (p.batch > 1 && in->stride_batch != 0) ? in->stride_batch : span;
  if (a.q_bat < span || a.q_bat % 8 != 0 || a.q_bat >= kMaxElems) return CSBP_ERR_INVALID;
  if (ws_bytes < kStatusBytes) return CSBP_ERR_WORKSPACE;
  // places in the cache are counted in 32 bits
  if (cache->pages * cache->page_size > 0x7fffffff) return CSBP_ERR_UNSUPPORTED;
  int sms = 0;
  if (!device_sms(sms)) sms = 152;
  const Cut cut = cut_of(p, *cache);
  const Places at = places(cut, cache->d, sms);
  if (ws_bytes < at.bytes) return CSBP_ERR_WORKSPACE;
  a.pages = static_cast<int32_t>(cache->pages);
  a.page_size = cache->page_size;
  a.Hkv = cache->Hkv;
  a.table_pages = p.table_pages;
  a.k = static_cast<const uint8_t*>(cache->k);
  a.v = static_cast<const uint8_t*>(cache->v);
  a.k_scale = static_cast<const uint8_t*>(cache->k_scale);
  a.v_scale = static_cast<const uint8_t*>(cache->v_scale);
  a.batch = p.batch;
  a.queries = p.queries;
  a.Hq = p.Hq;
  a.G = p.Hq / cache->Hkv;
  a.causal = p.causal;
  // a window that no position can leave is none
  a.window = p.window >= p.table_pages * cache->page_size ? 0 : p.window;
  a.sinks = p.sinks;
  a.scale_log2 = p.scale * 1.4426950408889634f;
  a.q = static_cast<const __nv_bfloat16*>(in->q);
  a.table = in->table;
  a.length = in->length;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  a.heads = cut.heads;
  a.slices = cut.slices;
  a.head_blocks = cut.head_blocks;
  a.row_tiles = cut.row_tiles;
  a.wide_scales = aligned(cache->k_scale, 4) && aligned(cache->v_scale, 4) &&
                  cache->Hkv * (cache->d / kGroup) % 4 == 0;
  a.by_page = Divisor::of(static_cast<uint32_t>(cache->page_size));
  a.by_G = Divisor::of(static_cast<uint32_t>(a.G));
  a.by_row_tiles = Divisor::of(static_cast<uint32_t>(cut.row_tiles));
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.part_o = reinterpret_cast<float*>(ws + kStatusBytes);
  a.part_z = reinterpret_cast<float*>(ws + at.part_z);
  a.pieces = reinterpret_cast<int2*>(ws + at.pieces);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool half = cut.tile_rows == 8;
  const cudaError_t e = cache->d == 128
                            ? (half ? launch<128, true>(a, cut, sms, s) : launch<128, false>(a, cut, sms, s))
                            : (half ? launch<64, true>(a, cut, sms, s) : launch<64, false>(a, cut, sms, s));
  return e == cudaSuccess ? CSBP_OK : CSBP_ERR_CUDA;
}
