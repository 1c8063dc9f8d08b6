// Attention of a few new tokens per sequence over the quantised paged K/V cache
// (csbp_generate.h), for sm_103a: softmax(scale q K^T) V with K and V read where
// they lie, once, in E4M3.
//
// Rows and keys.  The query rows of one KV head of a sequence are (token, head of
// the group), flattened; a row tile is 8 or 16 of them.  A row tile reads the
// keys that any of its rows reads, sinks first, then the window (or all), in steps
// of 32 keys per warp.  A warp takes one KV head and every S-th step of 32 keys; the
// CTA's warps are H heads x S such slices, so that the scale bytes of a token's
// heads, which share a 32-byte sector, are read by one CTA at one time.
//
// Work.  The steps of all sequences and row tiles, end to end, form one list that
// is cut into equal shares, one per SM (or, where a token's heads take several CTAs,
// as many per group of SMs: the CTAs of a group read the same tokens at the same
// time, and sectors of scale bytes that they share come from DRAM once): every CTA adds
// the lengths up and finds its share itself, so that lengths never come to the host.  A
// row tile that is cut leaves normalised fp32 partials with their LSE in the workspace,
// which are joined exactly, by the last CTA that leaves one or by a second kernel
// ([Blog] "在线 softmax 合并：为什么分两段算仍是同一个注意力").
//
// Matrix products.  With so few rows the tensor-memory path would write every K and
// V value to shared memory once more, as bf16, and that alone would bound it: the
// products are m16n8k16 warp MMAs, whose operands go from the codes to registers
// with one conversion per two values (E4M3 to f16 is exact).  Keys or features are
// the 16 and query rows the 8, so that 8 rows waste nothing:
//   S^T = K Q^T  per group of 32 features in its own accumulator, which is then
//                scaled by the key's 2^e in fp32; Q is held in f16 with a power
//                of two per row (8 bits of mantissa, exact for elements down to
//                2^-23 of the row's largest).
//   O^T = V^T P^T  P is held in f16, as p 2^14 2^(e - E), with V's scale 2^e of the
//                key and group and E the largest so far, at most 2^14 above it: its
//                rounding is 2^-11 of p, or 2^-25 of the row's largest p below f16's
//                normal range.
// Scales of V farther apart than that would let a key wipe out others, in rows that do not
// read it or give it next to no weight, too.  They are rare (of a step's 32 keys a value
// 2^14 times another's largest): keys of a step that are near one another are summed by
// themselves then, and the sums before and after are put aside and joined in fp32.
// ldmatrix brings K's codes as four features of a key and, transposed, V's as four
// keys of a feature; which of the 16 keys is which row of the first product is
// chosen so that P^T needs one transposition of 8 x 8 for the second.
// Maxima, sums, O and everything that is scaled are fp32.  The tensor cores'
// accumulator drops what is below its last place at every MMA of 16 keys: after
// 2,048 of them (2^-13) O is put aside in the workspace and a new sum begun.
//
// What bounds it.  One query of 32 heads: 64 sequences of 8,192 keys, 8 heads of 128: 143
// us, 5.8 TB/s; 4 of 1,048,576, 4 heads: 490 us, 6.8 TB/s, the rate of a copy.  Beside
// the bytes a call has about 15 us: finding the share and the first pages (4), the ring
// filling and draining, the end of a piece and its joining (3 each).  A window of 1,024
// in 61 sequences takes 38.6 us of which the bytes are 20.  From 10 rows on, the MMAs, the
// conversions and the softmax bound it: 16 sequences of 16,000 keys, 8 heads, take 96
// us for 10 rows and 61 us more for every 16.
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
#include <type_traits>

#include "csbp_generate.h"
#include "csbp_internal.h"
#include "device_once.h"
#include "kv_cache.cuh"
#include "paged_work.cuh"
#include "ptx_sm100.cuh"

namespace csbp {
namespace {

using namespace paged;

constexpr size_t kStatusBytes = 256;
constexpr int kMostWarps = 12;
constexpr int kStages = 2;
constexpr int kKeys = 32;     // of a warp's step, two MMAs
// Rows of a head and sequence that go to row tiles of 16, which read the keys again
// each (from L2); more go to whole tiles (attn_paged_tiles.cu).  16 sequences of 16,000
// keys, 8 heads of 128: 20 / 40 / 45 / 60 rows take 153 / 217 / 218 / 279 us here and
// 247 / 246 / 245 / 246 there; 24 sequences with a window of 1,000, 2 heads of 64: 28 / 56
// rows 16.8 / 26.6 and 20.9 / 20.9.
constexpr int kMostRows = 48;
constexpr int kFlush = 1024;  // steps that one accumulator takes in
constexpr float kShift = 14.f;  // p is held as p 2^14; a row's maximum may lag by 2^1

// 8 x 8 f16 numbers, row g in lanes 4g .. 4g + 3: transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}
// Four 8 x 16-byte matrices: lane 4g + t gets bytes 4t .. of row g of each.
__device__ __forceinline__ void load_rows(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
// Two 16 x 16-byte matrices transposed: lane 4g + t gets rows 4t .. 4t + 3 of columns
// g and g + 8 of each.
__device__ __forceinline__ void load_columns(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Warps of a CTA, by its registers: 32 sums and 16 words of Q per lane and 8 rows.
__host__ __device__ constexpr int most_warps(int tiles) { return tiles == 1 ? 12 : 8; }

// Whether the CTAs join what was cut.  One query of 32 heads: 64 x 8,192 keys take 140 us
// so and 145 with a kernel of its own, 4 x 1,048,576 484 and 513, a window of 1,024 37.5
// either way, 3 x 1,000 keys of 2 heads 8.9 and 9.4; but with 16 rows to a tile, which one
// CTA joins, 16 sequences of 10 rows and 8 heads take 120 and 98.
__host__ __device__ constexpr bool joins_itself(int tile_rows) { return tile_rows == 8; }

// Pieces of cut items that a CTA has left, two at most, in shared memory.
struct Pieces {
  int entry[2], block[2];
  int first[2], n[2];  // CTAs first, first + lanes, .. have its n pieces
  int count, last;
};

// ------------------------------------------------------------ shared memory
template <int D, int NT>
struct Rows {
  static constexpr int kRows = 8 * NT;  // of a tile
  static constexpr int kGroups = D / 32;
  // a warp's ring stage: K codes, V codes, scale words (K, V), the step's record
  static constexpr int kCodes = kKeys * D;
  static constexpr int kWords = 2 * kCodes;
  static constexpr int kRecord = kWords + 2 * kKeys * 4;
  static constexpr int kStage = kRecord + 128;
  // the step's scales: fp32 of K [key][group], f16 of V [group][key]; the sum's first E
  static constexpr int kScales = kStages * kStage;
  static constexpr int kFirstTop = kScales + kKeys * kGroups * 6;
  // and when an item ends, in their place, 4 rows of the result [row][D + 4] and their
  // LSE (log2)
  static constexpr int kSum = kScales;
  static constexpr int kSumRow = D + 4;
  static constexpr int kSumZ = kSum + 4 * kSumRow * 4;
  static constexpr int kWarpBytes = (kSumZ + 16 + 127) / 128 * 128;
  static_assert((kMostWarps * 4 + sizeof(Cursor)) <= 192, "find_share beside Pieces");
  static_assert(kFirstTop + 4 <= kSumZ, "shared memory of a warp");
  static constexpr int kPieces = 192;
  static constexpr int kRoom = 256;  // find_share and Pieces, in front
  static constexpr int smem(int warps) { return kRoom + warps * kWarpBytes; }

  // Place of a key's 16-byte chunks: chunk c lies at c ^ this.  The rows that an
  // ldmatrix takes at once (K: 0, 1, 4, 5, .. or 2, 3, 6, 7, ..; V: 0 .. 7) lie in
  // different banks.
  static __device__ __forceinline__ int k_swizzle(int r) {
    return D == 128 ? (r & 1) | (r >> 1 & 6) : r >> 2 & 3;
  }
  static __device__ __forceinline__ int v_swizzle(int r) { return D == 128 ? r & 7 : r >> 1 & 3; }
};
static_assert(Rows<128, 1>::smem(most_warps(1)) <= 232448 &&
                  Rows<128, 2>::smem(most_warps(2)) <= 232448,
              "shared memory of a CTA");
static_assert(Rows<128, 1>::kWarpBytes % 128 == 0 && Rows<64, 1>::kWarpBytes % 64 == 0,
              "swizzled rows");

// Key (of 16) of row m of the first product: rows 2t, 2t + 1 and 2t + 8, 2t + 9 are
// the keys 4t .. 4t + 3 that lane quarter t has of V.
__device__ __forceinline__ int key_of(int m) { return (m & 6) << 1 | (m & 1) | (m >> 3) << 1; }
// and the row of a key
__device__ __forceinline__ int row_of_key(int r) { return (r >> 1 & 6) | (r & 1) | (r & 2) << 2; }

// Two scale bytes as fp32: 2^(byte - 127), 255 as NaN.
__device__ __forceinline__ void two_scales(uint32_t w, float& lo, float& hi) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.bf16x2.ue8m0x2 %0, a;\n}"
      : "=r"(r)
      : "r"(w));
  lo = __uint_as_float(r << 16);
  hi = __uint_as_float(r & 0xffff0000u);
}
// What a step is about, as the ring carries it.
struct Record {
  uint32_t there;    // which of its keys are there
  int j;             // the first of them
  int entry, block;  // (see Cursor)
  int step, n;       // of the entry's n
  int c;             // keys of the sequence
  uint32_t left;     // keys that are left of a step of which a part has been taken
};

// A step ahead: its record, and what the lane looked up for its key.
struct Ahead {
  Record r;
  int page, place;
};

// Weights of two sums with the LSE (log2) a and b in their join, and its LSE.  In full
// precision: where scales of V lie far apart this is done for every step.
__device__ __noinline__ float3 join_sums(float a, float b) {
  const float most = fmaxf(a, b), ref = most == -INFINITY ? 0.f : most;
  const float x = exp2f(a - ref), y = exp2f(b - ref), both = x + y;
  const float f = both == 0.f ? 0.f : 1.f / both;
  return make_float3(x * f, y * f, both == 0.f ? -INFINITY : ref + log2f(both));
}

// The largest of a warp's words, byte by byte.
__device__ __forceinline__ uint32_t warp_max4(uint32_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = __vmaxu4(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
// Whether a scale byte is more than 14 below `most`; one of 0 is not.
__device__ __forceinline__ bool far_below(uint32_t number, uint32_t most) {
  return at_least_u8x4(__vsubus4(most, number | __vcmpeq4(number, 0)), 0x0f0f0f0fu) != 0;
}
// Of the keys `there`, a lane each, the first and those whose scale bytes all lie within 7
// of its own; where its own is 0, within 14 of the largest.  (0 is near any.)
__device__ __noinline__ uint32_t near_first(uint32_t number, uint32_t most, uint32_t there) {
  const uint32_t first = __shfl_sync(0xffffffffu, number, __ffs(there) - 1);
  const uint32_t none = __vcmpeq4(first, 0), of = first | (most & none);
  const uint32_t lo = __vsubus4(of, 0x07070707u + (0x07070707u & none));
  const uint32_t hi = __vaddus4(of, 0x07070707u & ~none);
  return there & __ballot_sync(0xffffffffu,
                               at_least_u8x4(number | __vcmpeq4(number, 0), lo) == 0x80808080u &&
                                   at_least_u8x4(hi, number) == 0x80808080u);
}

template <int D, int NT>
struct Kernel {
  using L = Rows<D, NT>;
  static constexpr int kG = L::kGroups;

  const PagedParams& p;
  const int lane, g, t, slice, head_in;
  const uint32_t mem;  // the warp's shared memory

  // rows 8n + 2t and 8n + 2t + 1 at 2n and 2n + 1
  float acc[NT][D / 16][4];  // O^T: features 16f + g and + 8 of the two rows
  uint32_t q[NT][D / 16][2];
  float m[2 * NT], l[2 * NT], row_scale[2 * NT];
  int row_lo[2 * NT], row_hi[2 * NT];  // [lo, hi) of a row, besides the sinks
  int all_lo, all_hi;                  // of the rows of the tile alike
  uint32_t top;                        // E of each group, a byte each
  bool aside;                          // a sum has been put aside

  __device__ __forceinline__ Kernel(const PagedParams& p, const uint8_t* smem)
      : p(p), lane(threadIdx.x & 31), g(lane >> 2), t(lane & 3),
        slice(static_cast<int>(threadIdx.x >> 5) / p.heads),
        head_in(static_cast<int>(threadIdx.x >> 5) % p.heads),
        mem(smem_u32(smem)) {}

  __device__ __forceinline__ void look(Cursor& cur, Ahead& a) const {
    const bool front = cur.step < cur.r.n_first;
    a.r.j = (front ? 0 : cur.r.lo) +
            ((front ? cur.step : cur.step - cur.r.n_first) * p.slices + slice) * kKeys;
    const int j = a.r.j + lane, entry = p.by_page(j);
    a.place = j - entry * p.page_size;
    a.page = -1;
    if (j < (front ? cur.r.first : cur.r.hi))
      a.page = __ldg(p.table + static_cast<int64_t>(cur.b) * p.table_pages + entry);
    a.r.entry = cur.entry;
    a.r.block = cur.block;
    a.r.step = cur.step;
    a.r.n = cur.r.n;
    a.r.c = cur.r.c;
    if (++cur.step < cur.r.n) return;
    cur.step = 0;
    cur.block += p.lanes;
    if (cur.block < p.head_blocks) return;
    cur.block -= p.lanes * p.lane_blocks;
    ++cur.entry;
    cur.load(p, L::kRows);
  }

  // Starts the copies of a step into a stage of the ring.  A key that is not there
  // is zeros (copies of one row of the cache would make it a hot spot: 61 x 1 queries
  // with a window of 92 keys took 24 us).
  __device__ __forceinline__ void issue(const Ahead& a, int stage, uint2& pending) const {
    const uint32_t at = mem + stage * L::kStage;
    const int head = a.r.block * p.heads + head_in;
    const bool there = static_cast<uint32_t>(a.page) < static_cast<uint32_t>(p.pages) && head < p.Hkv;
    const uint32_t row =
        there ? static_cast<uint32_t>(a.page * p.page_size + a.place) * p.Hkv + head : 0;
    const uint32_t is = __ballot_sync(0xffffffffu, there);
    constexpr int kChunks = D / 16, kAtOnce = 32 / kChunks;
    const int chunk = lane % kChunks, r0 = lane / kChunks;
    const uint8_t *k = p.k + chunk * 16, *v = p.v + chunk * 16;
#pragma unroll
    for (int i = 0; i < kKeys / kAtOnce; ++i) {
      const int r = i * kAtOnce + r0;
      const uint64_t from = static_cast<uint64_t>(__shfl_sync(0xffffffffu, row, r)) * D;
      const int n = is >> r & 1 ? 16 : 0;
      copy16(at + r * D + (chunk ^ L::k_swizzle(r)) * 16, k + from, n);
      copy16(at + L::kCodes + r * D + (chunk ^ L::v_swizzle(r)) * 16, v + from, n);
    }
    // scale bytes
    const uint64_t place = static_cast<uint64_t>(row) * kG;
    if (p.wide_scales) {
      copy4(at + L::kWords + lane * 4, p.k_scale + (place & ~uint64_t(3)), there ? 4 : 0);
      copy4(at + L::kWords + (kKeys + lane) * 4, p.v_scale + (place & ~uint64_t(3)),
            there ? 4 : 0);
    } else {
      uint32_t w[2] = {0, 0};
      if (there)
#pragma unroll
        for (int e = 0; e < kG; ++e) {
          w[0] |= static_cast<uint32_t>(__ldg(p.k_scale + place + e)) << 8 * e;
          w[1] |= static_cast<uint32_t>(__ldg(p.v_scale + place + e)) << 8 * e;
        }
      pending = make_uint2(w[0], w[1]);  // stored a step later, so that nobody waits here
    }
    if (lane == 0) {
      asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at + L::kRecord), "r"(is),
                   "r"(a.r.j), "r"(a.r.entry), "r"(a.r.block)
                   : "memory");
      asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at + L::kRecord + 16),
                   "r"(a.r.step), "r"(a.r.n), "r"(a.r.c), "r"(0)
                   : "memory");
    }
  }
  __device__ __forceinline__ void store_pending(int stage, uint2 pending) const {
    if (p.wide_scales) return;
    sts32(mem + stage * L::kStage + L::kWords + lane * 4, pending.x);
    sts32(mem + stage * L::kStage + L::kWords + (kKeys + lane) * 4, pending.y);
  }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int f = 0; f < D / 16; ++f)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[n][f][k] = 0.f;
#pragma unroll
    for (int x = 0; x < 2 * NT; ++x) {
      l[x] = 0.f;
      // (not -inf: a difference with a masked score has to stay a number)
      m[x] = -3e38f;
    }
    top = 0;
    if (lane == 0) sts32(mem + L::kFirstTop, 0);
  }

  // Rows of a tile: queries to registers, and what each row reads.
  __device__ __forceinline__ void begin(const Record& cur) {
    const int head = min(cur.block * p.heads + head_in, p.Hkv - 1);
    const int b = p.by_row_tiles(cur.entry);
    const int rows = p.queries * p.G, row0 = (cur.entry - b * p.row_tiles) * L::kRows;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = min(row0 + 8 * n + g, rows - 1);
      const int i = p.by_G(r), gi = r - i * p.G;
      const __nv_bfloat16* src = p.q + b * p.q_bat + i * p.q_tok +
                                 (static_cast<int64_t>(head) * p.G + gi) * D + t * 4;
      uint2 raw[D / 16];
#pragma unroll
      for (int f = 0; f < D / 16; ++f) raw[f] = __ldg(reinterpret_cast<const uint2*>(src + f * 16));
      uint32_t most = 0;
#pragma unroll
      for (int f = 0; f < D / 16; ++f)
        most = max(max(most, max(raw[f].x & 0x7fffu, raw[f].x >> 16 & 0x7fffu)),
                   max(raw[f].y & 0x7fffu, raw[f].y >> 16 & 0x7fffu));
      most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
      // the largest element becomes 2^7 .. 2^8
      const int ex = max(static_cast<int>(most >> 7) - 127, -110);
      const float scale = __uint_as_float(static_cast<uint32_t>(127 + 7 - ex) << 23);
      // (not 0: a masked score times it has to stay -inf)
      const float back = fmaxf(p.scale_log2 * ldexpf(1.f, ex - 7), 1e-37f);
      row_scale[2 * n] = __shfl_sync(0xffffffffu, back, 8 * t);
      row_scale[2 * n + 1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);
#pragma unroll
      for (int f = 0; f < D / 16; ++f) {
        q[n][f][0] = pack_f16(__uint_as_float(raw[f].x << 16) * scale,
                              __uint_as_float(raw[f].x & 0xffff0000u) * scale);
        q[n][f][1] = pack_f16(__uint_as_float(raw[f].y << 16) * scale,
                              __uint_as_float(raw[f].y & 0xffff0000u) * scale);
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int at = cur.c - p.queries + static_cast<int>(p.by_G(min(row0 + 8 * n + 2 * t + x, rows - 1)));
        row_hi[2 * n + x] = p.causal ? at + 1 : cur.c;
        row_lo[2 * n + x] = window_begin(p, at);
      }
    }
    const int i0 = p.by_G(row0), i1 = p.by_G(min(row0 + L::kRows, rows) - 1);
    all_hi = p.causal ? cur.c - p.queries + i0 + 1 : cur.c;
    all_lo = window_begin(p, cur.c - p.queries + i1);
    aside = false;
    clear();
  }

  __device__ __forceinline__ bool reads(int x, int j) const {
    return j < row_hi[x] && (j >= row_lo[x] || j < p.sinks);
  }

  // Scales that are above E, far below it or NaN.  E becomes the largest so far, what was
  // summed under the old one is scaled, and `delta` is E - e, or 15 where a scale is that far
  // below because its byte is 0 (what is below 2^-118 counts as 0 there) or NaN.
  //
  // Where the scales do not lie within 2^14 of E, or E has risen since the sum's begin by
  // more than fp32 can follow, the sum so far is to be put aside first: all of `there` is left
  // for then.
  // Where they do not lie within 2^14 of one another, `there` becomes those of the first key
  // and the ones near it in each group.  Returns what is left.  (`fresh`: nothing has been
  // summed yet.)
  __device__ __forceinline__ uint32_t odd_scales(uint32_t word, bool fresh, uint32_t& there,
                                                 uint32_t& delta) {
    uint32_t left = 0;
    uint32_t number = there >> lane & 1 ? word & ~__vcmpeq4(word, 0xffffffffu) : 0;
    uint32_t now = warp_max4(__vmaxu4(number, top));  // (fresh: top is 0)
    if (__any_sync(0xffffffffu, far_below(number, now))) {
      if (!fresh) return there;
      left = there;
      there = near_first(number, now, there);
      left &= ~there;
      number = there >> lane & 1 ? number : 0;
      now = warp_max4(number);
    }
    uint32_t first = lds32(mem + L::kFirstTop);
    first |= now & __vcmpeq4(first, 0);
    // (nothing is borrowed; a fresh sum never waits for another)
    if (!fresh && at_least_u8x4(now - first, 0x41414141u)) return there;
    __syncwarp();
    if (lane == 0) sts32(mem + L::kFirstTop, first);
    if (!fresh) {
#pragma unroll
      for (int e = 0; e < kG; ++e) {
        const uint32_t by = (now >> 8 * e & 255) - (top >> 8 * e & 255);
        const float f = by < 127 ? __uint_as_float((127 - by) << 23) : 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[n][2 * e + k][c] *= f;
      }
    }
    top = now;
    delta = there >> lane & 1 ? __vminu4(now - number, 0x0f0f0f0fu) : 0;
    return left;
  }

  // NaN in V (codes, or `v_word`'s scales): NaN in the sums of the rows that read the
  // key, and 0 in the place of the codes, for the rows that do not.
  __device__ __forceinline__ void mark_nan(const Record& cur, uint32_t v, uint32_t v_word) {
#pragma unroll 1
    for (int r = 0; r < kKeys; ++r) {
      const uint32_t scale = __shfl_sync(0xffffffffu, v_word, r);
      if (!(cur.there >> r & 1)) continue;
      const uint32_t row = v + r * D;
#pragma unroll
      for (int f = 0; f < D / 16; ++f)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          // feature 16f + 8k + g
          uint32_t code;
          asm volatile("ld.shared.u8 %0, [%1];"
                       : "=r"(code)
                       : "r"(row + (((f ^ L::v_swizzle(r)) << 4) | 8 * k | g))
                       : "memory");
          if ((code & 0x7f) != 0x7f && (scale >> 8 * (f / 2) & 255) != 255) continue;
#pragma unroll
          for (int x = 0; x < 2 * NT; ++x)
            if (reads(x, cur.j + r)) acc[x >> 1][f][2 * k + (x & 1)] = NAN;
        }
    }
    __syncwarp();
#pragma unroll 1
    for (int i = lane * 4; i < kKeys * D; i += 128) {
      const uint32_t w = lds32(v + i);
      if (nan_codes(w)) sts32(v + i, w & ~nan_codes(w));
    }
    __syncwarp();
  }

  // The keys `cur.there` of a step.  Those that are left for a sum of their own (see
  // odd_scales; none as a rule) go to its record in the ring, and `in_sum`, the steps in the
  // sum so far, becomes what has this one put aside.
  __device__ __forceinline__ void step(const Record& cur, int stage, int& in_sum) {
    const uint32_t at = mem + stage * L::kStage;
    const uint32_t scales = mem + L::kScales, v_scales = scales + kKeys * kG * 4;
    // ------- the step's scales, a key per lane
    uint32_t k_word = lds32(at + L::kWords + lane * 4);
    uint32_t v_word = lds32(at + L::kWords + (kKeys + lane) * 4);
    uint32_t there = cur.there;
    const bool upper = D == 64 && p.wide_scales && ((cur.block * p.heads + head_in) & 1);
    if (D == 64 && p.wide_scales) {  // its half of the word
      k_word = upper ? k_word >> 16 : k_word & 0xffffu;
      v_word = upper ? v_word >> 16 : v_word & 0xffffu;
    }
    const bool is_there = there >> lane & 1;
    uint32_t delta = is_there ? top - v_word : 0;
    // f16 holds 2^-delta to delta = 14
    const uint32_t odd = (delta + (kG == 4 ? 0x71717171u : 0x7171u)) | delta;
    const bool other = is_there && ((odd | ~at_least_u8x4(top, v_word)) & 0x80808080u) != 0;
    bool bad = false;
    if (__any_sync(0xffffffffu, other)) {
      bad = __any_sync(0xffffffffu, is_there && any_byte_255(v_word));
      const uint32_t left = odd_scales(v_word, in_sum == 0, there, delta);
      if (left) {
        in_sum = kFlush - 1;
        if (lane == 0) sts32(at + L::kRecord + 28, left);
        __syncwarp();
        if (left == cur.there) return;
      }
    }
    {
      float f[4];
      two_scales(k_word, f[0], f[1]);
      const uint32_t to = scales + ((lane & 16) + row_of_key(lane & 15)) * kG * 4;
      if constexpr (kG == 4) {
        two_scales(k_word >> 16, f[2], f[3]);
        asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(to), "f"(f[0]), "f"(f[1]),
                     "f"(f[2]), "f"(f[3])
                     : "memory");
      } else {
        asm volatile("st.shared.v2.f32 [%0], {%1,%2};" ::"r"(to), "f"(f[0]), "f"(f[1]) : "memory");
      }
      // 2^-delta in f16: only the upper byte, 4 (15 - delta), 0 for 15
      const uint32_t h = 0x3c3c3c3cu - 4 * delta;
#pragma unroll
      for (int e = 0; e < kG; ++e)
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(v_scales + e * (2 * kKeys) + lane * 2),
                     "h"(static_cast<uint16_t>(__byte_perm(h, 0, 0x0004 | e << 4)))
                     : "memory");
    }
    __syncwarp();

    // ------- S^T = K Q^T: of each 16 keys those of rows g and g + 8
    float s[2][NT][4];
    const int r_k = key_of(lane & 15);
    const uint32_t k0 = at + r_k * D + (((lane >> 4) ^ L::k_swizzle(r_k)) << 4);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float ks[2][kG];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t from = scales + (16 * u + 8 * k + g) * kG * 4;
        if constexpr (kG == 4)
          asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                       : "=f"(ks[k][0]), "=f"(ks[k][1]), "=f"(ks[k][2]), "=f"(ks[k][3])
                       : "r"(from)
                       : "memory");
        else
          asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];"
                       : "=f"(ks[k][0]), "=f"(ks[k][1])
                       : "r"(from)
                       : "memory");
      }
#pragma unroll
      for (int e = 0; e < kG; ++e) {
        uint32_t w[4];
        load_rows(w, (k0 ^ (e << 5)) + 16 * u * D);
        uint32_t a[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          a[k] = f16_low(w[k]);
          a[4 + k] = f16_high(w[k]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float c[4] = {0.f, 0.f, 0.f, 0.f};
          mma(c, a[0], a[1], a[4], a[5], q[n][2 * e][0], q[n][2 * e][1]);
          mma(c, a[2], a[3], a[6], a[7], q[n][2 * e + 1][0], q[n][2 * e + 1][1]);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            s[u][n][k] = e == 0 ? c[k] * ks[k >> 1][0] : fmaf(c[k], ks[k >> 1][e], s[u][n][k]);
        }
      }
    }

    // ------- mask
    const bool inside = there == 0xffffffffu && cur.j + kKeys <= all_hi &&
                        (cur.j >= all_lo || cur.j + kKeys <= p.sinks);
    if (!inside) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = 16 * (k >> 1) + key_of(8 * (k & 1) + g);
        const bool here = there >> r & 1;
#pragma unroll
        for (int x = 0; x < 2 * NT; ++x)
          if (!here || !reads(x, cur.j + r)) s[k >> 1][x >> 1][2 * (k & 1) + (x & 1)] = -INFINITY;
      }
    }

    // ------- softmax (scores before the row's scale, which is positive)
    float most[2 * NT];
    bool grows = false;
#pragma unroll
    for (int x = 0; x < 2 * NT; ++x) {
      const int n = x >> 1, k = x & 1;
      most[x] = fmaxf(fmaxf(s[0][n][k], s[0][n][2 + k]), fmaxf(s[1][n][k], s[1][n][2 + k])) *
                row_scale[x];
      grows |= most[x] > m[x] + 1.f;
    }
    if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
      for (int x = 0; x < 2 * NT; ++x) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1)
          most[x] = fmaxf(most[x], __shfl_xor_sync(0xffffffffu, most[x], o));
        // (a row's own maximum says when it is brought up to date, not the others')
        const float now = most[x] > m[x] + 1.f ? most[x] : m[x];
        const float f = now == m[x] ? 1.f : ex2_approx(m[x] - now);
        m[x] = now;
        l[x] *= f;
#pragma unroll
        for (int e = 0; e < D / 16; ++e) {
          acc[x >> 1][e][x & 1] *= f;
          acc[x >> 1][e][2 + (x & 1)] *= f;
        }
      }
    }
    float pr[2][NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int x = 2 * n + (k & 1);
#pragma unroll
        for (int u = 0; u < 2; ++u)
          pr[u][n][k] = ex2_approx(fmaf(s[u][n][k], row_scale[x], kShift - m[x]));
      }
#pragma unroll
      for (int k = 0; k < 2; ++k)
        l[2 * n + k] += (pr[0][n][k] + pr[0][n][2 + k]) + (pr[1][n][k] + pr[1][n][2 + k]);
    }

    // ------- NaN in V where some row does not read the key
    const uint32_t v_codes = at + L::kCodes;
    if (!inside) {
      uint32_t found = 0;
#pragma unroll
      for (int i = 0; i < kKeys * D / 512; ++i) {
        uint4 w;
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                     : "r"(v_codes + i * 512 + lane * 16)
                     : "memory");
        found |= nan_codes(w.x) | nan_codes(w.y) | nan_codes(w.z) | nan_codes(w.w);
      }
      bad |= __any_sync(0xffffffffu, found != 0);
    }
    if (bad) mark_nan(cur, v_codes, v_word);

    // ------- P^T: row g, keys 4t .. 4t + 3 of each 16, under V's scales of each group,
    // and O^T += V^T P^T
    const int r_v = lane & 15;
    const uint32_t v0 = v_codes + r_v * D + (((lane >> 4) ^ L::v_swizzle(r_v)) << 4);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t b[NT][kG][2];
      {
        uint2 vs[kG];
#pragma unroll
        for (int e = 0; e < kG; ++e) vs[e] = lds64(v_scales + e * (2 * kKeys) + 32 * u + 8 * t);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint32_t b0 = transpose8(pack_f16(pr[u][n][0], pr[u][n][1]));
          const uint32_t b1 = transpose8(pack_f16(pr[u][n][2], pr[u][n][3]));
#pragma unroll
          for (int e = 0; e < kG; ++e) {
            b[n][e][0] = mul_f16x2(b0, vs[e].x);
            b[n][e][1] = mul_f16x2(b1, vs[e].y);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < kG; ++e) {
        uint32_t w[4], a[8];
        load_columns(w, (v0 ^ (e << 5)) + 16 * u * D);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          a[k] = f16_low(w[k]);
          a[4 + k] = f16_high(w[k]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma(acc[n][2 * e], a[0], a[1], a[4], a[5], b[n][e][0], b[n][e][1]);
          mma(acc[n][2 * e + 1], a[2], a[3], a[6], a[7], b[n][e][0], b[n][e][1]);
        }
      }
    }
    __syncwarp();  // the stage and the scales have been read
  }

  // What the registers hold as a normalised O and its LSE, joined with what was put
  // aside: O stays in `acc`, z[x] is the LSE (log2) of row x.
  __device__ __forceinline__ void normalise(float (&z)[2 * NT]) {
    const int64_t at =
        (static_cast<int64_t>(blockIdx.x) * (p.heads * p.slices) + (threadIdx.x >> 5)) * L::kRows;
#pragma unroll
    for (int x = 0; x < 2 * NT; ++x) {
      const int n = x >> 1, row = 8 * n + 2 * t + (x & 1);
      float sum = l[x];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      z[x] = sum == 0.f ? -INFINITY : m[x] - kShift + lg2_approx(sum);
      float mine = 1.f, old = 0.f;
      if (aside) {
        const float3 both = join_sums(p.aside_z[at + row], z[x]);
        old = both.x;
        mine = both.y;
        z[x] = both.z;
      }
      const float inv = sum == 0.f ? 0.f : __fdividef(1.f, sum);
#pragma unroll
      for (int f = 0; f < D / 16; ++f) {
        // 2^(E - 127), in two steps: one could lie below fp32's range
        const int ex = static_cast<int>(top >> 8 * (f / 2) & 255);
        const float f0 = __uint_as_float(static_cast<uint32_t>(ex / 2 + 64) << 23);
        const float f1 = __uint_as_float(static_cast<uint32_t>(ex - ex / 2 + 63) << 23);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float& o = acc[n][f][2 * k + (x & 1)];
          o = o * inv * f0 * f1;
          if (aside) o = o * mine + p.aside_o[(at + row) * D + 16 * f + 8 * k + g] * old;
        }
      }
    }
  }

  // Puts a normalised sum aside and begins another.
  __device__ __forceinline__ void put_aside(const float (&z)[2 * NT]) {
    const int64_t at =
        (static_cast<int64_t>(blockIdx.x) * (p.heads * p.slices) + (threadIdx.x >> 5)) * L::kRows;
    __syncwarp();
#pragma unroll
    for (int x = 0; x < 2 * NT; ++x) {
      const int n = x >> 1, row = 8 * n + 2 * t + (x & 1);
      if (g == 0) p.aside_z[at + row] = z[x];
#pragma unroll
      for (int f = 0; f < D / 16; ++f)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          p.aside_o[(at + row) * D + 16 * f + 8 * k + g] = acc[n][f][2 * k + (x & 1)];
    }
    __syncwarp();
    aside = true;
    clear();
  }

  // The rows of a piece, joined over the slices, 4 rows at a time by way of shared
  // memory: to the outputs where the piece is the whole of a row's keys (`part` < 0),
  // else to a place among the partials.
  __device__ __forceinline__ void finish(const Record& cur, int part, const float (&z)[2 * NT],
                                         uint8_t* warps) {
    const int head = cur.block * p.heads + head_in;
    const int b = p.by_row_tiles(cur.entry), row0 = (cur.entry - b * p.row_tiles) * L::kRows;
    const int rows = min(L::kRows, p.queries * p.G - row0);
    const auto sync = [&] {
      if (p.slices > 1)
        __syncthreads();
      else
        __syncwarp();
    };
    uint8_t* mine = warps + (threadIdx.x >> 5) * L::kWarpBytes;
    const uint8_t* first = warps + head_in * L::kWarpBytes;  // slice 0
    const int stride = p.heads * L::kWarpBytes;
#pragma unroll
    for (int n = 0; n < 2 * NT; ++n) {  // rows 4n .. 4n + 3: those of the lanes t / 2 = n % 2
      if (4 * n >= rows) break;
      if (t >> 1 == (n & 1)) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int row = 2 * (t & 1) + x;
          float* to = reinterpret_cast<float*>(mine + L::kSum) + row * L::kSumRow + g;
#pragma unroll
          for (int f = 0; f < D / 16; ++f) {
            to[16 * f] = acc[n / 2][f][x];
            to[16 * f + 8] = acc[n / 2][f][2 + x];
          }
          if (g == 0) reinterpret_cast<float*>(mine + L::kSumZ)[row] = z[n / 2 * 2 + x];
        }
      }
      sync();
      constexpr int kLanes = D / 4;
#pragma unroll 1
      for (int y = slice * 32 + lane; y < min(4, rows - 4 * n) * kLanes; y += p.slices * 32) {
        if (head >= p.Hkv) break;
        const int row = y / kLanes, f = y % kLanes * 4;
        float most = -INFINITY;
#pragma unroll 1
        for (int s = 0; s < p.slices; ++s)
          most = fmaxf(most, reinterpret_cast<const float*>(first + s * stride + L::kSumZ)[row]);
        const float ref = most == -INFINITY ? 0.f : most;
        float both = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int s = 0; s < p.slices; ++s) {
          const float zs = reinterpret_cast<const float*>(first + s * stride + L::kSumZ)[row];
          if (zs == -INFINITY) continue;  // it has read nothing
          const float w = ex2_approx(zs - ref);
          const float4 v = *reinterpret_cast<const float4*>(
              reinterpret_cast<const float*>(first + s * stride + L::kSum) + row * L::kSumRow + f);
          both += w;
          o.x = fmaf(w, v.x, o.x);
          o.y = fmaf(w, v.y, o.y);
          o.z = fmaf(w, v.z, o.z);
          o.w = fmaf(w, v.w, o.w);
        }
        const float inv = both == 0.f ? 0.f : __fdividef(1.f, both);
        const float lse = both == 0.f ? -INFINITY : ref + lg2_approx(both);
        o.x *= inv;
        o.y *= inv;
        o.z *= inv;
        o.w *= inv;
        if (part < 0) {
          const int q_row = row0 + 4 * n + row, i = p.by_G(q_row);
          const int h = head * p.G + q_row - i * p.G;
          const int64_t token = static_cast<int64_t>(b) * p.queries + i;
          *reinterpret_cast<uint2*>(p.o + (token * p.Hq + h) * D + f) =
              make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
          if (f == 0)
            p.lse[(static_cast<int64_t>(b) * p.Hq + h) * p.queries + i] = lse * 0.6931471805599453f;
        } else {
          const int64_t at =
              (static_cast<int64_t>(part) * p.heads + head_in) * L::kRows + 4 * n + row;
          *reinterpret_cast<float4*>(p.part_o + at * D + f) = o;
          if (f == 0) p.part_z[at] = lse;
        }
      }
      sync();
    }
  }
};

// 4 features (f ..) of U rows that were cut into n pieces, of which piece k lies at
// at[u] + k step (+ begin for the first) among the partials; (b, q_row, head)[u] is what
// they are, b < 0 for none.  (From L2: other CTAs wrote them, perhaps in this launch.)
struct JoinedRow {
  int b, q_row, head;
};
template <int D, int U>
__device__ __forceinline__ void join_rows(const PagedParams& p, int n, const int64_t (&at)[U],
                                          int64_t step, int64_t begin,
                                          const JoinedRow (&row)[U], int f) {
  float m[U], both[U];
  float4 o[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    m[u] = -INFINITY;
    both[u] = 0.f;
    o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
#pragma unroll 2
  for (int k = 0; k < n; ++k) {
    float z[U];
    float4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t x = at[u] + k * step + (k == 0 ? begin : 0);
      z[u] = __ldcg(p.part_z + x);
      v[u] = __ldcg(reinterpret_cast<const float4*>(p.part_o + x * D + f));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // (a piece that has read nothing is O = 0, LSE = -inf)
      const float most = fmaxf(m[u], z[u]), ref = most == -INFINITY ? 0.f : most;
      const float old = ex2_approx(m[u] - ref), w = ex2_approx(z[u] - ref);
      m[u] = most;
      both[u] = fmaf(both[u], old, w);
      o[u].x = fmaf(w, v[u].x, o[u].x * old);
      o[u].y = fmaf(w, v[u].y, o[u].y * old);
      o[u].z = fmaf(w, v[u].z, o[u].z * old);
      o[u].w = fmaf(w, v[u].w, o[u].w * old);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (row[u].b < 0) continue;
    const float inv = both[u] == 0.f ? 0.f : __fdividef(1.f, both[u]);
    const float z = both[u] == 0.f ? -INFINITY : m[u] + lg2_approx(both[u]);
    const int i = p.by_G(row[u].q_row), h = row[u].head * p.G + row[u].q_row - i * p.G;
    const int64_t token = static_cast<int64_t>(row[u].b) * p.queries + i;
    *reinterpret_cast<uint2*>(p.o + (token * p.Hq + h) * D + f) = make_uint2(
        pack_bf16x2(o[u].x * inv, o[u].y * inv), pack_bf16x2(o[u].z * inv, o[u].w * inv));
    if (f == 0)
      p.lse[(static_cast<int64_t>(row[u].b) * p.Hq + h) * p.queries + i] = z * 0.6931471805599453f;
  }
}

// Joins the pieces of an item.  The whole CTA calls it.
template <int D, int R>
__device__ __forceinline__ void join_item(const PagedParams& p, int entry, int block, int first,
                                          int n) {
  constexpr int kLanes = D / 4;
  const int b = p.by_row_tiles(entry), tile = entry - b * p.row_tiles;
  const int rows = min(R, p.queries * p.G - tile * R);
  // the first piece is where the item begins, the others are their CTAs' first
  const int64_t piece = static_cast<int64_t>(p.heads) * R;
  constexpr int U = 2;
  const int stride = blockDim.x / kLanes, all = p.heads * rows;
  for (int x0 = threadIdx.x / kLanes; x0 < all; x0 += U * stride) {
    int64_t at[U];
    JoinedRow row[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int x = min(x0 + u * stride, all - 1);
      const int head_in = x / rows, r = x - head_in * rows, head = block * p.heads + head_in;
      at[u] = 2 * first * piece + head_in * R + r;
      row[u] = JoinedRow{x0 + u * stride < all && head < p.Hkv ? b : -1, tile * R + r, head};
    }
    join_rows<D, U>(p, n, at, 2 * p.lanes * piece, piece, row, threadIdx.x % kLanes * 4);
  }
}

// The last CTA to have left a piece of an item joins them, in their order.  At the end,
// where the CTA has its registers for that.
template <int D, int R>
__device__ __forceinline__ void join_pieces(const PagedParams& p, Pieces& cut) {
  __syncthreads();
  if (threadIdx.x == 0) {
    int last = 0;
    for (int x = 0; x < cut.count; ++x) {
      int* arrived = p.arrived + static_cast<int64_t>(cut.entry[x]) * p.head_blocks + cut.block[x];
      // releases the CTA's pieces, acquires the others'; wraps to 0, for the next launch
      uint32_t before;
      asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;"
                   : "=r"(before)
                   : "l"(arrived), "r"(cut.n[x] - 1)
                   : "memory");
      if (before == static_cast<uint32_t>(cut.n[x] - 1)) last |= 1 << x;
    }
    cut.last = last;
  }
  __syncthreads();
#pragma unroll 1
  for (int x = 0; x < 2; ++x)
    if (cut.last >> x & 1)
      join_item<D, R>(p, cut.entry[x], cut.block[x], cut.first[x], cut.n[x]);
}

template <int D, int NT>
__global__ void __launch_bounds__(most_warps(NT) * 32, 1)
    paged_rows_kernel(const __grid_constant__ PagedParams p) {
  using L = Rows<D, NT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr bool kFused = joins_itself(L::kRows);
  if (!kFused) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint8_t* warps = smem + L::kRoom;
  Pieces& cut = *reinterpret_cast<Pieces*>(smem + L::kPieces);
  if (threadIdx.x == 0) cut.count = 0;
  Kernel<D, NT> k(p, warps + (threadIdx.x >> 5) * L::kWarpBytes);
  Cursor cursor{};
  const Share share =
      find_share<L::kRows, kMostWarps>(p, reinterpret_cast<uint32_t*>(smem), cursor);
  if (share.begin >= share.end) return;
  const int steps = static_cast<int>(share.end - share.begin);
  Ahead next;
  k.look(cursor, next);
  uint2 pending = make_uint2(0, 0);
  int in_sum = 0, stage = 0;
  // two rounds that only start copies, then one for each step
#pragma unroll 1
  for (int i = -kStages; i < steps;) {
    Record r;
    if (i >= 0) {
      __syncwarp();
      asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(r.there), "=r"(r.j), "=r"(r.entry), "=r"(r.block)
                   : "r"(k.mem + stage * L::kStage + L::kRecord)
                   : "memory");
      asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(r.step), "=r"(r.n), "=r"(r.c), "=r"(r.left)
                   : "r"(k.mem + stage * L::kStage + L::kRecord + 16)
                   : "memory");
      if (i == 0 || r.step == 0 || r.left) {
        if (!r.left) {
          k.begin(r);
          in_sum = 0;
        } else {
          __syncwarp();  // (all lanes have read the record)
          if (k.lane == 0) sts32(k.mem + stage * L::kStage + L::kRecord + 28, 0);
        }
      }
      copies_wait<kStages - 1>();
      __syncwarp();
      k.step(r, stage, in_sum);
      const bool ends = r.step + 1 == r.n || i + 1 == steps;
      if (ends || ++in_sum == kFlush) {
        float z[2 * NT];
        k.normalise(z);
        const uint32_t left = lds32(k.mem + stage * L::kStage + L::kRecord + 28);
        if (!ends || left) {
          k.put_aside(z);
          in_sum = 0;
          if (left) {  // the step once more, with the keys that are left
            if (k.lane == 0) sts32(k.mem + stage * L::kStage + L::kRecord, left);
            continue;
          }
        } else {
          // a CTA leaves at most two partials: where an item ends or goes through (0)
          // and where one begins (1); the latter knows how many there are
          const bool starts = r.step <= i;
          const bool whole = starts && r.step + 1 == r.n;
          k.finish(r, whole ? -1 : 2 * static_cast<int>(blockIdx.x) + (starts ? 1 : 0), z, warps);
          if (!kFused && starts && threadIdx.x == 0)
            p.pieces[static_cast<int64_t>(r.entry) * p.head_blocks + r.block] =
                make_int2(static_cast<int>(blockIdx.x),
                          1 + static_cast<int>((r.n - 1 - r.step + share.per - 1) / share.per));
          if (kFused && !whole && threadIdx.x == 0) {
            const uint32_t first = share.begin + i - r.step, last = first + r.n - 1;
            const int x = cut.count++, c = first / share.per;  // (of the lane's CTAs)
            cut.entry[x] = r.entry;
            cut.block[x] = r.block;
            cut.first[x] = c * p.lanes + static_cast<int>(blockIdx.x) % p.lanes;
            cut.n[x] = static_cast<int>(last / share.per) - c + 1;
          }
        }
      }
    }
    // (scale words of the step before: nobody waits for them)
    if (i > -kStages) k.store_pending(stage ^ 1, pending);
    if (i + kStages < steps) {
      k.issue(next, stage, pending);
      if (i + kStages + 1 < steps) k.look(cursor, next);
    }
    copies_commit();
    ++i;
    stage ^= 1;
  }
  copies_wait<0>();
  if (kFused) join_pieces<D, L::kRows>(p, cut);
}

// Two E4M3 codes of a word's low or high half as fp32.
__device__ __forceinline__ float2 two_codes(uint32_t f16x2) {
  return __half22float2(*reinterpret_cast<const __half2*>(&f16x2));
}

// Rows from .. from + rows of a whole tile in fp32, from the keys themselves: where scales
// lie too far apart for f16 operands, in K among the keys of a tile or in V.  Two rows to
// each of 4 warps; a lane takes a key's scores, then D / 32 features of O.  (Rare, and not
// made for speed: 16 sequences of 16,384 keys and 160 rows for each of 8 heads of 128, all
// of them so, take 27 ms.)
constexpr int kExactRows = 8;
template <int D>
__device__ __noinline__ void exact_rows(const PagedParams& p, int entry, int head, int from,
                                        int rows) {
  __shared__ __align__(16) float queries[kExactRows][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = p.by_row_tiles(entry), tile = entry - b * p.row_tiles;
  const Range r = range_of(p, b, tile, kPairRows);
  const int32_t* table = p.table + static_cast<int64_t>(b) * p.table_pages;
  const bool has[2] = {2 * warp < rows, 2 * warp + 1 < rows};
  float row_scale[2];
  int lo[2], hi[2], token[2], h[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int row = tile * kPairRows + from + min(2 * warp + x, rows - 1);
    token[x] = p.by_G(row);
    h[x] = head * p.G + row - token[x] * p.G;
    const int at = r.c - p.queries + token[x];
    hi[x] = p.causal ? at + 1 : r.c;
    lo[x] = window_begin(p, at);
    // the largest element becomes 1 .. 2, so that no product passes fp32's range before the
    // scales are in it
    const __nv_bfloat16* q =
        p.q + b * p.q_bat + token[x] * p.q_tok + static_cast<int64_t>(h[x]) * D;
    float most = 0.f;
    for (int c = lane; c < D; c += 32) most = fmaxf(most, fabsf(__bfloat162float(q[c])));
    const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(most));
    const int ex = max(static_cast<int>(bits >> 23) - 127, -110);
    const float scale = ldexpf(1.f, -ex);
    for (int c = lane; c < D; c += 32) queries[2 * warp + x][c] = __bfloat162float(q[c]) * scale;
    row_scale[x] = fmaxf(p.scale_log2 * ldexpf(1.f, ex), 1e-44f);
  }
  __syncwarp();
  // sums of 32 x 32 keys and of all before them, so that no sum takes in very many terms; O
  // in units of 2^-24, so that a sum of the largest values does not pass fp32's range
  constexpr int F = D / 32;
  float m[2] = {-INFINITY, -INFINITY}, l[2][2] = {}, o[2][2][F] = {};
#pragma unroll 1
  for (int i0 = 0; i0 < r.keys(); i0 += 32) {
    // ------- a key per lane
    const int i = i0 + lane, j = i < r.keys() ? r.key(i) : 0, page_at = p.by_page(j);
    const int page = i < r.keys() ? __ldg(table + page_at) : -1;
    const bool there = static_cast<uint32_t>(page) < static_cast<uint32_t>(p.pages);
    const uint32_t place =
        there ? static_cast<uint32_t>(page * p.page_size + j - page_at * p.page_size) * p.Hkv + head
              : 0;
    float s[2] = {0.f, 0.f};
    if (there) {
#pragma unroll 1
      for (int e = 0; e < F; ++e) {
        const uint4* codes =
            reinterpret_cast<const uint4*>(p.k + static_cast<uint64_t>(place) * D) + 2 * e;
        float sum[2] = {0.f, 0.f};
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
          const uint4 w = __ldg(codes + k);
          const uint32_t word[4] = {w.x, w.y, w.z, w.w};
          const float* q = &queries[2 * warp][32 * e + 16 * k];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float2 a = two_codes(f16_low(word[y])), c = two_codes(f16_high(word[y]));
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float4 f = *reinterpret_cast<const float4*>(q + x * D + 4 * y);
              sum[x] = fmaf(a.x, f.x, fmaf(a.y, f.y, fmaf(c.x, f.z, fmaf(c.y, f.w, sum[x]))));
            }
          }
        }
        const int byte = __ldg(p.k_scale + static_cast<uint64_t>(place) * F + e);
        const float scale = byte == 255 ? NAN : ldexpf(1.f, byte - 127);
        s[0] = fmaf(sum[0], scale, s[0]);
        s[1] = fmaf(sum[1], scale, s[1]);
      }
    }
    uint32_t reads[2];
    float w[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const bool read = has[x] && there && j < hi[x] && (j >= lo[x] || j < p.sinks);
      reads[x] = __ballot_sync(0xffffffffu, read);
      s[x] = read ? s[x] * row_scale[x] : -INFINITY;
      float most = s[x];
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
      most = fmaxf(most, m[x]);
      const float ref = most == -INFINITY ? 0.f : most, old = exp2f(m[x] - ref);
      m[x] = most;
      w[x] = exp2f(s[x] - ref);
      const bool full = (i0 & 1023) == 0;  // 32 x 32 keys are in the first sum
      l[x][1] = (l[x][1] + (full ? l[x][0] : 0.f)) * old;
      l[x][0] = fmaf(full ? 0.f : l[x][0], old, w[x]);
#pragma unroll
      for (int f = 0; f < F; ++f) {
        o[x][1][f] = (o[x][1][f] + (full ? o[x][0][f] : 0.f)) * old;
        o[x][0][f] = full ? 0.f : o[x][0][f] * old;
      }
    }
    // ------- F features per lane
    for (uint32_t any = reads[0] | reads[1]; any; any &= any - 1) {
      const int k = __ffs(any) - 1;
      const uint64_t at = static_cast<uint64_t>(__shfl_sync(0xffffffffu, place, k));
      const float w0 = __shfl_sync(0xffffffffu, w[0], k), w1 = __shfl_sync(0xffffffffu, w[1], k);
      const int byte = __ldg(p.v_scale + at * F + lane * F / 32);
      const float scale = byte == 255 ? NAN : ldexpf(1.f, byte - 127 - 24);
      float v[F];
      if constexpr (F == 4) {
        const uint32_t word = __ldg(reinterpret_cast<const uint32_t*>(p.v + at * D) + lane);
        const float2 a = two_codes(f16_low(word)), c = two_codes(f16_high(word));
        v[0] = a.x;
        v[1] = a.y;
        v[2] = c.x;
        v[3] = c.y;
      } else {
        const uint32_t word = __ldg(reinterpret_cast<const uint16_t*>(p.v + at * D) + lane);
        const float2 a = two_codes(f16_low(word));
        v[0] = a.x;
        v[1] = a.y;
      }
#pragma unroll
      for (int f = 0; f < F; ++f) {
        v[f] *= scale;
        if (reads[0] >> k & 1) o[0][0][f] = fmaf(w0, v[f], o[0][0][f]);
        if (reads[1] >> k & 1) o[1][0][f] = fmaf(w1, v[f], o[1][0][f]);
      }
    }
  }
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    float sum = l[x][0] + l[x][1];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (!has[x]) continue;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    float y[F];
#pragma unroll
    for (int f = 0; f < F; ++f) y[f] = (o[x][0][f] + o[x][1][f]) * inv * 0x1p24f;
    const int64_t at = (static_cast<int64_t>(b) * p.queries + token[x]) * p.Hq + h[x];
    uint32_t* to = reinterpret_cast<uint32_t*>(p.o + at * D) + lane * (F / 2);
#pragma unroll
    for (int f = 0; f < F; f += 2) to[f / 2] = pack_bf16x2(y[f], y[f + 1]);
    if (lane == 0)
      p.lse[(static_cast<int64_t>(b) * p.Hq + h[x]) * p.queries + token[x]] =
          sum == 0.f ? -INFINITY : (m[x] + log2f(sum)) * 0.6931471805599453f;
  }
}

// Joins the pieces where a launch does not do so itself; a CTA per head and 8 rows.  (In 48
// registers, so that 20,480 CTAs that find nothing to do take 18 us, not 20.)
template <int D>
__global__ void __launch_bounds__(128, 10)
    paged_join_kernel(const __grid_constant__ PagedParams p, int tile_rows) {
  constexpr int kLanes = D / 4;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int item = blockIdx.x, chunks = tile_rows / 8;
  const int head_in = blockIdx.y / chunks, from = (blockIdx.y - head_in * chunks) * 8;
  const int2 piece = p.pieces[item];
  if (piece.y == 1 || piece.y == 0) return;
  const int entry = item / p.head_blocks, block = item - entry * p.head_blocks;
  const int b = p.by_row_tiles(entry), tile = entry - b * p.row_tiles;
  const int head = block * p.heads + head_in;
  const int rows = min(8, p.queries * p.G - tile * tile_rows - from);
  if (rows <= 0 || head >= p.Hkv) return;
  if (tile_rows == kPairRows) {
    bool far = piece.y < 0;
    for (int k = threadIdx.x; k < piece.y; k += blockDim.x)
      far |= p.far[2 * (piece.x + k * p.lanes) + (k == 0)] != 0;
    if (__syncthreads_or(far)) {
      exact_rows<D>(p, entry, head, from, rows);
      return;
    }
  }
  constexpr int U = 8 * kLanes / 128;
  const int64_t size = static_cast<int64_t>(p.heads) * tile_rows;  // of a piece
  int64_t at[U];
  JoinedRow row[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = threadIdx.x / kLanes + u * (128 / kLanes);
    at[u] = 2 * piece.x * size + head_in * tile_rows + from + min(r, rows - 1);
    row[u] = JoinedRow{r < rows ? b : -1, tile * tile_rows + from + r, head};
  }
  join_rows<D, U>(p, piece.y, at, 2 * p.lanes * size, size, row, threadIdx.x % kLanes * 4);
}

// ------------------------------------------------------------------- host
// How the heads and rows of a problem are cut up: H x S warps to a CTA, as many
// as can be with as few heads of the last CTA missing.
struct Cut {
  int heads, slices, head_blocks, row_tiles, tile_rows, step_keys;
  int64_t items;
  bool tiles;  // whole row tiles
};

Cut cut_of(const csbp_paged_problem& p, const csbp_kv_cache& c) {
  Cut r{};
  const int64_t rows = static_cast<int64_t>(p.queries) * (p.Hq / c.Hkv);
  r.tiles = rows > kMostRows;
  r.tile_rows = r.tiles ? kPairRows : rows <= 8 ? 8 : 16;
  r.row_tiles = static_cast<int>((rows + r.tile_rows - 1) / r.tile_rows);
  r.items = static_cast<int64_t>(p.batch) * r.row_tiles * c.Hkv;
  r.heads = r.slices = 1;
  r.head_blocks = c.Hkv;
  r.step_keys = kTileKeys;
  if (r.tiles) return r;
  const int most = most_warps(r.tile_rows / 8);
  double best = 0;
  for (int h = 1; h <= std::min(most, c.Hkv); ++h) {
    const int blocks = (c.Hkv + h - 1) / h, s = most / h;
    const double busy = static_cast<double>(h) * s * c.Hkv / (static_cast<double>(blocks) * h);
    if (busy >= best) {
      best = busy;
      r.heads = h;
      r.slices = s;
      r.head_blocks = blocks;
    }
  }
  r.items = static_cast<int64_t>(p.batch) * r.row_tiles * r.head_blocks;
  r.step_keys = kKeys * r.slices;
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
  const int64_t keys = static_cast<int64_t>(p->table_pages) * c->page_size;
  const Cut cut = cut_of(*p, *c);
  if ((keys / cut.step_keys + 3) * cut.head_blocks > 0x7fffffff / (cut.items / cut.head_blocks))
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
  size_t part_z, aside_o, aside_z, far, pieces, bytes;
};
Places places(const Cut& cut, int d, int sms) {
  const size_t rows = static_cast<size_t>(2) * sms * cut.heads * cut.tile_rows;
  Places r;
  r.part_z = kStatusBytes + round256(rows * d * 4);
  const size_t sums = static_cast<size_t>(sms) * cut.heads * cut.slices * cut.tile_rows;
  r.aside_o = r.part_z + round256(rows * 4);
  r.aside_z = r.aside_o + round256(sums * d * 4);
  r.far = r.aside_z + round256(sums * 4);
  r.pieces = r.far + round256(cut.tiles ? static_cast<size_t>(2) * sms * sizeof(int) : 0);
  r.bytes = r.pieces + round256(static_cast<size_t>(cut.items) * sizeof(int2));
  return r;
}

template <int D, int NT>
cudaError_t launch(const PagedParams& p, const Cut& cut, cudaStream_t stream) {
  using L = Rows<D, NT>;
  static PerDeviceOnce configured;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!configured.run(dev, [&](int) {
        e = cudaFuncSetAttribute(paged_rows_kernel<D, NT>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 L::smem(most_warps(NT)));
        return e == cudaSuccess;
      }))
    return e != cudaSuccess ? e : cudaErrorInvalidDevice;
  const int warps = cut.heads * cut.slices;
  paged_rows_kernel<D, NT><<<p.lanes * p.lane_ctas, warps * 32, L::smem(warps), stream>>>(p);
  return cudaGetLastError();
}

cudaError_t join(const PagedParams& p, const Cut& cut, int d, cudaStream_t stream) {
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(cut.items),
                     static_cast<unsigned>(cut.heads * (cut.tile_rows / 8)));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return d == 128 ? cudaLaunchKernelEx(&cfg, paged_join_kernel<128>, p, cut.tile_rows)
                  : cudaLaunchKernelEx(&cfg, paged_join_kernel<64>, p, cut.tile_rows);
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
  // places in the cache are counted in 31 bits, heads of them in 32
  if (cache->pages * cache->page_size >
      std::min<int64_t>(0x7fffffff, 0xffffffffll / cache->Hkv))
    return CSBP_ERR_UNSUPPORTED;
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
  a.lanes = cut.head_blocks <= sms / 8 ? cut.head_blocks : 1;
  a.lane_ctas = sms / a.lanes;
  a.lane_blocks = cut.head_blocks / a.lanes;
  a.by_lanes = Divisor::of(static_cast<uint32_t>(a.lanes));
  a.wide_scales = aligned(cache->k_scale, 4) && aligned(cache->v_scale, 4) &&
                  cache->Hkv * (cache->d / kGroup) % 4 == 0;
  a.by_page = Divisor::of(static_cast<uint32_t>(cache->page_size));
  a.by_G = Divisor::of(static_cast<uint32_t>(a.G));
  a.by_row_tiles = Divisor::of(static_cast<uint32_t>(cut.row_tiles));
  a.step_keys = cut.step_keys;
  a.by_step = Divisor::of(static_cast<uint32_t>(cut.step_keys));
  a.status = static_cast<int*>(workspace);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.part_o = reinterpret_cast<float*>(ws + kStatusBytes);
  a.part_z = reinterpret_cast<float*>(ws + at.part_z);
  a.aside_o = reinterpret_cast<float*>(ws + at.aside_o);
  a.aside_z = reinterpret_cast<float*>(ws + at.aside_z);
  a.far = reinterpret_cast<int*>(ws + at.far);
  a.pieces = reinterpret_cast<int2*>(ws + at.pieces);
  a.arrived = reinterpret_cast<int*>(ws + at.pieces);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const auto run = [&](auto d) {
    constexpr int D = decltype(d)::value;
    return cut.tile_rows == 8 ? launch<D, 1>(a, cut, s) : launch<D, 2>(a, cut, s);
  };
  const int timed = timer_begin(13, stream);
  cudaError_t e = cut.tiles         ? launch_tiles(a, cache->d, s)
                  : cache->d == 128 ? run(std::integral_constant<int, 128>())
                                    : run(std::integral_constant<int, 64>());
  timer_end(timed, stream);
  if (e != cudaSuccess) return CSBP_ERR_CUDA;
  if (joins_itself(cut.tile_rows)) return CSBP_OK;
  const int joined = timer_begin(14, stream);
  e = join(a, cut, cache->d, s);
  timer_end(joined, stream);
  return e == cudaSuccess ? CSBP_OK : CSBP_ERR_CUDA;
}
