// Attention over the quantised paged K/V cache for more query rows than the warp
// MMAs of attn_paged.cu carry (csbp_generate.h): blocks that are denoised, drafts of
// wide groups, chunks of prompts; on tcgen05 with its accumulators in TMEM.
//
// Rows.  The query rows of one KV head of a sequence, (token, head of the group)
// flattened, in row tiles of 128; a CTA works on two of them ("slots") against the
// keys that any of their rows reads, in tiles of 128 keys.  A last single row tile
// goes to both slots, which take the key tiles in turn; slot 0 joins the two sums at
// the end (`alternate`).  The list of steps (a pair of row tiles, a key tile, a KV
// head) is cut as in attn_paged.cu (paged_work.cuh), with as many partials and the same
// joining kernel.
//
// Operands.  K, V and Q are f16 in shared memory, P f16 in TMEM, all under powers of
// two that fp32 takes back: E4M3 codes are exact in f16, and so are their group
// scales 2^(e - E) to 2^-22, with E the largest scale byte of the K tile, and of
// V twice the largest so far in the feature group (O is rescaled when one grows past
// that, and when the maximum of a row has grown by 2^5.9).  P is p 2^10, rounded to
// 2^-11 of itself (2^-35 of the row's largest at least).  Where scales lie farther apart
// (a value 2^22 times the largest of another group of 32) the small ones would be lost, in
// rows that do not read the large one too: such an item is worked out again in fp32, by the
// kernel that joins the pieces.
//
// Keys.  One warp looks the pages up and starts the copies of K's codes and the scale
// bytes into a ring of three half tiles, another those of V's (cp.async: one bulk copy
// per key takes 58 clocks of the issuing warp each); five warps write K and V as f16
// into 128-byte-swizzled tiles: one for K (S(t) of both slots is done long before
// K(t + 1) is wanted) and two for V.  An alternate piece, which has one Q tile, puts
// every other K in the place of the second.  One thread issues the MMAs, two warpgroups
// do the softmax, a row per thread, as in the training forward.
//
// What bounds it.  16 sequences of 16,384 keys, 8 heads of 128, 160 rows: 264 us, where
// the bytes take 63 and the MMAs 115 (of 2 x 128 rows); a chunk of 2,000 tokens in a
// window of 1,024: 180 us, MMAs 40.  A pair of row tiles takes a key tile in 4,600
// clocks: two softmax rows of 128 scores per thread (1,800 clocks alone, 3,700 both at
// once), P V, and the next S, with a handover of 300 to 400 clocks between them, and
// beside that the conversion of K and V (3,500).  An item of a window costs 12,000 more
// for its result and the next Q.
//
// Keys that a row does not read are masked.  Where some row of the pair does not read
// a key of a tile, NaN in V is written as 0 and remembered: the rows that read it are
// marked when they are stored.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "csbp_internal.h"
#include "device_once.h"
#include "mbar_spin.cuh"
#include "paged_work.cuh"
#include "pair_math.cuh"
#include "ptx_sm100.cuh"

namespace csbp {
namespace paged {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = 5;  // converters
constexpr float kThreshold = 5.9f;  // log2: a row's maximum may lag by that
constexpr float kShift = 10.f;     // P = p 2^10 (2^15.9 at most)
constexpr int kHeadroom = 7;       // K and V operands: codes times up to 2^7
constexpr int kFlush = 512;        // key tiles that one accumulator takes in
constexpr int kHalves = 3;         // of the ring
constexpr int kInfos = 8;
// Per-warpgroup register budgets (setmaxnreg): issuer, copies and converters, softmax.  Their
// sum must not exceed the launch allocation (checked on the host).
constexpr uint32_t kRegsLow = 64;
constexpr uint32_t kRegsSoftmax = 192;
constexpr int kRegsNeeded = 256 * kRegsLow + 256 * kRegsSoftmax;

template <int D>
struct Tiles {
  static constexpr int kTileBytes = kTile * D * 2;  // Q, K or V tile (f16)
  static constexpr int kBoxBytes = kTile * 128;     // its 64-feature boxes
  static constexpr int kHalf = kTile * D;           // codes
  static constexpr int kQ = 0;                      // 2 slots
  static constexpr int kK = kQ + 2 * kTileBytes;
  static constexpr int kV = kK + kTileBytes;
  static constexpr int kRing = kV + 2 * kTileBytes;
  static constexpr int kWords = kRing + kHalves * kHalf;  // [3 tiles][K, V][key] scale words
  static constexpr int kInfo = kWords + 3 * 2 * kTile * 4;
  static constexpr int kRows = kInfo + kInfos * 64;  // [3 tiles][key] place in the cache
  static constexpr int kBar = kRows + 3 * kTile * 4;
  // barriers; those of K and V are [2] by tile
  static constexpr int bQFull = 0;                  // [2] per slot: it begins a piece
  static constexpr int bKFull = 2, bKEmpty = 4, bVFull = 6, bVEmpty = 8;
  static constexpr int bSFull = 10, bPFull = 12, bPvDone = 14;  // [2] per slot
  static constexpr int bDrain = 16;
  static constexpr int bInfo = 17;                  // [2] by tile
  static constexpr int bRows = 19;                  // [2] by tile: places of its keys
  static constexpr int bFull = 21;                  // [kHalves] codes are there
  static constexpr int bFree = bFull + kHalves;     // and have been converted
  static constexpr int kBars = bFree + kHalves;
  static constexpr int kMisc = kBar + kBars * 8;    // TMEM base, abort flag
  static constexpr int kRedo = kMisc + 8;           // [kInfos] by item
  static constexpr int kFar = kRedo + kInfos * 4;   // [kInfos] by item
  static constexpr int kCursor = (kFar + kInfos * 4 + 15) / 16 * 16;  // of each softmax warp
  static constexpr int kScale = kCursor + 8 * 48;  // [2 slots][row] of Q
  static constexpr int kJoin = kScale + 2 * kTile * 4;  // [row] of an alternate piece's slot 1
  static constexpr int kSmem = kJoin + kTile * 16;
  static constexpr uint32_t kColO = 256;            // O of slot s at kColO + D s
};
static_assert(Tiles<128>::kSmem <= 232448, "shared memory of a CTA");

// What is known about a tile, in shared memory.
struct Info {
  uint32_t there[4];  // which keys are there
  float k_factor;     // of S
  uint32_t k_top;     // E of K
  uint32_t top;       // E of V, a byte per group
  int at, cut, j0;    // its first place in the list; the first [0, cut) of its keys are
                      // sinks (at ..), the others keys j0 + their place in the tile
  int edge;           // some row does not read some key
  int upper;          // the scale bytes are the upper half of their words
  int item;           // the CTA's pieces so far
  int first;          // of a piece
  int k_at;           // where K goes
  int k_after;        // the tile whose S has to be done by then
};
static_assert(sizeof(Info) == 64, "");

__device__ __forceinline__ void copies_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// One arrival when the lane's cp.async copies so far are done.
__device__ __forceinline__ void arrive_after_copies(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major) {
  return (1u << 4)                                   // D: f32; A and B: f16
         | (static_cast<uint32_t>(b_mn_major) << 16)  // B major-ness
         | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// True in one thread of a warp; keeps what it passes to MMAs in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(yes));
  return yes != 0;
}

// 8 consecutive fp32 TMEM columns of this thread's lane, times f.
__device__ __forceinline__ void tmem_scale8(uint32_t at, float f) {
  float r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
      : "r"(at)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] *= f;
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n\t"
      "tcgen05.wait::st.sync.aligned;\n" ::"r"(at),
      "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7])
      : "memory");
}

__device__ __forceinline__ void lds128(uint32_t a, uint32_t* r) {
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
// 16 columns of the thread's lane.
__device__ __forceinline__ void tmem_ld16(uint32_t at, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
        "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]),
        "=f"(r[14]), "=f"(r[15])
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 3, 256;" ::: "memory"); }

// A CTA's part of one item.
struct Piece {
  int b, head, tile;  // sequence, KV head, pair of row tiles
  int k0, count, n;   // its steps, of the item's n
  int rows;           // of the pair
  bool alternate;
};

__device__ __forceinline__ Piece piece_of(const PagedParams& p, const Cursor& cur, int left) {
  Piece x;
  x.b = cur.b;
  x.head = cur.block;
  x.tile = cur.entry - cur.b * p.row_tiles;
  x.k0 = cur.step;
  x.n = cur.r.n;
  x.count = min(cur.r.n - cur.step, left);
  x.rows = min(kPairRows, p.queries * p.G - x.tile * kPairRows);
  x.alternate = x.rows <= kTile;
  return x;
}
__device__ __forceinline__ void next_item(const PagedParams& p, Cursor& cur) {
  cur.step = 0;
  cur.block += p.lanes;
  if (cur.block < p.head_blocks) return;
  cur.block -= p.lanes * p.lane_blocks;
  ++cur.entry;
  cur.load(p, kPairRows);
}

// A warp's cursor while its registers hold scores.
__device__ __forceinline__ void keep_cursor(uint32_t at, const Cursor& c) {
  if ((threadIdx.x & 31) == 0) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(c.entry), "r"(c.block),
                 "r"(c.step), "r"(c.b)
                 : "memory");
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at + 16), "r"(c.r.c), "r"(c.r.first),
                 "r"(c.r.lo), "r"(c.r.hi)
                 : "memory");
    asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(at + 32), "r"(c.r.n_first), "r"(c.r.n)
                 : "memory");
  }
  __syncwarp();
}
__device__ __forceinline__ Cursor kept_cursor(uint32_t at) {
  Cursor c;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(c.entry), "=r"(c.block), "=r"(c.step), "=r"(c.b)
               : "r"(at)
               : "memory");
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(c.r.c), "=r"(c.r.first), "=r"(c.r.lo), "=r"(c.r.hi)
               : "r"(at + 16)
               : "memory");
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];"
               : "=r"(c.r.n_first), "=r"(c.r.n)
               : "r"(at + 32)
               : "memory");
  return c;
}

// 2^(kHeadroom - delta) in f16, both halves; 0 below 2^-24, NaN for a byte of 255.  Where
// it takes E4M3's last bit below 2^-24 a 1 goes to `far` in shared memory (a byte of 0,
// below 2^-118, aside).
__device__ __noinline__ uint32_t operand_scale(int top, int byte, uint32_t far) {
  const int delta = top - byte;
  if (delta > kHeadroom + 15 && byte != 0 && byte != 255) sts32(far, 1);
  const uint32_t h = byte == 255 ? 0x7fffu
                     : delta <= kHeadroom + 14 ? static_cast<uint32_t>(kHeadroom + 15 - delta) << 10
                     : delta <= kHeadroom + 24 ? 1u << (kHeadroom + 24 - delta)
                                               : 0u;
  return h | h << 16;
}

// Keys that all rows of a pair read, besides the sinks: [lo, hi).
struct Common {
  int lo, hi;
};
__device__ __forceinline__ Common common_of(const PagedParams& p, int c, int tile) {
  const int first = tile * kPairRows, last = min(first + kPairRows, p.queries * p.G) - 1;
  Common x;
  x.hi = p.causal ? c - p.queries + static_cast<int>(p.by_G(first)) + 1 : c;
  x.lo = window_begin(p, c - p.queries + static_cast<int>(p.by_G(last)));
  return x;
}
// Whether some row of the pair does not read some key of a tile, going by the places of its
// keys: the first `cut` are sinks, the others keys j0 + their place in it.  (The first
// sinks are read by all rows.)
__device__ __forceinline__ bool edge_of(const PagedParams& p, const Common& x, int cut, int j0) {
  return cut < kTileKeys && !(j0 + kTileKeys <= x.hi &&
                              (j0 + cut >= x.lo || j0 + kTileKeys <= p.sinks));
}

// -------------------------------------------------------------------- copies
// Two warps: one looks keys up and copies K and the scale bytes, one copies V and works
// the scales' maxima out once they are there.
template <int D>
struct Copier {
  using L = Tiles<D>;
  const PagedParams& p;
  uint8_t* const smem;
  const uint32_t mem;
  const int lane;
  uint64_t* const bars;
  int* const abort_flag;

  __device__ __forceinline__ Copier(const PagedParams& p, uint8_t* smem, uint64_t* bars,
                                    int* abort_flag)
      : p(p), smem(smem), mem(smem_u32(smem)), lane(threadIdx.x & 31), bars(bars),
        abort_flag(abort_flag) {}

  __device__ __forceinline__ bool wait(int bar, int parity) const {
    return mbar_wait_warp(&bars[bar], parity & 1, p.status, abort_flag);
  }

  // Starts the copies of K's or V's codes of tile t.  (One copy of the code for both
  // warps, and a loop: what the roles of this kernel run per tile has to fit the
  // instruction cache together.)
  __device__ __noinline__ void copy(const uint8_t* codes, int t, int half) const {
    constexpr int kChunks = D / 16, kAtOnce = 32 / kChunks, kBatch = 32 / kAtOnce;
    const int chunk = lane % kChunks, r0 = lane / kChunks;
    const uint8_t* src = codes + chunk * 16;
    uint32_t to = mem + L::kRing + half * L::kHalf + r0 * D + chunk * 16;
    uint32_t rows = mem + L::kRows + (t % 3) * (kTile * 4) + r0 * 4;
    uint32_t word = mem + L::kInfo + (t % kInfos) * 64;
#pragma unroll 1
    for (int x = 0; x < 4; ++x, to += 32 * D, rows += 128, word += 4) {  // 32 keys
      uint32_t row[kBatch];
      const uint32_t there = lds32(word) >> r0;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) row[i] = lds32(rows + i * kAtOnce * 4);
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        copy16(to + i * kAtOnce * D, src + static_cast<uint64_t>(row[i]) * D,
               there >> i * kAtOnce & 1 ? 16 : 0);
    }
    arrive_after_copies(smem_u32(&bars[L::bFull + half]));
  }

  __device__ __forceinline__ void run_k(Cursor& cur, int steps) {
    int page[4], place[4];  // of keys lane + 32 x of the next tile
    const auto look = [&] {
      const int i0 = cur.step * kTileKeys + lane, end = cur.r.keys();
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int j = cur.r.key(i0 + 32 * x), entry = p.by_page(j);
        place[x] = j - entry * p.page_size;
        page[x] = -1;
        if (i0 + 32 * x < end) page[x] = __ldg(p.table + static_cast<int64_t>(cur.b) * p.table_pages + entry);
      }
    };
    int item = 0, m = 0;
    Common common{};
    bool begins = true, alternate = false;
    look();
#pragma unroll 1
    for (int t = 0; t < steps; ++t) {
      // (the places and scale words of tile t - 3 are free: V(t - 3) had been converted
      // when the codes of K(t - 1) were copied)
      const int h = 2 * t;
      Info& info = reinterpret_cast<Info*>(smem + L::kInfo)[t % kInfos];
      if (begins) {
        const int tile = cur.entry - cur.b * p.row_tiles;
        alternate = p.queries * p.G - tile * kPairRows <= kTile;
        m = 0;
        common = common_of(p, cur.r.c, tile);
      }
      const int at = cur.step * kTileKeys, cut = min(max(cur.r.first - at, 0), kTileKeys);
      const int j0 = at - cur.r.first + cur.r.lo;  // (of a key that is no sink)
      bool edge = edge_of(p, common, cut, j0);
      uint32_t rows = mem + L::kRows + (t % 3) * (kTile * 4) + lane * 4;
      uint32_t words = mem + L::kWords + (t % 3) * (2 * kTile * 4) + lane * 4;
      uint32_t there[4];
#pragma unroll
      for (int x = 0; x < 4; ++x, rows += 128, words += 128) {
        const bool is = static_cast<uint32_t>(page[x]) < static_cast<uint32_t>(p.pages);
        const uint32_t row =
            is ? static_cast<uint32_t>(page[x] * p.page_size + place[x]) * p.Hkv + cur.block : 0;
        there[x] = __ballot_sync(0xffffffffu, is);
        edge |= there[x] != ~0u;
        sts32(rows, row);
        const uint64_t at = static_cast<uint64_t>(row) * (D / 32);
        if (p.wide_scales) {
          copy4(words, p.k_scale + (at & ~uint64_t(3)), is ? 4 : 0);
          copy4(words + kTile * 4, p.v_scale + (at & ~uint64_t(3)), is ? 4 : 0);
        } else {
          uint32_t k = 0, v = 0;
          if (is)
#pragma unroll
            for (int e = 0; e < D / 32; ++e) {
              k |= static_cast<uint32_t>(__ldg(p.k_scale + at + e)) << 8 * e;
              v |= static_cast<uint32_t>(__ldg(p.v_scale + at + e)) << 8 * e;
            }
          sts32(words, k);
          sts32(words + kTile * 4, v);
        }
      }
      if (lane == 0) {
#pragma unroll
        for (int x = 0; x < 4; ++x) info.there[x] = there[x];
        info.at = at;
        info.cut = cut;
        info.j0 = j0;
        info.edge = edge;
        info.upper = D == 64 && p.wide_scales && (cur.block & 1);
        info.item = item;
        info.first = begins;
        // (the second Q tile is free when slot 1 has stored the piece before, which passes
        // through it, and the MMAs before are done: so it is when the first S of this piece
        // is, which waits for slot 1's arrival on its bQFull, in every piece)
        info.k_at = alternate && (m & 1) ? L::kQ + L::kTileBytes : L::kK;
        info.k_after = alternate && m > 1 ? t - 2 : t - 1;
      }
      ++m;
      // V(t - 2) had the half tile (and all that waited for bRows of t - 2 are past it)
      if (h >= kHalves && !wait(L::bFree + h % kHalves, h / kHalves - 1)) return;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[L::bRows + (t & 1)]);
      copy(p.k, t, h % kHalves);
      if (t + 1 < steps) {
        begins = ++cur.step == cur.r.n;
        if (begins) {
          next_item(p, cur);
          ++item;
        }
        look();
      }
    }
  }

  // The scale bytes of a key (D = 64: its head's half of a word).
  __device__ __forceinline__ uint32_t word(int t, int kv, int key, bool upper) const {
    const uint32_t w = lds32(mem + L::kWords + ((t % 3) * 2 + kv) * (kTile * 4) + key * 4);
    return D == 128 ? w : upper ? w >> 16 : w & 0xffffu;
  }

  __device__ __forceinline__ void run_v(int steps) {
    uint32_t top = 0, first = 0;  // E, and E when a piece began
#pragma unroll 1
    for (int t = 0; t < steps; ++t) {
      const int h = 2 * t + 1;
      if (!wait(L::bRows + (t & 1), t >> 1)) return;
      if (h >= kHalves && !wait(L::bFree + h % kHalves, h / kHalves - 1)) return;
      copy(p.v, t, h % kHalves);
      // the scales
      if (!wait(L::bFull + (h - 1) % kHalves, (h - 1) / kHalves)) return;
      Info& info = reinterpret_cast<Info*>(smem + L::kInfo)[t % kInfos];
      const bool upper = D == 64 && info.upper, begins = info.first;
      uint32_t k = 0, v = 0;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        uint32_t a = word(t, 0, lane + 32 * x, upper), b = word(t, 1, lane + 32 * x, upper);
        if (any_byte_255(a) || any_byte_255(b)) {
          a &= ~__vcmpeq4(a, 0xffffffffu);
          b &= ~__vcmpeq4(b, 0xffffffffu);
        }
        k = __vmaxu4(k, a);
        v = __vmaxu4(v, b);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v = __vmaxu4(v, __shfl_xor_sync(0xffffffffu, v, o));
      k = max(max(k & 255, k >> 8 & 255), max(k >> 16 & 255, k >> 24));
      k = __reduce_max_sync(0xffffffffu, k);
      // (twice as much as now, so that a little growth does not rescale O)
      bool far = false;
      if (begins) {
        top = first = __vaddus4(v, 0x01010101u);
      } else if (__vmaxu4(top, v) != top) {
        top = __vmaxu4(top, __vaddus4(v, 0x01010101u));
        // O follows E by 2^64 (and any way from a byte of 1, that of zeros: then it is nothing)
        const uint32_t zeros = __vcmpleu4(first, 0x01010101u);
        first = (first & ~zeros) | (top & zeros);
        far = at_least_u8x4(top - first, 0x41414141u) != 0;
      }
      if (lane == 0) {
        info.k_factor = ldexpf(1.f, static_cast<int>(k) - 127 - kHeadroom);
        info.k_top = k;
        info.top = top;
        if (begins) reinterpret_cast<volatile int*>(smem + L::kRedo)[info.item % kInfos] = 0;
        if (begins || far)
          reinterpret_cast<volatile int*>(smem + L::kFar)[info.item % kInfos] = far;
        mbar_arrive(&bars[L::bInfo + (t & 1)]);
      }
      __syncwarp();
    }
  }
};

// ---------------------------------------------------------------- converters
template <int D>
struct Converter {
  using L = Tiles<D>;
  const PagedParams& p;
  uint8_t* const smem;
  const uint32_t mem;
  const int warp, lane;

  __device__ __forceinline__ Converter(const PagedParams& p, uint8_t* smem)
      : p(p), smem(smem), mem(smem_u32(smem)), warp(static_cast<int>(threadIdx.x >> 5) - 3),
        lane(threadIdx.x & 31) {}

  // Codes of half tile `half` to f16 in the operand tile at `tile`, under E `top`.
  // kEdge: NaN is written as 0; whether there was any.
  template <bool kEdge>
  __device__ __forceinline__ bool convert(uint32_t from, uint32_t bytes, uint32_t top,
                                          uint32_t tile, uint32_t far) const {
    // 4 rows of 8 pieces of 16 codes (D = 64: 8 of 4) at a time, so that 8 lanes read
    // and write different banks
    constexpr int kAtOnce = D == 128 ? 4 : 8;
    const int r0 = D == 128 ? (lane >> 4) * 2 + (lane >> 2 & 1) : lane >> 2;
    const int c = D == 128 ? (lane & 3) + 4 * ((lane >> 2 ^ lane >> 3) & 1) : lane & 3;
    const int e = static_cast<int>(top >> 8 * (c >> 1) & 255);
    from += c * 16;
    bytes += c >> 1;
    tile += (c >> 2) * L::kBoxBytes;
    bool found = false;
    constexpr int kBatch = 3;  // loaded together
#pragma unroll 1
    for (int q0 = warp; q0 < kTile / kAtOnce; q0 += kBatch * kWarps) {
      uint32_t w[kBatch][4], byte[kBatch];
#pragma unroll
      for (int x = 0; x < kBatch; ++x) {
        const int r = min(q0 + x * kWarps, kTile / kAtOnce - 1) * kAtOnce + r0;
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[x][0]), "=r"(w[x][1]), "=r"(w[x][2]), "=r"(w[x][3])
                     : "r"(from + r * D)
                     : "memory");
        asm volatile("ld.shared.u8 %0, [%1];" : "=r"(byte[x]) : "r"(bytes + r * 4) : "memory");
      }
#pragma unroll
      for (int x = 0; x < kBatch; ++x) {
        if (x > 0 && q0 + x * kWarps >= kTile / kAtOnce) break;  // (the same for the warp)
        const int r = (q0 + x * kWarps) * kAtOnce + r0;
        if (kEdge) {
          uint32_t bad = byte[x] == 255;
#pragma unroll
          for (int k = 0; k < 4; ++k) bad |= nan_codes(w[x][k]);
          if (bad) {
            found = true;
            if (byte[x] == 255) byte[x] = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) w[x][k] &= ~nan_codes(w[x][k]);
          }
        }
        // 2^(headroom - (E - e)) in f16, the normal ones at once
        const int field = kHeadroom + 15 - e + static_cast<int>(byte[x]);
        uint32_t s = static_cast<uint32_t>(field) * 0x04000400u;
        if (field <= 0 || byte[x] == 255) s = operand_scale(e, static_cast<int>(byte[x]), far);
        const uint32_t to = tile + sw128_offset(r, 2 * (c & 3));
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(to),
                     "r"(mul_f16x2(f16_low(w[x][0]), s)), "r"(mul_f16x2(f16_high(w[x][0]), s)),
                     "r"(mul_f16x2(f16_low(w[x][1]), s)), "r"(mul_f16x2(f16_high(w[x][1]), s))
                     : "memory");
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(to ^ 16),
                     "r"(mul_f16x2(f16_low(w[x][2]), s)), "r"(mul_f16x2(f16_high(w[x][2]), s)),
                     "r"(mul_f16x2(f16_low(w[x][3]), s)), "r"(mul_f16x2(f16_high(w[x][3]), s))
                     : "memory");
      }
    }
    return found;
  }

  __device__ __forceinline__ void run(int steps, uint64_t* bars, int* abort_flag) {
    int half = 0, use = 0;
    bool ok = true;
#pragma unroll 1
    for (int h = 0; ok && h < 2 * steps; ++h) {
      const int t = h >> 1, kv = h & 1;
      const Info& info = reinterpret_cast<const Info*>(smem + L::kInfo)[t % kInfos];
      // (what is known of a tile is known when its K is there)
      ok = kv == 0 ? mbar_wait_warp(&bars[L::bInfo + (t & 1)], (t >> 1) & 1, p.status, abort_flag)
                   : mbar_wait_warp(&bars[L::bFull + half], use & 1, p.status, abort_flag);
      const int after = kv ? t - 2 : info.k_after;
      if (ok && after >= 0)
        ok = mbar_wait_warp(&bars[(kv ? L::bVEmpty : L::bKEmpty) + (after & 1)], after >> 1 & 1,
                            p.status, abort_flag);
      if (!ok) break;
      const uint32_t from = mem + L::kRing + half * L::kHalf;
      const uint32_t bytes = mem + L::kWords + ((t % 3) * 2 + kv) * (kTile * 4) +
                             (D == 64 && info.upper ? 2 : 0);
      const uint32_t top = kv ? info.top : info.k_top * 0x01010101u;
      const uint32_t tile = mem + (kv ? L::kV + (t & 1) * L::kTileBytes : info.k_at);
      const uint32_t far = mem + L::kFar + info.item % kInfos * 4;
      if (kv && info.edge) {
        if (convert<true>(from, bytes, top, tile, far))
          reinterpret_cast<volatile int*>(smem + L::kRedo)[info.item % kInfos] = 1;
      } else {
        convert<false>(from, bytes, top, tile, far);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bars[(kv ? L::bVFull : L::bKFull) + (t & 1)]);
        mbar_arrive(&bars[L::bFree + half]);
      }
      if (++half == kHalves) {
        half = 0;
        ++use;
      }
    }
  }
};

// ------------------------------------------------------------- softmax rows
// What a softmax thread's row is.
struct RowAt {
  int i, h;    // query and head
  int lo, hi;  // keys [lo, hi) of it, besides the sinks
};
__device__ __forceinline__ RowAt row_at(const PagedParams& p, const Piece& x, int c, int row) {
  const int r = min(x.tile * kPairRows + row, p.queries * p.G - 1);
  RowAt a;
  a.i = p.by_G(r);
  a.h = x.head * p.G + r - a.i * p.G;
  const int at = c - p.queries + a.i;
  a.hi = p.causal ? at + 1 : c;
  a.lo = window_begin(p, at);
  return a;
}

// Starts the copies of the warp's 32 rows of Q to rows `to0` .. of the tile at `tile`;
// `a` is the lane's row.
template <int D>
__device__ __noinline__ void copy_query(const PagedParams& p, const Piece x, const RowAt a,
                                        uint32_t tile, int to0) {
  constexpr int kChunks = D / 8, kAtOnce = 32 / kChunks;
  const int lane = threadIdx.x & 31, c = lane % kChunks;
  const int64_t mine = x.b * p.q_bat + a.i * p.q_tok + static_cast<int64_t>(a.h) * D;
  tile += (c >> 3) * Tiles<D>::kBoxBytes;
#pragma unroll 4
  for (int r = lane / kChunks; r < 32; r += kAtOnce) {
    const int64_t from = __shfl_sync(0xffffffffu, mine, r);
    copy16(tile + sw128_offset(to0 + r, c & 7), p.q + from + c * 8, 16);
  }
}

// That row `to` of the tile as f16 with its largest element as 2^7 .. 2^8 (and the
// copies of the warp waited for); returns what its scores are to be multiplied by.
template <int D>
__device__ __noinline__ float convert_query(const PagedParams& p, uint32_t tile, int to) {
  copies_wait_all();
  __syncwarp();
  uint32_t most = 0;
#pragma unroll 4
  for (int k = 0; k < D / 8; ++k) {
    uint32_t w[4];
    lds128(tile + (k >> 3) * Tiles<D>::kBoxBytes + sw128_offset(to, k & 7), w);
#pragma unroll
    for (int e = 0; e < 4; ++e) most = __vmaxu2(most, w[e] & 0x7fff7fffu);
  }
  most = max(most & 0xffffu, most >> 16);
  const int ex = max(static_cast<int>(most >> 7) - 127, -110);
  const float f = __uint_as_float(static_cast<uint32_t>(127 + 7 - ex) << 23);
#pragma unroll 4
  for (int k = 0; k < D / 8; ++k) {
    const uint32_t at = tile + (k >> 3) * Tiles<D>::kBoxBytes + sw128_offset(to, k & 7);
    uint32_t w[4];
    lds128(at, w);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = pack_f16(__uint_as_float(w[e] << 16) * f, __uint_as_float(w[e] & 0xffff0000u) * f);
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3])
                 : "memory");
  }
  fence_proxy_async_smem();
  __syncwarp();
  return p.scale_log2 * ldexpf(1.f, ex - 7);
}

// Features (of chunk c, a bit each) that are NaN in some key that the row reads of those
// tiles of the piece from which NaN has been taken out: those at an edge, or with a key
// that is not there.  (The others carry it through the MMAs.  All keys of a long text, each
// byte by itself, would take longer than the waits of the other roles allow.)
template <int D>
__device__ __noinline__ uint32_t nan_features(const PagedParams& p, const Piece x, const Range r,
                                              const RowAt a, int c) {
  uint32_t bad = 0;
  const Common common = common_of(p, r.c, x.tile);
  const int32_t* table = p.table + static_cast<int64_t>(x.b) * p.table_pages;
  const auto missing = [&](int j, int end) {  // whether one of keys [j, end) is
    bool some = false;
    for (int entry = p.by_page(j); j < end && !some; j = ++entry * p.page_size)
      some = static_cast<uint32_t>(__ldg(table + entry)) >= static_cast<uint32_t>(p.pages);
    return some;
  };
  for (int k = x.k0; k < x.k0 + x.count; ++k) {
    const int at = k * kTileKeys, cut = min(max(r.first - at, 0), kTileKeys);
    const int j0 = at - r.first + r.lo, end = min(at + kTileKeys, r.keys());
    if (!edge_of(p, common, cut, j0) && end == at + kTileKeys && !missing(at, at + cut) &&
        !missing(j0 + cut, j0 + kTileKeys))
      continue;
    for (int i = at; i < end; ++i) {
      const int j = r.key(i);
      if (!(j < a.hi && (j >= a.lo || j < p.sinks))) continue;
      const int entry = p.by_page(j);
      const int pg = __ldg(table + entry);
      if (static_cast<uint32_t>(pg) >= static_cast<uint32_t>(p.pages)) continue;
      const uint64_t slot = static_cast<uint32_t>(pg * p.page_size + j - entry * p.page_size);
      const uint64_t place = slot * p.Hkv + x.head;
      if (__ldg(p.v_scale + place * (D / 32) + c) == 255) bad = ~0u;
      const uint4* codes = reinterpret_cast<const uint4*>(p.v + place * D + c * 32);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 v = __ldg(codes + h);
        const uint32_t nan[4] = {nan_codes(v.x), nan_codes(v.y), nan_codes(v.z), nan_codes(v.w)};
        if (nan[0] | nan[1] | nan[2] | nan[3])
#pragma unroll
          for (int e = 0; e < 16; ++e) bad |= (nan[e / 4] >> 8 * (e % 4) & 1) << (16 * h + e);
      }
    }
  }
  return bad;
}

// What a row has summed.
struct Sum {
  float m, l;    // largest score (log2) and sum of P under it
  uint32_t top;  // E of each feature group
  int tiles;     // key tiles in the accumulator
  bool aside;    // and earlier ones in `aside_o`, `aside_z`
};

// ... and the LSE of it (log2).
__device__ __forceinline__ float lse_of(const Sum& sum) {
  return sum.tiles > 0 && sum.l != 0.f ? sum.m - kShift + log2f(sum.l) : -INFINITY;
}

// What slot 1 of an alternate piece leaves for slot 0, beside its O.
struct Join {
  float z, inv;  // LSE, 1 / l
  uint32_t top;
  int what;      // bit 0: it has summed something, bit 1: it has put something aside
};

// 2^(E - 127 - headroom) of feature group g in two factors: one could lie below fp32's
// range.
__device__ __forceinline__ float2 unit_of(uint32_t top, int g) {
  const int ex = static_cast<int>(top >> 8 * g & 255);
  return make_float2(__uint_as_float(static_cast<uint32_t>(ex / 2 + 64) << 23),
                     __uint_as_float(static_cast<uint32_t>(ex - ex / 2 + 63 - kHeadroom) << 23));
}

// Stores a row's normalised O and its LSE, joined with what was put aside and, of an
// alternate piece (`other`), with slot 1's.  To the outputs (`part` = -1), a place among
// the partials, or aside (kAside).  Whole warps; `o_at` is the warp's O.  On their way
// to outputs and partials the rows pass through the Q tile at `tile`, so that they are
// written as wholes: 32 rows' 16 bytes at a time took 1,500 clocks per 16 columns.  (What
// is put aside, in the middle of a piece, does not.)
constexpr int kAside = -2;
template <int D>
__device__ __noinline__ void store_sum(const PagedParams& p, const Piece x, const Range r,
                                       const RowAt a, const Sum sum, uint32_t o_at, int s, int row,
                                       int part, bool redo, uint32_t tile, const Join* other) {
  tc_fence_after_sync();
  float* const aside_o = p.aside_o + static_cast<int64_t>(blockIdx.x) * kPairRows * D;
  float* const aside_z = p.aside_z + static_cast<int64_t>(blockIdx.x) * kPairRows;
  const int mine = s * kTile + row, others = kTile + row;
  const bool here = sum.tiles > 0;
  Join o1{-INFINITY, 0.f, 0, 0};
  if (other) o1 = other[row];
  const float z = lse_of(sum);
  const float z_mine = sum.aside ? aside_z[mine] : -INFINITY;
  const float z_other = o1.what & 2 ? aside_z[others] : -INFINITY;
  const float most = fmaxf(fmaxf(z, o1.z), fmaxf(z_mine, z_other));
  const float ref = most == -INFINITY ? 0.f : most;
  float w = exp2f(z - ref), w1 = exp2f(o1.z - ref);
  float w_mine = exp2f(z_mine - ref), w_other = exp2f(z_other - ref);
  const float all = w + w1 + w_mine + w_other, inv = all == 0.f ? 0.f : 1.f / all;
  // (NaN in a sum goes on to all of the row)
  w = z == -INFINITY ? 0.f : w * inv / sum.l;
  w1 = o1.z == -INFINITY ? 0.f : w1 * inv * o1.inv;
  w_mine *= inv;
  w_other *= inv;
  const float lse = all == 0.f ? -INFINITY : ref + log2f(all);
  const bool valid = x.tile * kPairRows + (x.alternate ? 0 : s * kTile) + row < p.queries * p.G;
  const int64_t token = static_cast<int64_t>(x.b) * p.queries + a.i;
  const int64_t place = static_cast<int64_t>(part) * kPairRows + (x.alternate ? 0 : s * kTile) + row;
  // where the row goes, in bytes
  uint8_t* const base = reinterpret_cast<uint8_t*>(part == -1 ? static_cast<void*>(p.o) : p.part_o);
  const int64_t row_at = part != -1 ? place * D * 4 : valid ? (token * p.Hq + a.h) * D * 2 : -1;
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    float o[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = 0.f;
    if (here) {
      tmem_ld32(o_at + c, o);
      const float2 u = unit_of(sum.top, c / 32);
      const float f = w * u.x;
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = o[i] * f * u.y;
    }
    if (o1.what & 1) {
      const float2 u = unit_of(o1.top, c / 32);
      const float f = w1 * u.x;
#pragma unroll
      for (int k = 0; k < 32; k += 16) {
        float y[16];
        tmem_ld16(o_at + D + c + k, y);
#pragma unroll
        for (int i = 0; i < 16; ++i) o[k + i] = fmaf(y[i] * f, u.y, o[k + i]);
      }
    }
    if (sum.aside || (o1.what & 2)) {
#pragma unroll 1
      for (int k = 0; k < 2; ++k) {
        if (k == 0 ? z_mine == -INFINITY : z_other == -INFINITY) continue;
        const float f = k == 0 ? w_mine : w_other;
        const float4* v =
            reinterpret_cast<const float4*>(aside_o + (k == 0 ? mine : others) * D + c);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 y = v[i];
          o[4 * i] = fmaf(y.x, f, o[4 * i]);
          o[4 * i + 1] = fmaf(y.y, f, o[4 * i + 1]);
          o[4 * i + 2] = fmaf(y.z, f, o[4 * i + 2]);
          o[4 * i + 3] = fmaf(y.w, f, o[4 * i + 3]);
        }
      }
    }
    if (redo) {
      const uint32_t bad = valid ? nan_features<D>(p, x, r, a, c / 32) : 0;
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (bad >> i & 1) o[i] = NAN;
    }
    if (part == kAside) {
      float4* to = reinterpret_cast<float4*>(aside_o + mine * D + c);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        to[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
      continue;
    }
    const auto put = [&](int chunk, uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {
      asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(
                       tile + (chunk >> 3) * Tiles<D>::kBoxBytes + sw128_offset(row, chunk & 7)),
                   "r"(w0), "r"(w1), "r"(w2), "r"(w3)
                   : "memory");
    };
    if (part == -1) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        put(c / 8 + i, pack_bf16x2(o[8 * i], o[8 * i + 1]), pack_bf16x2(o[8 * i + 2], o[8 * i + 3]),
            pack_bf16x2(o[8 * i + 4], o[8 * i + 5]), pack_bf16x2(o[8 * i + 6], o[8 * i + 7]));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        put(c % (D / 2) / 4 + i, __float_as_uint(o[4 * i]), __float_as_uint(o[4 * i + 1]),
            __float_as_uint(o[4 * i + 2]), __float_as_uint(o[4 * i + 3]));
    }
    // the tile's rows have 2 D bytes: the whole row, or half of the fp32
    const int width = part == -1 ? D : D / 2;
    if ((c + 32) % width != 0) continue;
    constexpr int kChunks = D / 8, kAtOnce = 32 / kChunks;
    const int k = lane % kChunks;
    uint8_t* const to = base + (part == -1 ? 0 : (c + 32 - width) * 4) + k * 16;
    __syncwarp();
#pragma unroll 4
    for (int y = lane / kChunks; y < 32; y += kAtOnce) {
      const int64_t at = __shfl_sync(0xffffffffu, row_at, y);
      uint32_t v[4];
      lds128(tile + (k >> 3) * Tiles<D>::kBoxBytes + sw128_offset((row & ~31) + y, k & 7), v);
      if (at >= 0) *reinterpret_cast<uint4*>(to + at) = make_uint4(v[0], v[1], v[2], v[3]);
    }
    __syncwarp();
  }
  if (part == kAside)
    aside_z[mine] = lse;
  else if (part >= 0)
    p.part_z[place] = lse;
  else if (valid)
    p.lse[(static_cast<int64_t>(x.b) * p.Hq + a.h) * p.queries + a.i] = lse * 0.6931471805599453f;
  tc_fence_before_sync();
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tiles_kernel(const __grid_constant__ PagedParams p) {
  using L = Tiles<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // the swizzled tiles need a 1024-aligned window
    if (threadIdx.x == 0) atomicExch(p.status, DEV_MISALIGNED);
    return;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint32_t* tmem_base_sh = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  int* abort_flag = reinterpret_cast<int*>(smem + L::kMisc + 4);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;

  Cursor cur{};
  const Share share =
      find_share<kPairRows, kThreads / 32>(p, reinterpret_cast<uint32_t*>(smem), cur);
  if (share.begin >= share.end) return;
  const int steps = static_cast<int>(share.end - share.begin);
  if (threadIdx.x == 0) {
    // arrivals: converter warps, a slot's softmax warps, the copying lanes, else one
    // arrival or commit
    for (int i = 0; i < L::kBars; ++i) {
      const auto is = [&](int bar) { return i == bar || i == bar + 1; };
      mbar_init(&bars[i], is(L::bQFull) || is(L::bPFull)                   ? 4
                          : is(L::bKFull) || is(L::bVFull) || i >= L::bFree ? kWarps
                          : i >= L::bFull                                   ? 32
                                                                            : 1);
    }
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_base_sh, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_base_sh;

  if (warp < 8) {
    setmaxnreg_dec<kRegsLow>();
    if (warp == 0 && elect_one()) {
      // ===================== MMA issuer
      constexpr uint32_t idesc_s = idesc_f16_f32(128, 128, false);
      constexpr uint32_t idesc_pv = idesc_f16_f32(128, D, true);
      bool ok = true;
      int npv0 = 0, npv1 = 0, pieces = 0;        // P V issued per slot, pieces so far
      int sum0 = 0, sum1 = 0;                    // key tiles in the accumulators
      // (descriptors are made where they are used: 64 registers hold few of them)
      const uint32_t base = smem_u32(smem);
      const auto desc_of = [&](uint32_t at, uint32_t lead) {
        asm volatile("" : "+r"(at));
        return sdesc_sw128(at, lead, 1024);
      };
      // S_s = Q K^T of Q tile sq
      auto issue_s = [&](int s, int sq, int k_at) {
        tc_fence_after_sync();
        const uint64_t q_desc = desc_of(base + L::kQ + sq * L::kTileBytes, 16);
        const uint64_t k_desc = desc_of(base + k_at, 16);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (k >> 2) * L::kBoxBytes + (k & 3) * 32;
          umma_bf16_ss(tmem + s * 128, sdesc_step(q_desc, off), sdesc_step(k_desc, off), idesc_s,
                       k > 0 ? 1u : 0u);
        }
        umma_commit(&bars[L::bSFull + s]);
      };
      // O_s += P_s V
      auto issue_pv = [&](int s, int v_at, uint32_t acc0) {
        tc_fence_after_sync();
        const uint64_t v_desc = desc_of(base + v_at, L::kBoxBytes);  // MN-major
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          umma_bf16_ts(tmem + L::kColO + s * D, tmem + s * 128 + k * 8, sdesc_step(v_desc, k * 2048),
                       idesc_pv, k > 0 ? 1u : acc0);
        umma_commit(&bars[L::bPvDone + s]);
      };
      int t = 0;  // key tiles so far
      for (int left = steps; ok && left > 0;) {
        const Piece x = piece_of(p, cur, left);
        const bool both = !x.alternate;
        const int count = x.count;
        ok = mbar_wait(&bars[L::bQFull], pieces & 1, p.status, abort_flag) &&
             mbar_wait(&bars[L::bQFull + 1], pieces & 1, p.status, abort_flag);
        ++pieces;
        sum0 = sum1 = 0;
        // S of tile m and P V of tile m - 1, of the slots that work on them, each as soon
        // as what it reads is there (a slot's S after its P V, which reads the P there):
        // the conversion of K and V waits for them
#pragma unroll 1
        for (int m = 0; ok && m <= count; ++m) {
          // bits 0, 1: S of the slots to be issued, 2, 3: P V
          uint32_t todo = both ? (m < count ? 3u : 0u) | (m > 0 ? 12u : 0u)
                               : (m < count ? 1u << (m & 1) : 0u) | (m > 0 ? 8u >> (m & 1) : 0u);
          bool k_full = false, v_full = false;
          uint64_t t0 = 0;
          int idle = 0;
          while (todo) {
            bool some = false;
            const int tk = t + m, tv = t + m - 1;  // K's and V's tile
            if (!v_full && (todo & 12))
              v_full = mbar_test_wait(&bars[L::bVFull + (tv & 1)], tv >> 1 & 1);
            if (!k_full && (todo & 3))
              k_full = mbar_test_wait(&bars[L::bKFull + (tk & 1)], tk >> 1 & 1);
#pragma unroll 1
            for (int s = 0; s < 2; ++s) {
              const int npv = s ? npv1 : npv0;
              if ((todo >> s & 4) && v_full && mbar_test_wait(&bars[L::bPFull + s], npv & 1)) {
                int sum = s ? sum1 : sum0;
                issue_pv(s, L::kV + (tv & 1) * L::kTileBytes, sum > 0 ? 1u : 0u);
                if (++sum == kFlush) sum = 0;
                if (s) {
                  ++npv1;
                  sum1 = sum;
                } else {
                  ++npv0;
                  sum0 = sum;
                }
                todo &= ~(4u << s);
                if (!(todo & 12)) umma_commit(&bars[L::bVEmpty + (tv & 1)]);
                some = true;
              } else if ((todo >> s & 1) && !(todo >> s & 4) && k_full &&
                         (npv == 0 || mbar_test_wait(&bars[L::bPvDone + s], (npv - 1) & 1))) {
                issue_s(s, both ? s : 0, !both && (m & 1) ? L::kQ + L::kTileBytes : L::kK);
                todo &= ~(1u << s);
                if (!(todo & 3)) umma_commit(&bars[L::bKEmpty + (tk & 1)]);
                some = true;
              }
            }
            // bounded, as every wait
            if (some) {
              idle = 0;
            } else if ((++idle & 63) == 0) {
              const uint64_t now = globaltimer_ns();
              if (idle == 64) t0 = now;
              if (*reinterpret_cast<volatile int*>(abort_flag) || now - t0 > 2000000000ull) {
                if (now - t0 > 2000000000ull) {
                  atomicExch(p.status, DEV_TIMEOUT);
                  *reinterpret_cast<volatile int*>(abort_flag) = 1;
                }
                ok = false;
                break;
              }
            }
          }
        }
        t += x.count;
        left -= x.count;
        if (left > 0) next_item(p, cur);
      }
      // drain every MMA this thread issued before the CTA may free TMEM
      umma_commit(&bars[L::bDrain]);
      mbar_wait(&bars[L::bDrain], 0, nullptr, nullptr, 500000000ull);
    } else if (warp == 1) {
      Copier<D>(p, smem, bars, abort_flag).run_k(cur, steps);
      copies_wait_all();
    } else if (warp == 2) {
      Copier<D>(p, smem, bars, abort_flag).run_v(steps);
      copies_wait_all();
    } else if (warp >= 3) {
      Converter<D>(p, smem).run(steps, bars, abort_flag);
    }
  } else {
    setmaxnreg_inc<kRegsSoftmax>();
    // ===================== softmax warpgroup of slot s
    const int s = (warp - 8) >> 2;
    const int row = threadIdx.x - 128 * (2 + s);
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t colS = s * 128, colO = L::kColO + s * D;
    bool ok = true;
    int n_s = 0;  // key tiles of this slot so far
    int t0 = 0;   // key tiles so far
    int item = 0;
    const uint32_t kept = smem_u32(smem + L::kCursor + (warp - 8) * 48);
    keep_cursor(kept, cur);
    const uint32_t s_at = tmem + lane_base + colS, o_at = tmem + lane_base + colO;
    const uint32_t q_tile = smem_u32(smem + L::kQ + s * L::kTileBytes);
    float* const q_scale = reinterpret_cast<float*>(smem + L::kScale) + s * kTile;
    for (int left = steps; left > 0; ++item) {
      int count, stride, hi, lo;
      bool has_rows;
      {
        const Cursor cur = kept_cursor(kept);
        const Piece x = piece_of(p, cur, left);
        const int first_row = x.alternate ? 0 : s * kTile;
        has_rows = first_row + (warp & 3) * 32 < x.rows;  // warp-uniform
        const RowAt a = row_at(p, x, cur.r.c, first_row + row);
        if (has_rows && (s == 0 || !x.alternate)) {
          copy_query<D>(p, x, a, q_tile, row & ~31);
          q_scale[row] = convert_query<D>(p, q_tile, row);
        }
        // (all lanes have stored the piece before and written what the other slot may read)
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::bQFull + s]);
        hi = a.hi;
        lo = a.lo;
        count = x.count;
        stride = x.alternate ? 2 : 1;
      }
      float row_scale = q_scale[row];
      Sum sum{-INFINITY, 0.f, 0, 0, false};
      // the last P V of this slot
      const auto last_done = [&] {
        if (n_s > 0 && ok)
          ok = mbar_wait_warp(&bars[L::bPvDone + s], (n_s - 1) & 1, p.status, abort_flag);
      };

#pragma unroll 1
      for (int m = stride == 2 ? s : 0; ok && m < count; m += stride) {
        if (sum.tiles == kFlush) {
          last_done();
          if (!ok) break;
          if (has_rows) {
            const Cursor cur = kept_cursor(kept);
            const Piece x = piece_of(p, cur, left);
            store_sum<D>(p, x, cur.r, row_at(p, x, cur.r.c, (x.alternate ? 0 : s * kTile) + row), sum, o_at, s, row, kAside, false, 0, nullptr);
          }
          sum = Sum{-INFINITY, 0.f, 0, 0, true};
        }
        if (!mbar_wait_warp(&bars[L::bSFull + s], n_s & 1, p.status, abort_flag)) {
          ok = false;
          break;
        }
        ++n_s;
        if (!has_rows) {  // nothing to do, but the MMA counts four warps
          ++sum.tiles;
          if (lane == 0) mbar_arrive(&bars[L::bPFull + s]);
          continue;
        }
        if (stride == 2 && m == 1) row_scale = q_scale[row - s * kTile];  // slot 0's Q
        tc_fence_after_sync();
        const Info& info = reinterpret_cast<const Info*>(smem + L::kInfo)[(t0 + m) % kInfos];
        // (not 0: a masked score times it has to stay -inf)
        const float mult = fmaxf(row_scale * info.k_factor, 1e-37f);
        float sv[kTile];
#pragma unroll
        for (int c = 0; c < kTile / 32; c += 2)
          tmem_ld32x2(s_at + c * 32, s_at + (c + 1) * 32,
                      sv + c * 32, sv + (c + 1) * 32);
        if (info.edge) {
          const uint32_t there[4] = {info.there[0], info.there[1], info.there[2], info.there[3]};
          const auto first = [&](int n, int q) -> uint32_t {  // those of word q among the first n
            n = min(max(n - 32 * q, 0), 32);
            return n == 32 ? ~0u : (1u << n) - 1;
          };
          const int cut = info.cut, at = info.at, j0 = info.j0;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t sinks = first(cut, q);
            const uint32_t reads =
                there[q] &
                ((sinks & first(hi - at, q)) |
                 (~sinks & first(hi - j0, q) &
                  (~first(lo - j0, q) | (p.window ? first(p.sinks - j0, q) : 0u))));
            if (!__all_sync(0xffffffffu, reads == ~0u))
#pragma unroll
            for (int c = 0; c < 32; ++c)
              sv[32 * q + c] = reads >> c & 1 ? sv[32 * q + c] : -INFINITY;
          }
        }
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < kTile; c += 2) mx4[c / 2 % 4] = fmax3(mx4[c / 2 % 4], sv[c], sv[c + 1]);
        const float mx = fmax3(fmaxf(mx4[0], mx4[1]), mx4[2], mx4[3]);
        const float m_new = fmaxf(sum.m, mx * mult);
        // A row's maximum is brought up to date where it has grown by too much itself: what
        // other rows of the warp read does not say when.  (false while both are -inf)
        const bool need = m_new > sum.m + kThreshold;
        const uint32_t now = info.top;
        if (sum.tiles > 0 && (now != sum.top || __any_sync(0xffffffffu, need))) {
          // O holds the P V so far, under the old maximum and E (its last P V is done:
          // this S was issued after it)
          const float alpha = need ? exp2f(sum.m - m_new) : 1.f;
#pragma unroll 1
          for (int c = 0; c < D / 8; ++c) {  // (8 at a time: the scores are in registers)
            const int by = static_cast<int>((now >> 8 * (c / 4) & 255) - (sum.top >> 8 * (c / 4) & 255));
            tmem_scale8(o_at + c * 8,
                        alpha * (by < 127 ? __uint_as_float(static_cast<uint32_t>(127 - by) << 23) : 0.f));
          }
        }
        sum.top = now;
        if (need) {
          sum.l *= exp2f(sum.m - m_new);  // 0 when sum.m was -inf
          sum.m = m_new;
        }
        const float ref = (sum.m == -INFINITY ? 0.f : sum.m) - kShift;
        const uint64_t mult2 = f2_pack(mult, mult), neg = f2_pack(-ref, -ref);
        uint64_t rs2 = f2_pack(0.f, 0.f);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float packed[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(sv[half * 64 + 2 * c], sv[half * 64 + 2 * c + 1]), mult2, neg),
                      x0, x1);
            const float e0 = ex2_approx(x0), e1 = ex2_approx(x1);
            rs2 = f2_add(rs2, f2_pack(e0, e1));
            packed[c] = __uint_as_float(pack_f16(e0, e1));
          }
          tmem_st32(s_at + half * 32, packed);
        }
        float rs0, rs1;
        f2_unpack(rs2, rs0, rs1);
        sum.l += rs0 + rs1;
        ++sum.tiles;
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::bPFull + s]);
      }
      // ------- the piece's end
      last_done();
      Cursor cur = kept_cursor(kept);
      const Piece x = piece_of(p, cur, left);
      const RowAt a = row_at(p, x, cur.r.c, (x.alternate ? 0 : s * kTile) + row);
      const int later = x.n - x.k0 - x.count;  // steps of the item in later shares
      const bool starts = x.k0 == 0;
      const int part =
          starts && later == 0 ? -1 : 2 * static_cast<int>(blockIdx.x) + (starts ? 1 : 0);
      Join* const other = reinterpret_cast<Join*>(smem + L::kJoin);
      if (x.alternate) {  // slot 0 stores for both
        if (s == 1)
          other[row] = Join{lse_of(sum), 1.f / sum.l, sum.top,
                            (sum.tiles > 0 ? 1 : 0) | (sum.aside ? 2 : 0)};
        tc_fence_before_sync();
        if (s == 1 && sum.aside) __threadfence_block();
        softmax_sync();
      }
      // (known when the last V is in its tile: both slots' last P V are done by now)
      const bool redo = reinterpret_cast<volatile int*>(smem + L::kRedo)[item % kInfos] != 0;
      if (threadIdx.x == 256) {
        const int far = reinterpret_cast<volatile int*>(smem + L::kFar)[item % kInfos];
        if (part >= 0) p.far[part] = far;
        if (starts)
          p.pieces[static_cast<int64_t>(cur.entry) * p.head_blocks + cur.block] =
              make_int2(static_cast<int>(blockIdx.x),
                        part < 0 && far ? -1
                                        : 1 + static_cast<int>((later + share.per - 1) / share.per));
      }
      if (ok && has_rows && !(x.alternate && s == 1))
        store_sum<D>(p, x, cur.r, a, sum, o_at, s, row, part, redo, q_tile,
                     x.alternate ? other : nullptr);
      tc_fence_before_sync();
      if (x.alternate) softmax_sync();  // what slot 1 has summed has been read
      t0 += x.count;
      left -= x.count;
      if (left > 0) {
        next_item(p, cur);
        keep_cursor(kept, cur);
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t launch(const PagedParams& p, cudaStream_t stream) {
  static PerDeviceOnce configured;
  static int launch_regs[PerDeviceOnce::kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!configured.run(dev, [&](int device) {
        e = cudaFuncSetAttribute(paged_tiles_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Tiles<D>::kSmem);
        if (e != cudaSuccess) return false;
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, paged_tiles_kernel<D>);
        if (e != cudaSuccess) return false;
        launch_regs[device] = fa.numRegs;
        return true;
      }))
    return e != cudaSuccess ? e : cudaErrorInvalidDevice;
  // setmaxnreg.inc would wait forever if the budgets exceeded the launch allocation
  if (launch_regs[dev] * kThreads < kRegsNeeded) return cudaErrorInvalidConfiguration;
  paged_tiles_kernel<D><<<p.lanes * p.lane_ctas, kThreads, Tiles<D>::kSmem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tiles(const PagedParams& p, int d, cudaStream_t stream) {
  return d == 128 ? launch<128>(p, stream) : launch<64>(p, stream);
}

}  // namespace paged
}  // namespace csbp
