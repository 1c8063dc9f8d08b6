// Attention of a batch that shares a long prefix (csbp_generate.h), for
// sm_103a: softmax(scale q K^T) V over the prefix keys, which all sequences
// read, and each sequence's own keys.
//
// Rows.  The query rows of one KV head are (sequence, token, head of the
// group), flattened in that order; a row tile is 128 consecutive ones, so the
// prefix K/V pass through the tensor cores once per 128 rows however they
// divide into sequences, tokens and heads.  The softmax warps copy the tile's
// rows into shared memory themselves, which takes any
// token or batch stride and any group size.
//
// Keys.  A row tile reads all prefix key tiles, then the own key tiles of each
// sequence that has rows in it, masked to that sequence's rows.  Own keys of
// short sequences fill few rows of the MMA, but no more than they would in
// row tiles of their own, and one softmax covers all of a row's keys.
//
// Work.  A job is two row tiles ("slots") of one head group with all their key
// tiles; a prefix key tile is loaded once for both, and each slot has its own
// softmax warpgroup, so that one slot's MMAs run under the other's softmax.  A
// job with one row tile left gives it to both slots, which take the key tiles
// in turn and are joined at the end (`alternate`).  The jobs, end to end, form
// one list that is cut into equal shares, one per CTA and SM, wherever the cuts
// fall: a CTA works through the pieces of its share.  A job that is cut leaves
// a normalised fp32 partial and its LSE per piece in the workspace, and a
// second kernel joins them exactly ([Blog] "在线 softmax 合并：为什么分两段算仍是同一个注意力").
//
// Runs.  The tensor cores' accumulator drops what is below its last place, a
// little in each of a tile's eight steps and always towards zero: O over T key
// tiles came out small by T 2^-21 of itself (V = 1: 0.5 % over a million keys,
// 18 % over 40 million, and nothing is added any more from 2^26 equal weights on).
// So a row reads about 2,048 tiles in a piece, 2^-10, and never more than twice as
// many: where an equal share could hold more, every job is cut into `runs` of one
// length, each with a partial of its own.
//
// Roles (384 threads), as in the training forward: one thread of warp 0
// TMA producer, one of warp 1 MMA issuer, warp 2 works out the pieces ahead of
// the others, warps 4..7 and 8..11 softmax of slot 0 and 1 (thread t = row t = TMEM
// lane t).  P is the TMEM A operand of P V, as bf16 pairs over the first 64
// columns of its S (d = 128) or in columns of its own (d = 64); its rounding to
// bf16 is the one that the tensor cores ask for, maxima and sums stay fp32.  O is
// rescaled only when a row's maximum grows by more than 2^8.  Warps without a row
// of their own take no part.  Own rows past a sequence's end may hold NaN: their
// scores are masked, and the softmax warps clear their V rows in shared memory
// before the MMA that would multiply them by P = 0.  Where another masked V is
// not finite, the rows it reached are summed again at the end of the share.
//
// Bound.  Long prefixes with enough rows: the chain S -> softmax -> P V of a slot
// and the issuer's barriers, as in the training forward (tensor pipe 55 % active
// at d = 128, 34 % at 64; issue slots 35 % and 44 %).  Few rows: HBM.  Small
// calls: a start of about 4 us, an end of 3.5, and the second kernel.  Measured:
//   1,048,576 keys, 4 x 16 queries, 32 / 8 heads of 128   790 us, 1390 TFLOP/s
//     (0.72 of the measured bf16 rate), 869 us and 1265 call after call, where the
//     power cap lowers the clocks; heads of 64            606 us
//   16,384 keys, 16 x 32 queries of 40 / 8 heads, own keys up to 1024   167 us
//   65,536 keys, 8 x 1 queries, 32 / 8 heads   48.8 us, 5.5 TB/s (0.81 of a copy)
//   8,192 keys, 8 x 1 queries, 32 / 8 heads    18.4 us
// A kernel without tensor cores took 41,000 us at the second and 7,200 at 8192
// keys; one job per CTA without cuts 46 us there, 342 at the second.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "csbp_generate.h"
#include "csbp_internal.h"
#include "device_once.h"
#include "divisor.cuh"
#include "generate_internal.h"
#include "mbar_spin.cuh"
#include "pair_math.cuh"
#include "ptx_sm100.cuh"

namespace csbp {
namespace {

constexpr size_t kStatusBytes = 256;
constexpr int64_t kMaxElems = int64_t(1) << 39;
constexpr int kThreads = 384;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
// Per-warpgroup register budgets (setmaxnreg): producer / MMA, softmax.
// Their sum must not exceed the launch allocation (checked on the host).
constexpr uint32_t kRegsLow = 112;
constexpr uint32_t kRegsSoftmax = 192;
constexpr int kRegsNeeded = 128 * kRegsLow + 256 * kRegsSoftmax;

// tma_load_3d with an L2 policy.
__device__ __forceinline__ void tma_load_3d_hint(void* smem_dst, const void* tmap, uint64_t* bar,
                                                 int x, int y, int z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
}

// True in one thread of a warp (all of it calls this).  With this test, and the
// warp's number the same in all lanes for the compiler, it keeps what the MMAs and
// copies of that thread take in uniform registers; `lane == 0` cost 4 to 25 % (a
// million keys: 861 against 829 us, 8 x 1 queries over 65536 keys with heads of 64
// 47 against 35).
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(yes));
  return yes != 0;
}

// How the rows and keys of a problem are cut up (host and device).
struct Plan {
  int32_t gs, n_groups;   // query heads per row group, groups of them
  int32_t seq_rows;       // rows of one sequence: queries x gs
  int32_t row_tiles;      // per head group
  int32_t pairs;          // jobs per head group
  int32_t parts;          // most pieces of a job
  int32_t ctas;           // shares
  int32_t runs;           // of a job; 1: jobs are cut where shares end
  // the list: jobs of equal length `full` in units of time, the first
  // `len_prefix` of each for its prefix tiles and the rest for the own tiles.
  // Its entries are runs, of length `len`.
  uint32_t len, full, len_prefix, total, snap;
  // share length in 32.32 fixed point, and reciprocals that only guess or cut
  // the same way everywhere
  uint64_t step;
  float inv_step;
  float inv_prefix, inv_own;
  Divisor by_gs, by_queries, by_seq_rows, by_pairs, by_len, by_runs, by_per_kv;

  // start of share c; a cut that would leave a piece shorter than `snap` moves to
  // the end of the job (of the run before it, where there are runs)
  __host__ __device__ uint32_t share(uint32_t c) const {
    if (c >= static_cast<uint32_t>(ctas)) return total;
    const uint32_t x = static_cast<uint32_t>((c * step) >> 32);
    const uint32_t start = by_len(x) * len, past = x - start;
    return past < snap ? start : len - past < snap ? start + len : x;
  }
  // the share that holds place x of the list
  __host__ __device__ int share_of(uint32_t x) const {
    int c = static_cast<int>(static_cast<float>(x) * inv_step);
    c = c < ctas ? c : ctas - 1;
    while (share(c) > x) --c;
    while (share(c + 1) <= x) ++c;
    return c;
  }

  // The piece at place `at` of a share that ends at `end`: its job and run, and
  // the range of the job's places.
  struct Piece {
    uint32_t job, run, x0, x1;
  };
  __host__ __device__ Piece piece(uint32_t at, uint32_t end) const {
    const uint32_t entry = by_len(at), start = entry * len;
    Piece r{entry, 0, at - start, end - start < len ? end - start : len};
    if (runs > 1) {
      r.job = by_runs(entry);
      r.run = entry - r.job * runs;
      r.x0 += r.run * len;
      r.x1 += r.run * len;
    }
    return r;
  }
};

// The jobs that are cut and how many pieces each has; at most one per cut.  (With
// runs all jobs are, each into its runs, and the list is empty.)
struct CutJobs {
  static constexpr int kMost = 255;  // as many CTAs, and pieces
  int32_t n;
  uint32_t job[kMost];
  uint8_t parts[kMost];
};

struct PrefixParams {
  Plan plan;
  int32_t batch, queries, prefix_len, own_max, Hq, causal;
  float scale_log2;
  const __nv_bfloat16* q;
  uint32_t q_tok, q_bat;  // strides in 16-byte units
  const __nv_bfloat16 *k_prefix, *v_prefix, *k_own, *v_own;
  int64_t tok[4], bat[4];  // element strides of those four
  const int32_t* own_len;
  __nv_bfloat16* o;   // [batch][queries][Hq][d]
  float* lse;         // [batch][Hq][queries]
  float* part_o;      // [parts][batch x queries x Hq][d]
  float* part_lse;    // [parts][batch x queries x Hq]
  int* status;
};

// A CTA's piece of a job.  Warp 2 works the pieces out ahead of the others and
// leaves them in a ring of two in shared memory.
struct Unit {
  int valid;           // 0: the share is done
  int group, part;
  int direct;          // the whole of its rows' keys
  int alternate;       // one row tile, both slots
  int m0, m1;          // range of the job's key-tile list
  int np;              // prefix key tiles of the job
  int row0[2];         // first flattened row of a slot's tile
  int rows[2];         // its rows
  int seq0[2];         // first of the sequences with rows in it
  int seqs[2];         // their number
  int own[2];          // their own key tiles, together
  // a slot's key tiles in the range: n_pre prefix tiles from t_pre on, then
  // n_own own tiles from t_own on, in steps of 1 (alternate: 2)
  int n_pre[2], t_pre[2], n_own[2], t_own[2];
  int keys[2][kTile];       // own keys of each sequence
  int upto[2][kTile + 1];   // own key tiles of the sequences before it

  // Whether slot s's Q tile is read.  One that is not signals nothing: its softmax
  // could be two pieces ahead of the issuer, where parities say the same again.
  __device__ __forceinline__ bool q_used(int s) const {
    return alternate ? s == 0 && m0 < m1 : n_pre[s] + n_own[s] > 0;
  }

  // Which slots read the m-th key tile of the list, and its number among the
  // prefix tiles or the slot's own tiles: prefix tiles first, then the two
  // slots' own tiles in turn.
  __device__ __forceinline__ void at(int m, bool& prefix, int& t, bool& in0, bool& in1) const {
    prefix = m < np;
    if (prefix) {
      t = m;
      in0 = !alternate || !(m & 1);
      in1 = !alternate || (m & 1);
      return;
    }
    const int x = m - np;
    if (alternate) {
      t = x;
      in0 = !(m & 1);
    } else {
      const int both = min(own[0], own[1]);
      in0 = x < 2 * both ? !(x & 1) : own[0] > own[1];
      t = x < 2 * both ? x >> 1 : x - both;
    }
    in1 = !in0;
  }
  // Place in the list of slot s's own tile t.
  __device__ __forceinline__ int place(int s, int t) const {
    const int both = min(own[0], own[1]);
    return np + (alternate ? t : t < both ? 2 * t + s : t + both);
  }
  // Own tiles of slot s among the first x of the list's own tiles.
  __device__ __forceinline__ int own_before(int s, int x) const {
    const int both = min(own[0], own[1]);
    if (x < 2 * both) return (x + 1 - s) >> 1;
    return own[s] > own[1 - s] ? x - both : both;
  }
  // Sequence (from seq0 on) that slot s's own tile t belongs to.
  __device__ __forceinline__ int sequence(int s, int t) const {
    int lo = 0, hi = seqs[s] - 1;
    while (lo < hi) {  // last one that starts at or before t
      const int mid = (lo + hi + 1) >> 1;
      if (upto[s][mid] <= t)
        lo = mid;
      else
        hi = mid - 1;
    }
    return lo;
  }
};

constexpr int kUnitBytes = (sizeof(Unit) + 15) / 16 * 16;

template <int D>
struct PrefixLayout {
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kTileBytes = kTile * D * 2;  // Q/K/V tile (bf16)
  static constexpr int kBoxBytes = kTile * 64 * 2;  // one 64-column TMA box
  static constexpr int kQ = 0;                      // 2 slots
  static constexpr int kK = kQ + 2 * kTileBytes;
  static constexpr int kV = kK + kStages * kTileBytes;
  static constexpr int kBar = kV + kStages * kTileBytes;
  // barriers
  static constexpr int bQFull = 0;                  // [2] per slot
  static constexpr int bKFull = bQFull + 2;         // [stage]
  static constexpr int bKEmpty = bKFull + kStages;
  static constexpr int bVFull = bKEmpty + kStages;
  static constexpr int bVEmpty = bVFull + kStages;
  static constexpr int bSFull = bVEmpty + kStages;  // [2] per slot
  static constexpr int bPFull = bSFull + 2;         // [2] (the slot's softmax warps)
  static constexpr int bPvDone = bPFull + 2;        // [2]
  static constexpr int bMerge = bPvDone + 2;        // slot 1's (max, sum) are in shared memory
  static constexpr int bJoined = bMerge + 1;        // slot 0 has read them and slot 1's O
  static constexpr int bUnitFull = bJoined + 1;     // [2] pieces worked out
  static constexpr int bUnitEmpty = bUnitFull + 2;  // [2] and used by all roles
  static constexpr int bDrain = bUnitEmpty + 2;
  static constexpr int kBars = bDrain + 1;
  static constexpr int kMisc = kBar + kBars * 8;    // tmem base, abort flag, redo flag
  static constexpr int kMl = (kMisc + 12 + 15) / 16 * 16;  // slot 1's max and sum, 128 rows
  static constexpr int kUnits = kMl + kTile * 8;    // ring of two pieces
  static constexpr int kDynSmem = kUnits + 2 * kUnitBytes;
  static constexpr uint32_t kColO = 256;            // O of slot s at kColO + D s
  // P of slot s: D = 64 leaves columns for it, where it is not over its S and the
  // next S need not wait for the PV (a million keys, 16 tokens of 4 sequences and
  // 32 heads: 604 us; 685 with P over S)
  static constexpr bool kOwnP = D == 64;
  static constexpr uint32_t kColP = kOwnP ? kColO + 2 * D : 0;
  static constexpr uint32_t kStepP = kOwnP ? kTile / 2 : kTile;
};

// Key tiles before place x of a job: prefix tiles by place alone (so that
// loading can start before any own length is known), own tiles by share.
__device__ __forceinline__ int prefix_before(const Plan& pl, int np, uint32_t x) {
  if (x >= pl.len_prefix) return np;
  return min(np, static_cast<int>(static_cast<float>(x) * pl.inv_prefix * static_cast<float>(np)));
}
// An own tile that comes while the other slot has none left takes longer than one
// that has its turn with the other slot's.  It counts kAlone of one: 64 x 1 queries
// over up to 2,048 own keys take 78 us with 1, 68 with 1.2, 62 with 1.4, 63 with
// 1.6; 24 x 16 over up to 8,192 72, 69, 66, 69.
constexpr float kAlone = 1.4f;
__device__ __forceinline__ int tiles_before(const Plan& pl, int np, int in_turn, int alone,
                                            uint32_t x) {
  if (x < pl.len_prefix) return prefix_before(pl, np, x);
  if (x == pl.full) return np + in_turn + alone;
  const float both = static_cast<float>(in_turn);
  const float t = static_cast<float>(x - pl.len_prefix) * pl.inv_own *
                  (both + kAlone * static_cast<float>(alone));
  return np + min(in_turn + alone, static_cast<int>(t <= both ? t : both + (t - both) / kAlone));
}

// The piece at place `at` of the list, in a share that ends at `end`; moves
// `at` to its end.  One whole warp.
__device__ __forceinline__ void make_unit(const PrefixParams& p, uint32_t& at, uint32_t end,
                                          Unit& u) {
  const int lane = threadIdx.x & 31;
  const Plan& pl = p.plan;
  if (at >= end) {
    if (lane == 0) u.valid = 0;
    __syncwarp();
    return;
  }
  const Plan::Piece piece = pl.piece(at, end);
  const uint32_t start = at - piece.x0;  // of the job, where shares cut it
  at += piece.x1 - piece.x0;
  const int group = pl.by_pairs(piece.job);
  const int pair = piece.job - group * pl.pairs;
  const bool alternate = 2 * pair + 1 >= pl.row_tiles;
  const int np = (p.prefix_len + kTile - 1) / kTile;
  int own[2];
#pragma unroll 1
  for (int s = 0; s < 2; ++s) {
    const int row0 = (2 * pair + (alternate ? 0 : s)) * kTile;
    const int rows = min(kTile, p.batch * pl.seq_rows - row0);
    const int seq0 = pl.by_seq_rows(row0);
    const int seqs = pl.by_seq_rows(row0 + rows - 1) - seq0 + 1;
    own[s] = s == 1 && alternate ? own[0] : 0;
    // (alternate: both slots go by slot 0's tables)
    for (int k0 = 0; k0 < (s == 1 && alternate ? 0 : seqs); k0 += 32) {
      const int k = k0 + lane;
      int keys = 0;
      if (k < seqs && p.own_max > 0)
        keys = min(max(__ldg(p.own_len + seq0 + k), 0), p.own_max);
      const int n = (keys + kTile - 1) / kTile;
      int sum = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
      }
      if (k < seqs) {
        u.keys[s][k] = keys;
        u.upto[s][k] = own[s] + sum - n;
      }
      own[s] += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) {
      u.row0[s] = row0;
      u.rows[s] = rows;
      u.seq0[s] = seq0;
      u.seqs[s] = seqs;
      u.own[s] = own[s];
    }
  }
  if (lane == 0) {
    u.valid = 1;
    u.group = group;
    u.part = pl.runs > 1 ? piece.run : static_cast<int>(blockIdx.x) - pl.share_of(start);
    u.direct = piece.x0 == 0 && piece.x1 == pl.full;
    u.alternate = alternate;
    u.np = np;
    const int in_turn = alternate ? own[0] : 2 * min(own[0], own[1]);
    const int alone = alternate ? 0 : abs(own[0] - own[1]);
    u.m0 = tiles_before(pl, np, in_turn, alone, piece.x0);
    u.m1 = tiles_before(pl, np, in_turn, alone, piece.x1);
    const int p0 = min(u.m0, np), p1 = min(u.m1, np);
    const int o0 = max(u.m0, np) - np, o1 = max(u.m1, np) - np;
#pragma unroll 1
    for (int s = 0; s < 2; ++s) {
      if (alternate) {  // places of the list with the slot's parity
        u.t_pre[s] = p0 + ((p0 ^ s) & 1);
        u.n_pre[s] = max(0, p1 - u.t_pre[s] + 1) >> 1;
        u.t_own[s] = o0 + (((np + o0) ^ s) & 1);
        u.n_own[s] = max(0, o1 - u.t_own[s] + 1) >> 1;
      } else {
        u.t_pre[s] = p0;
        u.n_pre[s] = p1 - p0;
        u.t_own[s] = u.own_before(s, o0);
        u.n_own[s] = u.own_before(s, o1) - u.t_own[s];
      }
    }
  }
  __syncwarp();
}

// A row of a tile: sequence b, token i, head h.
struct Row {
  uint32_t token;
  int b, i, h;
};
__device__ __forceinline__ Row row_at(const PrefixParams& p, int group, uint32_t flat) {
  Row r;
  r.token = p.plan.by_gs(flat);
  r.b = p.plan.by_queries(r.token);
  r.i = r.token - r.b * p.queries;
  r.h = group * p.plan.gs + static_cast<int>(flat - r.token * p.plan.gs);
  return r;
}

// Its place in q, in 16-byte units.
template <int D>
__device__ __forceinline__ uint32_t q_place(const PrefixParams& p, const Row& r) {
  return r.b * p.q_bat + r.i * p.q_tok + r.h * (D / 8);
}

// A warp's 32 Q rows into the 128-byte-swizzled tile of 64-feature boxes, from
// row `row0` on, D / 8 lanes to a row.  `mine`: place of the lane's own row in
// q, in 16-byte units.
template <int D>
__device__ __forceinline__ void copy_q(const PrefixParams& p, uint32_t mine, uint8_t* tile,
                                       int row0) {
  constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
  const int lane = threadIdx.x & 31, chunk = lane % kLanes;
  const uint4* src = reinterpret_cast<const uint4*>(p.q) + chunk;
  uint8_t* dst = tile + (chunk >> 3) * (kTile * 128);
  uint4 v[kLanes];
#pragma unroll
  for (int t = 0; t < kLanes; ++t)
    v[t] = __ldg(src + __shfl_sync(0xffffffffu, mine, t * kAtOnce + lane / kLanes));
#pragma unroll
  for (int t = 0; t < kLanes; ++t)
    *reinterpret_cast<uint4*>(dst + sw128_offset(row0 + t * kAtOnce + lane / kLanes, chunk & 7)) =
        v[t];
}

// acc += sum_j 2^(scale q.k_j - ref) v_j over keys [from, to) of one head, for
// two rows at once: 16 lanes to a row, lane l with features (l % 16) D / 16 .. (k
// and v point there); 4 keys in flight.  The rows' ranges may differ.
template <int D>
__device__ __forceinline__ void walk_keys(const float (&q)[D / 16], float (&acc)[D / 16],
                                          const __nv_bfloat16* k, const __nv_bfloat16* v,
                                          int64_t k_tok, int64_t v_tok, int from, int to,
                                          float scale, float ref) {
  constexpr int kN = D / 16, kBatch = 4;
  using Chunk = std::conditional_t<D == 128, uint4, uint2>;
  int most = to - from;
  most = max(most, __shfl_xor_sync(0xffffffffu, most, 16));
#pragma unroll 1
  for (int j0 = 0; j0 < most; j0 += kBatch) {
    float s[kBatch];
    Chunk vv[kBatch];
#pragma unroll
    for (int t = 0; t < kBatch; ++t) {
      s[t] = 0.f;
      const int64_t j = from + j0 + t < to ? from + j0 + t : 0;  // (in place of no load)
      const Chunk kk = __ldg(reinterpret_cast<const Chunk*>(k + j * k_tok));
      vv[t] = __ldg(reinterpret_cast<const Chunk*>(v + j * v_tok));
      const __nv_bfloat162* x = reinterpret_cast<const __nv_bfloat162*>(&kk);
#pragma unroll
      for (int e = 0; e < kN / 2; ++e) {
        const float2 y = __bfloat1622float2(x[e]);
        s[t] = fmaf(q[2 * e], y.x, fmaf(q[2 * e + 1], y.y, s[t]));
      }
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
#pragma unroll
      for (int t = 0; t < kBatch; ++t) s[t] += __shfl_xor_sync(0xffffffffu, s[t], o);
#pragma unroll
    for (int t = 0; t < kBatch; ++t) {
      const float w = exp2f(fmaf(s[t], scale, -ref));
      if (from + j0 + t >= to) continue;
      const __nv_bfloat162* x = reinterpret_cast<const __nv_bfloat162*>(&vv[t]);
#pragma unroll
      for (int e = 0; e < kN / 2; ++e) {
        const float2 y = __bfloat1622float2(x[e]);
        acc[2 * e] = fmaf(w, y.x, acc[2 * e]);
        acc[2 * e + 1] = fmaf(w, y.y, acc[2 * e + 1]);
      }
    }
  }
}

// Barrier 3: the eight softmax warps.
__device__ __forceinline__ void softmax_warps_sync() { asm volatile("bar.sync 3, 256;" ::: "memory"); }
__device__ __forceinline__ bool softmax_warps_and(bool x) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 3, 256, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(all)
      : "r"(static_cast<uint32_t>(x))
      : "memory");
  return all != 0;
}

// The rows of a share's pieces that came out not finite where masked keys can
// have done that, summed again over the keys that they read alone; their LSE
// is right (a score is masked before it is used).  By the softmax warps, when
// the whole share is done: the other roles have ended, so no wait of theirs
// runs out.  It is there to be right, not fast: 64 sequences of 8 tokens over
// 65536 keys (32 heads of 64) take 33 ms in place of 0.4 when one own V is NaN.
template <int D>
__device__ __forceinline__ void sum_again(const PrefixParams& p, uint32_t at, uint32_t end, Unit& u) {
  constexpr int kN = D / 16;
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - 4;
  const int f0 = (lane & 15) * kN;
  const int64_t all = static_cast<int64_t>(p.batch) * p.queries * p.Hq;
  while (true) {
    if (warp == 0) make_unit(p, at, end, u);
    softmax_warps_sync();
    if (!u.valid) return;
    const int64_t head = static_cast<int64_t>(p.plan.by_per_kv(u.group)) * D + f0;
#pragma unroll 1
    for (int i = warp; i < kTile; i += 8) {  // two rows
      const int s = i >= kTile / 2, row = 2 * i - s * kTile + (lane >> 4);
      const bool valid = row < u.rows[s] && !(u.alternate && s == 1) &&
                         (u.seqs[s] > 1 || p.causal) && u.m1 > max(u.m0, u.np);
      const Row x = row_at(p, u.group, u.row0[s] + min(row, max(u.rows[s] - 1, 0)));
      const int64_t r = static_cast<int64_t>(x.token) * p.Hq + x.h;
      const int64_t place = r * D + f0;
      bool need = false;
      float lse = 0.f;
      if (valid) {
        lse = u.direct ? p.lse[(static_cast<int64_t>(x.b) * p.Hq + x.h) * p.queries + x.i]
                       : p.part_lse[u.part * all + r];
        if (lse > -INFINITY) {  // it has keys, and no score is NaN
          float finite = 0.f;
#pragma unroll
          for (int c = 0; c < kN; ++c)
            finite = fmaf(u.direct ? __bfloat162float(p.o[place + c])
                                   : p.part_o[u.part * all * D + place + c],
                          0.f, finite);
          need = finite != finite;
        }
      }
      const uint32_t found = __ballot_sync(0xffffffffu, need);
      if (found == 0) continue;
      need = (found >> (lane & 16)) & 0xffffu;
      float q[kN], acc[kN];
      const __nv_bfloat16* qr = p.q + static_cast<int64_t>(q_place<D>(p, x)) * 8 + f0;
#pragma unroll
      for (int c = 0; c < kN; ++c) {
        q[c] = __bfloat162float(qr[c]);
        acc[c] = 0.f;
      }
      const float ref = lse * 1.4426950408889634f;
      const int pre0 = min(u.m0, u.np) * kTile;
      const int pre1 = min(p.prefix_len, min(u.m1, u.np) * kTile);
      walk_keys<D>(q, acc, p.k_prefix + head, p.v_prefix + head, p.tok[0], p.tok[1], pre0,
                   need ? pre1 : pre0, p.scale_log2, ref);
      // the piece's part of the sequence's own tiles
      const int sq = x.b - u.seq0[s], before = u.upto[s][sq];
      const int o0 = u.alternate ? max(u.m0, u.np) - u.np : u.t_own[s];
      const int o1 = u.alternate ? max(u.m1, u.np) - u.np : o0 + u.n_own[s];
      int hi = u.keys[s][sq];
      if (p.causal) hi = min(hi, hi - p.queries + x.i + 1);
      const int own0 = max(o0 - before, 0) * kTile;
      walk_keys<D>(q, acc, p.k_own + x.b * p.bat[2] + head, p.v_own + x.b * p.bat[3] + head,
                   p.tok[2], p.tok[3], own0, need ? min(hi, max(o1 - before, 0) * kTile) : own0,
                   p.scale_log2, ref);
#pragma unroll
      for (int c = 0; c < kN; ++c) {
        if (!need) continue;
        if (u.direct)
          p.o[place + c] = __float2bfloat16_rn(acc[c]);
        else
          p.part_o[u.part * all * D + place + c] = acc[c];
      }
    }
    softmax_warps_sync();
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap tm_kp, const __grid_constant__ CUtensorMap tm_vp,
                  const __grid_constant__ CUtensorMap tm_ko, const __grid_constant__ CUtensorMap tm_vo,
                  const PrefixParams p) {
  using Lay = PrefixLayout<D>;
  constexpr int kStages = Lay::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // layout above needs a 1024-aligned window
    if (threadIdx.x == 0) atomicExch(p.status, DEV_MISALIGNED);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::kBar);
  uint32_t* tmem_base_sh = reinterpret_cast<uint32_t*>(smem + Lay::kMisc);
  int* abort_flag = reinterpret_cast<int*>(smem + Lay::kMisc + 4);
  // set when a row may have taken in keys that it does not read
  volatile int* redo = reinterpret_cast<volatile int*>(smem + Lay::kMisc + 8);
  float2* ml = reinterpret_cast<float2*>(smem + Lay::kMl);
  const auto unit_at = [&](int k) -> Unit& {
    return *reinterpret_cast<Unit*>(smem + Lay::kUnits + (k & 1) * kUnitBytes);
  };

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);  // (see elect_one)
  const int lane = threadIdx.x & 31;
  // the kernel that joins the pieces may take its place on the GPU; it waits
  // for this one's end before it reads
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  uint32_t reached = p.plan.share(blockIdx.x);
  const uint32_t share_end = p.plan.share(blockIdx.x + 1);
  const Plan::Piece first = p.plan.piece(reached, share_end);
  const int first_group = p.plan.by_pairs(first.job);
  const int first_pair = first.job - first_group * p.plan.pairs;
  // Set-up, with the first piece's Q and K/V already on their way: memory takes
  // a few us to answer all SMs at once.  The two halves of the CTA meet at
  // barrier 2 when the barriers and TMEM are there.
  if (warp >= 4) {
    // (rows past the last are copies of it: finite, and never stored)
    const int flat = min(2 * first_pair * kTile + static_cast<int>(threadIdx.x) - 128,
                         p.batch * p.plan.seq_rows - 1);
    copy_q<D>(p, q_place<D>(p, row_at(p, first_group, flat)),
              smem + Lay::kQ + (warp >= 8 ? Lay::kTileBytes : 0), (warp & 3) * 32);
    fence_proxy_async_smem();
    asm volatile("bar.sync 2, %0;" ::"n"(kThreads) : "memory");
  } else {
    if (warp == 0 && lane == 0) {
      prefetch_tmap(&tm_kp);
      prefetch_tmap(&tm_vp);
      prefetch_tmap(&tm_ko);
      prefetch_tmap(&tm_vo);
      for (int i = 0; i < Lay::kBars; ++i) mbar_init(&bars[i], 1);
      for (int s = 0; s < 2; ++s) {  // the four warps of a slot
        mbar_init(&bars[Lay::bQFull + s], 4);
        mbar_init(&bars[Lay::bPFull + s], 4);
      }
      mbar_init(&bars[Lay::bMerge], 4);
      mbar_init(&bars[Lay::bJoined], 4);
      // producer, issuer and eight softmax warps
      mbar_init(&bars[Lay::bUnitEmpty], 10);
      mbar_init(&bars[Lay::bUnitEmpty + 1], 10);
      *abort_flag = 0;
      *redo = 0;
      fence_mbarrier_init();
    }
    if (warp == 1) {
      tmem_alloc(tmem_base_sh, 512);
      tmem_relinquish();
    }
    tc_fence_before_sync();
    asm volatile("bar.sync 1, 128;" ::: "memory");
    asm volatile("bar.arrive 2, %0;" ::"n"(kThreads) : "memory");
  }
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_base_sh;
  bool ok = true;

  if (warp < 4) {
    setmaxnreg_dec<kRegsLow>();
    if (warp == 0 && elect_one()) {
      // ===================== TMA producer
      int nk = 0, nv = 0;  // K / V tiles whose loads were issued
      int early = 0;       // of the first piece, before its own lengths are known
      // Keys that are read once need not push anything else out of L2, this
      // kernel's own code above all
      uint64_t policy;
      if (p.plan.pairs == 1)
        asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
      else
        asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
      auto load = [&](int buf, int full, const CUtensorMap* map, int st, int x, int tile, int z) {
        mbar_arrive_expect_tx(&bars[full + st], Lay::kTileBytes);
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          tma_load_3d_hint(smem + buf + st * Lay::kTileBytes + c * Lay::kBoxBytes, map,
                           &bars[full + st], x + c * 64, tile * kTile, z, policy);
      };
      if (reached < share_end) {
        const int np = (p.prefix_len + kTile - 1) / kTile;
        const int p0 = prefix_before(p.plan, np, first.x0);
        const int p1 = prefix_before(p.plan, np, first.x1);
        early = min(kStages, p1 - p0);
        const int x = p.plan.by_per_kv(first_group) * D;
        for (; nk < early; ++nk, ++nv) {
          load(Lay::kK, Lay::bKFull, &tm_kp, nk, x, p0 + nk, 0);
          load(Lay::kV, Lay::bVFull, &tm_vp, nk, x, p0 + nk, 0);
        }
      }
      for (int k = 0; ok; ++k) {
        ok = mbar_wait(&bars[Lay::bUnitFull + (k & 1)], (k >> 1) & 1, p.status, abort_flag);
        if (!ok) break;
        const Unit& u = unit_at(k);
        if (!u.valid) break;
        const int x = p.plan.by_per_kv(u.group) * D;
        const int m1 = u.m1;
        for (int m = u.m0 + (k == 0 ? early : 0); m < m1; ++m) {
          const int st = nk % kStages, use = nk / kStages;
          bool prefix, in0, in1;
          int tile, z = 0;
          u.at(m, prefix, tile, in0, in1);
          if (!prefix) {
            const int s = u.alternate || in0 ? 0 : 1;
            const int q = u.sequence(s, tile);
            tile -= u.upto[s][q];
            z = u.seq0[s] + q;
          }
          if (use > 0)
            ok = mbar_wait(&bars[Lay::bKEmpty + st], (use - 1) & 1, p.status, abort_flag);
          if (!ok) break;
          load(Lay::kK, Lay::bKFull, prefix ? &tm_kp : &tm_ko, st, x, tile, z);
          ++nk;
          if (use > 0)
            ok = mbar_wait(&bars[Lay::bVEmpty + st], (use - 1) & 1, p.status, abort_flag);
          if (!ok) break;
          load(Lay::kV, Lay::bVFull, prefix ? &tm_vp : &tm_vo, st, x, tile, z);
          ++nv;
        }
        if (ok) mbar_arrive(&bars[Lay::bUnitEmpty + (k & 1)]);
      }
      if (!ok) {
        // drain: wait (ignoring the abort flag) for the loads already issued
        for (int j = max(0, nk - kStages); j < nk; ++j)
          mbar_wait(&bars[Lay::bKFull + j % kStages], (j / kStages) & 1, nullptr, nullptr,
                    200000000ull);
        for (int j = max(0, nv - kStages); j < nv; ++j)
          mbar_wait(&bars[Lay::bVFull + j % kStages], (j / kStages) & 1, nullptr, nullptr,
                    200000000ull);
      }
    } else if (warp == 2) {
      // ===================== pieces of the share, one or two ahead
      for (int k = 0; ok && (k == 0 || unit_at(k - 1).valid); ++k) {
        if (k >= 2)
          ok = mbar_wait_warp(&bars[Lay::bUnitEmpty + (k & 1)], ((k >> 1) - 1) & 1, p.status,
                              abort_flag);
        if (!ok) break;
        make_unit(p, reached, share_end, unit_at(k));
        if (lane == 0) mbar_arrive(&bars[Lay::bUnitFull + (k & 1)]);
      }
    } else if (warp == 1 && elect_one()) {
      // ===================== MMA issuer
      constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, false, false);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, false, true);
      int npv[2] = {0, 0};      // PVs issued per slot
      int nq0 = 0, nq1 = 0;     // Q tiles taken
      bool fresh[2] = {};       // no PV of this piece yet: the next one overwrites O
      // S_s = Q K^T of Q tile sq and ring stage st into slot s's S columns
      auto issue_s = [&](int s, int st, int sq) -> bool {
        if (!Lay::kOwnP && npv[s] > 0 &&
            !mbar_wait_spin(&bars[Lay::bPvDone + s], (npv[s] - 1) & 1, p.status, abort_flag))
          return false;  // its last PV still reads the P held there
        tc_fence_after_sync();
        const uint64_t q_desc =
            sdesc_sw128(smem_u32(smem + Lay::kQ + sq * Lay::kTileBytes), 16, 1024);
        const uint64_t k_desc =
            sdesc_sw128(smem_u32(smem + Lay::kK + st * Lay::kTileBytes), 16, 1024);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (k >> 2) * Lay::kBoxBytes + (k & 3) * 32;
          umma_bf16_ss(tmem + s * 128, sdesc_step(q_desc, off), sdesc_step(k_desc, off), idesc_s,
                       k > 0 ? 1u : 0u);
        }
        umma_commit(&bars[Lay::bSFull + s]);
        return true;
      };
      auto p_ready = [&](int s) -> bool {
        return mbar_wait_spin(&bars[Lay::bPFull + s], npv[s] & 1, p.status, abort_flag);
      };
      // O_s += P_s V of ring stage st, P_s as bf16 pairs
      auto issue_pv = [&](int s, int st) -> bool {
        if (!Lay::kOwnP && !p_ready(s)) return false;
        tc_fence_after_sync();
        const uint64_t vb = sdesc_sw128(smem_u32(smem + Lay::kV + st * Lay::kTileBytes),
                                        Lay::kBoxBytes, 1024);  // V, MN-major B
        const uint32_t acc0 = fresh[s] ? 0u : 1u;
        fresh[s] = false;
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          umma_bf16_ts(tmem + Lay::kColO + s * D, tmem + Lay::kColP + s * Lay::kStepP + k * 8,
                       sdesc_step(vb, k * 2048),
                       idesc_pv, k > 0 ? 1u : acc0);
        umma_commit(&bars[Lay::bPvDone + s]);
        ++npv[s];
        return true;
      };
      int j = 0;  // key tiles so far
      for (int k = 0; ok; ++k) {
        ok = mbar_wait(&bars[Lay::bUnitFull + (k & 1)], (k >> 1) & 1, p.status, abort_flag);
        if (!ok) break;
        const Unit& u = unit_at(k);
        if (!u.valid) break;
        const int m0 = u.m0, m1 = u.m1, np = u.np, own0 = u.own[0], own1 = u.own[1];
        const int both = 2 * min(own0, own1);
        const bool alternate = u.alternate;
        const bool q0_full = u.q_used(0), q1_full = u.q_used(1);
        mbar_arrive(&bars[Lay::bUnitEmpty + (k & 1)]);
        if (m0 >= m1) continue;
        const int q1 = alternate ? 0 : 1;  // Q tile of slot 1
        if (q0_full) ok = mbar_wait(&bars[Lay::bQFull], nq0++ & 1, p.status, abort_flag);
        if (ok && q1_full) ok = mbar_wait(&bars[Lay::bQFull + 1], nq1++ & 1, p.status, abort_flag);
        if (!ok) break;
        fresh[0] = fresh[1] = true;
        bool prev0 = false, prev1 = false;
        int st = 0, pst = 0;
        auto v_ready = [&] {  // of the tile before
          return mbar_wait(&bars[Lay::bVFull + pst], ((j - 1) / kStages) & 1, p.status, abort_flag);
        };
        // Step m issues S of tile m and PV of tile m - 1; the last one PV only.
        for (int m = m0; m <= m1; ++m) {
          const bool more = m < m1;
          pst = st;
          st = j % kStages;
          // as in Unit::at
          const bool in0 = more && (alternate ? !(m & 1)
                                    : m < np  ? true
                                    : m - np < both ? !((m - np) & 1)
                                                    : own0 > own1);
          const bool in1 = more && ((!alternate && m < np) || !in0);
          // A tile that goes to the other slot than the one before (or none):
          // S_0, S_1, PV_0, PV_1, so that this S runs under the softmax of the
          // tile before.  Else PV_0, S_0, PV_1, S_1: each slot's softmax runs
          // under the other's MMAs.
          const bool apart = !((in0 && prev0) || (in1 && prev1));
          // (one copy of each group's code: the kernel's size costs time)
          const bool pv = m > m0;
#pragma unroll 1
          for (int pass = 0; ok && pass < 2; ++pass) {
            const bool with_pv = pv && (pass == 1) == apart;
            const bool with_s = more && pass == 0;
            if constexpr (Lay::kOwnP) {
              // S may follow as soon as the S before it is read: before the PV
              if (with_s)
                ok = mbar_wait(&bars[Lay::bKFull + st], (j / kStages) & 1, p.status, abort_flag);
              if (ok && with_pv) ok = v_ready();
              if (ok && with_pv && prev0) ok = p_ready(0);
              if (ok && with_s && in0) ok = issue_s(0, st, 0);
              if (ok && with_pv && prev0) ok = issue_pv(0, pst);
              if (ok && with_pv && prev1) ok = p_ready(1);
              if (ok && with_s && in1) ok = issue_s(1, st, q1);
              if (ok && with_pv && prev1) ok = issue_pv(1, pst);
              if (ok && with_pv) umma_commit(&bars[Lay::bVEmpty + pst]);
              if (ok && with_s) umma_commit(&bars[Lay::bKEmpty + st]);
            } else {
              if (with_pv) {
                ok = v_ready();
                if (ok && prev0) ok = issue_pv(0, pst);
              }
              if (ok && with_s) {
                ok = mbar_wait(&bars[Lay::bKFull + st], (j / kStages) & 1, p.status, abort_flag);
                if (ok && in0) ok = issue_s(0, st, 0);
              }
              if (ok && with_pv) {
                if (prev1) ok = issue_pv(1, pst);
                if (ok) umma_commit(&bars[Lay::bVEmpty + pst]);
              }
              if (ok && with_s) {
                if (in1) ok = issue_s(1, st, q1);
                if (ok) umma_commit(&bars[Lay::bKEmpty + st]);
              }
            }
            if (!apart) break;
          }
          if (!ok) break;
          prev0 = in0;
          prev1 = in1;
          if (more) ++j;
        }
      }
      // drain every MMA this thread issued before the CTA may free TMEM
      umma_commit(&bars[Lay::bDrain]);
      mbar_wait(&bars[Lay::bDrain], 0, nullptr, nullptr, 500000000ull);
    }
  } else {
    setmaxnreg_inc<kRegsSoftmax>();
    // ===================== softmax warpgroup of slot s
    const int s = (warp - 4) >> 2;
    const int row = threadIdx.x - 128 * (1 + s);
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t colS = s * 128;
    const uint32_t colP = Lay::kColP + s * Lay::kStepP;
    const uint32_t colO = Lay::kColO + s * D;
    const float sl2 = p.scale_log2;
    int n_mine = 0, n_other = 0;  // key tiles of this and the other slot so far
    int j0 = 0;                   // key tiles of the pieces before
    int n_joined = 0;             // pieces that both slots worked on
    for (int k = 0; ok; ++k) {
      ok = mbar_wait_warp(&bars[Lay::bUnitFull + (k & 1)], (k >> 1) & 1, p.status, abort_flag);
      if (!ok) break;
      const Unit& u = unit_at(k);  // the next one goes to the other record
      if (!u.valid) break;
      const int rows = u.rows[s];
      const bool has_rows = (warp & 3) * 32 < rows;  // warp-uniform
      const bool row_valid = row < rows;
      // own keys this row reads: positions [0, own_hi) of its sequence, the
      // my_seq-th of the tile
      const int sl = u.alternate ? 0 : s;  // both slots go by slot 0's tables
      int my_seq, own_hi;
      {
        const Row at = row_at(p, u.group, u.row0[s] + (row_valid ? row : 0));
        my_seq = at.b - u.seq0[sl];
        own_hi = u.keys[sl][my_seq];
        if (p.causal) own_hi = min(own_hi, own_hi - p.queries + at.i + 1);
        if (u.q_used(s)) {
          if (k > 0) {  // the first one is there
            copy_q<D>(p, q_place<D>(p, at), smem + Lay::kQ + s * Lay::kTileBytes,
                      (warp & 3) * 32);
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[Lay::bQFull + s]);
        }
      }
      const int n_pre = u.n_pre[s], n_tiles = n_pre + u.n_own[s];
      const int step = u.alternate ? 2 : 1;
      int y = n_pre > 0 ? u.t_pre[s] : u.t_own[s];
      float m_ref = -INFINITY;
      float l = 0.f;
      for (int t = 0; t < n_tiles; ++t, y = t == n_pre ? u.t_own[s] : y + step) {
        const bool prefix = t < n_pre;
        // this row reads columns [0, hi) of the tile; v_rows of its keys exist
        int tile = y, v_rows = kTile;
        int left = p.prefix_len;
        if (!prefix) {
          const int q = u.sequence(sl, y);
          tile -= u.upto[sl][q];
          v_rows = u.keys[sl][q] - tile * kTile;
          left = q == my_seq && row_valid ? own_hi : 0;
        }
        const int hi = min(left - tile * kTile, kTile);
        // The last PV read the P columns and wrote O (P over S: this S was
        // issued after it).
        const auto pv_done = [&]() -> bool {
          if (!Lay::kOwnP || n_mine + t == 0) return true;
          const bool done =
              mbar_wait_warp(&bars[Lay::bPvDone + s], (n_mine + t - 1) & 1, p.status, abort_flag);
          tc_fence_after_sync();
          return done;
        };
        if (!mbar_wait_warp(&bars[Lay::bSFull + s], (n_mine + t) & 1, p.status, abort_flag)) {
          ok = false;
          break;
        }
        if (!has_rows) {  // nothing to do, but the MMA counts four warps
          if (lane == 0) mbar_arrive(&bars[Lay::bPFull + s]);
          continue;
        }
        tc_fence_after_sync();
        const auto clear_v = [&]() -> bool {
          // the rest of the V tile may hold NaN, and P = 0 would not keep it out
          const int j = j0 + u.place(s, y) - u.m0, st = j % kStages;
          if (!mbar_wait_warp(&bars[Lay::bVFull + st], (j / kStages) & 1, p.status, abort_flag))
            return false;
          const int warps = (rows + 31) / 32;
          uint8_t* v = smem + Lay::kV + st * Lay::kTileBytes;
          const uint4 zero = make_uint4(0, 0, 0, 0);
          // 16-byte chunks [v_rows x 8, 128 x 8) of each 64-feature box
#pragma unroll 1
          for (int c = 0; c < D / 64; ++c)
#pragma unroll 1
            for (int k = v_rows * 8 + (warp & 3) * 32 + lane; k < kTile * 8; k += warps * 32)
              *reinterpret_cast<uint4*>(v + c * Lay::kBoxBytes + k * 16) = zero;
          fence_proxy_async_smem();
          return true;
        };
        if (__all_sync(0xffffffffu, hi <= 0)) {  // another sequence's keys: P = 0
          if (!pv_done()) {
            ok = false;
            break;
          }
          float zero[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) zero[c] = 0.f;
          tmem_st32(tmem + lane_base + colP, zero);
          tmem_st32(tmem + lane_base + colP + 32, zero);
          if (v_rows < kTile && !clear_v()) {
            ok = false;
            break;
          }
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[Lay::bPFull + s]);
          continue;
        }
        float sv[kTile];
#pragma unroll
        for (int c = 0; c < kTile / 32; c += 2)
          tmem_ld32x2(tmem + lane_base + colS + c * 32, tmem + lane_base + colS + (c + 1) * 32,
                      sv + c * 32, sv + (c + 1) * 32);
        // bit q: no row of this warp reads 32-column chunk q (warp-uniform)
        uint32_t dead = 0;
        if (__any_sync(0xffffffffu, hi < kTile)) {
#pragma unroll
          for (int q = 0; q < kTile / 32; ++q) {
            const int c0 = q * 32;
            if (__all_sync(0xffffffffu, hi <= c0)) dead |= 1u << q;
            if (!__all_sync(0xffffffffu, hi >= c0 + 32)) {
#pragma unroll
              for (int c = c0; c < c0 + 32; ++c) sv[c] = c < hi ? sv[c] : -INFINITY;
            }
          }
        }
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // (one chain: 829 us, this 803)
#pragma unroll
        for (int q = 0; q < kTile / 32; ++q) {
          if (dead & (1u << q)) continue;
#pragma unroll
          for (int c = q * 32; c < q * 32 + 32; c += 2)
            mx4[c / 2 % 4] = fmax3(mx4[c / 2 % 4], sv[c], sv[c + 1]);
        }
        const float mx = fmax3(fmaxf(mx4[0], mx4[1]), mx4[2], mx4[3]);
        // scores stay unscaled: the scale is positive, so the row max of the
        // scaled scores is the scaled max, and each exponent below takes the
        // scale in one fused multiply-add
        const float m_new = fmaxf(m_ref, mx * sl2);
        const bool need = m_new > m_ref + kRescaleThreshold;  // false while both are -inf
        if (!pv_done()) {
          ok = false;
          break;
        }
        if (__any_sync(0xffffffffu, need)) {
          // (a row without a key so far has O = 0)
          if (t > 0 && __any_sync(0xffffffffu, need && m_ref != -INFINITY)) {
            // O holds the PVs so far, scaled by the old reference
            const float alpha = need ? exp2f(m_ref - m_new) : 1.f;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              float o[32];
              tmem_ld32(tmem + lane_base + colO + c * 32, o);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] *= alpha;
              tmem_st32(tmem + lane_base + colO + c * 32, o);
            }
          }
          if (need) {
            l *= exp2f(m_ref - m_new);  // 0 when m_ref was -inf
            m_ref = m_new;
          }
        }
        const float mref_safe = (m_ref == -INFINITY) ? 0.f : m_ref;
        // exponent arguments and the row sum two lanes per instruction
        const uint64_t sl2x2 = f2_pack(sl2, sl2);
        const uint64_t negm = f2_pack(-mref_safe, -mref_safe);
        uint64_t rs2 = f2_pack(0.f, 0.f);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float packed[32];
          if (((dead >> (2 * half)) & 3u) == 3u) {
#pragma unroll
            for (int c = 0; c < 32; ++c) packed[c] = 0.f;
            tmem_st32(tmem + lane_base + colP + half * 32, packed);
            continue;
          }
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(sv[half * 64 + 2 * c], sv[half * 64 + 2 * c + 1]), sl2x2, negm),
                      x0, x1);
            const float e0 = ex2_approx(x0);
            const float e1 = ex2_approx(x1);
            rs2 = f2_add(rs2, f2_pack(e0, e1));
            packed[c] = __uint_as_float(pack_bf16x2(e0, e1));
          }
          tmem_st32(tmem + lane_base + colP + half * 32, packed);
        }
        float rs0, rs1;
        f2_unpack(rs2, rs0, rs1);
        l += rs0 + rs1;
        if (v_rows < kTile && !clear_v()) {
          ok = false;
          break;
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[Lay::bPFull + s]);
      }
      // ---- epilogue: wait for the last PV, join the slots, normalise, store
      const bool any_mine = n_tiles > 0;
      n_mine += n_tiles;
      n_other += u.n_pre[1 - s] + u.n_own[1 - s];
      j0 += u.m1 - u.m0;
      if (ok && any_mine)
        ok = mbar_wait_warp(&bars[Lay::bPvDone + s], (n_mine - 1) & 1, p.status, abort_flag);
      float w0 = 1.f, w1 = 0.f;  // weights of this slot's O and, joined, slot 1's
      const bool join = u.alternate && u.m0 < u.m1;
      const bool any_other = join && u.n_pre[1 - s] + u.n_own[1 - s] > 0;
      if (join && s == 1) {
        if (ok) {
          ml[row] = make_float2(m_ref, l);
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[Lay::bMerge]);
          // its O and `ml` are read by slot 0, which stores for both
          ok = mbar_wait_warp(&bars[Lay::bJoined], n_joined++ & 1, p.status, abort_flag);
        }
      } else if (join) {
        ok = ok && mbar_wait_warp(&bars[Lay::bMerge], n_joined++ & 1, p.status, abort_flag);
        if (ok && any_other)
          ok = mbar_wait_warp(&bars[Lay::bPvDone + 1], (n_other - 1) & 1, p.status, abort_flag);
        if (ok) {
          const float2 other = ml[row];
          const float top = fmaxf(m_ref, other.x);
          const float safe = (top == -INFINITY) ? 0.f : top;
          w0 = exp2f(m_ref - safe);
          w1 = exp2f(other.x - safe);
          l = l * w0 + other.y * w1;
          m_ref = top;
        }
      }
      if (ok && has_rows && !(u.alternate && s == 1)) {
        tc_fence_after_sync();
        // l is 0 without any key, NaN with a score that is
        const float inv_l = l == 0.f ? 0.f : 1.f / l;
        w0 = any_mine ? w0 * inv_l : 0.f;
        w1 *= inv_l;
        const float lse = l == 0.f ? -INFINITY : (m_ref + log2f(l)) * 0.69314718055994531f;
        // the row again: kept over the loop above it would cost registers there
        int own_row = u.row0[s] + (row_valid ? row : 0);
        asm volatile("" : "+r"(own_row));
        const Row at = row_at(p, u.group, own_row);
        const int r = row_valid ? static_cast<int>(at.token) * p.Hq + at.h : -1;
        const int64_t all = static_cast<int64_t>(p.batch) * p.queries * p.Hq;
        if (u.direct || __any_sync(0xffffffffu, l != 0.f)) {
          // The warp's rows, 2 D bytes of each at a time (D / 2 fp32 columns or
          // all D in bf16), through the Q tile, whose MMAs are complete: D / 8
          // lanes then store a row's bytes together.  Each warp stays in the
          // places of its own Q rows: others may be loading the next piece's.
          constexpr int kChunks = D / 8, kAtOnce = 32 / kChunks;
          uint8_t* stage = smem + Lay::kQ + s * Lay::kTileBytes;
          const int n_rows = min(32, rows - (warp & 3) * 32);
          const auto place = [&](int rr, int chunk) {
            return reinterpret_cast<uint4*>(stage + (chunk >> 3) * Lay::kBoxBytes +
                                            sw128_offset((warp & 3) * 32 + rr, chunk & 7));
          };
          const auto put = [&](int chunk, uint4 v) { *place(lane, chunk) = v; };
          const auto store_rows = [&](uint8_t* out, int pitch) {
            __syncwarp();
            const int chunk = lane & (kChunks - 1);
            out += chunk * 16;
            constexpr int kBatch = 4;
#pragma unroll 1
            for (int r0 = lane / kChunks; r0 - lane / kChunks < n_rows; r0 += kBatch * kAtOnce) {
              uint4 v[kBatch];
              int to[kBatch];
#pragma unroll
              for (int t = 0; t < kBatch; ++t) {
                to[t] = __shfl_sync(0xffffffffu, r, (r0 + t * kAtOnce) & 31);
                v[t] = *place((r0 + t * kAtOnce) & 31, chunk);
              }
#pragma unroll
              for (int t = 0; t < kBatch; ++t)
                if (r0 + t * kAtOnce < n_rows)
                  *reinterpret_cast<uint4*>(out + static_cast<int64_t>(to[t]) * pitch) = v[t];
            }
            __syncwarp();
          };
          float finite = 0.f;  // NaN once an element is not finite
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            const uint32_t col = half * (D / 2);
            float o[D / 2];
            const auto load_o = [&](uint32_t from, float* v) {
              if (D == 128)
                tmem_ld32x2(tmem + lane_base + from + col, tmem + lane_base + from + col + 32, v,
                            v + 32);
              else
                tmem_ld32(tmem + lane_base + from + col, v);
            };
            if (any_mine) {
              load_o(colO, o);
#pragma unroll
              for (int k = 0; k < D / 2; ++k) o[k] *= w0;
            } else {
#pragma unroll
              for (int k = 0; k < D / 2; ++k) o[k] = 0.f;
            }
            if (any_other) {
              float o1[D / 2];
              load_o(Lay::kColO + D, o1);
#pragma unroll
              for (int k = 0; k < D / 2; ++k) o[k] = fmaf(o1[k], w1, o[k]);
            }
            // without a key O is 0, not 0 times what masked keys left in it
#pragma unroll
            for (int k = 0; k < D / 2; ++k) o[k] = l == 0.f ? 0.f : o[k];
#pragma unroll
            for (int k = 0; k < D / 2; ++k) finite = fmaf(o[k], 0.f, finite);
            if (u.direct) {
#pragma unroll
              for (int k = 0; k < D / 16; ++k)
                put(half * (D / 16) + k, make_uint4(pack_bf16x2(o[8 * k], o[8 * k + 1]),
                                                    pack_bf16x2(o[8 * k + 2], o[8 * k + 3]),
                                                    pack_bf16x2(o[8 * k + 4], o[8 * k + 5]),
                                                    pack_bf16x2(o[8 * k + 6], o[8 * k + 7])));
              if (half == 0) continue;  // both halves fill the rows
            } else {
#pragma unroll
              for (int k = 0; k < D / 8; ++k)
                put(k, make_uint4(__float_as_uint(o[4 * k]), __float_as_uint(o[4 * k + 1]),
                                  __float_as_uint(o[4 * k + 2]), __float_as_uint(o[4 * k + 3])));
            }
            store_rows(u.direct ? reinterpret_cast<uint8_t*>(p.o)
                                : reinterpret_cast<uint8_t*>(p.part_o + u.part * all * D) +
                                      half * (D * 2),
                       u.direct ? D * 2 : D * 4);
          }
          // The MMA multiplies a row's P = 0 by masked keys too, those of other
          // sequences in its tile and later ones of its own, and 0 times an
          // infinity or NaN among their V is NaN (see sum_again).
          if (finite != finite && l == l && (u.seqs[sl] > 1 || p.causal) && u.m1 > max(u.m0, u.np))
            *redo = 1;
        }
        if (row_valid) {
          if (u.direct)
            p.lse[(static_cast<int64_t>(at.b) * p.Hq + at.h) * p.queries + at.i] = lse;
          else
            p.part_lse[u.part * all + r] = lse;
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if (join && s == 0 && ok) mbar_arrive(&bars[Lay::bJoined]);
        mbar_arrive(&bars[Lay::bUnitEmpty + (k & 1)]);
      }
    }
    // (the K ring is free: every MMA of both slots is complete)
    if (softmax_warps_and(ok) && *redo) {
      uint32_t cta;  // (kept apart from the start's: it would cost registers above)
      asm volatile("mov.u32 %0, %%ctaid.x;" : "=r"(cta));
      sum_again<D>(p, p.plan.share(cta), p.plan.share(cta + 1),
                   *reinterpret_cast<Unit*>(smem + Lay::kK));
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// Joins the pieces' partials: `blocks` CTAs for each cut job, and W warps work on
// a (query, head) row of it, each on every W-th piece.  Lanes hold the pieces' LSE in
// turn for the maximum and the weights, then d / 32 features each, with the loads of
// kBatch pieces in flight; the first of them are issued before the LSE is there.
// It is launched while the attention kernel still runs and waits for its end here,
// so its own start costs nothing.  It adds 9 us to 157 at 16 x 32 queries over
// 16,384 keys and 10 to 141 at 64 x 64 over 2,048 (12 and 32 with warps for the
// rows of all jobs, which had to find their pieces), 2 to 3 to the smallest calls.
template <int D, int W>
__global__ void __launch_bounds__(256)
    prefix_merge_kernel(const __grid_constant__ PrefixParams p, const __grid_constant__ CutJobs cut,
                        int blocks) {
  constexpr int kN = D / 32, kBatch = W == 1 ? 4 : 8;
  struct alignas(kN * 4) Part {
    float x[kN];
  };
  __shared__ Part joined[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Plan& pl = p.plan;
  const int n = static_cast<int>(blockIdx.x) / blocks;
  const uint32_t job = pl.runs > 1 ? n : cut.job[n];
  const int parts = pl.runs > 1 ? pl.runs : cut.parts[n];
  const uint32_t group = pl.by_pairs(job);
  const int i = (static_cast<int>(blockIdx.x) - n * blocks) * (8 / W) + warp / W;  // row of the job
  const int flat = static_cast<int>(job - group * pl.pairs) * (2 * kTile) + i;
  if (i >= 2 * kTile || flat >= p.batch * pl.seq_rows) return;
  const uint32_t token = pl.by_gs(flat);
  const uint32_t h = group * pl.gs + (flat - token * pl.gs);
  const int64_t rows = static_cast<int64_t>(p.batch) * p.queries * p.Hq;
  const int64_t r = static_cast<int64_t>(token) * p.Hq + h;
  const Part* part = reinterpret_cast<const Part*>(p.part_o + r * D) + lane;
  const int64_t step = rows * 32;  // from a piece to the next
  asm volatile("griddepcontrol.wait;" ::: "memory");
  Part v[kBatch];
  const int first = warp % W;
#pragma unroll
  for (int t = 0; t < kBatch; ++t)
    if (first + t * W < min(parts, 32)) v[t] = part[(first + t * W) * step];
  float top = -INFINITY;
#pragma unroll 1
  for (int k = lane; k < parts; k += 32) top = fmaxf(top, p.part_lse[k * rows + r]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float ref = top == -INFINITY ? 0.f : top;
  Part acc{};
  float sum = 0.f;
#pragma unroll 1
  for (int k0 = 0; k0 < parts; k0 += 32) {
    const float zk = k0 + lane < parts ? p.part_lse[(k0 + lane) * rows + r] : -INFINITY;
    const float w = expf(zk - ref);
    sum += w;
    const int n = min(32, parts - k0);
#pragma unroll 1
    for (int k1 = first; k1 < n; k1 += kBatch * W) {
      if (k0 + k1 > first) {
#pragma unroll
        for (int t = 0; t < kBatch; ++t)
          if (k1 + t * W < n) v[t] = part[(k0 + k1 + t * W) * step];
      }
#pragma unroll
      for (int t = 0; t < kBatch; ++t) {
        const int k = k1 + t * W;
        const float wk = __shfl_sync(0xffffffffu, w, k & 31);
        // a piece without a key of this row left no partial
        if (k >= n || wk == 0.f) continue;
#pragma unroll
        for (int c = 0; c < kN; ++c) acc.x[c] = fmaf(wk, v[t].x[c], acc.x[c]);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (W > 1) {
    joined[warp][lane] = acc;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / W), "n"(W * 32) : "memory");
    if (warp % W != 0) return;
#pragma unroll
    for (int k = 1; k < W; ++k)
#pragma unroll
      for (int c = 0; c < kN; ++c) acc.x[c] += joined[warp + k][lane].x[c];
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  struct alignas(kN * 2) Out {
    uint32_t x[kN / 2];
  } out;
#pragma unroll
  for (int c = 0; c < kN; c += 2) out.x[c / 2] = pack_bf16x2(acc.x[c] * inv, acc.x[c + 1] * inv);
  reinterpret_cast<Out*>(p.o + r * D)[lane] = out;
  if (lane == 0) {
    const uint32_t b = pl.by_queries(token);
    p.lse[(static_cast<int64_t>(b) * p.Hq + h) * p.queries + (token - b * p.queries)] =
        sum == 0.f ? -INFINITY : top + logf(sum);
  }
}

// How the problem is cut up on a GPU with `sms` SMs; false if it is too large
// for 32-bit places in the list.
bool make_plan(const csbp_prefix_problem& p, int sms, Plan& pl, CutJobs& cut) {
  const int G = p.Hq / p.Hkv;
  pl.gs = G;
  while (pl.gs > kTile || G % pl.gs != 0) --pl.gs;  // the largest divisor up to 128
  pl.n_groups = p.Hq / pl.gs;
  pl.seq_rows = p.queries * pl.gs;
  const int64_t rows = static_cast<int64_t>(p.batch) * pl.seq_rows;
  const int np = (p.prefix_len + kTile - 1) / kTile;
  pl.row_tiles = static_cast<int32_t>((rows + kTile - 1) / kTile);
  pl.pairs = (pl.row_tiles + 1) / 2;
  const int64_t jobs = static_cast<int64_t>(pl.pairs) * pl.n_groups;
  // (row tile, sequence) pairs of a head group that share rows: every tile and
  // every sequence starts one, together where both start
  int64_t both = kTile;
  while (pl.seq_rows % both != 0) both /= 2;  // rows between common starts: lcm
  both = static_cast<int64_t>(pl.seq_rows) * (kTile / both);
  const int64_t meets = pl.row_tiles + p.batch - (rows + both - 1) / both;
  // Lengths, in eighths of the time of a key tile read by one slot (1.1 to 1.4
  // us measured, D = 128): a prefix key tile of two slots takes 13 (1.8 us), the
  // start and the end of a piece 40.  Own keys count as 5/8 of the room for
  // them.
  constexpr int64_t kOne = 8, kTwo = 13, kEnds = 40, kJoin = 36;
  constexpr int64_t kMostTiles = 2048;  // that a row reads in a piece (see Runs above)
  const int64_t own_mean = (static_cast<int64_t>(p.own_max) * 5 / 8 + kTile - 1) / kTile;
  int64_t len_prefix = np * (pl.row_tiles == 1 ? kOne : kTwo) + kEnds;
  int64_t len = len_prefix + (meets * own_mean * kOne + pl.pairs - 1) / pl.pairs;
  int64_t total = jobs * len;
  // a share of at least two key tiles
  pl.ctas = static_cast<int32_t>(std::max<int64_t>(
      1, std::min<int64_t>(std::min(sms, CutJobs::kMost), (total - jobs * kEnds) / (2 * kOne))));
  // Whole jobs, one per CTA, where that ends as soon: a cut costs the joining
  // of its pieces (5 us, the second kernel).  More CTAs than SMs then start as
  // others end.
  const bool whole = (jobs + sms - 1) / sms * len <= total / pl.ctas + kEnds + kJoin;
  // Runs, where a row could read more than kMostTiles in one piece: of all numbers
  // up to about twice the least, the one with which the CTA with most runs ends
  // first.  (A row reads the prefix and its own sequence's keys.  Where those alone
  // can be too many, all sequences of a job may be as long as their room, which
  // puts `dense` times as many own tiles into a unit as the list assumes.)
  const int64_t own_most = (static_cast<int64_t>(p.own_max) + kTile - 1) / kTile;
  double dense = 1.0;
  if (own_most > kMostTiles) {
    const int64_t seqs = std::min<int64_t>(p.batch, (kTile + pl.seq_rows - 2) / pl.seq_rows + 1);
    dense = std::max(1.0, static_cast<double>(2 * seqs * own_most * kOne) /
                              static_cast<double>(len - len_prefix));
  }
  int64_t runs = 1;
  const int64_t longest = static_cast<int64_t>(kMostTiles * kTwo / dense);  // of a piece
  if (np + own_most > kMostTiles && (whole ? len : std::min(len, total / pl.ctas)) > longest) {
    const int64_t least = (len + longest - 1) / longest;
    int64_t best = INT64_MAX;
    for (int64_t r = least; r <= 2 * least + 16; ++r) {
      const int64_t time = (jobs * r + sms - 1) / sms * ((len + r - 1) / r + kEnds);
      if (time < best) {
        best = time;
        runs = r;
      }
    }
    len = (len + runs - 1) / runs;
    pl.ctas = static_cast<int32_t>(std::min<int64_t>(sms, jobs * runs));
    total = jobs * runs * len;
  }
  while (total >= int64_t(1) << 30 && len > 1) {  // coarser units: 32-bit places
    len_prefix = (len_prefix + 1) / 2;
    len = (len + 1) / 2;
    total = jobs * runs * len;
  }
  if (total >= int64_t(1) << 30) return false;
  pl.runs = static_cast<int32_t>(runs);
  pl.len = static_cast<uint32_t>(len);
  pl.full = static_cast<uint32_t>(len * runs);
  pl.total = static_cast<uint32_t>(total);
  pl.len_prefix = static_cast<uint32_t>(len_prefix);
  pl.inv_prefix = 1.f / static_cast<float>(len_prefix);
  pl.inv_own = pl.full > len_prefix ? 1.f / static_cast<float>(pl.full - len_prefix) : 0.f;
  pl.by_gs = Divisor::of(pl.gs);
  pl.by_queries = Divisor::of(p.queries);
  pl.by_seq_rows = Divisor::of(pl.seq_rows);
  pl.by_pairs = Divisor::of(pl.pairs);
  pl.by_len = Divisor::of(pl.len);
  pl.by_runs = Divisor::of(pl.runs);
  pl.by_per_kv = Divisor::of(G / pl.gs);  // row groups of a KV head
  pl.snap = 0;
  if (whole && runs == 1) {
    pl.ctas = static_cast<int32_t>(jobs);
    pl.step = static_cast<uint64_t>(len) << 32;
  } else {
    // rounded up, so that a share that is a whole number of jobs ends with one
    pl.step = ((static_cast<uint64_t>(total) << 32) + pl.ctas - 1) / pl.ctas;
    pl.snap = runs > 1 ? pl.len  // every cut moves to the end of a run
                       : static_cast<uint32_t>(std::min<int64_t>(kEnds, total / pl.ctas / 3));
  }
  pl.inv_step = static_cast<float>(4294967296.0 / static_cast<double>(pl.step));
  // the cuts inside jobs
  pl.parts = pl.runs;
  cut.n = 0;
  for (int c = 1; !whole && runs == 1 && c < pl.ctas; ++c) {
    const uint32_t x = pl.share(c), job = pl.by_len(x);
    if (x == job * pl.len) continue;
    if (cut.n == 0 || cut.job[cut.n - 1] != job) {
      cut.job[cut.n] = job;
      cut.parts[cut.n++] = 1;
    }
    pl.parts = std::max<int32_t>(pl.parts, ++cut.parts[cut.n - 1]);
  }
  return true;
}

bool device_sms(int& sms) {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess &&
         cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess &&
         sms > 0;
}

size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

size_t part_lse_offset(const csbp_prefix_problem& p, const Plan& pl) {
  const size_t rows = static_cast<size_t>(p.batch) * p.queries * p.Hq;
  return kStatusBytes + (pl.parts > 1 ? round256(pl.parts * rows * p.d * 4) : 0);
}

size_t workspace_bytes(const csbp_prefix_problem& p, const Plan& pl) {
  const size_t rows = static_cast<size_t>(p.batch) * p.queries * p.Hq;
  return part_lse_offset(p, pl) + (pl.parts > 1 ? round256(pl.parts * rows * 4) : 0);
}

template <int D>
cudaError_t launch(const CUtensorMap* maps, const PrefixParams& p, const CutJobs& cut, int sms,
                   cudaStream_t stream) {
  using Lay = PrefixLayout<D>;
  // the shared-memory limit is a per-device attribute: set it once on each
  // device, and read the kernel's register count there
  static PerDeviceOnce configured;
  static int launch_regs[PerDeviceOnce::kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!configured.run(dev, [&](int device) {
        e = cudaFuncSetAttribute(prefix_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Lay::kDynSmem);
        if (e != cudaSuccess) return false;
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, prefix_kernel<D>);
        if (e != cudaSuccess) return false;
        launch_regs[device] = fa.numRegs;
        return true;
      }))
    return e != cudaSuccess ? e : cudaErrorInvalidDevice;
  // setmaxnreg.inc would wait forever if the budgets exceeded the launch
  // allocation: refuse to launch instead
  if (launch_regs[dev] * kThreads < kRegsNeeded) return cudaErrorInvalidConfiguration;
  const int timed = timer_begin(13, stream);
  prefix_kernel<D><<<p.plan.ctas, kThreads, Lay::kDynSmem, stream>>>(maps[0], maps[1], maps[2], maps[3],
                                                              p);
  e = cudaGetLastError();
  timer_end(timed, stream);
  const int jobs = p.plan.runs > 1 ? p.plan.pairs * p.plan.n_groups : cut.n;
  if (e != cudaSuccess || jobs == 0) return e;
  const int per_job = std::min(2 * kTile, p.batch * p.plan.seq_rows);
  const int64_t rows = static_cast<int64_t>(jobs) * per_job;
  // few rows have many pieces (the keys were split to fill the GPU): more warps
  // to a row, up to about 32 warps per SM in all
  const int warps = rows <= 4 * sms ? 8 : rows <= 8192 ? 2 : 1;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  const int blocks = (per_job * warps + 7) / 8;
  cfg.gridDim = dim3(static_cast<unsigned>(jobs) * blocks);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  const int joined = timer_begin(14, stream);
  e = warps == 8   ? cudaLaunchKernelEx(&cfg, prefix_merge_kernel<D, 8>, p, cut, blocks)
      : warps == 2 ? cudaLaunchKernelEx(&cfg, prefix_merge_kernel<D, 2>, p, cut, blocks)
                   : cudaLaunchKernelEx(&cfg, prefix_merge_kernel<D, 1>, p, cut, blocks);
  timer_end(joined, stream);
  return e;
}

// Pointers and element strides of the five tensors (q, prefix K and V, own
// K and V).
struct Tensors {
  const void* t[5];
  int64_t tok[5], bat[5];
};

csbp_status validate(const csbp_prefix_problem* p) {
  if (!p) return CSBP_ERR_INVALID;
  if (p->batch < 1 || p->queries < 1 || p->prefix_len < 0 || p->own_max < 0 || p->Hq < 1 ||
      p->Hkv < 1 || p->Hq % p->Hkv != 0)
    return CSBP_ERR_INVALID;
  if (p->causal != 0 && p->causal != 1) return CSBP_ERR_INVALID;
  if (!(p->scale > 0.f) || p->scale > 3.0e38f) return CSBP_ERR_INVALID;
  if (p->d != 64 && p->d != 128) return CSBP_ERR_UNSUPPORTED;
  // every tensor stays below 2^39 elements, tested by division
  const int64_t rows = static_cast<int64_t>(p->batch) * p->queries;
  const int64_t lim = (kMaxElems - 1) / p->d;
  if (p->Hq > lim || rows > lim / p->Hq || p->prefix_len > lim / p->Hkv ||
      static_cast<int64_t>(p->batch) * p->own_max > lim / p->Hkv)
    return CSBP_ERR_UNSUPPORTED;
  // rows are counted in 32 bits
  if (rows * p->Hq > 0x3fffffff) return CSBP_ERR_UNSUPPORTED;
  // so are keys, up to the end of their last tile
  if (p->prefix_len > 0x7fffffff - kTile || p->own_max > 0x7fffffff - kTile)
    return CSBP_ERR_UNSUPPORTED;
  return CSBP_OK;
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

csbp_status check_inputs(const csbp_prefix_problem* p, const csbp_prefix_inputs* in,
                         Tensors& a) {
  if (!in || !in->q) return CSBP_ERR_INVALID;
  if (p->prefix_len > 0 && (!in->k_prefix || !in->v_prefix)) return CSBP_ERR_INVALID;
  if (p->own_max > 0 && (!in->k_own || !in->v_own || !in->own_len)) return CSBP_ERR_INVALID;
  if (!aligned(in->own_len, 4)) return CSBP_ERR_INVALID;
  const void* ptr[5] = {in->q, in->k_prefix, in->v_prefix, in->k_own, in->v_own};
  const int64_t len[5] = {p->queries, p->prefix_len, p->prefix_len, p->own_max, p->own_max};
  for (int i = 0; i < 5; ++i) {
    a.t[i] = ptr[i];
    a.tok[i] = a.bat[i] = 0;
    if (len[i] == 0) continue;
    if (!aligned(ptr[i], 16)) return CSBP_ERR_INVALID;
    if (in->stride_tok[i] < 0 || in->stride_batch[i] < 0) return CSBP_ERR_INVALID;
    const int64_t row = static_cast<int64_t>(i == 0 ? p->Hq : p->Hkv) * p->d;
    a.tok[i] = in->stride_tok[i] != 0 ? in->stride_tok[i] : row;
    if (a.tok[i] < row || a.tok[i] % 8 != 0 || a.tok[i] > (kMaxElems - 1) / len[i])
      return CSBP_ERR_INVALID;
    const bool prefix = i == 1 || i == 2;
    a.bat[i] = (!prefix && p->batch > 1 && in->stride_batch[i] != 0) ? in->stride_batch[i]
                                                                     : len[i] * a.tok[i];
    if (a.bat[i] < len[i] * a.tok[i] || a.bat[i] % 8 != 0 || a.bat[i] >= kMaxElems)
      return CSBP_ERR_INVALID;
  }
  return CSBP_OK;
}

// K or V [n][rows][Hkv][d] as {Hkv d, rows, n}, boxes of 64 features x 128 rows.
bool kv_map(CUtensorMap* m, const Tensors& t, int i, const csbp_prefix_problem& p, int64_t rows,
            int64_t n) {
  const uint64_t dims[3] = {static_cast<uint64_t>(p.Hkv) * p.d, static_cast<uint64_t>(rows),
                            static_cast<uint64_t>(n)};
  const uint64_t strides[2] = {static_cast<uint64_t>(t.tok[i]) * 2,
                               static_cast<uint64_t>(t.bat[i]) * 2};
  const uint32_t box[3] = {64, kTile, 1};
  return encode_map_3d(m, t.t[i], dims, strides, box);
}

}  // namespace
}  // namespace csbp

using namespace csbp;

extern "C" size_t csbp_prefix_workspace_bytes(const csbp_prefix_problem* problem) {
  if (validate(problem) != CSBP_OK) return 0;
  int sms = 0;
  if (!device_sms(sms)) sms = 152;  // no GPU: the GB300's count
  Plan pl{};
  CutJobs cut;
  return make_plan(*problem, sms, pl, cut) ? workspace_bytes(*problem, pl) : 0;
}

extern "C" csbp_status csbp_attn_prefix(const csbp_prefix_problem* problem,
                                        const csbp_prefix_inputs* in, void* o, float* lse,
                                        void* workspace, size_t ws_bytes, void* stream) {
  csbp_status st = validate(problem);
  if (st != CSBP_OK) return st;
  Tensors t{};
  if ((st = check_inputs(problem, in, t)) != CSBP_OK) return st;
  if (!o || !lse || !workspace || !aligned(o, 16) || !aligned(lse, 16) || !aligned(workspace, 16))
    return CSBP_ERR_INVALID;
  if (ws_bytes < kStatusBytes) return CSBP_ERR_WORKSPACE;
  const csbp_prefix_problem& p = *problem;
  // places in q are counted in 32 bits, in units of 16 bytes
  if (t.bat[0] > (int64_t(1) << 34) / p.batch) return CSBP_ERR_UNSUPPORTED;
  int sms = 0;
  if (!device_sms(sms)) return CSBP_ERR_CUDA;
  Plan pl{};
  CutJobs cut{};
  if (!make_plan(p, sms, pl, cut)) return CSBP_ERR_UNSUPPORTED;
  if (ws_bytes < workspace_bytes(p, pl)) return CSBP_ERR_WORKSPACE;
  CUtensorMap maps[4] = {};  // prefix K and V, own K and V
  if (p.prefix_len > 0 && (!kv_map(&maps[0], t, 1, p, p.prefix_len, 1) ||
                           !kv_map(&maps[1], t, 2, p, p.prefix_len, 1)))
    return CSBP_ERR_CUDA;
  if (p.own_max > 0 && (!kv_map(&maps[2], t, 3, p, p.own_max, p.batch) ||
                        !kv_map(&maps[3], t, 4, p, p.own_max, p.batch)))
    return CSBP_ERR_CUDA;
  // the maps of absent tensors are never used
  if (p.prefix_len == 0 && p.own_max > 0) maps[0] = maps[1] = maps[2];
  if (p.own_max == 0 && p.prefix_len > 0) maps[2] = maps[3] = maps[0];

  uint8_t* ws = static_cast<uint8_t*>(workspace);
  PrefixParams a{};
  a.plan = pl;
  a.batch = p.batch;
  a.queries = p.queries;
  a.prefix_len = p.prefix_len;
  a.own_max = p.own_max;
  a.Hq = p.Hq;
  a.causal = p.causal;
  a.scale_log2 = p.scale * 1.4426950408889634f;
  a.q = static_cast<const __nv_bfloat16*>(t.t[0]);
  a.q_tok = static_cast<uint32_t>(t.tok[0] / 8);
  a.q_bat = static_cast<uint32_t>(t.bat[0] / 8);
  const __nv_bfloat16** kv[4] = {&a.k_prefix, &a.v_prefix, &a.k_own, &a.v_own};
  for (int i = 0; i < 4; ++i) {
    *kv[i] = static_cast<const __nv_bfloat16*>(t.t[i + 1]);
    a.tok[i] = t.tok[i + 1];
    a.bat[i] = t.bat[i + 1];
  }
  a.own_len = in->own_len;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  a.part_o = reinterpret_cast<float*>(ws + kStatusBytes);
  a.part_lse = reinterpret_cast<float*>(ws + part_lse_offset(p, pl));
  a.status = reinterpret_cast<int*>(ws);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = p.d == 128 ? launch<128>(maps, a, cut, sms, s)
                                   : launch<64>(maps, a, cut, sms, s);
  return e == cudaSuccess ? CSBP_OK : CSBP_ERR_CUDA;
}
