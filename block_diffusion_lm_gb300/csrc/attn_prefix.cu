// Attention of a batch that shares a long prefix (csbp_generate.h), for
// sm_103a: softmax(scale q K^T) V over the prefix keys, which all sequences
// read, and each sequence's own keys.
//
// Rows.  The query rows of one KV head are (sequence, token, head of the
// group), flattened in that order; a row tile is 128 consecutive ones, so the
// prefix K/V pass through the tensor cores once per 128 rows however they
// divide into sequences, tokens and heads.  The softmax warps copy the tile's
// rows into shared memory themselves (a row per thread, zeros for the rest),
// which takes any token or batch stride and any group size.  Where row tiles
// kept inside sequences need (nearly) no more of them than tiles packed over
// sequences, a tile's keys are the prefix and then its sequence's own keys, in
// one softmax (`fused`); else the prefix runs on packed tiles and the own keys
// on separate units with tiles inside sequences.
//
// Units.  One CTA owns two row tiles ("slots") of one head group and a range
// of their key tiles; a key tile that both read is loaded once.  Each slot has
// its own softmax warpgroup, so that one slot's MMAs run under the other's
// softmax.  A CTA with one row tile left gives it to both slots, which take
// the key tiles in turn and are joined at the end (`alternate`).  Where the
// row tiles alone do not fill the GPU, the key tiles are split over CTAs too,
// each of which leaves a normalised fp32 partial and its LSE in the
// workspace, and a second kernel joins them exactly ([Blog] "在线 softmax 合并：
// 为什么分两段算仍是同一个注意力").
//
// Roles (384 threads), as in the training forward: warp 0 lane 0 TMA
// producer, warp 1 lane 0 MMA issuer, warps 4..7 and 8..11 softmax of slot 0
// and 1 (thread t = row t = TMEM lane t).  P overwrites the first 64 columns of
// its S as bf16 pairs and is the TMEM A operand of P V; O is rescaled only
// when a row's maximum grows by more than 2^8.  Warps without a row of their
// own take no part.  Own rows past a sequence's end may hold NaN: their scores
// are masked, and the softmax warps clear their V rows in shared memory before
// the MMA that would multiply them by P = 0.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "csbp_generate.h"
#include "csbp_internal.h"
#include "device_once.h"
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

// How the rows and keys of a problem are cut up (host and device).
struct Plan {
  int32_t gs, n_groups;   // query heads per row group, groups of them
  int32_t seq_rows;       // rows of one sequence: queries x gs
  int32_t tiles_seq;      // row tiles of one sequence
  int32_t fused;          // 1: tiles inside sequences read the prefix and the own keys
  int32_t row_tiles;      // of the shared units, per head group
  int32_t pairs;          // CTAs of the shared units per head group and key range
  int32_t splits;         // key ranges of the shared units
  int32_t own_pairs;      // CTAs per head group and range of the own units; 0: none
  int32_t own_splits;
  int32_t parts;          // splits + own splits; 1: written directly
};

struct PrefixParams {
  Plan plan;
  int32_t batch, queries, prefix_len, own_max, Hq, G, causal;
  float scale_log2;
  const __nv_bfloat16* q;
  int64_t q_tok, q_bat;  // element strides
  const int32_t* own_len;
  __nv_bfloat16* o;   // [batch][queries][Hq][d]
  float* lse;         // [batch][Hq][queries]
  float* part_o;      // [parts][batch x queries x Hq][d]
  float* part_lse;    // [parts][batch x queries x Hq]
  int* status;
};

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
  static constexpr int bDrain = bMerge + 1;
  static constexpr int kBars = bDrain + 1;
  static constexpr int kMisc = kBar + kBars * 8;    // tmem base, abort flag
  static constexpr int kMl = (kMisc + 8 + 15) / 16 * 16;  // slot 1's max and sum, 128 rows
  static constexpr int kDynSmem = kMl + kTile * 8;
  static constexpr uint32_t kColO = 256;            // O of slot s at kColO + D s
};

// One CTA's work, the same for all its threads.
struct Unit {
  int group, part;
  bool alternate;      // one row tile, both slots
  int64_t row0[2];     // first flattened row of a slot's tile
  int rows[2];         // its rows
  int seq[2];          // its sequence (fused and own units)
  int np;              // prefix key tiles
  int c[2], nc[2];     // own keys and key tiles of a slot's sequence
  int m0, m1;          // this CTA's range of the key-tile list

  // The m-th key tile of the list: prefix tiles first, then the two slots'
  // own tiles in turn.  Returns which slots read it.
  __device__ void at(int m, bool& prefix, int& tile, bool& in0, bool& in1) const {
    prefix = m < np;
    if (prefix) {
      tile = m;
      in0 = !alternate || !(m & 1);
      in1 = !alternate || (m & 1);
      return;
    }
    const int x = m - np;
    if (alternate) {
      tile = x;
      in0 = !(m & 1);
    } else {
      const int both = 2 * min(nc[0], nc[1]);
      in0 = x < both ? !(x & 1) : nc[0] > nc[1];
      tile = x < both ? x >> 1 : x - (both >> 1);
    }
    in1 = !in0;
  }
};

__device__ __forceinline__ Unit unit_of(const PrefixParams& p) {
  const Plan& pl = p.plan;
  Unit u;
  int64_t i = blockIdx.x;
  const int64_t shared = static_cast<int64_t>(pl.pairs) * pl.n_groups * pl.splits;
  const bool own = i >= shared;
  if (own) i -= shared;
  const int per = own ? pl.own_pairs : pl.pairs;
  const int pair = static_cast<int>(i % per);
  i /= per;
  u.group = static_cast<int>(i % pl.n_groups);
  const int split = static_cast<int>(i / pl.n_groups);
  u.part = own ? pl.splits + split : split;
  u.alternate = 2 * pair + 1 >= (own ? p.batch * pl.tiles_seq : pl.row_tiles);
  u.np = own ? 0 : (p.prefix_len + kTile - 1) / kTile;
  const bool inside = own || pl.fused;  // tiles inside sequences
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int tile = 2 * pair + (u.alternate ? 0 : s);
    int64_t end;
    if (inside) {
      u.seq[s] = tile / pl.tiles_seq;
      const int64_t first = static_cast<int64_t>(u.seq[s]) * pl.seq_rows;
      u.row0[s] = first + static_cast<int64_t>(tile - u.seq[s] * pl.tiles_seq) * kTile;
      end = first + pl.seq_rows;
    } else {
      u.seq[s] = 0;
      u.row0[s] = static_cast<int64_t>(tile) * kTile;
      end = static_cast<int64_t>(p.batch) * pl.seq_rows;
    }
    u.rows[s] = static_cast<int>(min(static_cast<int64_t>(kTile), end - u.row0[s]));
    u.c[s] = inside && p.own_max > 0 ? min(max(__ldg(p.own_len + u.seq[s]), 0), p.own_max) : 0;
    u.nc[s] = (u.c[s] + kTile - 1) / kTile;
  }
  const int64_t total = static_cast<int64_t>(u.np) + u.nc[0] + (u.alternate ? 0 : u.nc[1]);
  const int n = own ? pl.own_splits : pl.splits;
  u.m0 = static_cast<int>(total * split / n);
  u.m1 = static_cast<int>(total * (split + 1) / n);
  return u;
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
  float2* ml = reinterpret_cast<float2*>(smem + Lay::kMl);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const Unit u = unit_of(p);
  // the kernel that joins the parts may take its place on the GPU; it waits
  // for this one's end before it reads
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (threadIdx.x == 0) {
    for (int i = 0; i < Lay::kBars; ++i) mbar_init(&bars[i], 1);
    // arrivals of a slot's warps: all four load Q, those with rows make P
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars[Lay::bQFull + s], 4);
      mbar_init(&bars[Lay::bPFull + s], (u.rows[s] + 31) / 32);
    }
    mbar_init(&bars[Lay::bMerge], (u.rows[1] + 31) / 32);
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_base_sh, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_base_sh;
  const int kvh = u.group * p.plan.gs / p.G;

  if (warp < 4) {
    setmaxnreg_dec<kRegsLow>();
    if (warp == 0 && lane == 0 && u.m0 < u.m1) {
      // ===================== TMA producer
      int nk = 0, nv = 0;  // K / V tiles whose loads were issued
      bool ok = true;
      auto load = [&](int buf, int full, const CUtensorMap* map, int st, int tile, int z) {
        mbar_arrive_expect_tx(&bars[full + st], Lay::kTileBytes);
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          tma_load_3d(smem + buf + st * Lay::kTileBytes + c * Lay::kBoxBytes, map, &bars[full + st],
                      kvh * D + c * 64, tile * kTile, z);
      };
      for (int m = u.m0; m < u.m1; ++m) {
        const int j = m - u.m0, st = j % kStages, use = j / kStages;
        bool prefix, in0, in1;
        int tile;
        u.at(m, prefix, tile, in0, in1);
        const int z = prefix ? 0 : in0 ? u.seq[0] : u.seq[1];
        if (use > 0)
          ok = mbar_wait(&bars[Lay::bKEmpty + st], (use - 1) & 1, p.status, abort_flag);
        if (!ok) break;
        load(Lay::kK, Lay::bKFull, prefix ? &tm_kp : &tm_ko, st, tile, z);
        nk = j + 1;
        if (use > 0)
          ok = mbar_wait(&bars[Lay::bVEmpty + st], (use - 1) & 1, p.status, abort_flag);
        if (!ok) break;
        load(Lay::kV, Lay::bVFull, prefix ? &tm_vp : &tm_vo, st, tile, z);
        nv = j + 1;
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
    } else if (warp == 1 && lane == 0 && u.m0 < u.m1) {
      // ===================== MMA issuer
      constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, false, false);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, false, true);
      bool ok = true;
      for (int s = 0; s < (u.alternate ? 1 : 2) && ok; ++s)
        ok = mbar_wait(&bars[Lay::bQFull + s], 0, p.status, abort_flag);
      int npv[2] = {0, 0};  // PV issued per slot
      // S_s = Q_s K^T of ring stage st into slot s's S columns
      auto issue_s = [&](int s, int st) -> bool {
        if (npv[s] > 0 &&
            !mbar_wait_spin(&bars[Lay::bPvDone + s], (npv[s] - 1) & 1, p.status, abort_flag))
          return false;  // its last PV still reads the P held there
        tc_fence_after_sync();
        const int sq = u.alternate ? 0 : s;
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
      // O_s += P_s V of ring stage st, P_s (bf16 pairs) in slot s's S columns
      auto issue_pv = [&](int s, int st) -> bool {
        if (!mbar_wait_spin(&bars[Lay::bPFull + s], npv[s] & 1, p.status, abort_flag)) return false;
        tc_fence_after_sync();
        const uint64_t vb = sdesc_sw128(smem_u32(smem + Lay::kV + st * Lay::kTileBytes),
                                        Lay::kBoxBytes, 1024);  // V, MN-major B
        const uint32_t acc0 = npv[s] > 0 ? 1u : 0u;
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          umma_bf16_ts(tmem + Lay::kColO + s * D, tmem + s * 128 + k * 8, sdesc_step(vb, k * 2048),
                       idesc_pv, k > 0 ? 1u : acc0);
        umma_commit(&bars[Lay::bPvDone + s]);
        ++npv[s];
        return true;
      };
      bool prev0 = false, prev1 = false;
      int j = 0;
      for (int m = u.m0; m < u.m1 && ok; ++m, ++j) {
        const int st = j % kStages, pst = (j + kStages - 1) % kStages;
        bool prefix, in0, in1;
        int tile;
        u.at(m, prefix, tile, in0, in1);
        auto k_ready = [&] {
          return mbar_wait(&bars[Lay::bKFull + st], (j / kStages) & 1, p.status, abort_flag);
        };
        auto v_ready = [&] {  // of the tile before
          return mbar_wait(&bars[Lay::bVFull + pst], ((j - 1) / kStages) & 1, p.status, abort_flag);
        };
        if (!((in0 && prev0) || (in1 && prev1))) {
          // the tile before went to the other slot: this S runs under its softmax
          ok = k_ready();
          if (ok && in0) ok = issue_s(0, st);
          if (ok && in1) ok = issue_s(1, st);
          if (!ok) break;
          umma_commit(&bars[Lay::bKEmpty + st]);
          if (j > 0) {
            ok = v_ready();
            if (ok && prev0) ok = issue_pv(0, pst);
            if (ok && prev1) ok = issue_pv(1, pst);
            if (!ok) break;
            umma_commit(&bars[Lay::bVEmpty + pst]);
          }
        } else {
          // PV_0 of the tile before, S_0, PV_1, S_1: each slot's softmax runs
          // under the other's MMAs
          ok = v_ready();
          if (ok && prev0) ok = issue_pv(0, pst);
          if (ok) ok = k_ready();
          if (ok && in0) ok = issue_s(0, st);
          if (ok && prev1) ok = issue_pv(1, pst);
          if (!ok) break;
          umma_commit(&bars[Lay::bVEmpty + pst]);
          if (in1) ok = issue_s(1, st);
          if (!ok) break;
          umma_commit(&bars[Lay::bKEmpty + st]);
        }
        prev0 = in0;
        prev1 = in1;
      }
      if (ok && j > 0) {
        const int pst = (j - 1) % kStages;
        ok = mbar_wait(&bars[Lay::bVFull + pst], ((j - 1) / kStages) & 1, p.status, abort_flag);
        if (ok && prev0) ok = issue_pv(0, pst);
        if (ok && prev1) ok = issue_pv(1, pst);
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
    const uint32_t colO = Lay::kColO + s * D;
    const int rows = s ? u.rows[1] : u.rows[0];
    const int c_own = s ? u.c[1] : u.c[0];
    // this thread's row: (sequence b, token i, head h)
    const bool row_valid = row < rows;
    const int64_t flat = (s ? u.row0[1] : u.row0[0]) + (row_valid ? row : 0);
    const int64_t token = flat / p.plan.gs;
    const int b = static_cast<int>(token / p.queries);
    const int i = static_cast<int>(token - static_cast<int64_t>(b) * p.queries);
    const int h = u.group * p.plan.gs + static_cast<int>(flat - token * p.plan.gs);
    if (s == 0 || !u.alternate) {
      // Q row into the 128-byte-swizzled tile, zeros below the last row
      const uint4* src = reinterpret_cast<const uint4*>(p.q + b * p.q_bat + i * p.q_tok +
                                                        static_cast<int64_t>(h) * D);
      uint8_t* dst = smem + Lay::kQ + s * Lay::kTileBytes;
#pragma unroll
      for (int k = 0; k < D / 8; ++k) {
        const uint4 v = row_valid ? __ldg(src + k) : make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(dst + (k >> 3) * Lay::kBoxBytes + sw128_offset(row, k & 7)) = v;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[Lay::bQFull + s]);
    }
    if ((warp & 3) * 32 < rows) {  // a warp with rows
      const float sl2 = p.scale_log2;
      // own keys this row reads: positions [0, own_hi)
      const int own_hi = p.causal ? min(c_own, c_own - p.queries + i + 1) : c_own;
      float m_ref = -INFINITY;
      float l = 0.f;
      int n_tiles = 0;  // of this slot, so far
      bool ok = true;
      for (int m = u.m0; m < u.m1; ++m) {
        bool prefix, in0, in1;
        int tile;
        u.at(m, prefix, tile, in0, in1);
        if (!(s == 0 ? in0 : in1)) continue;
        if (!mbar_wait_warp(&bars[Lay::bSFull + s], n_tiles & 1, p.status, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        float sv[kTile];
#pragma unroll
        for (int c = 0; c < kTile / 32; c += 2)
          tmem_ld32x2(tmem + lane_base + colS + c * 32, tmem + lane_base + colS + (c + 1) * 32,
                      sv + c * 32, sv + (c + 1) * 32);
        // this row reads columns [0, hi) of the tile
        const int64_t left = static_cast<int64_t>(prefix ? p.prefix_len : own_hi) -
                             static_cast<int64_t>(tile) * kTile;
        const int hi = static_cast<int>(min(left, static_cast<int64_t>(kTile)));
        // bit q: no row of this warp reads 32-column chunk q (warp-uniform)
        uint32_t dead = 0;
        if (__any_sync(0xffffffffu, hi < kTile)) {
#pragma unroll
          for (int q = 0; q < kTile / 32; ++q) {
            const int c0 = q * 32;
            if (__all_sync(0xffffffffu, hi <= c0)) {
              dead |= 1u << q;
#pragma unroll
              for (int c = c0; c < c0 + 32; ++c) sv[c] = -INFINITY;
            } else if (!__all_sync(0xffffffffu, hi >= c0 + 32)) {
#pragma unroll
              for (int c = c0; c < c0 + 32; ++c) sv[c] = c < hi ? sv[c] : -INFINITY;
            }
          }
        }
        float mx = -INFINITY;
#pragma unroll
        for (int q = 0; q < kTile / 32; ++q) {
          if (dead & (1u << q)) continue;
#pragma unroll
          for (int c = q * 32; c < q * 32 + 32; c += 2) mx = fmax3(mx, sv[c], sv[c + 1]);
        }
        // scores stay unscaled: the scale is positive, so the row max of the
        // scaled scores is the scaled max, and each exponent below takes the
        // scale in one fused multiply-add
        const float m_new = fmaxf(m_ref, mx * sl2);
        const bool need = m_new > m_ref + kRescaleThreshold;  // false while both are -inf
        if (n_tiles > 0 && __any_sync(0xffffffffu, need)) {
          // O holds the PVs so far, scaled by the old reference; the last is
          // complete: the S this tile read was issued after it
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
            tmem_st32(tmem + lane_base + colS + half * 32, packed);
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
          tmem_st32(tmem + lane_base + colS + half * 32, packed);
        }
        float rs0, rs1;
        f2_unpack(rs2, rs0, rs1);
        l += rs0 + rs1;
        const int v_rows = c_own - tile * kTile;  // V rows of this own tile that exist
        if (!prefix && v_rows < kTile) {
          // the rest may hold NaN, and P = 0 would not keep it out: clear it
          const int j = m - u.m0, st = j % kStages;
          if (!mbar_wait_warp(&bars[Lay::bVFull + st], (j / kStages) & 1, p.status, abort_flag)) {
            ok = false;
            break;
          }
          const int warps = (rows + 31) / 32;
          uint8_t* v = smem + Lay::kV + st * Lay::kTileBytes;
          const uint4 zero = make_uint4(0, 0, 0, 0);
          // 16-byte chunks [v_rows x 8, 128 x 8) of each 64-feature box
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            for (int k = v_rows * 8 + (warp & 3) * 32 + lane; k < kTile * 8; k += warps * 32)
              *reinterpret_cast<uint4*>(v + c * Lay::kBoxBytes + k * 16) = zero;
          fence_proxy_async_smem();
        }
        ++n_tiles;
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[Lay::bPFull + s]);
      }
      // ---- epilogue: wait for the last PV, join the slots, normalise, store
      if (ok && n_tiles > 0)
        ok = mbar_wait_warp(&bars[Lay::bPvDone + s], (n_tiles - 1) & 1, p.status, abort_flag);
      float w0 = 1.f, w1 = 0.f;  // weights of this slot's O and, joined, slot 1's
      int n_other = 0;
      if (u.alternate) {
        if (s == 1) {
          if (ok) {
            ml[row] = make_float2(m_ref, l);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[Lay::bMerge]);
          }
          ok = false;  // slot 0 stores for both
        } else {
          // tiles m0 .. m1 - 1 went to the slots in turn
          n_other = (u.m1 - u.m0) - n_tiles;
          ok = ok && mbar_wait_warp(&bars[Lay::bMerge], 0, p.status, abort_flag);
          if (ok && n_other > 0)
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
      }
      if (ok) {
        tc_fence_after_sync();
        const float inv_l = (l > 0.f) ? 1.f / l : 0.f;
        w0 = n_tiles > 0 ? w0 * inv_l : 0.f;
        w1 *= inv_l;
        const float lse = (l > 0.f) ? (m_ref + log2f(l)) * 0.69314718055994531f : -INFINITY;
        const bool direct = p.plan.parts == 1;
        const int64_t r = token * p.Hq + h;
        const int64_t all = static_cast<int64_t>(p.batch) * p.queries * p.Hq;
        if (direct || __any_sync(0xffffffffu, l > 0.f)) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            float o[32];
            if (n_tiles > 0) {
              tmem_ld32(tmem + lane_base + colO + c * 32, o);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] *= w0;
            } else {
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = 0.f;
            }
            if (n_other > 0) {
              float o1[32];
              tmem_ld32(tmem + lane_base + Lay::kColO + D + c * 32, o1);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = fmaf(o1[k], w1, o[k]);
            }
            if (row_valid && direct) {
              __nv_bfloat16* dst = p.o + r * D + c * 32;
#pragma unroll
              for (int k = 0; k < 32; k += 8) {
                uint4 v;
                v.x = pack_bf16x2(o[k], o[k + 1]);
                v.y = pack_bf16x2(o[k + 2], o[k + 3]);
                v.z = pack_bf16x2(o[k + 4], o[k + 5]);
                v.w = pack_bf16x2(o[k + 6], o[k + 7]);
                *reinterpret_cast<uint4*>(dst + k) = v;
              }
            } else if (row_valid) {
              float* dst = p.part_o + (u.part * all + r) * D + c * 32;
#pragma unroll
              for (int k = 0; k < 32; k += 4)
                *reinterpret_cast<float4*>(dst + k) =
                    make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
            }
          }
        }
        if (row_valid) {
          if (direct)
            p.lse[(static_cast<int64_t>(b) * p.Hq + h) * p.queries + i] = lse;
          else
            p.part_lse[u.part * all + r] = lse;
        }
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// Joins the key ranges' partials: `W` warps per (query, head) row, each for
// every W-th part.  Lanes hold the parts' LSE in turn for the maximum and the
// weights, then d / 32 features each.  It is launched while the attention
// kernel still runs and waits for it here, so its own start costs nothing.
// Few rows have many parts (the GPU was filled by splitting the keys), so a row
// gets a CTA of its own and its parts are loaded side by side.
template <int D, int W>
__global__ void __launch_bounds__(256) prefix_merge_kernel(PrefixParams p) {
  constexpr int kN = D / 32;
  __shared__ float4 joined[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t rows = static_cast<int64_t>(p.batch) * p.queries * p.Hq;
  const int64_t r = blockIdx.x * static_cast<int64_t>(8 / W) + warp / W;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (W == 1 && r >= rows) return;
  const int parts = p.plan.parts;
  const float* z = p.part_lse + r;
  float top = -INFINITY;
  for (int k = lane; k < parts; k += 32) top = fmaxf(top, z[k * rows]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float ref = top == -INFINITY ? 0.f : top;
  float acc[kN] = {};
  float sum = 0.f;
  for (int k0 = 0; k0 < parts; k0 += 32) {
    const float zk = k0 + lane < parts ? z[(k0 + lane) * rows] : -INFINITY;
    const float w = expf(zk - ref);
    sum += w;
    const int n = min(32, parts - k0);
    for (int k1 = warp % W; k1 < n; k1 += 4 * W) {
      float v[4][kN];
      float wk[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int k = k1 + t * W;
        wk[t] = __shfl_sync(0xffffffffu, w, k & 31);
        if (k >= n) wk[t] = 0.f;
        // a range without a key of this row left no partial
        const float* src = p.part_o + ((k0 + k) * rows + r) * D + lane * kN;
#pragma unroll
        for (int c = 0; c < kN; c += 2) {
          const float2 x = wk[t] > 0.f ? *reinterpret_cast<const float2*>(src + c)
                                       : make_float2(0.f, 0.f);
          v[t][c] = x.x;
          v[t][c + 1] = x.y;
        }
      }
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int c = 0; c < kN; ++c) acc[c] = fmaf(wk[t], v[t][c], acc[c]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (W > 1) {
    float* mine = reinterpret_cast<float*>(&joined[warp][lane]);
#pragma unroll
    for (int c = 0; c < kN; ++c) mine[c] = acc[c];
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int k = 1; k < W; ++k)
#pragma unroll
      for (int c = 0; c < kN; ++c) acc[c] += reinterpret_cast<const float*>(&joined[k][lane])[c];
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  uint32_t out[kN / 2];
#pragma unroll
  for (int c = 0; c < kN; c += 2) out[c / 2] = pack_bf16x2(acc[c] * inv, acc[c + 1] * inv);
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + r * D) + lane * (kN / 2);
#pragma unroll
  for (int c = 0; c < kN / 2; ++c) dst[c] = out[c];
  if (lane == 0) {
    const int64_t bi = r / p.Hq;
    const int h = static_cast<int>(r - bi * p.Hq);
    const int64_t b = bi / p.queries;
    p.lse[(b * p.Hq + h) * p.queries + (bi - b * p.queries)] =
        sum > 0.f ? top + logf(sum) : -INFINITY;
  }
}

// How the problem is cut up on a GPU with `sms` SMs.
Plan make_plan(const csbp_prefix_problem& p, int sms) {
  Plan pl{};
  const int G = p.Hq / p.Hkv;
  pl.gs = G;
  while (pl.gs > kTile || G % pl.gs != 0) --pl.gs;  // the largest divisor up to 128
  pl.n_groups = p.Hq / pl.gs;
  pl.seq_rows = p.queries * pl.gs;
  pl.tiles_seq = static_cast<int32_t>((static_cast<int64_t>(pl.seq_rows) + kTile - 1) / kTile);
  const int64_t packed = (static_cast<int64_t>(p.batch) * pl.seq_rows + kTile - 1) / kTile;
  const int64_t inside = static_cast<int64_t>(p.batch) * pl.tiles_seq;
  const int np = (p.prefix_len + kTile - 1) / kTile;
  const int own_tiles = (p.own_max + kTile - 1) / kTile;
  pl.fused = p.prefix_len == 0 || (p.own_max > 0 && inside * 7 <= packed * 8) ? 1 : 0;
  pl.row_tiles = static_cast<int32_t>(pl.fused ? inside : packed);
  pl.pairs = (pl.row_tiles + 1) / 2;
  const bool own_units = !pl.fused && p.own_max > 0;
  pl.own_pairs = own_units ? static_cast<int32_t>((inside + 1) / 2) : 0;
  // Key ranges.  Costs in key-tile times of one CTA: a CTA costs its tiles
  // and about kOver more to start and store, and the partials of each range
  // are written and read once at the rate at which K/V stream in.
  constexpr double kOver = 3.0;
  const double rows = static_cast<double>(p.batch) * p.queries * p.Hq;
  const double join = rows * p.d * 8 / (static_cast<double>(sms) * kTile * p.d * 4);
  auto best = [&](int64_t ctas, int tiles, bool alone) {
    int pick = 1;
    double cost = 1e300;
    for (int n = 1; n <= std::min(std::max(tiles, 1), 2 * sms); ++n) {
      const double waves = std::ceil(static_cast<double>(ctas * n) / sms);
      const double c = waves * (std::ceil(static_cast<double>(tiles) / n) + kOver) +
                       (n > 1 || !alone ? join * n + kOver : 0.0);
      if (c < cost * 0.999) {
        cost = c;
        pick = n;
      }
    }
    return pick;
  };
  const int fused_tiles = np + (pl.fused ? own_tiles * 2 : 0);
  pl.splits = best(static_cast<int64_t>(pl.pairs) * pl.n_groups, fused_tiles, !own_units);
  pl.own_splits =
      own_units ? best(static_cast<int64_t>(pl.own_pairs) * pl.n_groups, 2 * own_tiles, false) : 0;
  pl.parts = pl.splits + pl.own_splits;
  return pl;
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
  return kStatusBytes + round256(pl.parts > 1 ? pl.parts * rows * p.d * 4 : 0);
}

size_t workspace_bytes(const csbp_prefix_problem& p, const Plan& pl) {
  const size_t rows = static_cast<size_t>(p.batch) * p.queries * p.Hq;
  return part_lse_offset(p, pl) + round256(pl.parts > 1 ? pl.parts * rows * 4 : 0);
}

template <int D>
cudaError_t launch(const CUtensorMap* maps, const PrefixParams& p, unsigned grid,
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
  prefix_kernel<D><<<grid, kThreads, Lay::kDynSmem, stream>>>(maps[0], maps[1], maps[2], maps[3],
                                                              p);
  e = cudaGetLastError();
  timer_end(timed, stream);
  if (e != cudaSuccess || p.plan.parts == 1) return e;
  const int64_t rows = static_cast<int64_t>(p.batch) * p.queries * p.Hq;
  const bool wide = rows <= 4096;  // a CTA per row
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(wide ? rows : (rows + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  const int joined = timer_begin(14, stream);
  e = wide ? cudaLaunchKernelEx(&cfg, prefix_merge_kernel<D, 8>, p)
           : cudaLaunchKernelEx(&cfg, prefix_merge_kernel<D, 1>, p);
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
  // row and tile counts of a head group fit 32 bits
  if (rows * (p->Hq / p->Hkv) > 0x3fffffff) return CSBP_ERR_UNSUPPORTED;
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
  return workspace_bytes(*problem, make_plan(*problem, sms));
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
  int sms = 0;
  if (!device_sms(sms)) return CSBP_ERR_CUDA;
  const Plan pl = make_plan(p, sms);
  if (ws_bytes < workspace_bytes(p, pl)) return CSBP_ERR_WORKSPACE;
  const int64_t grid = static_cast<int64_t>(pl.n_groups) *
                       (static_cast<int64_t>(pl.pairs) * pl.splits +
                        static_cast<int64_t>(pl.own_pairs) * pl.own_splits);
  const int64_t rows = static_cast<int64_t>(p.batch) * p.queries * p.Hq;
  if (grid > 0x7fffffff || rows / 8 >= 0x7fffffff) return CSBP_ERR_UNSUPPORTED;

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
  a.G = p.Hq / p.Hkv;
  a.causal = p.causal;
  a.scale_log2 = p.scale * 1.4426950408889634f;
  a.q = static_cast<const __nv_bfloat16*>(t.t[0]);
  a.q_tok = t.tok[0];
  a.q_bat = t.bat[0];
  a.own_len = in->own_len;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  a.part_o = reinterpret_cast<float*>(ws + kStatusBytes);
  a.part_lse = reinterpret_cast<float*>(ws + part_lse_offset(p, pl));
  a.status = reinterpret_cast<int*>(ws);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = p.d == 128 ? launch<128>(maps, a, static_cast<unsigned>(grid), s)
                                   : launch<64>(maps, a, static_cast<unsigned>(grid), s);
  return e == cudaSuccess ? CSBP_OK : CSBP_ERR_CUDA;
}
