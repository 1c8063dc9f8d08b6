// Appending to the quantised paged K/V cache with the position rotation on the
// way (csbp_generate.h): K is rotated and quantised, V quantised, Q rotated, in
// one launch.
//
// Angles.  A pair turns by pos x freq.  At far positions that product needs more
// bits than fp32 has (position 10^6, frequency 1: an ulp is 0.06), so it is taken
// in fixed point: `turns` holds freq / 2 pi modulo 1 in units of 2^-64 of a turn,
// and pos x turns modulo 2^64 is the angle modulo a whole turn, exact but for
// the 2^-65 of `turns` times pos.
//
// Scales.  A rotated value has an error of up to 2^-21 (|a| + |b|) in fp32, which
// is nothing to its code, but could decide a scale where the group's largest
// magnitude lies next to 448 x 2^e.  Such groups (one in 10^5) are worked out
// again in 64 bits, so that the scale is that of the rotation itself, and written
// once more where it is another; after the others, as a call among them cost the
// loop 50 registers.
//
// HBM bounds it: 3 + 1/32 bytes per value of K and V, 4 of Q.  A warp holds one
// token and goes through its heads, so that an angle's sine and cosine are worked
// out once for all heads that the warp takes; d / 16 lanes hold a head, each 8
// features and the 8 that they are rotated with.  131,042 tokens of 48 heads of
// 128: 380 us, 5.8 TB/s; 2,048 of 56 heads: 12.7 us; 8 tokens of 48 heads: 3.4.
// What counts for many tokens is how many loads are in flight: 24 warps per SM in CTAs of
// 4 (of 8 warps: 392 us), the next step's K or V loaded while one is encoded (406), sines
// and cosines in shared memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "csbp_generate.h"
#include "csbp_internal.h"
#include "kv_cache.cuh"
#include "ptx_sm100.cuh"

namespace csbp {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxD = 512;  // d / 16 lanes of one warp

struct AppendArgs {
  CacheArgs c;
  int32_t d, Hkv, Hq;
  int32_t turned;  // lanes of a head whose features are rotated: rotary dim / 16
  int32_t interleaved;
  const uint64_t* turns;
  const __nv_bfloat16* q;
  __nv_bfloat16* q_out;
  int64_t q_tok[2], q_bat[2];
  int32_t lanes;             // of a head: d / 16, up to the next power of two
  int32_t kv_steps, q_steps;  // steps of a warp for K (and for V), and for Q
  int32_t parts;              // warps that share a token's steps
  int32_t clear;              // rows of q_out that take no part become zeros
};

// 2 x 8 bf16 values of a lane as they lie in memory.
struct Raw {
  uint4 lo, hi;
};
__device__ __forceinline__ float value(const uint4& v, int e) {
  const uint32_t w = e < 2 ? v.x : e < 4 ? v.y : e < 6 ? v.z : v.w;
  return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
}

// Scale byte of a group whose largest magnitude is `top`: 448 = 1.75 x 2^8, so
// the exponent less 8, one more above 1.75.
__device__ __forceinline__ int scale_byte(float top) {
  return max(0, static_cast<int>((__float_as_uint(top) + 0x1fffffu) >> 23) - 8);
}
__device__ __forceinline__ int scale_byte(double top) {
  const int64_t bits = __double_as_longlong(top) + 0xfffffffffffffll / 4;
  return max(0, static_cast<int>(bits >> 52) - (1023 - 127) - 8);
}

// E4M3 of 8 values under the scale byte; NaN stays NaN.
__device__ __forceinline__ uint2 encode8(const float* y, int byte) {
  const float inv = __uint_as_float(static_cast<uint32_t>(254 - byte) << 23);  // 2^-e
  uint32_t two[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(c)
        : "f"(y[2 * k + 1] * inv), "f"(y[2 * k] * inv));
    two[k] = c;
  }
  return make_uint2(two[0] | two[1] << 16, two[2] | two[3] << 16);
}

// Pairs of a lane: (lo[e], hi[e]), or neighbours of lo and of hi; pair e turns
// by angle e either way.
template <class T>
__device__ __forceinline__ void rotate(T* lo, T* hi, const T* c, const T* s, bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      T* p = e < 4 ? lo + 2 * e : hi + 2 * (e - 4);
      const T a = p[0], b = p[1];
      p[0] = a * c[e] - b * s[e];
      p[1] = a * s[e] + b * c[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const T a = lo[e], b = hi[e];
      lo[e] = a * c[e] - b * s[e];
      hi[e] = a * s[e] + b * c[e];
    }
  }
}

__device__ __forceinline__ void lds_f4(uint32_t a, float* r) {
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3])
               : "r"(a)
               : "memory");
}

struct Encoded {
  int byte[2];
  uint2 code[2];
};

// The lane's 16 rotated K values in 64 bits, their groups' scale bytes and the
// codes.  The whole warp calls it; `top` is the warp's room for the largest
// magnitude of each chunk of 8 features.
__device__ __noinline__ Encoded encode_exact(const uint64_t* turns, int64_t pos, bool turned,
                                             bool interleaved, Raw raw, int c0, int c1,
                                             double* top) {
  double lo[8], hi[8];
  for (int e = 0; e < 8; ++e) {
    lo[e] = value(raw.lo, e);
    hi[e] = value(raw.hi, e);
  }
  if (turned) {
    double c[8], s[8];
    for (int e = 0; e < 8; ++e) {
      const int64_t turn = static_cast<int64_t>(static_cast<uint64_t>(pos) * turns[e]);
      sincospi(static_cast<double>(turn) * 0x1p-63, &s[e], &c[e]);
    }
    rotate(lo, hi, c, s, interleaved);
  }
  double m0 = 0.0, m1 = 0.0;
  float f0[8], f1[8];
  for (int e = 0; e < 8; ++e) {
    // infinities (past fp32's range too) to NaN, which the maxima pass over
    const float x = static_cast<float>(lo[e]), y = static_cast<float>(hi[e]);
    f0[e] = fmaf(x, 0.f, x);
    f1[e] = fmaf(y, 0.f, y);
    if (f0[e] == f0[e]) m0 = fmax(m0, fabs(lo[e]));
    if (f1[e] == f1[e]) m1 = fmax(m1, fabs(hi[e]));
  }
  __syncwarp();
  top[c0] = m0;
  top[c1] = m1;
  __syncwarp();
  for (int e = 1; e < 4; ++e) {
    m0 = fmax(m0, top[c0 ^ e]);
    m1 = fmax(m1, top[c1 ^ e]);
  }
  __syncwarp();
  Encoded r;
  r.byte[0] = scale_byte(m0);
  r.byte[1] = scale_byte(m1);
  r.code[0] = encode8(f0, r.byte[0]);
  r.code[1] = encode8(f1, r.byte[1]);
  return r;
}

// A lane's two chunks of a head.
__device__ __forceinline__ Raw load(const __nv_bfloat16* row, int x0, int x1, bool has) {
  Raw r{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  if (has) {
    r.lo = reinterpret_cast<const uint4*>(row)[x0];
    r.hi = reinterpret_cast<const uint4*>(row)[x1];
  }
  return r;
}

// Codes of one of a lane's chunks, and the scale byte by the first lane of its group.
__device__ __forceinline__ void store(uint8_t* codes, uint8_t* scales, int chunk, int byte,
                                      uint2 code) {
  reinterpret_cast<uint2*>(codes)[chunk] = code;
  if ((chunk & 3) == 0) scales[chunk >> 2] = static_cast<uint8_t>(byte);
}
// Codes and scale bytes of a lane's two chunks.
__device__ __forceinline__ void store(const AppendArgs& a, bool v, int64_t slot, int head, int x0,
                                      int x1, const Encoded& x) {
  const int64_t row = slot * a.Hkv + head;
  uint8_t* codes = (v ? a.c.codes[1] : a.c.codes[0]) + row * a.d;
  uint8_t* scales = (v ? a.c.scales[1] : a.c.scales[0]) + row * (a.d / kGroup);
  store(codes, scales, x0, x.byte[0], x.code[0]);
  store(codes, scales, x1, x.byte[1], x.code[1]);
}

__global__ void __launch_bounds__(kThreads, 6) cache_append_kernel(const __grid_constant__ AppendArgs a) {
  // per chunk of 8 features of the heads in a step: magnitude and pair size (or a
  // 64-bit magnitude)
  __shared__ __align__(16) float2 room[kWarps][64];
  __shared__ float4 angle[4][kThreads];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int64_t token = item / a.parts;
  const int part = static_cast<int>(item - token * a.parts);
  Row r;
  const int64_t b = token / a.c.rows;
  r.b = static_cast<int>(b);
  r.i = static_cast<int>(token - b * a.c.rows);
  // the same for the whole warp
  if (b >= a.c.batch) return;
  r.takes_part = !a.c.count || r.i < __ldg(a.c.count + r.b);
  const int at_once = 32 / a.lanes;
  const int l = lane & (a.lanes - 1), head0 = lane / a.lanes;
  const bool here = l < a.d / 16, turned = l < a.turned;
  // chunks of 8 features that the lane holds: a chunk and the one that it is rotated
  // with, or neighbours
  const bool split = turned && !a.interleaved;
  const int c0 = split ? l : 2 * l, c1 = split ? l + a.turned : 2 * l + 1;
  __nv_bfloat16* const out = a.q_out + r.b * a.q_bat[1] + r.i * a.q_tok[1];
  if (!r.takes_part) {
    if (a.clear)
      for (int step = part; step < a.q_steps; step += a.parts) {
        const int head = step * at_once + head0;
        if (!here || head >= a.Hq) continue;
        uint4* dst = reinterpret_cast<uint4*>(out + static_cast<int64_t>(head) * a.d);
        dst[c0] = dst[c1] = make_uint4(0, 0, 0, 0);
      }
    return;
  }
  const int64_t slot = slot_of(a.c, r);
  const int64_t pos = static_cast<int64_t>(__ldg(a.c.start + r.b)) + r.i;

  const uint64_t* turns = a.turns + 8 * l;
  if (turned) {
    float cosine[8], sine[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint64_t turn = static_cast<uint64_t>(pos) * __ldg(turns + e);
      sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &sine[e],
                &cosine[e]);
    }
    angle[0][threadIdx.x] = make_float4(cosine[0], cosine[1], cosine[2], cosine[3]);
    angle[1][threadIdx.x] = make_float4(cosine[4], cosine[5], cosine[6], cosine[7]);
    angle[2][threadIdx.x] = make_float4(sine[0], sine[1], sine[2], sine[3]);
    angle[3][threadIdx.x] = make_float4(sine[4], sine[5], sine[6], sine[7]);
  }
  // (from shared memory each time: the registers hold a step's loads instead)
  const uint32_t angles = smem_u32(&angle[0][threadIdx.x]);
  const auto turn_pairs = [&](float* lo, float* hi) {
    float c[8], s[8];
    lds_f4(angles, c);
    lds_f4(angles + kThreads * 16, c + 4);
    lds_f4(angles + 2 * kThreads * 16, s);
    lds_f4(angles + 3 * kThreads * 16, s + 4);
    rotate(lo, hi, c, s, a.interleaved != 0);
  };

  // ------- Q, two heads of a lane at a time
  const __nv_bfloat16* q = a.q + r.b * a.q_bat[0] + r.i * a.q_tok[0];
#pragma unroll 1
  for (int step = part; step < a.q_steps; step += 2 * a.parts) {
    Raw raw[2];
    bool has[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int head = (step + k * a.parts) * at_once + head0;
      has[k] = here && head < a.Hq;
      raw[k] = load(q + static_cast<int64_t>(head) * a.d, c0, c1, has[k]);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (!has[k]) continue;
      float lo[8], hi[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        lo[e] = value(raw[k].lo, e);
        hi[e] = value(raw[k].hi, e);
      }
      if (turned) turn_pairs(lo, hi);
      uint32_t w[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(lo[2 * e], lo[2 * e + 1]);
        const __nv_bfloat162 y = __floats2bfloat162_rn(hi[2 * e], hi[2 * e + 1]);
        w[e] = *reinterpret_cast<const uint32_t*>(&x);
        w[4 + e] = *reinterpret_cast<const uint32_t*>(&y);
      }
      uint4* dst = reinterpret_cast<uint4*>(
          out + static_cast<int64_t>((step + k * a.parts) * at_once + head0) * a.d);
      dst[c0] = make_uint4(w[0], w[1], w[2], w[3]);
      dst[c1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
  if (slot < 0) return;  // the same for the whole warp

  // ------- K and V
  // steps that have a scale to be worked out in 64 bits, one bit for every 32nd
  uint32_t again = 0;
  float2* mine = room[warp] + head0 * 2 * a.lanes;
  const auto fetch = [&](int step) {
    const bool v = step >= a.kv_steps;
    const int head = (v ? step - a.kv_steps : step) * at_once + head0;
    const __nv_bfloat16* src = (v ? a.c.src[1] + r.b * a.c.bat[1] + r.i * a.c.tok[1]
                                  : a.c.src[0] + r.b * a.c.bat[0] + r.i * a.c.tok[0]) +
                               static_cast<int64_t>(head) * a.d;
    return load(src, v ? 2 * l : c0, v ? 2 * l + 1 : c1,
                here && head < a.Hkv && step < 2 * a.kv_steps);
  };
  Raw next = fetch(part);
#pragma unroll 1
  for (int step = part; step < 2 * a.kv_steps; step += a.parts) {
    const bool v = step >= a.kv_steps, turn = !v && turned;
    const int head = (v ? step - a.kv_steps : step) * at_once + head0;
    const bool has = here && head < a.Hkv;
    const int x0 = v ? 2 * l : c0, x1 = v ? 2 * l + 1 : c1;
    const Raw raw = next;
    next = fetch(step + a.parts);
    float lo[8], hi[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      lo[e] = value(raw.lo, e);
      hi[e] = value(raw.hi, e);
    }
    float n0 = 0.f, n1 = 0.f;  // largest |a| + |b| of the pairs in a chunk
    if (turn) {
      if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          n0 = fmaxf(n0, fabsf(lo[2 * e]) + fabsf(lo[2 * e + 1]));
          n1 = fmaxf(n1, fabsf(hi[2 * e]) + fabsf(hi[2 * e + 1]));
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) n0 = fmaxf(n0, fabsf(lo[e]) + fabsf(hi[e]));
        n1 = n0;
      }
      turn_pairs(lo, hi);
    }
    float m0 = 0.f, m1 = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      lo[e] = fmaf(lo[e], 0.f, lo[e]);  // infinities to NaN, which the maxima pass over
      hi[e] = fmaf(hi[e], 0.f, hi[e]);
      m0 = fmaxf(m0, fabsf(lo[e]));
      m1 = fmaxf(m1, fabsf(hi[e]));
    }
    // largest of the four chunks of a group
    __syncwarp();
    mine[x0] = make_float2(m0, n0);
    mine[x1] = make_float2(m1, n1);
    __syncwarp();
#pragma unroll
    for (int e = 1; e < 4; ++e) {
      const float2 x = mine[x0 ^ e], y = mine[x1 ^ e];
      m0 = fmaxf(m0, x.x);
      n0 = fmaxf(n0, x.y);
      m1 = fmaxf(m1, y.x);
      n1 = fmaxf(n1, y.y);
    }
    Encoded x;
    x.byte[0] = scale_byte(m0);
    x.byte[1] = scale_byte(m1);
    n0 *= 0x1p-20f;  // twice the bound on the error of a rotated value; 0 for V
    n1 *= 0x1p-20f;
    const bool near = scale_byte(m0 + n0) != scale_byte(fmaxf(m0 - n0, 0.f)) ||
                      scale_byte(m1 + n1) != scale_byte(fmaxf(m1 - n1, 0.f));
    again |= static_cast<uint32_t>(near) << ((step / a.parts) & 31);
    x.code[0] = encode8(lo, x.byte[0]);
    x.code[1] = encode8(hi, x.byte[1]);
    if (!has) continue;
    store(a, v, slot, head, x0, x1, x);
  }

  // ------- scales next to a border, and their codes, once more
  again = __reduce_or_sync(0xffffffffu, again);
  if (again == 0) return;
  __syncwarp();
#pragma unroll 1
  for (int step = part; step < a.kv_steps; step += a.parts) {
    if (!(again >> ((step / a.parts) & 31) & 1)) continue;
    const int head = step * at_once + head0;
    const bool has = here && head < a.Hkv;
    const __nv_bfloat16* src =
        a.c.src[0] + r.b * a.c.bat[0] + r.i * a.c.tok[0] + static_cast<int64_t>(head) * a.d;
    const Encoded x = encode_exact(turns, pos, turned, a.interleaved != 0, load(src, c0, c1, has),
                                   c0, c1, reinterpret_cast<double*>(mine));
    // groups whose scale is another; the step's other groups keep the codes of their fp32
    // values, whatever the heads are that share the step with them
    const int64_t at = slot * a.Hkv + head;
    uint8_t* scales = a.c.scales[0] + at * (a.d / kGroup);
    const volatile uint8_t* is = scales;
    const bool other0 = has && is[c0 >> 2] != x.byte[0], other1 = has && is[c1 >> 2] != x.byte[1];
    __syncwarp();
    if (other0) store(a.c.codes[0] + at * a.d, scales, c0, x.byte[0], x.code[0]);
    if (other1) store(a.c.codes[0] + at * a.d, scales, c1, x.byte[1], x.code[1]);
  }
}

}  // namespace
}  // namespace csbp

using namespace csbp;

// freq / 2 pi modulo 1 in units of 2^-64, from 1 / 2 pi as a sum of two doubles:
// the first product and its error are exact, what is left out is below 2^-85 of
// a turn for frequencies up to 2^20.
extern "C" csbp_status csbp_rotary_turns(const double* freq, int32_t n, uint64_t* turns) {
  if (n < 0 || (n > 0 && (!freq || !turns))) return CSBP_ERR_INVALID;
  for (int i = 0; i < n; ++i)
    if (!(std::fabs(freq[i]) <= 0x1p20)) return CSBP_ERR_INVALID;
  constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;  // 1 / 2 pi
  for (int i = 0; i < n; ++i) {
    const double f = std::fabs(freq[i]);
    const volatile double product = f * kHi;  // (rounded, not fused with what follows)
    const double p = product, part = p - std::floor(p);  // exact
    const double rest = std::fma(f, kHi, -p) + f * kLo;
    const double units = std::ldexp(part, 64), whole = std::floor(units);
    const long long more = std::llrint((units - whole) + std::ldexp(rest, 64));
    const uint64_t turn = static_cast<uint64_t>(whole) + static_cast<uint64_t>(more);
    turns[i] = freq[i] < 0 ? 0 - turn : turn;
  }
  return CSBP_OK;
}

extern "C" csbp_status csbp_cache_append(const csbp_kv_cache* cache, const csbp_cache_rows* rows,
                                         const csbp_rotary* rotary, const void* k, const void* v,
                                         const csbp_append_queries* queries, void* stream) {
  AppendArgs a{};
  csbp_status st = make_args(cache, rows, k, v, a.c);
  if (st != CSBP_OK) return st;
  if (!rotary || rotary->dim < 16 || rotary->dim > cache->d || rotary->dim % 16 != 0 ||
      rotary->interleaved < 0 || rotary->interleaved > 1 || !rotary->turns ||
      !aligned(rotary->turns, 8))
    return CSBP_ERR_INVALID;
  if (queries && (queries->Hq < 0 || queries->clear < 0 || queries->clear > 1))
    return CSBP_ERR_INVALID;
  if (a.c.batch == 0) return CSBP_OK;
  if (cache->d > kMaxD) return CSBP_ERR_UNSUPPORTED;
  a.c.src[0] = static_cast<const __nv_bfloat16*>(k);
  a.c.src[1] = static_cast<const __nv_bfloat16*>(v);
  a.d = cache->d;
  a.Hkv = cache->Hkv;
  a.turned = rotary->dim / 16;
  a.interleaved = rotary->interleaved;
  a.turns = rotary->turns;
  if (queries && queries->Hq > 0) {
    if (!queries->q || !queries->out || !aligned(queries->q, 16) || !aligned(queries->out, 16))
      return CSBP_ERR_INVALID;
    if (queries->Hq > 65536) return CSBP_ERR_UNSUPPORTED;
    a.Hq = queries->Hq;
    a.clear = queries->clear;
    a.q = static_cast<const __nv_bfloat16*>(queries->q);
    a.q_out = static_cast<__nv_bfloat16*>(queries->out);
    const int64_t row = static_cast<int64_t>(a.Hq) * a.d;
    if (static_cast<int64_t>(rows->batch) * rows->rows > (kMaxElems - 1) / row)
      return CSBP_ERR_UNSUPPORTED;
    for (int i = 0; i < 2; ++i) {
      const int64_t tok = queries->stride_tok[i], bat = queries->stride_batch[i];
      if (tok < 0 || bat < 0) return CSBP_ERR_INVALID;
      a.q_tok[i] = tok != 0 ? tok : row;
      if (a.q_tok[i] < row || a.q_tok[i] % 8 != 0 || a.q_tok[i] > (kMaxElems - 1) / rows->rows)
        return CSBP_ERR_INVALID;
      const int64_t span = a.q_tok[i] * rows->rows;
      a.q_bat[i] = (rows->batch > 1 && bat != 0) ? bat : span;
      if (a.q_bat[i] < span || a.q_bat[i] % 8 != 0 || a.q_bat[i] >= kMaxElems)
        return CSBP_ERR_INVALID;
    }
  }
  a.lanes = 2;
  while (a.lanes * 16 < a.d) a.lanes *= 2;
  const int at_once = 32 / a.lanes;
  a.kv_steps = (a.Hkv + at_once - 1) / at_once;
  a.q_steps = (a.Hq + at_once - 1) / at_once;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return CSBP_ERR_CUDA;
  // few tokens are shared among warps, up to 32 per SM: then latency counts, and
  // the sines and cosines that each of them works out do not (2,048 tokens of 56
  // heads: 24 per SM 14.8 us, 32 12.7, 48 15.4)
  const int64_t tokens = static_cast<int64_t>(a.c.batch) * a.c.rows;
  a.parts = static_cast<int32_t>(
      std::max<int64_t>(1, std::min<int64_t>(2 * a.kv_steps + a.q_steps, 32 * sms / tokens)));
  const int64_t grid = (tokens * a.parts + kWarps - 1) / kWarps;
  if (grid > 0x7fffffff) return CSBP_ERR_UNSUPPORTED;
  const int timed = timer_begin(11, stream);
  cache_append_kernel<<<static_cast<unsigned>(grid), kThreads, 0,
                        static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  timer_end(timed, stream);
  return e == cudaSuccess ? CSBP_OK : CSBP_ERR_CUDA;
}
