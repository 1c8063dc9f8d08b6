// Attention of a few new tokens per sequence over the quantised paged K/V cache
// (csbp_generate.h), for sm_103a.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "csbp_generate.h"
#include "csbp_internal.h"
#include "kv_cache.cuh"

namespace csbp {
namespace {

constexpr size_t kStatusBytes = 256;
constexpr int kWarps = 4;

struct PagedParams {
  int64_t pages;
  int32_t page_size, Hkv, d;
  const uint8_t *k, *v, *k_scale, *v_scale;
  int32_t batch, queries, table_pages, Hq, causal, window, sinks;
  float scale_log2;
  const __nv_bfloat16* q;
  int64_t q_tok, q_bat;
  const int32_t *table, *length;
  __nv_bfloat16* o;
  float* lse;
};

__device__ __forceinline__ float scale_value(uint32_t byte) {
  return byte == 255 ? NAN : ldexpf(1.f, static_cast<int>(byte) - 127);
}

template <int N>
__device__ __forceinline__ void decode(const uint8_t* codes, float scale, float* x) {
#pragma unroll
  for (int e = 0; e < N; e += 2) {
    uint32_t h2;
    const uint16_t two = *reinterpret_cast<const uint16_t*>(codes + e);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(two));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
    x[e] = f.x * scale;
    x[e + 1] = f.y * scale;
  }
}

// One query row per CTA; its warps take the keys in turn and are joined.
template <int D>
__global__ void __launch_bounds__(kWarps * 32) paged_kernel(const PagedParams p) {
  constexpr int N = D / 32;
  __shared__ float sm[kWarps], sz[kWarps], so[kWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t row = blockIdx.x;
  const int h = static_cast<int>(row % p.Hq);
  row /= p.Hq;
  const int i = static_cast<int>(row % p.queries), b = static_cast<int>(row / p.queries);
  const int hk = h / (p.Hq / p.Hkv);
  const int c = min(max(__ldg(p.length + b), 0), p.table_pages * p.page_size);
  const int64_t t = static_cast<int64_t>(c) - p.queries + i;
  const int hi = static_cast<int>(p.causal ? max(t + 1, int64_t(0)) : c);
  const int lo = p.window ? static_cast<int>(max(t - p.window + 1, int64_t(0))) : 0;
  float q[N], acc[N] = {}, m = -INFINITY, z = 0.f;
  for (int e = 0; e < N; ++e)
    q[e] = __bfloat162float(p.q[b * p.q_bat + i * p.q_tok + int64_t(h) * D + lane * N + e]);
  for (int j = warp; j < hi; j += kWarps) {
    if (j < lo && j >= p.sinks) {
      j = lo - kWarps + ((warp - lo) % kWarps + kWarps) % kWarps;
      continue;
    }
    const int64_t page = __ldg(p.table + int64_t(b) * p.table_pages + j / p.page_size);
    if (page < 0 || page >= p.pages) continue;
    const int64_t at = (page * p.page_size + j % p.page_size) * p.Hkv + hk;
    float k[N], v[N], s = 0.f;
    decode<N>(p.k + at * D + lane * N, scale_value(p.k_scale[at * (D / 32) + lane * N / 32]), k);
    decode<N>(p.v + at * D + lane * N, scale_value(p.v_scale[at * (D / 32) + lane * N / 32]), v);
    for (int e = 0; e < N; ++e) s = fmaf(q[e], k[e], s);
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= p.scale_log2;
    const float top = s > m ? s : m;  // (NaN stays out of it)
    const float ref = top == -INFINITY ? 0.f : top;
    const float old = exp2f(m - ref), w = exp2f(s - ref);
    z = z * old + w;
    for (int e = 0; e < N; ++e) acc[e] = fmaf(w, v[e], acc[e] * old);
    m = top;
  }
  if (lane == 0) {
    sm[warp] = m;
    sz[warp] = z;
  }
  for (int e = 0; e < N; ++e) so[warp][lane * N + e] = acc[e];
  __syncthreads();
  if (warp) return;
  float top = -INFINITY;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w]);
  const float ref = top == -INFINITY ? 0.f : top;
  z = 0.f;
  for (int e = 0; e < N; ++e) acc[e] = 0.f;
  for (int w = 0; w < kWarps; ++w) {
    const float f = exp2f(sm[w] - ref);
    z += sz[w] * f;
    for (int e = 0; e < N; ++e) acc[e] += so[w][lane * N + e] * f;
  }
  const bool none = z == 0.f;
  for (int e = 0; e < N; ++e)
    p.o[(int64_t(b) * p.queries + i) * p.Hq * D + int64_t(h) * D + lane * N + e] =
        __float2bfloat16_rn(none ? 0.f : acc[e] / z);
  if (lane == 0)
    p.lse[(int64_t(b) * p.Hq + h) * p.queries + i] =
        none ? -INFINITY : (ref + log2f(z)) * 0.6931471805599453f;
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
  // keys and rows are counted in 32 bits
  if (static_cast<int64_t>(p->table_pages) * c->page_size > 0x7fffffff - 1024)
    return CSBP_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(p->batch) * p->queries > 0x3fffffff / p->Hq)
    return CSBP_ERR_UNSUPPORTED;
  return CSBP_OK;
}

}  // namespace
}  // namespace csbp

using namespace csbp;

extern "C" size_t csbp_paged_workspace_bytes(const csbp_paged_problem* problem,
                                             const csbp_kv_cache* cache) {
  if (validate(problem, cache) != CSBP_OK) return 0;
  return kStatusBytes;
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
  if (ws_bytes < csbp_paged_workspace_bytes(problem, cache)) return CSBP_ERR_WORKSPACE;
  a.pages = cache->pages;
  a.page_size = cache->page_size;
  a.Hkv = cache->Hkv;
  a.d = cache->d;
  a.k = static_cast<const uint8_t*>(cache->k);
  a.v = static_cast<const uint8_t*>(cache->v);
  a.k_scale = static_cast<const uint8_t*>(cache->k_scale);
  a.v_scale = static_cast<const uint8_t*>(cache->v_scale);
  a.batch = p.batch;
  a.queries = p.queries;
  a.table_pages = p.table_pages;
  a.Hq = p.Hq;
  a.causal = p.causal;
  a.window = p.window;
  a.sinks = p.sinks;
  a.scale_log2 = p.scale * 1.4426950408889634f;
  a.q = static_cast<const __nv_bfloat16*>(in->q);
  a.table = in->table;
  a.length = in->length;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  const unsigned grid = static_cast<unsigned>(p.batch) * p.queries * p.Hq;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int timed = timer_begin(13, stream);
  if (cache->d == 128)
    paged_kernel<128><<<grid, kWarps * 32, 0, s>>>(a);
  else
    paged_kernel<64><<<grid, kWarps * 32, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  timer_end(timed, stream);
  return e == cudaSuccess ? CSBP_OK : CSBP_ERR_CUDA;
}
