// Attention of a batch that shares a long prefix (csbp_generate.h).
//
// One warp per (query, head): lanes hold d/32 features each, walk the prefix
// keys and the sequence's own keys, and keep the running maximum and sum of
// the softmax in fp32.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "csbp_generate.h"
#include "csbp_internal.h"

namespace csbp {
namespace {

constexpr size_t kStatusBytes = 256;
constexpr int64_t kMaxElems = int64_t(1) << 39;

struct PrefixArgs {
  int32_t batch, queries, prefix_len, own_max, Hq, Hkv, d, causal;
  float scale;
  const __nv_bfloat16* t[5];
  int64_t tok[5], bat[5];
  const int32_t* own_len;
  __nv_bfloat16* o;
  float* lse;
};

template <int D>
__global__ void __launch_bounds__(256) prefix_simple_kernel(PrefixArgs a) {
  constexpr int kN = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x * 8ll + (threadIdx.x >> 5);
  if (row >= static_cast<int64_t>(a.batch) * a.queries * a.Hq) return;
  const int h = static_cast<int>(row % a.Hq);
  const int64_t bi = row / a.Hq;
  const int i = static_cast<int>(bi % a.queries);
  const int64_t b = bi / a.queries;
  const int hk = h / (a.Hq / a.Hkv);
  float q[kN], acc[kN];
  for (int c = 0; c < kN; ++c) {
    q[c] = __bfloat162float(a.t[0][b * a.bat[0] + i * a.tok[0] + h * D + c * 32 + lane]) * a.scale;
    acc[c] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  auto walk = [&](const __nv_bfloat16* k, const __nv_bfloat16* v, int64_t kt, int64_t vt, int n) {
    for (int64_t j = 0; j < n; ++j) {
      float s = 0.f;
      for (int c = 0; c < kN; ++c) s += q[c] * __bfloat162float(k[j * kt + c * 32 + lane]);
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      const float top = fmaxf(m, s);
      const float old = m == -INFINITY ? 0.f : expf(m - top);
      const float w = expf(s - top);
      l = l * old + w;
      for (int c = 0; c < kN; ++c)
        acc[c] = acc[c] * old + w * __bfloat162float(v[j * vt + c * 32 + lane]);
      m = top;
    }
  };
  if (a.prefix_len > 0) walk(a.t[1] + hk * D, a.t[2] + hk * D, a.tok[1], a.tok[2], a.prefix_len);
  if (a.own_max > 0) {
    const int c = min(max(a.own_len[b], 0), a.own_max);
    const int n = a.causal ? min(c, max(c - a.queries + i + 1, 0)) : c;
    walk(a.t[3] + b * a.bat[3] + hk * D, a.t[4] + b * a.bat[4] + hk * D, a.tok[3], a.tok[4], n);
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  for (int c = 0; c < kN; ++c)
    a.o[row * D + c * 32 + lane] = __float2bfloat16_rn(acc[c] * inv);
  if (lane == 0)
    a.lse[(b * a.Hq + h) * a.queries + i] = l > 0.f ? m + logf(l) : -INFINITY;
}

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
  return CSBP_OK;
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Pointers and strides of the five tensors (q, prefix K and V, own K and V).
csbp_status check_inputs(const csbp_prefix_problem* p, const csbp_prefix_inputs* in,
                         PrefixArgs& a) {
  if (!in || !in->q) return CSBP_ERR_INVALID;
  if (p->prefix_len > 0 && (!in->k_prefix || !in->v_prefix)) return CSBP_ERR_INVALID;
  if (p->own_max > 0 && (!in->k_own || !in->v_own || !in->own_len)) return CSBP_ERR_INVALID;
  if (!aligned(in->own_len, 4)) return CSBP_ERR_INVALID;
  const void* ptr[5] = {in->q, in->k_prefix, in->v_prefix, in->k_own, in->v_own};
  const int64_t len[5] = {p->queries, p->prefix_len, p->prefix_len, p->own_max, p->own_max};
  for (int i = 0; i < 5; ++i) {
    a.t[i] = static_cast<const __nv_bfloat16*>(ptr[i]);
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

}  // namespace
}  // namespace csbp

using namespace csbp;

extern "C" size_t csbp_prefix_workspace_bytes(const csbp_prefix_problem* problem) {
  if (validate(problem) != CSBP_OK) return 0;
  return kStatusBytes;
}

extern "C" csbp_status csbp_attn_prefix(const csbp_prefix_problem* problem,
                                        const csbp_prefix_inputs* in, void* o, float* lse,
                                        void* workspace, size_t ws_bytes, void* stream) {
  csbp_status st = validate(problem);
  if (st != CSBP_OK) return st;
  PrefixArgs a{};
  if ((st = check_inputs(problem, in, a)) != CSBP_OK) return st;
  if (!o || !lse || !workspace || !aligned(o, 16) || !aligned(lse, 16) || !aligned(workspace, 16))
    return CSBP_ERR_INVALID;
  if (ws_bytes < csbp_prefix_workspace_bytes(problem)) return CSBP_ERR_WORKSPACE;
  const csbp_prefix_problem& p = *problem;
  a.batch = p.batch;
  a.queries = p.queries;
  a.prefix_len = p.prefix_len;
  a.own_max = p.own_max;
  a.Hq = p.Hq;
  a.Hkv = p.Hkv;
  a.d = p.d;
  a.causal = p.causal;
  a.scale = p.scale;
  a.own_len = in->own_len;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  const int64_t rows = static_cast<int64_t>(p.batch) * p.queries * p.Hq;
  const int64_t grid = (rows + 7) / 8;
  if (grid > 0x7fffffff) return CSBP_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int timed = timer_begin(13, stream);
  if (p.d == 128)
    prefix_simple_kernel<128><<<static_cast<unsigned>(grid), 256, 0, s>>>(a);
  else
    prefix_simple_kernel<64><<<static_cast<unsigned>(grid), 256, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  timer_end(timed, stream);
  return e == cudaSuccess ? CSBP_OK : CSBP_ERR_CUDA;
}
