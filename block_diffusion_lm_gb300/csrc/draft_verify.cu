// Verification of drafted tokens (csbp_generate.h): accept while
// u q(x) < p(x), then draw the next token from max(p - q, 0), or from p, by
// inverting its cumulative sum at r.
//
// The answers are whole numbers, so the arithmetic must not depend on the
// order of summation: u q and p are compared as exact products in 64 bits,
// and the sums carry about 2^-46 of their value.  64-bit adds run at 1/64 of
// the 32-bit rate here, so the pass over the vocabulary keeps each lane's sum
// as an unevaluated pair of fp32 numbers (error-free additions) and only the
// joining of lanes, and the search inside the one segment that holds the
// answer, are 64-bit.
#include <cuda_runtime.h>

#include <cstdint>

#include "csbp_generate.h"
#include "csbp_internal.h"

namespace csbp {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kCluster = 8;  // CTAs of one sequence, for long vocabularies

struct VerifyArgs {
  int32_t drafts, vocab;
  int64_t p_row, p_batch, q_row, q_batch;
  const float *p, *q, *u, *r;
  const int32_t *token, *length;
  int32_t *accepted, *out;
};

// Unevaluated sum hi + lo, |lo| small against hi.
struct Pair {
  float hi, lo;
};

// s += x + e, where e is a rounding remainder of x
__device__ __forceinline__ void add(Pair& s, float x, float e) {
  const float t = s.hi + x;
  const float b = t - s.hi;
  s.lo += ((s.hi - (t - b)) + (x - b)) + e;
  s.hi = t;
}

// The weight max(p - q, 0) as d + e exactly (e the remainder of the rounded
// difference d); 0 for a NaN.
__device__ __forceinline__ void add_residual(Pair& s, float p, float q) {
  const float d = p - q;
  const float b = d - p;
  const float e = (p - (d - b)) - (q + b);
  if (d > 0.f) add(s, d, e);
}

template <bool kResidual>
__device__ __forceinline__ void add_weight(Pair& s, float p, float q) {
  if (kResidual)
    add_residual(s, p, q);
  else if (p > 0.f)
    add(s, p, 0.f);
}

// This lane's share of w over [v0, v1), v0 a multiple of 4.  Rows that start on
// 16 bytes are read four at a time, with 4 loads of each row in flight.
template <bool kResidual>
__device__ __forceinline__ double lane_sum(const float* p, const float* q, int64_t v0, int64_t v1,
                                           int lane) {
  Pair s{0.f, 0.f};
  const uintptr_t low = reinterpret_cast<uintptr_t>(p) | (kResidual ? reinterpret_cast<uintptr_t>(q)
                                                                    : 0);
  int64_t v = v0;
  if ((low & 15u) == 0) {
    constexpr int kUnroll = 4;
    for (; v + 128 * kUnroll <= v1; v += 128 * kUnroll) {
      float4 x[kUnroll], y[kUnroll];
#pragma unroll
      for (int t = 0; t < kUnroll; ++t) {
        x[t] = __ldg(reinterpret_cast<const float4*>(p + v + t * 128) + lane);
        if (kResidual) y[t] = __ldg(reinterpret_cast<const float4*>(q + v + t * 128) + lane);
      }
#pragma unroll
      for (int t = 0; t < kUnroll; ++t) {
        if (!kResidual) y[t] = make_float4(0.f, 0.f, 0.f, 0.f);
        add_weight<kResidual>(s, x[t].x, y[t].x);
        add_weight<kResidual>(s, x[t].y, y[t].y);
        add_weight<kResidual>(s, x[t].z, y[t].z);
        add_weight<kResidual>(s, x[t].w, y[t].w);
      }
    }
  }
#pragma unroll 4
  for (v += lane; v < v1; v += 32)
    add_weight<kResidual>(s, __ldg(p + v), kResidual ? __ldg(q + v) : 0.f);
  return static_cast<double>(s.hi) + static_cast<double>(s.lo);
}

__device__ __forceinline__ double warp_sum(double t) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  return t;
}

__device__ __forceinline__ double weight(const float* p, const float* q, int64_t v) {
  const double w = static_cast<double>(__ldg(p + v)) - (q ? static_cast<double>(__ldg(q + v)) : 0.0);
  return w > 0.0 ? w : 0.0;
}

// Shared memory of a CTA.
struct Shared {
  double seg[kWarps];         // sums of the warps' segments, then of their parts
  double cta[kCluster];       // sums of the cluster's CTAs (each writes all copies)
  int first_bad;
  int found;
};

// Of n sums that follow a sum of `before`: the first one that carries it past
// `target`, with `before` moved to its start.  If rounding leaves none, the last
// with any weight.
__device__ __forceinline__ int crossing(const double* sums, int n, double target, double& before) {
  int last = 0;
  double at = before, last_at = before;
  for (int k = 0; k < n; ++k) {
    if (sums[k] > 0.0) {
      last = k;
      last_at = at;
      if (at + sums[k] > target) break;
    }
    at += sums[k];
  }
  before = last_at;
  return last;
}

__device__ __forceinline__ void store_cluster(double* local, uint32_t rank, double x) {
  uint32_t addr = static_cast<uint32_t>(__cvta_generic_to_shared(local)), remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(remote), "d"(x) : "memory");
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}

constexpr int kNobody = -3;  // another CTA of the cluster has the answer
constexpr int kNoWeight = -2;

// Smallest v with w_0 + .. + w_v > r x total (in one CTA of the cluster, kNobody
// in the others); -1 when the total is not finite, kNoWeight when it is 0.
// Every warp sums one contiguous segment of the vocabulary; the CTA whose part
// holds the answer finds the segment, lets its warps sum pieces of it in 64
// bits, and scans the piece.
// On entry the cluster's CTAs have arrived at its barrier (they all run, and
// have read what an earlier draw left).
template <int C>
__device__ int draw(const float* p, const float* q, int V, float r, int rank, Shared& sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t seg = (static_cast<int64_t>(V) + C * kWarps * 128 - 1) / (C * kWarps * 128) * 128;
  const int64_t start = (static_cast<int64_t>(rank) * kWarps + warp) * seg;
  const int64_t end = min(start + seg, static_cast<int64_t>(V));
  double t = 0.0;
  if (start < end)
    t = q ? lane_sum<true>(p, q, start, end, lane) : lane_sum<false>(p, q, start, end, lane);
  t = warp_sum(t);
  if (lane == 0) sh.seg[warp] = t;
  __syncthreads();
  if (C > 1) cluster_wait();
  if (warp == 0) {
    double mine = 0.0;
    for (int k = 0; k < kWarps; ++k) mine += sh.seg[k];
    if (C == 1) {
      if (lane == 0) sh.cta[0] = mine;
    } else if (lane < C) {
      store_cluster(&sh.cta[rank], lane, mine);
    }
  }
  if (C > 1)
    cluster_sync();
  else
    __syncthreads();
  double total = 0.0;
#pragma unroll
  for (int k = 0; k < C; ++k) total += sh.cta[k];
  if (!(total > 0.0)) return total == 0.0 ? kNoWeight : -1;
  if (!(total < 1e300)) return -1;
  const double target = static_cast<double>(r) * total;
  double before = 0.0;
  if (crossing(sh.cta, C, target, before) != rank) return kNobody;
  const int k = crossing(sh.seg, kWarps, target, before);
  __syncthreads();  // all have read the segments' sums
  // pieces of segment k, one per warp
  const int64_t s0 = (static_cast<int64_t>(rank) * kWarps + k) * seg;
  const int64_t s1 = min(s0 + seg, static_cast<int64_t>(V));
  const int64_t piece = (seg + kWarps - 1) / kWarps;  // a multiple of 8
  {
    double w = 0.0;
    const int64_t e = min(s0 + (warp + 1) * piece, s1);
    for (int64_t v = s0 + warp * piece + lane; v < e; v += 32) w += weight(p, q, v);
    w = warp_sum(w);
    if (lane == 0) sh.seg[warp] = w;
  }
  __syncthreads();
  if (warp == 0) {
    const int m = crossing(sh.seg, kWarps, target, before);
    const int64_t p0 = s0 + m * piece, p1 = min(p0 + piece, s1);
    int found = -1, positive = -1;
    for (int64_t c = p0; c < p1 && found < 0; c += 32) {
      const double w = c + lane < p1 ? weight(p, q, c + lane) : 0.0;
      double sum = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double x = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += x;
      }
      const unsigned over = __ballot_sync(0xffffffffu, w > 0.0 && before + sum > target);
      const unsigned any = __ballot_sync(0xffffffffu, w > 0.0);
      if (over)
        found = static_cast<int>(c) + __ffs(over) - 1;
      else if (any)
        positive = static_cast<int>(c) + 31 - __clz(any);
      before += __shfl_sync(0xffffffffu, sum, 31);
    }
    // two roundings of one sum can differ in their last bits
    if (lane == 0) sh.found = found >= 0 ? found : positive;
  }
  __syncthreads();
  return sh.found;
}

// C CTAs (a cluster) per sequence, each for a part of the vocabulary; all of
// them judge the drafts.
template <int C>
__global__ void __launch_bounds__(kThreads) draft_verify_kernel(VerifyArgs a) {
  __shared__ Shared sh;
  if (C > 1) cluster_arrive();
  const int64_t b = blockIdx.x / C;
  const int rank = static_cast<int>(blockIdx.x % C);
  int n = a.drafts;
  if (a.length) n = min(max(__ldg(a.length + b), 0), a.drafts);
  if (threadIdx.x == 0) sh.first_bad = n;
  __syncthreads();
  const int32_t* token = a.token + b * a.drafts;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int x = __ldg(token + i);
    bool ok = false;
    if (x >= 0 && x < a.vocab) {
      const double px = __ldg(a.p + b * a.p_batch + i * a.p_row + x);
      const double qx = __ldg(a.q + b * a.q_batch + i * a.q_row + x);
      ok = static_cast<double>(__ldg(a.u + b * a.drafts + i)) * qx < px;
    }
    if (!ok) atomicMin(&sh.first_bad, i);
  }
  __syncthreads();
  const int acc = sh.first_bad;
  const float* p = a.p + b * a.p_batch + acc * a.p_row;
  const float* q = acc < n ? a.q + b * a.q_batch + acc * a.q_row : nullptr;
  const float r = __ldg(a.r + b);
  int next = draw<C>(p, q, a.vocab, r, rank, sh);
  if (next == kNoWeight && q) {  // p <= q everywhere, the same in all CTAs
    if (C > 1)
      cluster_arrive();
    else
      __syncthreads();
    next = draw<C>(p, nullptr, a.vocab, r, rank, sh);
  }
  const bool writes = next >= 0 || (next != kNobody && rank == 0);
  if (writes) {
    int32_t* out = a.out + b * (static_cast<int64_t>(a.drafts) + 1);
    for (int i = threadIdx.x; i <= a.drafts; i += kThreads)
      out[i] = i < acc ? __ldg(token + i) : i == acc ? max(next, -1) : -1;
    if (threadIdx.x == 0) a.accepted[b] = acc;
  }
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Row and batch strides of `rows` rows: the given ones, or contiguous for 0.
bool strides(int64_t rows, int64_t batch, int64_t V, int64_t row, int64_t bat, int64_t& row_out,
             int64_t& bat_out) {
  constexpr int64_t kMax = int64_t(1) << 40;
  if (row < 0 || bat < 0) return false;
  row_out = row != 0 ? row : V;
  if (row_out < V || row_out > kMax / (rows > 0 ? rows : 1)) return false;
  bat_out = (batch > 1 && bat != 0) ? bat : rows * row_out;
  return bat_out >= rows * row_out && bat_out <= kMax;
}

}  // namespace
}  // namespace csbp

using namespace csbp;

extern "C" csbp_status csbp_draft_verify(const csbp_verify_problem* problem, const float* p,
                                         const float* q, const int32_t* token, const float* u,
                                         const float* r, const int32_t* length,
                                         int32_t* accepted, int32_t* out, void* stream) {
  if (!problem) return CSBP_ERR_INVALID;
  const csbp_verify_problem& c = *problem;
  if (c.batch < 0 || c.drafts < 0 || c.drafts > 4096 || c.vocab < 1) return CSBP_ERR_INVALID;
  VerifyArgs a{};
  if (!strides(static_cast<int64_t>(c.drafts) + 1, c.batch, c.vocab, c.p_row, c.p_batch, a.p_row,
               a.p_batch) ||
      !strides(c.drafts, c.batch, c.vocab, c.q_row, c.q_batch, a.q_row, a.q_batch))
    return CSBP_ERR_INVALID;
  if (c.batch == 0) return CSBP_OK;
  if (!p || !r || !accepted || !out) return CSBP_ERR_INVALID;
  if (c.drafts > 0 && (!q || !token || !u)) return CSBP_ERR_INVALID;
  const void* all[] = {p, q, token, u, r, length, accepted, out};
  for (const void* x : all)
    if (!aligned4(x)) return CSBP_ERR_INVALID;
  a.drafts = c.drafts;
  a.vocab = c.vocab;
  a.p = p;
  a.q = q;
  a.u = u;
  a.r = r;
  a.token = token;
  a.length = length;
  a.accepted = accepted;
  a.out = out;
  // one CTA reads about as fast as 1/100 of the GPU: a cluster per sequence
  // once every thread of one CTA would have more than four loads of a row
  const int ctas = c.vocab > 4 * 4 * kThreads ? kCluster : 1;
  if (static_cast<int64_t>(c.batch) * ctas > 0x7fffffff) return CSBP_ERR_UNSUPPORTED;
  cudaLaunchAttribute together{};
  together.id = cudaLaunchAttributeClusterDimension;
  together.val.clusterDim.x = static_cast<unsigned>(ctas);
  together.val.clusterDim.y = together.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(c.batch) * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = &together;
  cfg.numAttrs = 1;
  const int timed = timer_begin(15, stream);
  const cudaError_t e = ctas > 1 ? cudaLaunchKernelEx(&cfg, draft_verify_kernel<kCluster>, a)
                                 : cudaLaunchKernelEx(&cfg, draft_verify_kernel<1>, a);
  timer_end(timed, stream);
  return e == cudaSuccess ? CSBP_OK : CSBP_ERR_CUDA;
}
