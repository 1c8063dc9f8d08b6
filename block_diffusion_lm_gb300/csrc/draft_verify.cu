// Verification of drafted tokens (csbp_generate.h): accept while
// u q(x) < p(x), then draw the next token from max(p - q, 0), or from p, by
// inverting its cumulative sum at r.
//
// The answers are whole numbers, so the arithmetic must not depend on the
// order of summation: u q and p are compared as exact products in 64 bits,
// and the sums are kept to 2^-42 of their value at worst.  64-bit adds run at
// 1/64 of the 32-bit rate here, so the pass over the vocabulary keeps sums as
// unevaluated fp32 numbers (error-free additions, Knuth's two-sum) and only the
// joining of warps, and the search inside the one segment that holds the answer,
// are 64-bit.
//
// A sequence reads two rows of the vocabulary (p and q where its first draft
// was refused) or one, and answers with a few integers: HBM bounds a full batch
// (96 sequences of 131,072 tokens 22.0 us, 4.6 TB/s), the chain of three passes,
// each a load and a joining of warps, a small one (3 of 32,768 tokens 8.0 us).
// 64-bit sums throughout took 74 us at the first, one CTA per sequence 38, one
// running pair per lane, which is less exact, 21.4.
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

// Sums of weights w >= 0 are unevaluated: hi + lo in a tree, h + m + l over all
// of a lane's trees.  How far off they can be, with u = 2^-24 (half a step) and
// S the sum in question: a leaf has |lo| <= u S, a node of level k
// |lo| <= (k + 1) u S, and its two roundings of lo lose (2 k + 1) u^2 S at most.
// So 16 weights lose (3 + 5 + 7 + 9) u^2 S, however many trees follow (the third
// word keeps them to u^3), the step back to a pair u^2 S, and the five levels of
// a warp (3 + 5 + 7 + 9 + 11) u^2 S: 60 u^2 = 2^-42.1 in all, for any vocabulary;
// with roundings of either sign about 2^-47.  (One running pair per lane, whose lo
// collects the roundings of all its additions, is off by 2^-45 after 256 of them
// and by 2^-38 after 8,192.)
struct Pair {
  float hi, lo;
};
struct Sum {
  float h, m, l;
};

// a + b exactly
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float t = a + b;
  const float x = t - a;
  return {t, (a - (t - x)) + (b - x)};
}

// a + b of two such sums
__device__ __forceinline__ Pair join(Pair a, Pair b) {
  Pair s = two_sum(a.hi, b.hi);
  s.lo += a.lo + b.lo;
  return s;
}

__device__ __forceinline__ Pair join(const Pair (&a)[4]) {
  return join(join(a[0], a[1]), join(a[2], a[3]));
}

// s += x, with |m| <= u h and |l| <= u m kept
__device__ __forceinline__ void add(Sum& s, Pair x) {
  const Pair h = two_sum(s.h, x.hi), m = two_sum(s.m, x.lo), e = two_sum(m.hi, h.lo);
  const float l = s.l + (m.lo + e.lo);
  s.h = h.hi + e.hi;
  const float r = e.hi - (s.h - h.hi);
  s.m = r + l;
  s.l = l - (s.m - r);
}

// The weight exactly: p, or max(p - q, 0) as the rounded difference and its
// remainder.  0 for a NaN.
template <bool kResidual>
__device__ __forceinline__ Pair weight(float p, float q) {
  if (!kResidual) return {p > 0.f ? p : 0.f, 0.f};
  const float d = p - q;
  const float x = d - p;
  const float e = (p - (d - x)) - (q + x);
  return d > 0.f ? Pair{d, e} : Pair{0.f, 0.f};
}

// Sum over the warp, in lane 0 (other lanes have partial sums).
__device__ __forceinline__ double warp_sum(Pair s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Pair x{__shfl_down_sync(0xffffffffu, s.hi, o), __shfl_down_sync(0xffffffffu, s.lo, o)};
    s = join(s, x);
  }
  return static_cast<double>(s.hi) + static_cast<double>(s.lo);
}

// This lane's share of w over [v0, v1).  Rows that start on 16 bytes (v0 does
// too) are read four at a time, with 4 loads of each row in flight.
template <bool kResidual>
__device__ __forceinline__ Pair lane_sum(const float* p, const float* q, int64_t v0, int64_t v1,
                                         int lane) {
  Sum s{0.f, 0.f, 0.f};
  const uintptr_t low = reinterpret_cast<uintptr_t>(p + v0) |
                        (kResidual ? reinterpret_cast<uintptr_t>(q + v0) : 0);
  constexpr int kN = 4;
  int left = static_cast<int>(v1 - v0);
  p += v0;
  q += kResidual ? v0 : 0;
  if ((low & 15u) == 0) {
#pragma unroll 1
    for (; left >= 128 * kN; left -= 128 * kN, p += 128 * kN, q += kResidual ? 128 * kN : 0) {
      float4 x[kN], y[kN];
#pragma unroll
      for (int t = 0; t < kN; ++t) {
        x[t] = __ldg(reinterpret_cast<const float4*>(p + t * 128) + lane);
        y[t] = kResidual ? __ldg(reinterpret_cast<const float4*>(q + t * 128) + lane)
                         : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      Pair w[kN];
#pragma unroll
      for (int t = 0; t < kN; ++t) {
        const Pair four[4] = {weight<kResidual>(x[t].x, y[t].x), weight<kResidual>(x[t].y, y[t].y),
                              weight<kResidual>(x[t].z, y[t].z), weight<kResidual>(x[t].w, y[t].w)};
        w[t] = join(four);
      }
      add(s, join(w));
    }
  }
#pragma unroll 1
  for (; left >= 32 * kN; left -= 32 * kN, p += 32 * kN, q += kResidual ? 32 * kN : 0) {
    float x[kN], y[kN];
#pragma unroll
    for (int t = 0; t < kN; ++t) {
      x[t] = __ldg(p + t * 32 + lane);
      y[t] = kResidual ? __ldg(q + t * 32 + lane) : 0.f;
    }
    Pair w[kN];
#pragma unroll
    for (int t = 0; t < kN; ++t) w[t] = weight<kResidual>(x[t], y[t]);
    add(s, join(w));
  }
#pragma unroll 1
  for (int k = lane; k < left; k += 32)
    add(s, weight<kResidual>(__ldg(p + k), kResidual ? __ldg(q + k) : 0.f));
  return {s.h, s.m + s.l};
}

__device__ __forceinline__ Pair lane_sum(const float* p, const float* q, int64_t v0, int64_t v1,
                                         int lane) {
  return q ? lane_sum<true>(p, q, v0, v1, lane) : lane_sum<false>(p, q, v0, v1, lane);
}

__device__ __forceinline__ double weight(const float* p, const float* q, int64_t v) {
  const double w = static_cast<double>(__ldg(p + v)) - (q ? static_cast<double>(__ldg(q + v)) : 0.0);
  return w > 0.0 ? w : 0.0;
}

// Shared memory of a CTA.
struct Shared {
  double seg[kWarps];    // sums of the warps' segments, then of their pieces
  double cta[kCluster];  // sums of the cluster's CTAs (each writes all copies)
  double target, before;
  int first_bad;
  int found;
};

// x_0 + .. + x_lane
__device__ __forceinline__ double scan(double x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// A warp's lanes hold sums x that follow a sum of `before`: the first lane that
// carries it past `target`, with `before` moved to its start.  If rounding leaves
// none, the last with any weight.
__device__ __forceinline__ int crossing(double x, int lane, double target, double& before) {
  const double upto = before + scan(x, lane);
  const unsigned any = __ballot_sync(0xffffffffu, x > 0.0);
  const unsigned over = __ballot_sync(0xffffffffu, x > 0.0 && upto > target);
  const int k = over ? __ffs(over) - 1 : 31 - __clz(any | 1u);
  if (k > 0) before = __shfl_sync(0xffffffffu, upto, k - 1);
  return k;
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

constexpr int kNobody = -3;    // another CTA of the cluster has the answer
constexpr int kNoWeight = -2;  // all weights are 0
constexpr int kSearch = 0;     // in this CTA's part

template <int C>
__device__ int draw(const float* p, const float* q, int V, float r, int rank, Shared& sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t seg = (static_cast<int64_t>(V) + C * kWarps * 128 - 1) / (C * kWarps * 128) * 128;
  const int64_t start = (static_cast<int64_t>(rank) * kWarps + warp) * seg;
  const int64_t end = min(start + seg, static_cast<int64_t>(V));
  Pair mine{0.f, 0.f};
  if (start < end) mine = lane_sum(p, q, start, end, lane);
  const double t = warp_sum(mine);
  if (lane == 0) sh.seg[warp] = t;
  __syncthreads();
  if (C > 1) cluster_wait();
  // 64-bit arithmetic from here, in one warp only
  if (warp == 0) {
    const double all = scan(lane < kWarps ? sh.seg[lane] : 0.0, lane);
    const double x = __shfl_sync(0xffffffffu, all, kWarps - 1);
    if (C == 1) {
      if (lane == 0) sh.cta[0] = x;
    } else if (lane < C) {
      store_cluster(&sh.cta[rank], lane, x);
    }
    __syncwarp();  // the barrier wants whole warps
  }
  if (C > 1) {
    cluster_arrive();
    cluster_wait();
  }
  if (warp == 0) {
    const double x = lane < C ? sh.cta[lane] : 0.0;
    const double total = __shfl_sync(0xffffffffu, scan(x, lane), 31);
    const double target = static_cast<double>(r) * total;
    double before = 0.0;
    int state = kSearch;
    if (!(total > 0.0 && total < 1e300))
      state = total == 0.0 ? kNoWeight : -1;
    else if (crossing(x, lane, target, before) != rank)
      state = kNobody;
    int k = 0;
    if (state == kSearch)
      k = crossing(lane < kWarps ? sh.seg[lane] : 0.0, lane, target, before);
    __syncwarp();
    if (lane == 0) {
      sh.target = target;
      sh.before = before;
      sh.found = state == kSearch ? k : state;
    }
  }
  __syncthreads();
  const int k = sh.found;
  if (k < 0) return k;
  // pieces of segment k, one per warp
  const int64_t s0 = (static_cast<int64_t>(rank) * kWarps + k) * seg;
  const int64_t s1 = min(s0 + seg, static_cast<int64_t>(V));
  const int64_t piece = seg / kWarps;  // a multiple of 8
  {
    const int64_t v0 = s0 + warp * piece, v1 = min(v0 + piece, s1);
    const double w = warp_sum(v0 < v1 ? lane_sum(p, q, v0, v1, lane) : Pair{0.f, 0.f});
    if (lane == 0) sh.seg[warp] = w;
  }
  __syncthreads();
  if (warp == 0) {
    const double target = sh.target;
    double before = sh.before;
    const int m = crossing(lane < kWarps ? sh.seg[lane] : 0.0, lane, target, before);
    const int64_t p0 = s0 + m * piece, p1 = min(p0 + piece, s1);
    int found = -1, positive = -1;
    for (int64_t c = p0; c < p1 && found < 0; c += 32) {
      const double w = c + lane < p1 ? weight(p, q, c + lane) : 0.0;
      const double upto = before + scan(w, lane);
      const unsigned over = __ballot_sync(0xffffffffu, w > 0.0 && upto > target);
      const unsigned any = __ballot_sync(0xffffffffu, w > 0.0);
      if (over)
        found = static_cast<int>(c) + __ffs(over) - 1;
      else if (any)
        positive = static_cast<int>(c) + 31 - __clz(any);
      before = __shfl_sync(0xffffffffu, upto, 31);
    }
    // two roundings of one sum can differ in their last bits
    __syncwarp();
    if (lane == 0) sh.found = found >= 0 ? found : positive;
  }
  __syncthreads();
  return sh.found;
}

// C CTAs (a cluster) per sequence, each for a part of the vocabulary; all of
// them judge the drafts.  Three CTAs to an SM take 40 registers a thread.
template <int C>
__global__ void __launch_bounds__(kThreads, 3) draft_verify_kernel(VerifyArgs a) {
  __shared__ Shared sh;
  if (C > 1) cluster_arrive();
  const int64_t b = blockIdx.x / C;
  const int rank = static_cast<int>(blockIdx.x % C);
  const int32_t* token = a.token + b * a.drafts;
  const int n = a.length ? min(max(__ldg(a.length + b), 0), a.drafts) : a.drafts;
  const float r = __ldg(a.r + b);
  if (threadIdx.x == 0) sh.first_bad = n;
  __syncthreads();
  // tokens past the n-th are looked up too, so that they do not wait for n
  for (int i = threadIdx.x; i < a.drafts; i += kThreads) {
    const int x = __ldg(token + i);
    bool ok = false;
    if (x >= 0 && x < a.vocab) {
      const double px = __ldg(a.p + b * a.p_batch + i * a.p_row + x);
      const double qx = __ldg(a.q + b * a.q_batch + i * a.q_row + x);
      ok = static_cast<double>(__ldg(a.u + b * a.drafts + i)) * qx < px;
    }
    if (!ok && i < n) atomicMin(&sh.first_bad, i);
  }
  __syncthreads();
  const int acc = sh.first_bad;
  const float* p = a.p + b * a.p_batch + acc * a.p_row;
  const float* q = acc < n ? a.q + b * a.q_batch + acc * a.q_row : nullptr;
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
  // A cluster per sequence as large as all sequences' CTAs still run at once
  // (three to an SM), and with at least four 16-byte loads of a row per thread.
  // Measured, us, with 1, 2, 4 and 8 CTAs at a 131,072-token vocabulary:
  // 1 sequence 21.4, 15.0, 10.6, 9.7; 48 sequences 30.9, 19.1, 15.4, 14.0; 96
  // sequences 37.7, 27.1, 20.9, 24.3; 200 sequences 51.1, 40.0, 42.5, 49.0.  At
  // 8,000 tokens (3 sequences) 7.7, 8.1, 7.9, 7.9.
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return CSBP_ERR_CUDA;
  int ctas = 1;
  while (ctas < kCluster && static_cast<int64_t>(c.batch) * ctas * 2 <= 3 * sms &&
         static_cast<int64_t>(c.vocab) >= 2 * ctas * 16 * kThreads)
    ctas *= 2;
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
  const cudaError_t e = ctas == 8   ? cudaLaunchKernelEx(&cfg, draft_verify_kernel<8>, a)
                        : ctas == 4 ? cudaLaunchKernelEx(&cfg, draft_verify_kernel<4>, a)
                        : ctas == 2 ? cudaLaunchKernelEx(&cfg, draft_verify_kernel<2>, a)
                                    : cudaLaunchKernelEx(&cfg, draft_verify_kernel<1>, a);
  timer_end(timed, stream);
  return e == cudaSuccess ? CSBP_OK : CSBP_ERR_CUDA;
}
