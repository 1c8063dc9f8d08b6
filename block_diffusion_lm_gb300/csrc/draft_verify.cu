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

constexpr int kWarps = 32;
constexpr int kThreads = kWarps * 32;

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

__device__ __forceinline__ double weight(const float* p, const float* q, int v) {
  const double w = static_cast<double>(p[v]) - (q ? static_cast<double>(q[v]) : 0.0);
  return w > 0.0 ? w : 0.0;
}

// Smallest v with w_0 + .. + w_v > r x total, -1 without a usable total.
// Every warp sums one contiguous segment; then warp 0 finds the segment and
// scans it.
__device__ int draw(const float* p, const float* q, int V, float r, double* seg_sum,
                    int* answer) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int seg = ((V + kWarps * 32 - 1) / (kWarps * 32)) * 32;
  {
    const int64_t v0 = static_cast<int64_t>(warp) * seg;
    const int64_t v1 = v0 + seg < V ? v0 + seg : V;
    Pair s{0.f, 0.f};
    for (int64_t v = v0 + lane; v < v1; v += 32) {
      if (q)
        add_residual(s, __ldg(p + v), __ldg(q + v));
      else if (const float x = __ldg(p + v); x > 0.f)
        add(s, x, 0.f);
    }
    double t = static_cast<double>(s.hi) + static_cast<double>(s.lo);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (lane == 0) seg_sum[warp] = t;
  }
  __syncthreads();
  if (warp == 0) {
    double total = 0.0;
    for (int k = 0; k < kWarps; ++k) total += seg_sum[k];
    int found = -1;
    if (total > 0.0 && total < 1e300) {
      const double target = static_cast<double>(r) * total;
      double before = 0.0;
      int k = 0, last = 0;
      double last_before = 0.0;
      for (; k < kWarps; ++k) {
        if (seg_sum[k] > 0.0) {
          last = k;
          last_before = before;
        }
        if (before + seg_sum[k] > target) break;
        before += seg_sum[k];
      }
      if (k == kWarps) {  // r outside [0, 1): the last token that has weight
        k = last;
        before = last_before;
      }
      const int64_t v0 = static_cast<int64_t>(k) * seg;
      const int64_t v1 = v0 + seg < V ? v0 + seg : V;
      int positive = -1;
      for (int64_t c = v0; c < v1 && found < 0; c += 32) {
        const int64_t v = c + lane;
        const double w = v < v1 ? weight(p, q, static_cast<int>(v)) : 0.0;
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
      // the two roundings of one segment's sum can differ in their last bits
      if (found < 0) found = positive;
    }
    if (lane == 0) *answer = total > 0.0 ? found : -2;  // -2: no weight at all
  }
  __syncthreads();
  return *answer;
}

__global__ void __launch_bounds__(kThreads) draft_verify_kernel(VerifyArgs a) {
  __shared__ double seg_sum[kWarps];
  __shared__ int first_bad, answer;
  const int64_t b = blockIdx.x;
  int n = a.drafts;
  if (a.length) n = min(max(__ldg(a.length + b), 0), a.drafts);
  if (threadIdx.x == 0) first_bad = n;
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
    if (!ok) atomicMin(&first_bad, i);
  }
  __syncthreads();
  const int acc = first_bad;
  const float* p = a.p + b * a.p_batch + acc * a.p_row;
  const float* q = acc < n ? a.q + b * a.q_batch + acc * a.q_row : nullptr;
  const float r = __ldg(a.r + b);
  int next = draw(p, q, a.vocab, r, seg_sum, &answer);
  if (next == -2 && q) {  // p <= q everywhere
    __syncthreads();
    next = draw(p, nullptr, a.vocab, r, seg_sum, &answer);
  }
  if (next < 0) next = -1;
  int32_t* out = a.out + b * (static_cast<int64_t>(a.drafts) + 1);
  for (int i = threadIdx.x; i <= a.drafts; i += kThreads)
    out[i] = i < acc ? __ldg(token + i) : i == acc ? next : -1;
  if (threadIdx.x == 0) a.accepted[b] = acc;
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
  const int timed = timer_begin(15, stream);
  draft_verify_kernel<<<c.batch, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  timer_end(timed, stream);
  return e == cudaSuccess ? CSBP_OK : CSBP_ERR_CUDA;
}
