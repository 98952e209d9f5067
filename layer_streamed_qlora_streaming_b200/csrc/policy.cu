// Clipped policy loss with a KL term, from logits to loss, log-probabilities and dlogits (the surrogate
// of Schulman et al., "Proximal Policy Optimization Algorithms", 2017, with the per-token KL estimate
// k3 of Shao et al., "DeepSeekMath", 2024; formulas in policy.cuh). Its gradient:
//   dl/dlogp = -r A [u is r A] + beta (1 - exp(ref - logp)),  dlogits = w dl/dlogp (onehot(y) - softmax(x)).
// One CTA per row reads it twice: maximum and sum of exponentials, then dlogits.
#include "common.cuh"
#include "pdl.cuh"
#include "policy.cuh"

namespace lst {
namespace {

using bf16 = __nv_bfloat16;

// scratch: [0] rows done so far (as unsigned), then 4 floats a row, then the weight of each sequence's tokens
__host__ __device__ inline float* row_terms(float* scratch) { return scratch + 4; }
__host__ __device__ inline float* seq_weight(float* scratch, int64_t T) { return scratch + 4 + 4 * T; }

// exp(d) - d - 1 without its cancellation near zero: the power series there
__device__ __forceinline__ float k3_term(float d) {
  if (fabsf(d) < 0.125f) {
    float t = 1.f / 720.f;
    t = fmaf(t, d, 1.f / 120.f);
    t = fmaf(t, d, 1.f / 24.f);
    t = fmaf(t, d, 1.f / 6.f);
    t = fmaf(t, d, 0.5f);
    return t * d * d;
  }
  return expm1f(d) - d;
}

// One token's terms (l, kl, clipped, r) and dl/dlogp.
struct Token {
  float4 terms;
  float slope;
};
__device__ __forceinline__ Token policy_token(const PolicyArgs& a, int64_t t, float logp) {
  const float A = a.adv[a.adv_per_seq ? t / a.S : t];
  const float r = a.old_logp ? expf(logp - a.old_logp[t]) : 1.f;
  const float in = r * A, cl = fminf(fmaxf(r, 1.f - a.lo), 1.f + a.hi) * A;
  const bool cut = in > cl;  // the clip lowers the surrogate: no gradient
  float kl = 0.f, dkl = 0.f;
  if (a.ref_logp) {
    const float d = a.ref_logp[t] - logp;
    kl = k3_term(d);
    dkl = -expm1f(d);
  }
  return {make_float4(fmaf(a.beta, kl, -(cut ? cl : in)), kl, cut ? 1.f : 0.f, r), fmaf(a.beta, dkl, cut ? 0.f : -in)};
}

// One CTA: counts the mask and leaves the weight of a counted token of each sequence.
__global__ void __launch_bounds__(1024) k_policy_weights(const int32_t* __restrict__ mask, int64_t T, int S, int norm,
                                                         float* __restrict__ scratch) {
  pdl_wait();
  pdl_trigger();
  __shared__ int64_t part[32];
  __shared__ float common;
  float* w = seq_weight(scratch, T);
  const int64_t nseq = T / S;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t mine = 0;
  for (int64_t b = warp; b < nseq; b += 32) {
    int n = 0;
    for (int i = lane; i < S; i += 32) n += mask ? mask[b * S + i] != 0 : 1;
    n = __reduce_add_sync(0xffffffffu, n);
    mine += n;
    if (lane == 0) w[b] = norm == 1 ? (n ? 1.f / ((float)nseq * (float)n) : 0.f) : 1.f / (float)T;
  }
  if (lane == 0) part[warp] = mine;
  __syncthreads();
  if (threadIdx.x == 0) {
    reinterpret_cast<unsigned*>(scratch)[0] = 0;
    int64_t n = 0;
    for (int i = 0; i < 32; ++i) n += part[i];
    common = n ? 1.f / (float)n : 0.f;
  }
  __syncthreads();
  if (norm == 0)
    for (int64_t b = threadIdx.x; b < nseq; b += blockDim.x) w[b] = common;
}

// The last CTA of the call adds the row terms in a fixed order (fp64) and writes out.
__device__ __forceinline__ void finish_row(const PolicyArgs& a, int64_t t, float4 terms) {
  __shared__ bool last;
  __shared__ double part[4][32];
  if (threadIdx.x == 0) {
    reinterpret_cast<float4*>(row_terms(a.scratch))[t] = terms;
    __threadfence();
    last = atomicAdd(reinterpret_cast<unsigned*>(a.scratch), 1u) + 1u == (unsigned)a.T;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  const float4* rows = reinterpret_cast<const float4*>(row_terms(a.scratch));
  double s[4] = {0, 0, 0, 0};
  for (int64_t i = threadIdx.x; i < a.T; i += blockDim.x) {
    const float4 v = __ldcg(rows + i);
    s[0] += v.x;
    s[1] += v.y;
    s[2] += v.z;
    s[3] += v.w;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    for (int o = 16; o > 0; o >>= 1) s[e] += __shfl_xor_sync(0xffffffffu, s[e], o);
    if ((threadIdx.x & 31) == 0) part[e][threadIdx.x >> 5] = s[e];
  }
  __syncthreads();
  if (threadIdx.x < 4) {
    double v = 0;
    for (int i = 0; i < (int)(blockDim.x >> 5); ++i) v += part[threadIdx.x][i];
    a.out[threadIdx.x] = (float)v;
  }
}

__global__ void __launch_bounds__(512) k_policy_rows(const PolicyArgs a, int64_t row0) {
  pdl_wait();
  pdl_trigger();
  __shared__ float red[16];
  __shared__ float coef_s;
  const int64_t lrow = blockIdx.x, t = row0 + lrow;
  const float* x = a.logits + lrow * a.V;
  bf16* d = a.dlog ? a.dlog + lrow * a.V : nullptr;
  const int y = a.y[t];
  const bool counted = !a.mask || a.mask[t] != 0;
  const bool bad = counted && (y < 0 || y >= a.V);
  if (bad && threadIdx.x == 0) dev_fail(DEV_ERR_BAD_INDEX);
  if (!counted || bad) {
    if (d)
      for (int c = threadIdx.x; c < a.V; c += blockDim.x) d[c] = __float2bfloat16_rn(0.f);
    if (threadIdx.x == 0) a.logp[t] = 0.f;
    finish_row(a, t, make_float4(0.f, 0.f, 0.f, 0.f));
    return;
  }
  float m = -INFINITY, s = 0.f;
  for (int c = threadIdx.x; c < a.V; c += blockDim.x) m = fmaxf(m, x[c]);
  m = warp_max(m);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  for (int i = 0; i < (int)(blockDim.x >> 5); ++i) m = fmaxf(m, red[i]);
  for (int c = threadIdx.x; c < a.V; c += blockDim.x) s += expf(x[c] - m);
  s = warp_sum(s);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  s = 0.f;
  for (int i = 0; i < (int)(blockDim.x >> 5); ++i) s += red[i];
  const float ls = logf(s);
  float4 terms;
  if (threadIdx.x == 0) {
    const float logp = (x[y] - m) - ls;
    const Token k = policy_token(a, t, logp);
    const float w = seq_weight(a.scratch, a.T)[t / a.S];
    a.logp[t] = logp;
    coef_s = -w * k.slope;
    terms = make_float4(w * k.terms.x, w * k.terms.y, w * k.terms.z, w * k.terms.w);
  }
  __syncthreads();
  if (d) {
    const float coef = coef_s;
    for (int c = threadIdx.x; c < a.V; c += blockDim.x) {
      const float p = expf(x[c] - m - ls);
      d[c] = __float2bfloat16_rn(coef * (c == y ? p - 1.f : p));
    }
  }
  finish_row(a, t, terms);
}

}  // namespace

int64_t policy_scratch(int64_t T, int S) { return 4 + 4 * T + T / S; }

bool policy_args_ok(const PolicyArgs& a) {
  return a.T > 0 && a.T <= INT32_MAX && a.V > 0 && a.V <= kPolicyMaxV && a.S > 0 && a.T % a.S == 0 && a.lo >= 0.f &&
         a.lo <= 1.f && a.hi >= 0.f && a.beta >= 0.f && a.beta < INFINITY && (a.beta == 0.f || a.ref_logp) &&
         a.norm >= 0 && a.norm <= 2;
}

cudaError_t policy_begin(const PolicyArgs& a, cudaStream_t s) {
  if (!policy_args_ok(a)) return cudaErrorInvalidValue;
  const cudaError_t e = launch_k(k_policy_weights, dim3(1), dim3(1024), 0, s, 0, a.mask, a.T, a.S, a.norm, a.scratch);
  note_launch(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t policy_rows(const PolicyArgs& a, int64_t row0, int64_t rows, cudaStream_t s) {
  if (!policy_args_ok(a) || row0 < 0 || rows <= 0 || row0 + rows > a.T) return cudaErrorInvalidValue;
  const cudaError_t e = launch_k(k_policy_rows, dim3((unsigned)rows), dim3(512), 0, s, 0, a, row0);
  note_launch(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace lst
