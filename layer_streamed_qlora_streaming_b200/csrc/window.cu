// Causal GQA attention with a sliding window and sinks: key j of a sequence is visible to its query
// i when j <= i and (i - j < window or j < sinks).
//   s_ij = q_i . k_j / sqrt(hd),  P = softmax of s over the visible keys,  o_i = sum_j P_ij v_j,
//   lse_i = log sum_j exp s_ij;
//   D_i = do_i . o_i,  dS_ij = P_ij (do_i . v_j - D_i),
//   dq_i = sum_j dS_ij k_j / sqrt(hd),  dk_j = sum_{h, i} dS_ij q_i / sqrt(hd),  dv_j = sum_{h, i} P_ij do_i,
// the last two over the query heads h that share the kv head. One warp per row (query or key), its
// lanes along the head dimension, the sums of a row in one fixed order.
#include "common.cuh"
#include "pdl.cuh"
#include "ex2.cuh"
#include "window.cuh"

namespace lst {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

template <int N>
__device__ __forceinline__ void load_row(float (&x)[N], const __nv_bfloat16* p, int lane) {
#pragma unroll
  for (int e = 0; e < N; ++e) x[e] = __bfloat162float(p[lane + 32 * e]);
}
template <int N>
__device__ __forceinline__ float dot(const float (&a)[N], const float (&b)[N]) {
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < N; ++e) s += a[e] * b[e];
  return warp_sum(s);
}
// f(j) for the visible keys j of query i in ascending order
template <typename F>
__device__ __forceinline__ void each_key(int i, int window, int sinks, F f) {
  const int w0 = max(0, i - window + 1);
  for (int j = 0; j < min(sinks, w0); ++j) f(j);
  for (int j = w0; j <= i; ++j) f(j);
}

template <int HD>
__global__ void __launch_bounds__(256) k_window_fwd(const WinArgs p) {
  constexpr int N = HD / 32;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= p.T * p.hq) return;
  const int64_t t = row / p.hq, tok0 = t - t % p.S;
  const int h = (int)(row % p.hq), kvh = h / (p.hq / p.hkv), i = (int)(t % p.S);
  float q[N], o[N] = {}, m = -INFINITY, l = 0.f;
  load_row<N>(q, p.q + t * p.ldq + (int64_t)h * HD, lane);
  each_key(i, p.window, p.sinks, [&](int j) {
    float k[N], v[N];
    load_row<N>(k, p.k + (tok0 + j) * p.ldk + (int64_t)kvh * HD, lane);
    load_row<N>(v, p.v + (tok0 + j) * p.ldv + (int64_t)kvh * HD, lane);
    const float s = dot<N>(q, k) * p.scale;
    const float mn = fmaxf(m, s), c = expf(m - mn), e = expf(s - mn);
    m = mn;
    l = l * c + e;
#pragma unroll
    for (int x = 0; x < N; ++x) o[x] = o[x] * c + e * v[x];
  });
#pragma unroll
  for (int x = 0; x < N; ++x) {
    const float y = o[x] / l;
    p.o[t * p.ldo + (int64_t)h * HD + lane + 32 * x] = __float2bfloat16_rn(y);
    if (p.o32) p.o32[(t * p.hq + h) * HD + lane + 32 * x] = y;
  }
  if (lane == 0) p.lse[row] = m + logf(l);
}

// x * scale of one row (lane + 32 e its columns), the rotary embedding of position pos undone
template <int HD>
__device__ __forceinline__ void store_grad(__nv_bfloat16* dst, const float (&x)[HD / 32], const AttnBwdArgs& p, int pos,
                                           int lane) {
  constexpr int N = HD / 32, HALF = HD / 2;
#pragma unroll
  for (int e = 0; e < N / 2; ++e) {
    const int c = lane + 32 * e;
    float y1 = x[e] * p.scale, y2 = x[e + N / 2] * p.scale;
    if (p.rope_cos) {
      const float cs = p.rope_cos[(int64_t)pos * HALF + c], sn = p.rope_sin[(int64_t)pos * HALF + c];
      const float a = y1 * cs + y2 * sn;
      y2 = y2 * cs - y1 * sn;
      y1 = a;
    }
    dst[c] = __float2bfloat16_rn(y1);
    dst[c + HALF] = __float2bfloat16_rn(y2);
  }
}

template <int HD>
__global__ void __launch_bounds__(256) k_window_dq(const WinBwdArgs p) {
  constexpr int N = HD / 32;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= p.T * p.hq) return;
  const int64_t t = row / p.hq, tok0 = t - t % p.S;
  const int h = (int)(row % p.hq), kvh = h / (p.hq / p.hkv), i = (int)(t % p.S);
  float q[N], o[N], d[N], dq[N] = {};
  load_row<N>(q, p.q + t * p.ldq + (int64_t)h * HD, lane);
  load_row<N>(d, p.dout + t * p.lddo + (int64_t)h * HD, lane);
  if (p.o32) {
#pragma unroll
    for (int x = 0; x < N; ++x) o[x] = p.o32[(t * p.hq + h) * HD + lane + 32 * x];
  } else {
    load_row<N>(o, p.o + t * p.ldo + (int64_t)h * HD, lane);
  }
  const float D = dot<N>(d, o), lse = p.lse[row];
  if (lane == 0) p.D[row] = D;
  each_key(i, p.window, p.sinks, [&](int j) {
    float k[N], v[N];
    load_row<N>(k, p.k + (tok0 + j) * p.ldk + (int64_t)kvh * HD, lane);
    load_row<N>(v, p.v + (tok0 + j) * p.ldv + (int64_t)kvh * HD, lane);
    const float pr = expf(dot<N>(q, k) * p.scale - lse), ds = pr * (dot<N>(d, v) - D);
#pragma unroll
    for (int x = 0; x < N; ++x) dq[x] += ds * k[x];
  });
  store_grad<HD>(p.dq + t * p.lddq + (int64_t)h * HD, dq, p, i, lane);
}

template <int HD>
__global__ void __launch_bounds__(256) k_window_dkdv(const WinBwdArgs p) {
  constexpr int N = HD / 32;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= p.T * p.hkv) return;
  const int64_t t = row / p.hkv, tok0 = t - t % p.S;
  const int kvh = (int)(row % p.hkv), grp = p.hq / p.hkv, j = (int)(t % p.S);
  const int end = j < p.sinks ? p.S : (int)min((int64_t)p.S, (int64_t)j + p.window);
  float k[N], v[N], dk[N] = {}, dv[N] = {};
  load_row<N>(k, p.k + t * p.ldk + (int64_t)kvh * HD, lane);
  load_row<N>(v, p.v + t * p.ldv + (int64_t)kvh * HD, lane);
  for (int h = kvh * grp; h < (kvh + 1) * grp; ++h) {
    for (int i = j; i < end; ++i) {
      float q[N], d[N];
      load_row<N>(q, p.q + (tok0 + i) * p.ldq + (int64_t)h * HD, lane);
      load_row<N>(d, p.dout + (tok0 + i) * p.lddo + (int64_t)h * HD, lane);
      const int64_t at = (tok0 + i) * p.hq + h;
      const float pr = expf(dot<N>(q, k) * p.scale - p.lse[at]), ds = pr * (dot<N>(d, v) - p.D[at]);
#pragma unroll
      for (int x = 0; x < N; ++x) {
        dv[x] += pr * d[x];
        dk[x] += ds * q[x];
      }
    }
  }
  store_grad<HD>(p.dk + t * p.lddk + (int64_t)kvh * HD, dk, p, j, lane);
#pragma unroll
  for (int x = 0; x < N; ++x) p.dv[t * p.lddv + (int64_t)kvh * HD + lane + 32 * x] = __float2bfloat16_rn(dv[x]);
}

}  // namespace

bool window_shape_ok(int64_t T, int S, int hq, int hkv, int hd, int window, int sinks) {
  return (hd == 64 || hd == 128) && hq > 0 && hkv > 0 && hq % hkv == 0 && S > 0 && T > 0 && T % S == 0 &&
         T <= INT32_MAX && T * hq <= INT32_MAX && window >= 1 && sinks >= 0;
}

int64_t window_scratch(int64_t T, int S, int hq, int hkv, int hd, int window, int sinks) { return T * hq; }

cudaError_t window_fwd(const WinArgs& a, cudaStream_t s) {
  if (!window_shape_ok(a.T, a.S, a.hq, a.hkv, a.hd, a.window, a.sinks)) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)((a.T * a.hq + 7) / 8));
  const cudaError_t e = a.hd == 128 ? launch_k(k_window_fwd<128>, grid, dim3(256), 0, s, 0, a)
                                    : launch_k(k_window_fwd<64>, grid, dim3(256), 0, s, 0, a);
  note_launch(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t window_bwd(const WinBwdArgs& a, cudaStream_t s) {
  if (!window_shape_ok(a.T, a.S, a.hq, a.hkv, a.hd, a.window, a.sinks)) return cudaErrorInvalidValue;
  const dim3 gq((unsigned)((a.T * a.hq + 7) / 8)), gk((unsigned)((a.T * a.hkv + 7) / 8));
  cudaError_t e;
  if (a.hd == 128) {
    e = launch_k(k_window_dq<128>, gq, dim3(256), 0, s, 0, a);
    if (e == cudaSuccess) e = launch_k(k_window_dkdv<128>, gk, dim3(256), 0, s, 0, a);
  } else {
    e = launch_k(k_window_dq<64>, gq, dim3(256), 0, s, 0, a);
    if (e == cudaSuccess) e = launch_k(k_window_dkdv<64>, gk, dim3(256), 0, s, 0, a);
  }
  note_launch(2);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace lst
